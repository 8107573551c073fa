// sv_kv_shared_f16_1.cu -- shared-prefix attention kernels: f16, vectors of up to 128 components.
#include "sv_kv_shared.cuh"

namespace sv {

extern const SharedKernel shared_kernels_f16_1[3] = {kv_attend_shared_kernel<32, false, 1>,
                                              kv_attend_shared_kernel<64, false, 1>,
                                              kv_attend_shared_kernel<128, false, 1>};

}  // namespace sv
