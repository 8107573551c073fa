// sv_kv_shared_f16_2.cu -- shared-prefix attention kernels: f16, vectors of up to 256 components.
#include "sv_kv_shared.cuh"

namespace sv {

extern const SharedKernel shared_kernels_f16_2[3] = {kv_attend_shared_kernel<32, false, 2>,
                                              kv_attend_shared_kernel<64, false, 2>,
                                              kv_attend_shared_kernel<128, false, 2>};

}  // namespace sv
