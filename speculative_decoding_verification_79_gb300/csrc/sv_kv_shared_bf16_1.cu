// sv_kv_shared_bf16_1.cu -- shared-prefix attention kernels: bf16, vectors of up to 128 components.
#include "sv_kv_shared.cuh"

namespace sv {

extern const SharedKernel shared_kernels_bf16_1[3] = {kv_attend_shared_kernel<32, true, 1>,
                                              kv_attend_shared_kernel<64, true, 1>,
                                              kv_attend_shared_kernel<128, true, 1>};

}  // namespace sv
