// sv_kv_shared_bf16_2.cu -- shared-prefix attention kernels: bf16, vectors of up to 256 components.
#include "sv_kv_shared.cuh"

namespace sv {

extern const SharedKernel shared_kernels_bf16_2[3] = {kv_attend_shared_kernel<32, true, 2>,
                                              kv_attend_shared_kernel<64, true, 2>,
                                              kv_attend_shared_kernel<128, true, 2>};

}  // namespace sv
