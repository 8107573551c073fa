// sv_kv_shared.cuh -- cache attention of rows that hold the same pages for their first tokens
// (sm_103a). The kernel; its instances are in sv_kv_shared_*.cu, the rest in sv_kv_shared.cu.
//
// The softmax of a row splits at any token: with (m, s, o) the largest score, the sum of the
// exponentials and the weighted values of a part, parts join by weights 2^(m - max m). So the
// tokens that a group of rows shares are attended to by all its queries as if they were one row's
// (AT_GROUPS: a key tile is read once for 128 queries of the group instead of once a row), each
// row's other tokens by its own (AT_OWN), and a second kernel joins the two, or more where a query
// tile was cut between CTAs.
//
// Both parts are in one launch: the CTAs are divided between them by their work, counted in key
// tiles of their width. A CTA runs one of the two. Large groups are attended to by a launch behind
// it (sv_kv_group.cu).
//
// Bound as sv_kv_attend is: a query tile's chain of scores, weights and outputs, some 10,000 cycles
// whatever its keys, then 1,600 to 2,600 cycles a key tile. 64 rows of 64 queries on 740 tokens
// without a group take 69 us, sv_kv_attend 61: the counts of what is shared, a launch for large
// groups that ends at once, and the join. 64 chats of one token (8 heads of 8 queries, 60 to 1,500
// tokens of their own behind 8,100 common ones): 52 us for the rows' own tokens, 30 for the common
// ones, 10 for the join, 84 together, since each starts as CTAs of the one before end.
#pragma once
#include "sv_kv_attend.cuh"

namespace sv {

template <int W, bool BF16, int NDB>
__global__ void __launch_bounds__(AT_THREADS, 1)
    kv_attend_shared_kernel(const __grid_constant__ SharedArgs A, const __grid_constant__ AttendPlan P,
                            const __grid_constant__ CUtensorMap tmK,
                            const __grid_constant__ CUtensorMap tmV) {
  extern __shared__ unsigned char dsm_raw[];
  // (Barriers and the like are at the same place for both parts.)
  __shared__ alignas(16) unsigned char raw[sizeof(AtShared<AT_OWN, 128>)];
  __shared__ uint32_t s_groups[AT_LIVE];
  __shared__ int s_sum[AT_THREADS / 32];
  auto& sh = reinterpret_cast<AtShared<AT_OWN, W>&>(raw);
  at_setup(sh);
  kv_enter_ready(A.ready);
  const long long most = (long long)kv_ld(A.H.head + 1) * A.T * A.group;  // queries of the largest group
  const int rows = at_width(most), grid = gridDim.x;
  const AtCount own = at_count<AT_OWN>(A, sh.rows);
  AtCount common = {0, 0};
  if (!at_large(A, most)) common = at_count<AT_GROUPS>(A, s_groups);
  int own_before, before;
  const int own_total = at_block_sum(own.sum, sh.sum, &own_before);
  const int total = at_block_sum(common.sum, s_sum, &before);
  const float a = static_cast<float>(total) * at_cost(rows), b = static_cast<float>(own_total) * at_cost(W);
  const int ctas = total ? max(1, min(grid - 1, __float2int_rn(grid * (a / (a + b))))) : 0;
  const int cta = blockIdx.x;
  __syncthreads();  // (the sums are read; their place is used again)
  if (cta >= ctas)
    at_body<AT_OWN, W, BF16, NDB>(A, P, tmK, tmV, sh, sh.rows, dsm_raw, own, own_total, own_before,
                                  cta - ctas, grid - ctas);
  else if (W == 32 && rows == 32)
    at_body<AT_GROUPS, 32, BF16, NDB>(A, P, tmK, tmV, reinterpret_cast<AtShared<AT_GROUPS, 32>&>(raw),
                                      s_groups, dsm_raw, common, total, before, cta, ctas);
  else if (W == 32 && rows == 64)
    at_body<AT_GROUPS, 64, BF16, NDB>(A, P, tmK, tmV, reinterpret_cast<AtShared<AT_GROUPS, 64>&>(raw),
                                      s_groups, dsm_raw, common, total, before, cta, ctas);
  else
    at_body<AT_GROUPS, 128, BF16, NDB>(A, P, tmK, tmV, reinterpret_cast<AtShared<AT_GROUPS, 128>&>(raw),
                                       s_groups, dsm_raw, common, total, before, cta, ctas);
}

typedef void (*SharedKernel)(const SharedArgs, const AttendPlan, const CUtensorMap, const CUtensorMap);
// Kernels for rows of 32, 64 and 128 queries, by type and width.
extern const SharedKernel shared_kernels_f16_1[3], shared_kernels_f16_2[3], shared_kernels_bf16_1[3],
    shared_kernels_bf16_2[3];

}  // namespace sv
