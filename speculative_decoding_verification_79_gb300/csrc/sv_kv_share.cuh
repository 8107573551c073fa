// sv_kv_share.cuh -- attention of rows that share pages: the caller's buffer and the launches.
#pragma once
#include "sv_kv.cuh"

namespace sv {

// A query tile's partial results are in slots tile + c, for the CTAs c = first .. last.
struct KvSpan {
  int first, last;
};

// What sv_kv_share found, at the start of the caller's buffer (all zeros: no groups). Groups have
// two rows or more; the tokens that a group shares are a multiple of 128.
struct KvShare {
  int32_t* head;   // number of groups, rows of the largest
  int4* row;       // [batch] group (-1: alone), its rows, its tokens, the row's place in it
  int4* group;     // [batch / 2] first row in `order`, rows, tokens, its lowest row
  int32_t* order;  // [batch] rows by group
  int32_t* bad;    // [batch] set when a row's pages are no longer those of its group
  uint32_t* ready; // [KV_MAX_CTAS] see kv_enter_ready; 0 between calls
  int32_t* pages;  // [batch / 2, max_pages] the pages that a group's tokens are in
};
constexpr int KV_SHARE_HEAD = 64;

struct SharedArgs : AttendArgs {
  KvShare H;
  uint32_t* ready;  // H's, when the launch for rows has one for groups behind it
  int tiles;        // query tiles of a row at most
  int large;        // may large groups go to their own kernel?
  int always;       // is every group's common part shared (sv_set_share_always)?
  float row_cost, row_parts;  // (see at_rule)
  int reach;
  int own_rows;     // rows of a slot of partial results of rows
  KvSpan *own_span, *span;  // by query tile: of rows, of groups
  float *own_part, *part;
  float2 *own_stat, *stat;
};

// A launch that starts as CTAs of the one before it end, and reads nothing that that one writes,
// still has to see what earlier ones wrote. Those the one before has waited for, but that it then let
// this one start puts nothing in order. So each of its CTAs, once it has waited, releases a flag, and
// this launch's CTA of the same number takes it by an exchange, an acquire: what the releasing thread
// saw, the taker sees. (A flag of an earlier call is never met: one CTA's exchange took it, and no two
// read the same store.) A CTA that comes before its flag waits for the whole launch, and takes the flag
// then. Both launches have the same grid.
__device__ __forceinline__ void kv_enter_ready(uint32_t* ready) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (ready && threadIdx.x == 0)
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(ready + blockIdx.x), "r"(1u) : "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// (Whoever enters so waits by griddepcontrol.wait before it ends.)
__device__ __forceinline__ void kv_enter_behind(uint32_t* ready) {
  auto take = [&]() {
    uint32_t was = 0;
    if (threadIdx.x == 0)
      asm volatile("atom.exch.acq_rel.gpu.global.b32 %0, [%1], %2;"
                   : "=r"(was)
                   : "l"(ready + blockIdx.x), "r"(0u)
                   : "memory");
    return __syncthreads_or(was != 0) != 0;
  };
  if (!take()) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    take();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The caller's buffer for T tokens of `group` query heads a head: where its parts are (in A, from
// `base` on); returns its bytes.
size_t kv_share_layout(const KvCache& C, int T, int group, unsigned char* base, SharedArgs* A);
cudaError_t launch_kv_share(const KvCache& C, const KvScratch& S, const KvShare& H,
                            const int32_t* group, cudaStream_t st);
cudaError_t launch_kv_attend_shared(SharedArgs& A, sv_dtype dt, cudaStream_t st);

}  // namespace sv
