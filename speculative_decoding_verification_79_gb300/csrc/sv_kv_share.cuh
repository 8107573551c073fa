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
  int4* group;     // [batch / 2] first row in `order`, rows, tokens, the row whose pages are read
  int32_t* order;  // [batch] rows by group
  int32_t* bad;    // [batch] set when a row's pages are no longer those of its group
};
constexpr int KV_SHARE_HEAD = 64;

struct SharedArgs : AttendArgs {
  KvShare H;
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

// The caller's buffer for T tokens of `group` query heads a head: where its parts are (in A, from
// `base` on); returns its bytes.
size_t kv_share_layout(const KvCache& C, int T, int group, unsigned char* base, SharedArgs* A);
cudaError_t launch_kv_share(const KvCache& C, const KvScratch& S, const KvShare& H,
                            const int32_t* group, cudaStream_t st);
cudaError_t launch_kv_attend_shared(SharedArgs& A, sv_dtype dt, cudaStream_t st);

}  // namespace sv
