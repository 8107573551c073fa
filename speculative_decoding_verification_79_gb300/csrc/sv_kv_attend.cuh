// sv_kv_attend.cuh -- the cache attention's CTA: units of work, queries, weights, products and
// partial results, shared by its kernels (sv_kv_attend.cu, sv_kv_shared.cuh). What it computes,
// and what bounds it, is at the top of sv_kv_attend.cu.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <cmath>

#include "sv_device.cuh"
#include "sv_kv_share.cuh"

namespace sv {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // sv_markov.cu

// What a kernel attends with: all rows by themselves (sv_kv_attend); rows behind the tokens that
// they share with a group; or groups of rows over those tokens (sv_kv_attend_shared). "Rows" below
// are groups in the last.
enum AtMode { AT_ROWS, AT_OWN, AT_GROUPS };

constexpr int AT_KEYS = 128;     // tokens per key tile
constexpr int AT_PARTS = 4;      // threads of a query row copy
constexpr int AT_SM_WARPS = 4 * AT_PARTS;  // warps that form the weights
constexpr int AT_SM0 = 128;      // first of their threads, after copies, scores and outputs
constexpr int AT_SM_THREADS = 32 * AT_SM_WARPS;
constexpr int AT_THREADS = AT_SM0 + AT_SM_THREADS;
constexpr int AT_BLK = AT_KEYS * 128;  // 128 tokens x 128 bytes
constexpr int AT_MAX_RING = 8;   // most K tiles, and V tiles, in shared memory
constexpr int AT_INFO = 32;      // key tiles whose page data are kept
constexpr int AT_PTERMS = 3;     // e5m2 terms of a weight
// Warps of sv_kv_group.cu's CTA that form weights, and that convert values.
constexpr int GR_WEIGHTS = 16, GR_CONVERT = 4;
template <bool BF16>
constexpr int AT_QTERMS = BF16 ? 2 : 3;  // terms of a query: e4m3, then e5m2
// Weights are kept as 2^(x - m + 11): up to 2^15 before the reference must move (below
// e5m2's 57344). Their terms end at 2^-16, e5m2's smallest: a weight has its 11 bits down to
// 2^-17 of the reference's, below that a resolution of 2^-27 of it. A larger shift would leave
// less room for later maxima and move references in more tiles.
constexpr float AT_SHIFT = 11.f, AT_LIMIT = 15.f;

// Instruction descriptors of kind::f8f6f4 (float32 accumulator, M = 128), without N.
// Scores: A and B e4m3, K-major (A e5m2 for the later terms). Output: A e5m2 (tensor memory), B
// e4m3, MN-major.
constexpr uint32_t AT_IDESC_S = (1u << 4) | (8u << 24), AT_IDESC_E5M2_A = 1u << 7;
constexpr uint32_t AT_IDESC_O = (1u << 4) | (1u << 7) | (1u << 16) | (8u << 24);

// Descriptors are given as their low words (address and the unused leading offset) with the
// constant high word of the operands' layout. A from shared memory, or from tensor memory.
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t alo, uint32_t blo, uint32_t hi,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %3};\n\t"
      "mov.b64 b, {%2, %3};\n\tsetp.ne.u32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(alo), "r"(blo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t blo, uint32_t hi,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\tsetp.ne.u32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(blo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void tm_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tm_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Sixteen consecutive float32 columns of this thread's lane; complete after tm_wait_ld.
__device__ __forceinline__ void tm_ld16(uint32_t addr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15])
      : "r"(addr));
}
__device__ __forceinline__ void tm_st16(uint32_t addr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
      "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]),
      "f"(v[15])
      : "memory");
}
__device__ __forceinline__ void tm_ld8(uint32_t addr, float* v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                 "=f"(v[6]), "=f"(v[7])
               : "r"(addr));
}
__device__ __forceinline__ void tm_st2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b)
               : "memory");
}
__device__ __forceinline__ void tm_st4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
// The loaded registers are operands of the wait, so that no use of them moves above it.
template <int C>
__device__ __forceinline__ void tm_wait_ld(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < C; ++i) asm volatile("" : "+f"(v[i]));
}
__device__ __forceinline__ void tm_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Shared-memory matrix descriptor of an operand in 128-byte swizzled rows whose groups of
// eight (K-major: rows; MN-major: steps of K) follow each other. One swizzle atom covers the
// other dimension, so the leading offset is not used.
__device__ __forceinline__ uint32_t at_desc_lo(uint32_t addr) {
  return ((addr >> 4) & 0x3fffu) | (1u << 16);
}
constexpr uint32_t AT_HI = (1024 >> 4) | (1u << 14) | (2u << 29);

// One lane of a converged warp.
__device__ __forceinline__ bool at_elect() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void at_tma(void* dst, const CUtensorMap* map, int x, int y,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void fence_async_global() {
  asm volatile("fence.proxy.async.global;" ::: "memory");
}
__device__ __forceinline__ void at_bar(int id, int n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
// Barrier `id` of n threads; true everywhere when x is true anywhere.
__device__ __forceinline__ bool at_vote(int id, int n, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}

// ---------------------------------------------------------------------------
// Units of work.
// ---------------------------------------------------------------------------

// What a launch needs beside AttendArgs.
struct AttendPlan {
  int nk, nv;  // tiles of the rings
  int join;    // floats of the buffer in which row copies are added
};

// Row b of the batch (a group: the tokens it shares, no new ones, the queries of its rows).
struct AtRow {
  int len, n;    // cached and new tokens; n = 0 when the row's data is wrong
  int rows;      // query rows of a head
  int nrt, rr;   // query tiles, rows of each (the last may have fewer)
  int skip;      // first key tiles that are left to the group
  bool bad;
};

// What a call's key tiles cost with tiles of W query rows, in cycles.
__host__ __device__ constexpr int at_cost(int W) { return W == 32 ? 1600 : (W == 64 ? 1800 : 2600); }
__host__ __device__ constexpr int at_width(long long rows) {
  return rows <= 32 ? 32 : (rows <= 64 ? 64 : 128);
}

// Large groups are attended to by a kernel of their own, sv_kv_group.cu, in 2,400 cycles a key tile.
constexpr int AT_LARGE_COST = 2400;
__device__ __forceinline__ bool at_large(const SharedArgs& A, long long rows) {
  return A.large && at_width(rows) == 128;
}
// Key tiles that a group of n rows has in common, or 0 when its rows are better off alone. Sharing
// takes the group's query tiles, and for each row's own query tile results in parts, which are
// written, read and joined: some 3,000 cycles and 80 a query (10 us of 512 query tiles of 36
// queries). Beside that the call is longer by 5 us with a second kind of work in its launch and by
// 14 with another launch: what is gained in all (taking the groups to be alike) has to exceed that
// on 152 SMs. Shared and alone, us, with 8 heads: four rows of 128 queries on 3,000 common tokens
// 226 and 151 (such rows fill their products by themselves); 64 rows of 72 queries on 8,192, by
// twos 327 and 311, by fours 261 and 310; of 36 by 32 on 2,048 79 and 89, on 768 70 and 60; of 8
// by twos on 2,048 76 and 81, on 768 56 and 49; 8 rows of 36 by twos on 8,192 50 and 47.
// A group is priced by its own queries, although all of a call's run as the largest does: by what they
// then take, small ones beside a large one were left alone, one of 16 rows and 24 of two on 2,048 90
// us instead of 81, one and 8 on 8,192 98 instead of 83 (sv_kv_attend 72 and 105). Taking groups to be
// alike shares a large one among many small ones where it alone would not pay: one and 24 on 768
// tokens 56 us, all shared 59, sv_kv_attend 44.
// (The warps that plan ask this for every query tile, in every kernel of the call with the same answer:
// few instructions, each with its rounding said.)
constexpr float AT_KIND = 152 * 10000.f, AT_LAUNCH = 152 * 27000.f;
__device__ __forceinline__ int at_common(const SharedArgs& A, int n, int tokens) {
  const int keys = tokens / AT_KEYS;
  if (A.always) return keys;
  const int seen = min(keys, A.reach), all = n * A.T * A.group;
  const bool large = at_large(A, all);
  const float cost = large ? AT_LARGE_COST : at_cost(at_width(all));
  const float row = __fsub_rn(__fmul_rn(__int2float_rn(seen), A.row_cost), A.row_parts);
  const float alone = __fmul_rn(__int2float_rn(n), row);
  const float once = __fmul_rn(__fmul_rn(__int2float_rn((all + KV_ROWS - 1) / KV_ROWS), cost),
                               __int2float_rn(seen + KV_EXTRA));
  const float gain = __fmul_rn(__fsub_rn(alone, once), __int2float_rn(A.C.heads * kv_ld(A.H.head)));
  return gain > (large ? AT_LAUNCH : AT_KIND) ? keys : 0;
}
// What the rule takes from a call: a row's cost a key tile and for its parts, key tiles that a query
// sees at most (a window leaves out what is between the row's start and it).
inline void at_rule(SharedArgs* A) {
  const int rows = A->T * A->group;
  A->row_cost = static_cast<float>(A->tiles) * static_cast<float>(at_cost(at_width(rows)));
  A->row_parts = 3000.f * static_cast<float>(A->tiles) + 80.f * static_cast<float>(rows);
  const long long span = ((long long)A->window + AT_KEYS - 1) / AT_KEYS +
                         ((long long)A->sinks + AT_KEYS - 1) / AT_KEYS + 1;
  A->reach = A->window && span < 0x7fffffff ? static_cast<int>(span) : 0x7fffffff;
}
__device__ __forceinline__ int at_skip(const AttendArgs&, int) { return 0; }
__device__ __forceinline__ int at_skip(const SharedArgs& A, int b) {
  const int4 x = kv_ld(A.H.row + b);
  return x.x < 0 ? 0 : at_common(A, x.y, x.z);
}

template <AtMode M, typename Args>
__device__ __forceinline__ AtRow at_row(const Args& A, int b) {
  AtRow r;
  if constexpr (M == AT_GROUPS) {
    const int4 x = kv_ld(A.H.group + b);
    const int keys = at_common(A, x.y, x.z);
    r.len = keys * AT_KEYS;
    r.n = 0;
    r.rows = keys ? x.y * A.T * A.group : 0;
    r.nrt = (r.rows + KV_ROWS - 1) / KV_ROWS;
    r.rr = r.nrt ? (r.rows + r.nrt - 1) / r.nrt : 0;
    r.skip = 0;
    r.bad = false;
    return r;
  }
  r.skip = M == AT_OWN ? at_skip(A, b) : 0;
  r.len = kv_ld(A.C.len + b);
  r.n = A.n_new ? kv_ld(A.n_new + b) : A.T;
  r.bad = r.n < 0 || r.n > A.T || r.len < 0 ||
          (long long)r.len + r.n > (long long)A.C.max_pages << A.C.lgp;
  // (A row that was cut below what it shared: its group's tokens are no longer its own.)
  if (M == AT_OWN) r.bad = r.bad || r.len < r.skip * AT_KEYS;
  if (r.bad) r.n = 0;
  r.rows = r.n * A.group;
  r.nrt = (r.rows + KV_ROWS - 1) / KV_ROWS;
  r.rr = r.nrt ? (r.rows + r.nrt - 1) / r.nrt : 0;
  return r;
}

// The page of a row's token at `key` (of a group: one of those that it shares), -1 when out of range.
template <AtMode M, typename Args>
__device__ __forceinline__ int at_page(const Args& A, int b, int key) {
  if constexpr (M == AT_GROUPS) {
    const int p = kv_ld(A.H.pages + (size_t)b * A.C.max_pages + (key >> A.C.lgp));
    return p >= 0 && p < A.C.pages ? p : -1;
  }
  return kv_page(A.C, b, key);
}

// Query tile rt of a row: rows r0 .. r1 - 1, and the key tiles that any of them sees:
// `ns` from `s0` on near the row's start (sinks), then `lo` to `hi` - 1.
struct AtTile {
  int r0, r1;
  int end;            // keys below end are visible to some query
  int pos_lo, pos_hi; // bounds of the queries' positions
  int s0, ns, lo, hi;
  __device__ __forceinline__ int tiles() const { return ns + hi - lo; }
  __device__ __forceinline__ int key_tile(int i) const { return i < ns ? s0 + i : lo + i - ns; }
};

template <AtMode M, typename Args>
__device__ __forceinline__ AtTile at_tile(const Args& A, const AtRow& r, int b, int rt) {
  AtTile t;
  t.r0 = rt * r.rr;
  t.r1 = min(t.r0 + r.rr, r.rows);
  t.s0 = 0;
  if constexpr (M == AT_GROUPS) {  // every query sees these keys, as far as its window reaches
    t.pos_lo = t.pos_hi = t.end = r.len;
    t.hi = r.len / AT_KEYS;
    t.lo = t.ns = 0;
    if (A.window) {
      const int first = kv_ld(A.H.group + b).x, per = A.T * A.group;
      int lo = 0x7fffffff, hi = 0;
      for (int m = t.r0 / per; m <= (t.r1 - 1) / per; ++m) {
        const int len = max(kv_ld(A.C.len + kv_ld(A.H.order + first + m)), r.len);
        lo = min(lo, len);
        hi = max(hi, len);
      }
      t.pos_lo = lo;
      t.pos_hi = min(hi, 0x7ffffeff - A.T) + A.T - 1;
      t.lo = min(max(0, lo - A.window + 1) / AT_KEYS, t.hi);
      t.ns = min((min(A.sinks, r.len) + AT_KEYS - 1) / AT_KEYS, t.lo);
    }
    return t;
  }
  // (One query tile holds all tokens: no division.)
  const int t0 = rt ? t.r0 / A.group : 0, t1 = r.nrt == 1 ? r.n - 1 : (t.r1 - 1) / A.group;
  t.pos_lo = A.parent ? r.len : r.len + t0;
  t.pos_hi = A.parent ? r.len + r.n - 1 : r.len + t1;
  t.end = t.pos_hi + 1;
  t.hi = (t.end + AT_KEYS - 1) / AT_KEYS;  // (positions end 256 below 2^31)
  t.lo = 0;
  t.ns = 0;
  if (A.window) {
    t.lo = max(0, t.pos_lo - A.window + 1) / AT_KEYS;
    t.ns = min((min(A.sinks, t.end) + AT_KEYS - 1) / AT_KEYS, t.lo);
  }
  if (M == AT_OWN) {
    t.s0 = min(r.skip, t.ns);
    t.ns -= t.s0;
    t.lo = max(t.lo, r.skip);
  }
  return t;
}

// Query row i of row b's head: row of the batch, token, head of the group.
struct AtQuery {
  int b, t, gh;
};
template <AtMode M, typename Args>
__device__ __forceinline__ AtQuery at_query(const Args& A, int b, int i) {
  AtQuery q;
  q.b = b;
  if constexpr (M == AT_GROUPS) {
    const int per = A.T * A.group, m = i / per;
    q.b = kv_ld(A.H.order + kv_ld(A.H.group + b).x + m);
    i -= m * per;
  }
  q.t = i / A.group;
  q.gh = i - q.t * A.group;
  return q;
}

// Number of a query tile. A group's first is no less than the tiles of the groups before, each of
// which has at most one that is not full, and more than the first of the group before.
__device__ __forceinline__ int at_group_base(const SharedArgs& A, int g) {
  return static_cast<int>((long long)kv_ld(A.H.group + g).x * A.T * A.group / KV_ROWS) + g;
}
__device__ __forceinline__ int at_tile_no(const AttendArgs&, AtMode, int, int, int) { return 0; }
__device__ __forceinline__ int at_tile_no(const SharedArgs& A, AtMode m, int b, int rt, int h) {
  const int base = m == AT_OWN ? b * A.tiles : at_group_base(A, b);
  return (base + rt) * A.C.heads + h;
}

// Work is counted in key tiles, with KV_EXTRA more for each query tile: what its queries'
// conversion and its results cost. Its order is rows, query tiles, heads.

// Units of a query tile for one head, which may have no key that a group's window reaches, and of
// row b's query tile rt (0: none).
template <AtMode M>
__device__ __forceinline__ int at_units(const AtTile& t) {
  const int n = t.tiles();
  return M == AT_GROUPS && n == 0 ? 0 : KV_EXTRA + n;
}
template <AtMode M, typename Args>
__device__ __forceinline__ int at_units(const Args& A, int b, int rt) {
  const AtRow r = at_row<M>(A, b);
  return rt < r.nrt ? at_units<M>(at_tile<M>(A, r, b, rt)) : 0;
}
// Rows of the batch, or groups.
template <AtMode M, typename Args>
__device__ __forceinline__ int at_rows(const Args& A) {
  if constexpr (M == AT_GROUPS) return kv_ld(A.H.head);
  return A.C.batch;
}
// Query tiles of the largest row or group.
template <AtMode M, typename Args>
__device__ __forceinline__ int at_most_tiles(const Args& A) {
  long long rows = (long long)A.T * A.group;
  if constexpr (M == AT_GROUPS) rows *= kv_ld(A.H.head + 1);
  return static_cast<int>((rows + KV_ROWS - 1) / KV_ROWS);
}

// The first row after b that has queries (one exists), from a bit for each. A whole warp, a lane
// a word: an idle batch has thousands of rows without any, and looking their counts up one
// after the other took a call of 31 us to 950 (two rows of 20,000 tokens at the ends of 4,096).
constexpr int AT_LIVE = (SV_MAX_B + 31) / 32;
__device__ __forceinline__ int at_next_row(const uint32_t* rows, int batch, int b) {
  const int lane = threadIdx.x & 31, words = (batch + 31) / 32;
  for (int w0 = (b + 1) / 32; w0 < words; w0 += 32) {
    const int w = w0 + lane;
    uint32_t x = w < words ? rows[w] : 0;
    if (w == (b + 1) / 32) x &= ~0u << ((b + 1) % 32);
    const uint32_t found = __ballot_sync(0xffffffffu, x != 0);
    if (found) {
      const int first = __ffs(found) - 1;
      return (w0 + first) * 32 + __ffs(__shfl_sync(0xffffffffu, x, first)) - 1;
    }
  }
  return batch - 1;
}

// The units of this CTA, one query tile after the other: key tiles i0 .. i1 - 1 of the
// current one. Every role walks the same sequence.
template <AtMode M>
struct AtWalk {
  int b, h, rt;
  AtRow row;
  AtTile tile;
  int i0, i1;
  int base, at, end;  // first unit of the query tile, of the share in it, share's end

  // The share of the current query tile; false when it has no key tile.
  __device__ __forceinline__ bool settle() {
    const int stop = min(end, base + KV_EXTRA + tile.tiles());
    i0 = max(0, at - base - KV_EXTRA);
    i1 = max(0, stop - base - KV_EXTRA);
    return i1 > i0;
  }
  // From unit `rem` of query tile rt0 of row b0 (all heads). One thread does this for all; the
  // first query tile may have no key tile in the share (see first).
  template <typename Args>
  __device__ __forceinline__ void start(const Args& A, int b0, int rt0, int rem, int from, int to) {
    at = from;
    end = to;
    b = b0;
    rt = rt0;
    row = at_row<M>(A, b);
    tile = at_tile<M>(A, row, b, rt);
    const int per = at_units<M>(tile);
    h = rem / per;
    base = from - (rem - h * per);
    settle();
  }
  // For the warps that walk, before the first query tile.
  template <typename Args>
  __device__ __forceinline__ void first(const Args& A, const uint32_t* rows) {
    if (live() && i1 <= i0) next(A, rows);
  }
  __device__ __forceinline__ bool live() const { return at < end; }
  // A whole warp; `rows` has a bit for each row that has queries.
  template <typename Args>
  __device__ __noinline__ void next(const Args& A, const uint32_t* rows) {
    do {
      base += at_units<M>(tile);
      at = base;
      if (at >= end) return;
      if (++h == A.C.heads) {
        h = 0;
        if (++rt == row.nrt) {
          rt = 0;
          b = at_next_row(rows, at_rows<M>(A), b);  // (it exists: units are left)
          row = at_row<M>(A, b);
        }
        tile = at_tile<M>(A, row, b, rt);
      }
    } while (!settle());
  }
};

// Share c of n equal parts of `total` units begins at at_share(c); at_owner is the share that
// holds unit u.
__device__ __forceinline__ int at_share(int c, int total, int n) {
  const int per = total / n;
  return c * per + min(c, total - per * n);
}
__device__ __forceinline__ int at_owner(int u, int total, int n) {
  const int per = total / n, big = total - per * n;  // the first `big` shares have one more
  return u < big * (per + 1) ? u / (per + 1) : big + (u - big * (per + 1)) / per;
}

// A query tile's share as the product and weight warps read it from shared memory.
struct AtItem {
  int b, h, len, n;
  int r0, R;        // query rows r0 .. r0 + R - 1 of the head
  int i0, m;        // key tiles i0 .. i0 + m - 1 (m = 0: no more work)
  int tiles;        // of the query tile
  int end, pos_lo, pos_hi;  // as AtTile
  int s0, ns, lo;
  int bad;          // the row's tree is wrong
  int u0;           // unit of its first key tile
  int no;           // number of the query tile
  int part;         // its result is one of several, whichever keys this CTA saw
  __device__ __forceinline__ int key_tile(int i) const { return i < ns ? s0 + i : lo + i - ns; }
  // A tile is cut (some query does not see all of it) when its first key is cut_hi or above,
  // and when it has a key below cut_lo that is not a sink.
  __device__ __forceinline__ int cut_hi() const { return pos_lo - AT_KEYS + 2; }
  __device__ __forceinline__ int cut_lo(int window) const { return window ? pos_hi - window + 1 : 0; }
};

// The lowest n bits (none below 1, all from 32 on).
__device__ __forceinline__ uint32_t at_below(int n) {
  return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u);
}

// Two and four consecutive values, rounded to the output's type.
__device__ __forceinline__ uint32_t at_pack(float a, float b, int bf16) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  const __half2 y = __floats2half2_rn(a, b);
  return bf16 ? *reinterpret_cast<const uint32_t*>(&x) : *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ void at_store4(void* out, long long at, float4 y, int bf16) {
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) =
      make_uint2(at_pack(y.x, y.y, bf16), at_pack(y.z, y.w, bf16));
}

// Partial results: where (in vectors of four floats) components c .. c + 3 of row r are in
// slot `id` of `rows` rows. Rows are next to each other: their threads store, and the join reads,
// whole sectors. (Rows one after the other made the stores of 128 x 256 floats 9,000 cycles.)
__device__ __forceinline__ size_t at_part(int id, int r, int c, int dim, int rows = KV_ROWS) {
  return ((size_t)id * (dim / 4) + c / 4) * rows + r;
}

// log2 of a positive normal number (or NaN): its exponent, and the hardware's logarithm of the
// rest, which is good to 2^-22 there.
__device__ __forceinline__ float at_log2(float x) {
  const uint32_t u = __float_as_uint(x);
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(__uint_as_float((u & 0x7fffffu) | 0x3f800000u)));
  return x == x ? static_cast<float>(static_cast<int>(u >> 23) - 127) + y : x;
}

// Have `limit` cycles passed since the first call with *t0 == 0?
__device__ __forceinline__ bool at_expired(long long* t0, long long limit) {
  const long long t = clock64();
  if (*t0 == 0) *t0 = t;
  return t - *t0 > limit;
}

// The rest of a wait whose first probe (which suspends the thread for some microseconds at
// most) was in vain. Bounded: false (and a report) when it runs out or another one has. Not
// expanded at every wait: the kernel's loops share the instruction cache.
static __device__ __noinline__ bool at_wait_on(uint64_t* bar, uint32_t parity, volatile int* abort,
                                        const AttendArgs& A) {
  long long t0 = 0;
  while (!mbar_try(bar, parity)) {
    if (*abort) return false;
    if (at_expired(&t0, A.wait_limit)) {
      *abort = 1;
      kv_report(A.S.hdr, ST_TIMEOUT);
      return false;
    }
  }
  return true;
}

// After a wait gave up, products already issued must end before the accumulators are freed.
__device__ __forceinline__ void at_drain(uint64_t* bar, bool abort) {
  if (!abort) return;
  umma_commit(bar);
  const long long t0 = clock64();
  while (!mbar_test(bar, 0))
    if (clock64() - t0 > WAIT_CYCLES / 8) break;
}

// The queries of an item: half a warp takes a row, a lane eight components (sixteen above
// dim 128). at_fetch copies them, as they are, to where the lane's own terms will be, so
// that all rows are on their way at once; at_convert makes the terms: 8-bit in the layout of
// a K-major operand, in each of the row's copies (W rows apart). The factor of a row's
// scores is the power of two that its terms were divided by, times the call's scale; NaN
// when a component is infinite, which the saturating terms would not show. (Rows past the
// item's keep what they held: each row's results are its own.) Not expanded in place: once
// per query tile, and the kernel's loops share the instruction cache.
__device__ __forceinline__ uint32_t at_raw(int db, int row, int l16) {
  // The 16 bytes go to chunk l16 & 7 of the row in block 0 (l16 < 8) or 1 of the terms'
  // blocks; above dim 128 the second half of the row to blocks 2 and 3.
  return (2 * db + (l16 >> 3)) * AT_BLK + row * 128 + (l16 & 7) * 16;
}
template <AtMode M, typename Args>
__device__ __noinline__ void at_fetch(const Args& A, int ndb, const AtItem* it, unsigned char* Q) {
  const int hw = (threadIdx.x - AT_SM0) >> 4, l16 = threadIdx.x & 15;
#pragma unroll 1
  for (int row = hw; row < it->R; row += 2 * AT_SM_WARPS) {
    const AtQuery q = at_query<M>(A, it->b, it->r0 + row);
    const uint16_t* src = static_cast<const uint16_t*>(A.q) + q.b * A.q_row + q.t * A.q_tok +
                          (size_t)(it->h * A.group + q.gh) * A.C.dim;
    for (int db = 0; db < ndb; ++db) {
      const int d = db * 128 + l16 * 8;
      if (d < A.C.dim)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                         smem_addr(Q + at_raw(db, row, l16))),
                     "l"(src + d)
                     : "memory");
    }
  }
}
template <int W, bool BF16, int NDB>
__device__ __noinline__ void at_convert(const AttendArgs& A, const AtItem* it,
                                        unsigned char* Q, float* cs) {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  const int hw = (threadIdx.x - AT_SM0) >> 4, l16 = threadIdx.x & 15;
  const uint32_t half = 0xffffu << (threadIdx.x & 16);  // (the other half may have no row)
#pragma unroll 1
  for (int row = hw; row < it->R; row += 2 * AT_SM_WARPS) {
    float f[NDB][8];
    float a = 0.f;
#pragma unroll
    for (int db = 0; db < NDB; ++db) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (db * 128 + l16 * 8 < A.C.dim)
        x = *reinterpret_cast<const uint4*>(Q + at_raw(db, row, l16));
      const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&xw[e]));
        f[db][2 * e] = BF16 ? bf_lo(xw[e]) : y.x;
        f[db][2 * e + 1] = BF16 ? bf_hi(xw[e]) : y.y;
        a = fmaxf(a, fmaxf(fabsf(f[db][2 * e]), fabsf(f[db][2 * e + 1])));
      }
    }
    __syncwarp(half);  // the row is in registers: its place is free
#pragma unroll
    for (int s = 8; s; s >>= 1) a = fmaxf(a, __shfl_xor_sync(half, a, s));
    const float sc = kv_scale(a);
    const float inv = __uint_as_float((254u << 23) - __float_as_uint(sc));
#pragma unroll
    for (int db = 0; db < NDB; ++db) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = f[db][e] * inv;
      unsigned char* dst =
          Q + (size_t)db * AT_BLK + row * 128 + (((l16 >> 1) ^ (row & 7)) << 4) + (l16 & 1) * 8;
#pragma unroll
      for (int t = 0; t < AT_QTERMS<BF16>; ++t) {
        uint2 o;
        o.x = t ? e5m2x4(y[0], y[1], y[2], y[3]) : e4m3x4(y[0], y[1], y[2], y[3]);
        o.y = t ? e5m2x4(y[4], y[5], y[6], y[7]) : e4m3x4(y[4], y[5], y[6], y[7]);
#pragma unroll
        for (int c = 0; c < 128 / W; ++c)
          *reinterpret_cast<uint2*>(dst + (size_t)t * NDB * AT_BLK + c * W * 128) = o;
        const uint32_t ow[2] = {o.x, o.y};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 lo = t ? e5m2_to_f2(ow[e] & 0xffffu) : e4m3_to_f2(ow[e] & 0xffffu);
          const float2 hi = t ? e5m2_to_f2(ow[e] >> 16) : e4m3_to_f2(ow[e] >> 16);
          y[4 * e] -= lo.x;
          y[4 * e + 1] -= lo.y;
          y[4 * e + 2] -= hi.x;
          y[4 * e + 3] -= hi.y;
        }
      }
    }
    if (l16 == 0) cs[row] = it->bad || a == INFINITY ? NAN : sc * A.scale;
  }
  __syncwarp();
  fence_async();
}

// Bytes of x that are NaN (e4m3), as their upper bits.
__device__ __forceinline__ uint32_t at_nan4(uint32_t x) {
  return ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// The values of a cut tile, before they are multiplied: what weight 0 would not hide. Tokens
// from `end` on (whatever the page holds) are zeroed; a NaN is zeroed where it stands, and
// its token's bit set in `nans`: it becomes the weight of the queries that see it. One warp,
// eight lanes a token, 32 tokens at a time. (All weight warps stopping for it held up a cut
// tile by 4,000 cycles.)
static __device__ __noinline__ void at_check(unsigned char* v, int ndb, int end, uint32_t* nans) {
  const int lane = threadIdx.x & 31;
  if (lane < AT_KEYS / 32) nans[lane] = 0;
  __syncwarp();
#pragma unroll 1
  for (int blk = 0; blk < ndb * (AT_KEYS / 32); ++blk) {
    const int t0 = blk % (AT_KEYS / 32) * 32;
    uint4* p = reinterpret_cast<uint4*>(v + blk * 32 * 128) + lane;  // (tokens t0 + 4 u + lane / 8)
    if (t0 < end) {
      uint4 y[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) y[u] = p[32 * u];
      uint32_t nan = 0;
#pragma unroll
      for (int u = 0; u < 8; ++u)
        nan |= at_nan4(y[u].x) | at_nan4(y[u].y) | at_nan4(y[u].z) | at_nan4(y[u].w);
      if (__any_sync(0xffffffffu, nan != 0)) {
#pragma unroll 1
        for (int u = 0; u < 8; ++u) {
          uint4 x = p[32 * u];
          uint32_t* w = reinterpret_cast<uint32_t*>(&x);
          uint32_t has = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t m = at_nan4(w[i]);
            has |= m;
            w[i] &= ~((m >> 7) * 0xffu);
          }
          const int tok = t0 + 4 * u + (lane >> 3);
          if (!has || tok >= end) continue;
          p[32 * u] = x;
          atomicOr(&nans[tok / 32], 1u << (tok % 32));
        }
      }
    }
    if (t0 + 32 > end) {
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (t0 + 4 * u + (lane >> 3) >= end) p[32 * u] = make_uint4(0, 0, 0, 0);
    }
  }
  fence_async();
  __syncwarp();
}

// Waits for the copies of the last tiles 0 .. g - 1 of a ring of n.
static __device__ __noinline__ void at_land(uint64_t* full, int n, int g) {
  const long long t0 = clock64();
  for (int j = max(0, g - n); j < g; ++j)
    while (!mbar_test(&full[j % n], (j / n) & 1) && clock64() - t0 < WAIT_CYCLES / 4) {
    }
}

// The state of a CTA in shared memory.
template <AtMode M>
struct AtCommon {
  uint64_t kfull[AT_MAX_RING], kempty[AT_MAX_RING];
  uint64_t vfull[AT_MAX_RING], vempty[AT_MAX_RING], tinfo[AT_INFO];
  uint64_t sfull[3], pfull[3], pvdone[3], vchk[AT_MAX_RING], qfull, dfull[2], dempty[2], drain[2];
  uint64_t wfull[2], wempty[2], hfull[3];  // of sv_kv_group.cu: values in 16 bits, weights
  uint32_t tmem;
  int abort;
  AtWalk<M> walk;
  int total, sum[32];  // (of up to 32 warps)
  uint32_t rows[AT_LIVE];  // rows that have queries, a bit each
  // Per key tile and page of it: row of the pool (-1: none); key scale, log2 and inverse of
  // the value scale.
  int y[AT_INFO][8];
  float4 sc[AT_INFO][8];
  AtItem item[2];  // item k's description, at k & 1
};
template <AtMode M, int W>
struct AtShared : AtCommon<M> {
  // Item k's rows, at k & 1: factor of the score, position of the query, block nodes it sees
  // (trees), its row of the output.
  float c[2][W];
  int pos[2][W];
  unsigned long long see[2][W];
  long long out[2][W];
  int par[SV_MAX_TREE], tpos[SV_MAX_TREE];  // a tree: parents, positions
  unsigned long long tsee[SV_MAX_TREE];     // and what a node sees
  float top[AT_PARTS][128], l[AT_PARTS][128];  // largest scores, sums
  float2 stat[128];     // reference and sum of a row copy
  // Tokens of a cut tile with a NaN value, an entry per cut tile (no more of them than tiles
  // in V's ring are checked and not yet multiplied).
  uint32_t vnan[AT_MAX_RING][AT_KEYS / 32];
};

// Barriers and tensor memory, before anything of the call is read.
template <int WARPS = AT_SM_WARPS, typename Shared>
__device__ __forceinline__ void at_setup(Shared& sh) {
  const int tid = threadIdx.x;
  if (tid < AT_INFO) {
    mbar_init(&sh.tinfo[tid], 1);
    if (tid < AT_MAX_RING) {
      mbar_init(&sh.kfull[tid], 2);
      mbar_init(&sh.kempty[tid], 1);
      mbar_init(&sh.vfull[tid], 1);
      mbar_init(&sh.vempty[tid], 1);
      mbar_init(&sh.vchk[tid], 1);
    }
    if (tid < 3) {
      mbar_init(&sh.sfull[tid], 2);
      mbar_init(&sh.pfull[tid], AT_SM_WARPS);
      mbar_init(&sh.pvdone[tid], 1);
      mbar_init(&sh.hfull[tid], GR_WEIGHTS);
    }
    if (tid < 2) {
      mbar_init(&sh.dfull[tid], 1);
      mbar_init(&sh.dempty[tid], WARPS);
      mbar_init(&sh.drain[tid], 1);
      mbar_init(&sh.wfull[tid], GR_CONVERT);
      mbar_init(&sh.wempty[tid], 1);
    }
    if (tid == 0) {
      mbar_init(&sh.qfull, WARPS);
      *const_cast<volatile int*>(&sh.abort) = 0;
    }
    fence_mbar_init();
  }
  if (tid / 32 == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&sh.tmem)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}

// Sum of x over the CTA's threads; *before: of lower threads.
template <int THREADS = AT_THREADS>
__device__ __forceinline__ int at_block_sum(int x, int* sums, int* before) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int v = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += t;
  }
  static_assert(THREADS <= 1024, "an entry a warp");
  if (lane == 31) sums[w] = v;
  __syncthreads();
  int all = 0, pre = 0;
  for (int i = 0; i < THREADS / 32; ++i) {
    if (i < w) pre += sums[i];
    all += sums[i];
  }
  *before = pre + v - x;
  return all;
}

// The units of all rows' query tiles, counted by the threads in turn (all heads'): this thread's
// first and its sum; and a bit for each row that has queries.
struct AtCount {
  int mine, sum;
};
// Query tiles are looked at in a list: `nrt` entries for each row, as many as a row may have. Groups
// may be of very different sizes (one of 2,048 rows beside 1,024 of two would make 2^31 entries and
// more): beyond AT_LISTED entries theirs are by number, and an entry's group is looked for. (One
// token of such rows with 8 queries a head: 260 us instead of 522. By number always: a trip to memory
// or two more, 84.6 us instead of 83.7 for 64 chats behind one prompt, a round of eight groups 275.4
// instead of 272.2.)
constexpr int AT_LISTED = 2048;
static_assert(SV_MAX_B / 2 <= AT_LISTED, "groups of one query tile each are always listed");
struct AtPair {
  int b, rt;
};
template <AtMode M, typename Args>
__device__ __forceinline__ int at_pairs(const Args& A, int nrt) {
  const int n = at_rows<M>(A);
  if constexpr (M == AT_GROUPS)
    if ((long long)n * nrt > AT_LISTED) {  // (no less than any number; see at_group_base)
      const long long rows = (long long)kv_ld(A.H.head + 2) * A.T * A.group;
      return max(static_cast<int>(rows / KV_ROWS) + n, AT_LISTED + 1);
    }
  return n * nrt;
}
// (Not expanded in place: a launch's start waits for its code, which comes from memory.)
static __device__ __noinline__ AtPair at_pair_of(const SharedArgs& A, int p) {
  int b = 0;
  for (int end = kv_ld(A.H.head); end - b > 1;) {
    const int mid = (b + end) / 2;
    (at_group_base(A, mid) <= p ? b : end) = mid;
  }
  return AtPair{b, p - at_group_base(A, b)};
}
template <AtMode M, typename Args>
__device__ __forceinline__ AtPair at_pair(const Args& A, int p, int nrt, int pairs) {
  if constexpr (M == AT_GROUPS)
    if (__builtin_expect(pairs > AT_LISTED, 0)) return at_pair_of(A, p);
  const int b = p / nrt;
  return AtPair{b, p - b * nrt};
}
template <AtMode M, typename Args>
__device__ __forceinline__ int at_units_of(const Args& A, int p, int nrt, int pairs) {
  if (p >= pairs) return 0;
  if constexpr (M == AT_GROUPS) {
    const AtPair x = at_pair<M>(A, p, nrt, pairs);
    return at_units<M>(A, x.b, x.rt) * A.C.heads;
  }
  const int b = nrt == 1 ? p : p / nrt;
  return at_units<M>(A, b, p - b * nrt) * A.C.heads;
}
template <AtMode M, int THREADS = AT_THREADS, typename Args>
__device__ __forceinline__ AtCount at_count(const Args& A, uint32_t* rows) {
  const int tid = threadIdx.x, lane = tid & 31, nrt = at_most_tiles<M>(A), n = at_rows<M>(A);
  const int pairs = at_pairs<M>(A, nrt);
  AtCount a = {0, 0};
#pragma unroll 1
  for (int p = tid; p - lane < pairs; p += THREADS) {
    const int c = at_units_of<M>(A, p, nrt, pairs);
    if (p == tid) a.mine = c;
    a.sum += c;
    if (nrt == 1) {  // (p is the row)
      const uint32_t has = __ballot_sync(0xffffffffu, c != 0);
      if (lane == 0) rows[p / 32] = has;
    }
  }
  if (nrt > 1)
#pragma unroll 1
    for (int b = tid; b - lane < n; b += THREADS) {
      const uint32_t has = __ballot_sync(0xffffffffu, b < n && at_row<M>(A, b).rows > 0);
      if (lane == 0) rows[b / 32] = has;
    }
  return a;
}

// Do the rows of a group still hold its pages? Each weight warp of the grid looks at some of them,
// 256 pages of a row at a time; a row that does not becomes NaN when its parts are joined.
static __device__ __noinline__ void at_check_groups(const SharedArgs& A, int warp) {
  const KvCache& C = A.C;
  const int lane = threadIdx.x & 31, chunks = (C.max_pages + 255) / 256, step = gridDim.x * AT_SM_WARPS;
  for (int u = warp * gridDim.x + blockIdx.x; u < C.batch * chunks; u += step) {
    const int b = u / chunks, from = (u - b * chunks) * 256;
    const int4 x = kv_ld(A.H.row + b);
    const int pages = x.x < 0 ? 0 : at_common(A, x.y, x.z) << (7 - C.lgp);
    if (from >= pages) continue;
    const int32_t *mine = C.table + (size_t)b * C.max_pages, *its = A.H.pages + (size_t)x.x * C.max_pages;
    bool bad = pages > kv_ld(C.np + b) || pages > C.max_pages || pages << C.lgp > kv_ld(C.len + b);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int j = from + 32 * k + lane;
      if (j < min(pages, C.max_pages)) bad = bad || kv_ld(mine + j) != kv_ld(its + j);
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) {
      A.H.bad[b] = 1;
      kv_report(A.S.hdr, ST_DEVICE_INPUT);
    }
  }
}

// This CTA's share: the units of all rows' query tiles, cut into equal parts. The second pass over
// them finds the one where the share begins. The CTA's warps go on together.
template <AtMode M, int THREADS = AT_THREADS, typename Args, typename Shared>
__device__ __forceinline__ void at_begin(const Args& A, Shared& sh, AtCount count, int total, int before,
                                         int cta, int most_ctas) {
  const int tid = threadIdx.x;
  const int nrt = at_most_tiles<M>(A), pairs = at_pairs<M>(A, nrt);
  const int ctas = min(most_ctas, total);
  const int from = cta < ctas ? at_share(cta, total, ctas) : 0;
  const int to = cta < ctas ? at_share(cta + 1, total, ctas) : 0;
  if (tid == 0) {
    sh.total = total;
    if (from >= to) sh.walk.at = sh.walk.end = 0;
  }
  if (from < to) {
    int base = 0;
#pragma unroll 1
    for (int p0 = 0;; p0 += THREADS) {
      const int c = p0 == 0 ? count.mine : at_units_of<M>(A, p0 + tid, nrt, pairs);
      int all = total;
      if (pairs > THREADS) {  // (otherwise `before` is right already)
        __syncthreads();
        all = at_block_sum<THREADS>(c, sh.sum, &before);
      }
      if (from >= base + before && from < base + before + c) {
        // (One thread for all: its row's data and this code are at hand, which saves the
        // copies 3,000 cycles before their first page.)
        const AtPair x = at_pair<M>(A, p0 + tid, nrt, pairs);
        AtWalk<M> walk;
        walk.start(A, x.b, x.rt, from - base - before, from, to);
        sh.walk = walk;
      }
      base += all;
      if (base > from) break;
    }
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
}

__device__ __forceinline__ void at_prefetch(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}

// The warp that copies K tiles into their ring (of nk); returns how many it has issued. With tmV the
// pages of the chunk ahead, of K and V, are brought to L2 meanwhile.
template <AtMode M, int NDB, typename Args, typename Shared>
__device__ __forceinline__ int at_copy_keys(const Args& A, int nk, const CUtensorMap& tmK, Shared& sh,
                                            const uint32_t* s_rows, unsigned char* Ks,
                                            const CUtensorMap* tmV = nullptr) {
  constexpr int ndb = NDB, slot = ndb * AT_BLK;
  const KvCache& C = A.C;
  const int lane = threadIdx.x & 31;
  auto &kfull = sh.kfull, &kempty = sh.kempty;
  auto& tinfo = sh.tinfo;
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return mbar_try(bar, parity) || at_wait_on(bar, parity, const_cast<volatile int*>(&sh.abort), A);
  };
  // Pages are looked up for several tiles at a time, a page per lane and a
  // chunk ahead of their use; their data go to the other warps through a ring of entries,
  // one per tile, written before the tile's barrier is armed. (An entry is used again 32
  // tiles later, and K is never more than its ring and three steps ahead of the rest.)
  fence_async_global();  // (what earlier kernels stored, before copies read it)
  AtWalk<M> walk = sh.walk;
  walk.first(A, s_rows);
  const int ppt = AT_KEYS >> C.lgp;             // pages per tile
  const int tpc = min(32 / ppt, AT_INFO / 4);   // tiles per chunk
  const int mt = lane / ppt, sub = lane - mt * ppt;
  const size_t layer0 = (size_t)A.layer * C.pages;
  int n = 0, h = 0, page = -1;  // the chunk ahead: tiles, head, this lane's page
  bool used = false;
  int i = walk.live() ? walk.i0 : 0;
  auto look = [&]() {
    n = 0;
    if (!walk.live()) return;
    h = walk.h;
    n = min(tpc, walk.i1 - i);
    const int key = (mt < n ? walk.tile.key_tile(i + mt) : 0) * AT_KEYS + (sub << C.lgp);
    used = mt < n && key < walk.tile.end;
    page = used ? at_page<M>(A, walk.b, key) : -1;
    if (tmV && page >= 0)
      for (int db = 0; db < ndb; ++db) {
        at_prefetch(&tmK, db * 128, (page * C.heads + h) << C.lgp);
        at_prefetch(tmV, db * 128, (page * C.heads + h) << C.lgp);
      }
    i += n;
    if (i == walk.i1) {
      walk.next(A, s_rows);
      i = walk.live() ? walk.i0 : 0;
    }
  };
  int g = 0, q = 0, ph = 0;
  bool ok = true;
  look();
  while (ok && n) {
    const int count = n, head = h;
    const bool use = used;
    const int pg = page, y = pg >= 0 ? (pg * C.heads + head) << C.lgp : -1;
    const uint32_t held = __ballot_sync(0xffffffffu, y >= 0);
    for (int t = 0; t < count; ++t) {
      if (ph > 0 && !__all_sync(0xffffffffu, wait(&kempty[q], (ph - 1) & 1))) {
        ok = false;
        break;
      }
      if (lane == 0) {
        const uint32_t pages = __popc((held >> (t * ppt)) & ((1u << ppt) - 1u));
        mbar_arrive_expect_tx(&kfull[q], (pages << C.lgp) * 128u * ndb);
      }
      __syncwarp();
      if (mt == t && y >= 0) {
        unsigned char* dst = Ks + (size_t)q * slot + ((size_t)sub << C.lgp) * 128;
        for (int db = 0; db < ndb; ++db) at_tma(dst + db * AT_BLK, &tmK, db * 128, y, &kfull[q]);
      }
      if (t == 0) {  // the chunk's data, while its first tile is on its way
        float ks = 1.f, vs = 1.f;
        if (use) {
          if (pg >= 0) {
            ks = kv_ld(C.ks + (layer0 + pg) * C.heads + head);
            vs = kv_ld(C.vs + (layer0 + pg) * C.heads + head);
          }
          // A page out of range, or scales outside theirs: the scores become NaN.
          constexpr float LO = 5.421010862427522e-20f, HI = 18446744073709551616.f;  // 2^-64, 2^64
          if (pg < 0 || !(ks >= LO && ks <= HI && vs >= LO && vs <= HI)) {
            ks = NAN;
            vs = 1.f;
            kv_report(A.S.hdr, ST_DEVICE_INPUT);
          }
        }
        if (mt < count) {
          const int e = (g + mt) & (AT_INFO - 1);
          sh.y[e][sub] = y;
          sh.sc[e][sub] = make_float4(ks, log2f(vs), 1.f / vs, 0.f);
        }
        __syncwarp();
      }
      if (lane == 0) {  // (the second of kfull's arrivals: the tile's data are there)
        mbar_arrive(&kfull[q]);
        mbar_arrive(&tinfo[g & (AT_INFO - 1)]);
      }
      ++g;
      if (++q == nk) {
        q = 0;
        ++ph;
      }
      if (t == 0) look();
    }
  }
  return g;
}

// Where a mode's partial results are, and the rows of a slot.
template <AtMode M, typename Args>
__device__ __forceinline__ int at_slot_rows(const Args& A) {
  if constexpr (M == AT_OWN) return A.own_rows;
  return KV_ROWS;
}
template <AtMode M, typename Args>
__device__ __forceinline__ float2* at_stats(const Args& A) {
  if constexpr (M == AT_ROWS) return A.S.stat;
  else if constexpr (M == AT_OWN) return A.own_stat;
  else return A.stat;
}
template <AtMode M, typename Args>
__device__ __forceinline__ float* at_parts(const Args& A) {
  if constexpr (M == AT_ROWS) return A.S.part;
  else if constexpr (M == AT_OWN) return A.own_part;
  else return A.part;
}
template <AtMode M, typename Args>
__device__ __forceinline__ KvSpan* at_spans(const Args& A) {
  if constexpr (M == AT_OWN) return A.own_span;
  else return A.span;
}

// The work of one CTA, number `cta` of `most_ctas` that share it; `total` units in all, `before`
// this thread's of its count. (W, BF16 and NDB are template parameters because the loops' registers
// and instruction fetches matter: with the vector's width a variable, single tokens took 127 us
// instead of 120 and trees 173 instead of 166, as they were then.) W: rows of a copy (32, 64 or 128
// >= the query rows of a tile). BF16: type of the queries and outputs (else fp16). NDB: 128-byte
// blocks of a token's vector.
template <AtMode M, int W, bool BF16, int NDB, typename Args>
__device__ __forceinline__ void at_body(const Args& A, const AttendPlan& P, const CUtensorMap& tmK,
                                        const CUtensorMap& tmV, AtShared<M, W>& sh,
                                        const uint32_t* s_rows, unsigned char* dsm_raw,
                                        AtCount count, int total, int before, int cta,
                                        int most_ctas) {
  constexpr int COPIES = 128 / W;
  constexpr int NC = W / AT_PARTS;     // tokens of a thread
  constexpr int GC = NC < 16 ? NC : 16;  // taken at a time
  // Tensor memory: the output's accumulator, then three of scores (two above dim 128). A
  // tile's weights (32 columns a term) replace its scores.
  constexpr int ndb = NDB, nsb = ndb == 1 ? 3 : 2;
  constexpr uint32_t scol = 128 * ndb;
  auto &kfull = sh.kfull, &kempty = sh.kempty, &vfull = sh.vfull, &vempty = sh.vempty;
  auto& tinfo = sh.tinfo;
  auto &sfull = sh.sfull, &pfull = sh.pfull, &pvdone = sh.pvdone;
  auto& vchk = sh.vchk;
  auto& qfull = sh.qfull;
  auto &dfull = sh.dfull, &dempty = sh.dempty, &drain = sh.drain;
  volatile int& s_abort = *const_cast<volatile int*>(&sh.abort);
  auto& s_walk = sh.walk;
  auto& s_y = sh.y;
  auto& s_sc = sh.sc;
  auto& s_item = sh.item;
  auto& s_c = sh.c;
  auto& s_pos = sh.pos;
  auto& s_see = sh.see;
  auto& s_out = sh.out;
  auto &s_par = sh.par, &s_tpos = sh.tpos;
  auto& s_tsee = sh.tsee;
  auto &s_top = sh.top, &s_l = sh.l;
  auto& s_stat = sh.stat;
  auto& s_vnan = sh.vnan;

  unsigned char* dsm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(dsm_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const KvCache& C = A.C;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  constexpr int slot = ndb * AT_BLK;
  unsigned char* Qs = dsm;                                  // [terms][ndb][128][128]
  unsigned char* Ks = Qs + AT_QTERMS<BF16> * slot;          // [nk][ndb][128][128]
  unsigned char* Vs = Ks + (size_t)P.nk * slot;             // [nv][ndb][128][128]
  float* joinb = reinterpret_cast<float*>(Vs + (size_t)P.nv * slot);  // row copies being added

  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return mbar_try(bar, parity) || at_wait_on(bar, parity, &s_abort, A);
  };

  at_begin<M>(A, sh, count, total, before, cta, most_ctas);
  const uint32_t tmem = sh.tmem;

  int copied = 0;  // tiles whose copies this warp has issued
  if (w == 0) {
    copied = at_copy_keys<M, NDB>(A, P.nk, tmK, sh, s_rows, Ks);
  } else if (w == 1) {
    // ---- Scores of a tile.
    if (at_elect()) {
      const int ksteps = (C.dim + 31) / 32;
      const uint32_t qd = at_desc_lo(smem_addr(Qs)), ring0 = at_desc_lo(smem_addr(Ks));
      const uint32_t rstep = static_cast<uint32_t>(slot) >> 4;
      constexpr uint32_t ids = AT_IDESC_S | ((AT_KEYS / 8) << 17);
      bool ok = true;
      int q = 0, ph = 0, sb = 0, sph = 0;
      for (int item = 0; ok; ++item) {
        if (!wait(&qfull, item & 1)) break;
        const int m = s_item[item & 1].m;
        if (m == 0) break;
        for (int i = 0; i < m; ++i) {
          // An accumulator is free once the weights that replaced its scores are multiplied.
          if ((sph > 0 && !wait(&pvdone[sb], (sph - 1) & 1)) || !wait(&kfull[q], ph & 1)) {
            ok = false;
            break;
          }
          tm_fence_after();
          const uint32_t d = tmem + scol + sb * 128, kd = ring0 + q * rstep;
          uint32_t acc = 0;
          for (int t = 0; t < AT_QTERMS<BF16>; ++t)
            for (int db = 0; db < ndb; ++db) {
              const uint32_t id = t ? ids | AT_IDESC_E5M2_A : ids;
              const uint32_t al = qd + (t * ndb + db) * (AT_BLK >> 4), bl = kd + db * (AT_BLK >> 4);
              const int kn = ksteps - 4 * db;
              if (kn >= 4) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  umma_ss(d, al + 2 * k, bl + 2 * k, AT_HI, id, k ? 1u : acc);
              } else {
                for (int k = 0; k < kn; ++k)
                  umma_ss(d, al + 2 * k, bl + 2 * k, AT_HI, id, k ? 1u : acc);
              }
              acc = 1;
            }
          // (Two arrivals: the products' end, and what this thread has seen of the tile's data.)
          umma_commit(&sfull[sb]);
          mbar_arrive(&sfull[sb]);
          umma_commit(&kempty[q]);
          if (++sb == nsb) {
            sb = 0;
            ++sph;
          }
          if (++q == P.nk) {
            q = 0;
            ++ph;
          }
        }
      }
      at_drain(&drain[0], s_abort);
    }
  } else if (w == 2) {
    // ---- V copies, the values of cut tiles, and in the pauses planning: the next item's
    // description and rows.
    fence_async_global();
    AtWalk<M> walk = s_walk;
    walk.first(A, s_rows);
    const int ppt = AT_KEYS >> C.lgp;
    int k = 0, planned = 0;       // items planned, and their tiles
    bool more = true;
    int g = 0, q = 0, ph = 0;
    long long idle = 0;
    auto ready = [&](uint64_t* bar, int parity) {
      return __any_sync(0xffffffffu, mbar_test(bar, parity & 1)) != 0;
    };
    // Checked tiles, their place in the ring, and in their item ck. (No copy or plan passes
    // what is not checked.)
    int c = 0, cq = 0, cph = 0, ck = 0, ci = 0, cuts = 0;
    while (more || c < planned) {
      if (c < g && ready(&vfull[cq], cph)) {
        const AtItem& it = s_item[ck & 1];
        const int key0 = it.key_tile(it.i0 + ci) * AT_KEYS;
        if (key0 >= it.cut_hi() || (key0 < it.cut_lo(A.window) && key0 + AT_KEYS > A.sinks)) {
          at_check(Vs + (size_t)cq * slot, ndb, it.end - key0, s_vnan[cuts % AT_MAX_RING]);
          if (lane == 0) mbar_arrive(&vchk[cuts % AT_MAX_RING]);
          ++cuts;
        }
        if (++ci == it.m) {
          ci = 0;
          ++ck;
        }
        ++c;
        if (++cq == P.nv) {
          cq = 0;
          ++cph;
        }
        idle = 0;
        continue;
      }
      if (g < planned && g - c < P.nv && ready(&tinfo[g & (AT_INFO - 1)], g / AT_INFO) &&
          (ph == 0 || ready(&vempty[q], ph - 1))) {
        const int y = lane < ppt ? s_y[g & (AT_INFO - 1)][lane] : -1;
        const uint32_t pages = __popc(__ballot_sync(0xffffffffu, y >= 0));
        if (lane == 0) mbar_arrive_expect_tx(&vfull[q], (pages << C.lgp) * 128u * ndb);
        __syncwarp();
        if (y >= 0) {
          unsigned char* dst = Vs + (size_t)q * slot + ((size_t)lane << C.lgp) * 128;
          for (int db = 0; db < ndb; ++db) at_tma(dst + db * AT_BLK, &tmV, db * 128, y, &vfull[q]);
        }
        ++g;
        if (++q == P.nv) {
          q = 0;
          ++ph;
        }
        idle = 0;
        continue;
      }
      const int kb = k & 1;
      // (Item k's place is free once item k - 2 is done with.)
      if (!more || (k >= 2 && (ck < k - 1 || !ready(&dempty[kb], (k >> 1) - 1)))) {
        if (__any_sync(0xffffffffu, s_abort || at_expired(&idle, A.wait_limit))) {
          if (!s_abort) kv_report(A.S.hdr, ST_TIMEOUT);
          s_abort = 1;
          break;
        }
        __nanosleep(50);
        continue;
      }
      more = walk.live();
      const bool live = more;
      AtItem& it = s_item[kb];
      if (lane == 0) it.m = live ? walk.i1 - walk.i0 : 0;
      if (live) {
        const int R = walk.tile.r1 - walk.tile.r0;
        const int len = walk.row.len, nnew = walk.row.n;
        if (lane == 0) {
          it.b = walk.b;
          it.h = walk.h;
          it.len = len;
          it.n = nnew;
          it.r0 = walk.tile.r0;
          it.R = R;
          it.i0 = walk.i0;
          it.tiles = walk.tile.tiles();
          it.end = walk.tile.end;
          it.pos_lo = walk.tile.pos_lo;
          it.pos_hi = walk.tile.pos_hi;
          it.s0 = walk.tile.s0;
          it.ns = walk.tile.ns;
          it.lo = walk.tile.lo;
          it.u0 = walk.base + KV_EXTRA;
          if constexpr (M != AT_ROWS) {
            it.no = at_tile_no(A, M, walk.b, walk.rt, walk.h);
            it.part = M == AT_GROUPS || walk.row.skip > 0;
          }
        }
        bool badtree = false;
        const bool in_tree = M != AT_GROUPS && A.parent;
        if (in_tree) {
          __syncwarp();
          for (int t = lane; t < nnew; t += 32) {
            const int p = kv_ld(A.parent + (size_t)walk.b * A.T + t);
            badtree = badtree || (t > 0 && (p < 0 || p >= t));
            s_par[t] = p;
          }
          badtree = __any_sync(0xffffffffu, badtree);
          __syncwarp();
          if (badtree && lane == 0) kv_report(A.S.hdr, ST_DEVICE_INPUT);
        }
        if (in_tree && !badtree) {  // what a node of the tree sees, and its position
          for (int t = lane; t < nnew; t += 32) {
            unsigned long long see = 0;
            int up = 0;
            for (int i = t;; i = s_par[i]) {
              if (!A.window || up < A.window || len + i < A.sinks) see |= 1ull << i;
              if (i == 0) break;
              ++up;
            }
            s_tsee[t] = see;
            s_tpos[t] = len + up;
          }
          __syncwarp();
        }
#pragma unroll 1
        for (int r = lane; r < R; r += 32) {
          if constexpr (M == AT_GROUPS) {
            if (!A.window) continue;
            // (A tree that is wrong gives NaN to its row's own part.)
            const AtQuery q = at_query<M>(A, walk.b, walk.tile.r0 + r);
            int up = A.parent ? 0 : q.t;
            if (A.parent)
              for (int i = q.t; i > 0 && i < A.T && up < SV_MAX_TREE; ++up)
                i = kv_ld(A.parent + (size_t)q.b * A.T + i);
            s_pos[kb][r] = max(kv_ld(C.len + q.b), len) + up;
            continue;
          }
          const int t = (walk.tile.r0 + r) / A.group, gh = walk.tile.r0 + r - t * A.group;
          const bool tree = in_tree && !badtree;
          s_pos[kb][r] = tree ? s_tpos[t] : len + t;
          s_see[kb][r] = tree ? s_tsee[t] : ~0ull;  // (a bad tree's scores are NaN)
          s_out[kb][r] = ((long long)walk.b * A.T + t) * A.q_heads + walk.h * A.group + gh;
        }
        if (lane == 0) it.bad = badtree;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&dfull[kb]);
      if (live) planned += walk.i1 - walk.i0;
      if (live) walk.next(A, s_rows);
      ++k;
      idle = 0;
    }
    copied = g;
  } else if (w == 3) {
    // ---- Outputs: O += P V of a tile, while the next tile's scores multiply and its weights
    // form.
    if (at_elect()) {
      const uint32_t ring0 = at_desc_lo(smem_addr(Vs)), rstep = static_cast<uint32_t>(slot) >> 4;
      bool ok = true;
      int q = 0, ph = 0, sb = 0, sph = 0;
      for (int item = 0; ok; ++item) {
        if (!wait(&qfull, item & 1)) break;
        const int m = s_item[item & 1].m;
        if (m == 0) break;
        for (int i = 0; i < m; ++i) {
          if (!wait(&vfull[q], ph & 1) || !wait(&pfull[sb], sph & 1)) {
            ok = false;
            break;
          }
          tm_fence_after();
          const uint32_t pa = tmem + scol + sb * 128;
          for (int db = 0; db < ndb; ++db) {
            const uint32_t d = tmem + db * 128, vd = ring0 + q * rstep + db * (AT_BLK >> 4);
            const uint32_t ido = AT_IDESC_O | (static_cast<uint32_t>(min(128, C.dim - db * 128)) >> 3 << 17);
            const uint32_t acc = i > 0;
#pragma unroll
            for (int t = 0; t < AT_PTERMS; ++t)
#pragma unroll
              for (int k = 0; k < AT_KEYS / 32; ++k)
                umma_ts(d, pa + t * 32 + k * 8, vd + k * (4096 >> 4), AT_HI, ido, t + k ? 1u : acc);
          }
          umma_commit(&pvdone[sb]);
          umma_commit(&vempty[q]);
          if (++sb == nsb) {
            sb = 0;
            ++sph;
          }
          if (++q == P.nv) {
            q = 0;
            ++ph;
          }
        }
      }
      at_drain(&drain[1], s_abort);
    }
  } else {
    // ---- Weights and results.
    const int st = tid - AT_SM0, quad = w & 3, part = (w - 4) >> 2;
    const int row = quad * 32 + lane;             // lane of the accumulators
    const int copy = row / W, r = row % W;        // copy of query row r
    const int c0 = copy * W + part * NC;          // first of this thread's tokens
    const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    // Queries without a token and rows with wrong data: zeros or NaN. Neighbouring queries go
    // to different CTAs (the results of 32 may be half a megabyte), looked at by a lane each.
    const int queries = M == AT_GROUPS ? 0 : C.batch * A.T, spread = most_ctas * AT_SM_WARPS;
    const int first = most_ctas * (w - 4) + cta;
    for (int u0 = first; u0 < queries; u0 += 32 * spread) {
      const long long u = u0 + (long long)lane * spread;
      int fill = 0;
      if (u < queries) {
        const int b = static_cast<int>(u) / A.T, t = static_cast<int>(u) - b * A.T;
        const AtRow rw = at_row<M>(A, b);
        fill = rw.bad ? 2 : (t >= rw.n ? 1 : 0);
        if (rw.bad && t == 0) kv_report(A.S.hdr, ST_DEVICE_INPUT);
      }
      unsigned todo = __ballot_sync(0xffffffffu, fill != 0);
      while (todo) {
        const int j = __ffs(todo) - 1;
        todo &= todo - 1;
        const bool nan = __shfl_sync(0xffffffffu, fill, j) == 2;
        const long long at = (u0 + (long long)j * spread) * A.q_heads;
        const uint32_t x = nan ? 0x7fff7fffu : 0u;  // NaN in bf16 and fp16
        uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(A.out) + at * C.dim);
        for (int e = lane; e < A.q_heads * C.dim / 8; e += 32) o[e] = make_uint4(x, x, x, x);
        if (A.lse)
          for (int e = lane; e < A.q_heads; e += 32) A.lse[at + e] = nan ? NAN : -INFINITY;
      }
    }
    if constexpr (M != AT_ROWS) at_check_groups(A, w - 4);
    bool dead = false;  // a wait gave up: skip the work, keep meeting the other warps
    // A wait of these warps. Its lanes take up the answer together: loads and stores of the
    // accumulators, and the warps' barriers, are for converged warps, and `dead` has to be the
    // same in all of them.
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
    };
    // The queries of item k: on their way, and into shared memory; then the scores may begin.
    auto fetch = [&](int k) {
      if (!dead && !warp_wait(&dfull[k & 1], (k >> 1) & 1)) dead = true;
      if (!dead && s_item[k & 1].m > 0) at_fetch<M>(A, ndb, &s_item[k & 1], Qs);
    };
    auto convert = [&](int k) {
      if (!dead && s_item[k & 1].m > 0)
        at_convert<W, BF16, NDB>(A, &s_item[k & 1], Qs, s_c[k & 1]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&qfull);
    };
    // Is the output of the tile before done?
    int sb = 0, sph = 0;  // accumulator of the tile's scores, and its pass
    auto done = [&]() {
      const int b = sb ? sb - 1 : nsb - 1;
      return warp_wait(&pvdone[b], (sb ? sph : sph - 1) & 1);
    };
    fetch(0);
    convert(0);
    int g = 0, cuts = 0;  // key tiles, and cut ones
    bool opened = false;  // does a query tile that begins here go on in the next CTA?
    for (int item = 0;; ++item) {
      const int kb = item & 1;
      if (!dead && !warp_wait(&qfull, item & 1)) dead = true;
      // (The waits of a CTA give up together: see s_abort. Warps that saw the item must not
      // meet others that did not, so all of them agree first.)
      if (at_vote(5, AT_SM_THREADS, dead)) break;
      const AtItem& it = s_item[kb];
      const int m = it.m, len = it.len;
      if (m == 0) break;
      // Key tiles i < turn follow the row's start, the others the window; a tile is cut (some
      // query does not see all of it) from first key `cut_hi` on, and from `sinks` to `cut_lo`.
      int kt = it.key_tile(it.i0);
      const int turn = it.ns - it.i0, resume = it.lo;
      const int cut_hi = it.cut_hi(), cut_lo = it.cut_lo(A.window);
      const bool live = quad * 32 % W < it.R;  // does the warp have a query row?
      const bool real = r < it.R;
      const float cs = real ? s_c[kb][r] : 0.f;
      const int pos = real ? s_pos[kb][r] : -1;
      const unsigned long long see = real && M != AT_GROUPS ? s_see[kb][r] : 0;
      float l = 0.f, nm = 0.f;  // sum of the weights; 11 - reference
      bool unseen = real;       // has the row copy seen no key yet?

      // -- Key tiles.
#pragma unroll 1
      for (int i = 0; i < m; ++i, ++g) {
        if (i == turn) kt = resume;
        const int key0 = kt * AT_KEYS;
        ++kt;
        if (!dead && !warp_wait(&sfull[sb], sph & 1)) dead = true;
        tm_fence_after();
        if (i == m - 1) fetch(item + 1);  // (the last scores are done: the queries' place is free)
        // Is there a key of the tile that some query does not see?
        const bool cut = key0 >= cut_hi || (key0 < cut_lo && key0 + AT_KEYS > A.sinks);
        const uint32_t sa = tl + scol + sb * 128;
        if (live) {
          // This thread's scores as logarithms of their weights, sixteen tokens at a time.
          float x[NC];
#pragma unroll
          for (int c = 0; c < NC; c += GC) {
            if (GC == 16)
              tm_ld16(sa + c0 + c, x + c);
            else
              tm_ld8(sa + c0 + c, x + c);
          }
          tm_wait_ld<NC>(x);
          const float4* sc = s_sc[g & (AT_INFO - 1)];
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < NC; c += GC) {
            const float4 f = sc[(c0 + c) >> C.lgp];
            const float2 a = make_float2(f.x * cs, f.x * cs), b = make_float2(f.y + nm, f.y + nm);
#pragma unroll
            for (int e = c; e < c + GC; e += 2) {
              const float2 y = __ffma2_rn(make_float2(x[e], x[e + 1]), a, b);
              x[e] = y.x;
              x[e + 1] = y.y;
            }
          }
          if (__builtin_expect(cut, 0)) {
            // Which of this thread's NC tokens the query sees, as bits. A chain sees those up
            // to its position; a tree the cached ones and its own of the block.
            const int k0 = key0 + c0;
            uint32_t sees = at_below(M == AT_GROUPS || A.parent ? len - k0 : pos - k0 + 1);
            if (A.window) sees &= ~at_below(max(pos - k0 + 1, 0) - A.window) | at_below(A.sinks - k0);
            if (M != AT_GROUPS && A.parent) {
              const int o = k0 - len;
              if (o > -32 && o < 64)
                sees |= static_cast<uint32_t>(o >= 0 ? see >> o : see << -o) & at_below(len + it.n - k0);
            }
            if (!dead && !warp_wait(&vchk[cuts % AT_MAX_RING], (cuts / AT_MAX_RING) & 1)) dead = true;
            const uint32_t bad = s_vnan[cuts % AT_MAX_RING][c0 / 32] >> (c0 % 32);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              if ((bad >> c) & 1) x[c] = NAN;
              if (!((sees >> c) & 1)) x[c] = -INFINITY;
            }
          }
#pragma unroll
          for (int c = 0; c < NC; c += 2) top = max3(top, x[c], x[c + 1]);
          if (at_vote(1 + quad, 128, unseen || (real && top > AT_LIMIT))) {
            // Move references to the tile's largest scores; the outputs and sums so far shrink
            // by the difference.
            s_top[part][row] = top;
            at_bar(1 + quad, 128);
            const float d = fmaxf(fmaxf(s_top[0][row], s_top[1][row]),
                                  fmaxf(s_top[2][row], s_top[3][row]));  // over the reference - 11
            float move = 0.f, fac = 1.f;
            if (unseen) {  // nothing to shrink: the reference goes wherever the scores are
              if (d > -INFINITY) {
                move = d - AT_SHIFT;
                unseen = false;
              }
            } else if (real && d > AT_SHIFT) {
              move = d - AT_SHIFT;
              fac = exp2f(-move);
            }
            nm -= move;
            l *= fac;
#pragma unroll
            for (int c = 0; c < NC; ++c) x[c] -= move;
            __syncwarp();
            if (i > 0) {
              if (!dead && !done()) dead = true;
              tm_fence_after();
#pragma unroll 1
              for (int c = part * 16; c < C.dim; c += 64) {
                float o[16];
                tm_ld16(tl + c, o);
                tm_wait_ld<16>(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] *= fac;
                tm_st16(tl + c, o);
              }
            }
          }
          // Weights: 2^x, summed with the value scale taken out, rounded to fp16 (off by up to
          // 2^-11) and split. A term is the upper byte of what is left of the fp16 number,
          // rounded (halves away from zero); the rest after it is exact. Three terms hold all
          // of its 11 bits down to a weight of 2^-6; below, they end at e5m2's smallest, 2^-16,
          // so that a weight is off by up to 2^-17 (2^-28 of one at the reference). Cutting the
          // first term off instead saves an addition a pair (trees of 16 nodes 145.5 us instead
          // of 148.7), but the three are then off by up to 0.88 * 2^-10 on top.
#pragma unroll
          for (int c = 0; c < NC; c += GC) {
            uint32_t t[AT_PTERMS][GC / 2];
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < GC / 2; ++e) {
              const float2 p = make_float2(ex2(x[c + 2 * e]), ex2(x[c + 2 * e + 1]));
              sum = __fadd2_rn(sum, p);
              __half2 y = __floats2half2_rn(p.x, p.y);
#pragma unroll
              for (int k = 0; k < AT_PTERMS; ++k) {
                t[k][e] = *reinterpret_cast<const uint32_t*>(&y) + 0x00800080u;
                const uint32_t hi = t[k][e] & 0xff00ff00u;
                y = __hsub2(y, *reinterpret_cast<const __half2*>(&hi));
              }
            }
            l = fmaf(sum.x + sum.y, sc[(c0 + c) >> C.lgp].z, l);
#pragma unroll
            for (int k = 0; k < AT_PTERMS; ++k) {
              uint32_t v[GC / 4];
#pragma unroll
              for (int e = 0; e < GC / 4; ++e) v[e] = __byte_perm(t[k][2 * e], t[k][2 * e + 1], 0x7531);
              if constexpr (GC == 16)
                tm_st4(sa + k * 32 + (c0 + c) / 4, v[0], v[1], v[2], v[3]);
              else
                tm_st2(sa + k * 32 + (c0 + c) / 4, v[0], v[1]);
            }
          }
          // Tokens that belong to the row's other copies.
          if (COPIES > 1) {
#pragma unroll
            for (int c = 0; c < AT_KEYS / 16; c += AT_PARTS) {
              if ((c + part) * 16 / W == copy) continue;
#pragma unroll
              for (int k = 0; k < AT_PTERMS; ++k) tm_st4(sa + k * 32 + (c + part) * 4, 0, 0, 0, 0);
            }
          }
          tm_wait_st();
        }
        cuts += cut;
        tm_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[sb]);
        if (++sb == nsb) {
          sb = 0;
          ++sph;
        }
      }

      // -- The query tile's sums and outputs: the result when this CTA saw all its keys,
      // else partial results. The last scores are done, so the next queries go in first.
      s_l[part][row] = l;
      if (part == 0) s_stat[row].x = -nm;
      convert(item + 1);
      at_bar(5, AT_SM_THREADS);
      if (st < 128)
        s_stat[st].y = st % W < it.R ? s_l[0][st] + s_l[1][st] + (s_l[2][st] + s_l[3][st]) : 0.f;
      if (!dead && !done()) dead = true;
      tm_fence_after();
      at_bar(5, AT_SM_THREADS);
      const bool whole = m == it.tiles && (M == AT_ROWS || !it.part);
      // Partial results: two slots a CTA (it holds parts of two query tiles at most), or those of
      // the query tile.
      const int slot_id = M == AT_ROWS ? 2 * cta + (it.i0 == 0 ? 1 : 0) : it.no + cta;
      const int slot_rows = at_slot_rows<M>(A);
      float2* const part_stat = at_stats<M>(A) + (size_t)slot_id * slot_rows;
      float4* const parts = reinterpret_cast<float4*>(at_parts<M>(A));
      // Reference and sum over the row's copies, and this copy's factor. (The approximate
      // power and quotient are off by 2^-22; short code, since it comes from memory each time.)
      float ref = -INFINITY, sum = 0.f;
#pragma unroll 1
      for (int c = r; c < 128; c += W) {
        const float2 s2 = s_stat[c];
        if (s2.y == 0.f) continue;
        const float top = fmaxf(ref, s2.x);
        sum = fmaf(s2.y, ex2(s2.x - top), sum * ex2(ref - top));
        ref = top;
      }
      const float2 own = s_stat[row];
      float f = own.y == 0.f ? 0.f : ex2(own.x - ref);
      if (whole) f = sum == 0.f ? 0.f : __fdividef(f, sum);
      if (copy == 0 && part == 0 && real) {
        if (!whole)
          part_stat[r] = make_float2(ref, sum);
        else if (A.lse)
          A.lse[s_out[kb][r]] = sum == 0.f ? -INFINITY : (ref + at_log2(sum)) * 0.6931471805599453f;
      }
      // (Lanes without a query row skip what follows a load; all are together again at the next.)
      __syncwarp();
      if constexpr (COPIES == 1) {
        // A row's 16 components are whole sectors: straight from the accumulator.
#pragma unroll 1
        for (int c = part * 16; live && c < C.dim; c += 16 * AT_PARTS) {
          float o[16];
          tm_ld16(tl + c, o);
          tm_wait_ld<16>(o);
          if (real) {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = f == 0.f ? 0.f : o[e] * f;
            if (whole) {
              uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(A.out) +
                                                   s_out[kb][r] * C.dim + c);
#pragma unroll
              for (int e = 0; e < 16; e += 8)
                to[e / 8] = make_uint4(
                    at_pack(o[e], o[e + 1], BF16), at_pack(o[e + 2], o[e + 3], BF16),
                    at_pack(o[e + 4], o[e + 5], BF16), at_pack(o[e + 6], o[e + 7], BF16));
            } else {
              float4* to = parts + at_part(slot_id, r, c, C.dim, slot_rows);
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                to[e / 4 * slot_rows] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
          }
          __syncwarp();
        }
      } else {
        // Copies are added in shared memory, as many components at a time (a multiple of 8)
        // as fit there for the item's rows. (A row's stride is four floats more, so that
        // neither rows nor columns meet in a bank, 16 bytes at a time.)
        const int R = it.R, fit = (P.join / (COPIES * R) - 4) & ~7, line = min(fit, C.dim) + 4;
#pragma unroll 1
        for (int c = 0; c < C.dim; c += fit) {
          const int n = min(fit, C.dim - c);
#pragma unroll 1
          for (int d0 = part * 8; live && d0 < n; d0 += 16 * AT_PARTS) {
            float o[2][8];
            tm_ld8(tl + c + d0, o[0]);
            const int d1 = d0 + 8 * AT_PARTS;
            if (d1 < n) tm_ld8(tl + c + d1, o[1]);
            tm_wait_ld<16>(o[0]);
            if (real) {
              float* to = joinb + (copy * R + r) * line;
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                if (u && d1 >= n) break;
#pragma unroll
                for (int e = 0; e < 8; ++e) o[u][e] = f == 0.f ? 0.f : o[u][e] * f;
                float4* at = reinterpret_cast<float4*>(to + (u ? d1 : d0));
                at[0] = make_float4(o[u][0], o[u][1], o[u][2], o[u][3]);
                at[1] = make_float4(o[u][4], o[u][5], o[u][6], o[u][7]);
              }
            }
            __syncwarp();
          }
          at_bar(5, AT_SM_THREADS);
          // Four components to a thread: of a row in the result, of a column in partial results.
          const int wi = w - 4, inner = whole ? n / 4 : R, outer = whole ? R : n / 4;
#pragma unroll 1
          for (int a = wi; a < outer; a += AT_SM_WARPS)
#pragma unroll 1
            for (int b = lane; b < inner; b += 32) {
              const int rr = whole ? a : b, d = 4 * (whole ? b : a);
              float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int k = 0; k < COPIES; ++k) {
                const float4 x = *reinterpret_cast<const float4*>(joinb + (k * R + rr) * line + d);
                y.x += x.x;
                y.y += x.y;
                y.z += x.z;
                y.w += x.w;
              }
              if (whole)
                at_store4(A.out, s_out[kb][rr] * C.dim + c + d, y, BF16);
              else
                parts[at_part(slot_id, rr, c + d, C.dim, slot_rows)] = y;
            }
          __syncwarp();
          at_bar(5, AT_SM_THREADS);
        }
      }
      tm_fence_before();
      if constexpr (M == AT_ROWS) {
        if (!whole && it.i0 == 0) {  // the first of the CTAs that hold this query tile
          opened = true;
          if (st == 0) {
            const int all = sh.total, n = min(most_ctas, all);
            A.S.open[cta] = KvOpen{it.b, it.h, it.r0, it.R, at_owner(it.u0 + it.tiles - 1, all, n), 0};
          }
        }
      } else if (!whole && it.i0 == 0) {
        const int all = sh.total, n = min(most_ctas, all), last = at_owner(it.u0 + it.tiles - 1, all, n);
        if (M == AT_GROUPS || it.part) {
          if (st == 0) at_spans<M>(A)[it.no] = KvSpan{cta, last};
        } else {
          opened = true;
          if (st == 0) A.S.open[blockIdx.x] = KvOpen{it.b, it.h, it.r0, it.R, last - cta, it.no + cta};
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&dempty[kb]);
    }
    if (!opened && st == 0) A.S.open[blockIdx.x].R = 0;
  }

  tm_fence_before();
  __syncthreads();
  // After a wait gave up, what is on its way to shared memory lands before the CTA exits, also
  // the copies of a warp that was through before. (A stage's barrier whose last pass was
  // consumed answers at once.)
  if (s_abort) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (w == 0) at_land(kfull, P.nk, copied);
    if (w == 2) at_land(vfull, P.nv, copied);
  }
  if (w == 1) {
    __syncwarp();
    tm_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

// Shared memory of a CTA, and what the kernels' static arrays take of it (at most).
constexpr size_t AT_SMEM = 232448, AT_STATIC = 20480;

// What a launch needs beside its arguments (sv_kv_attend.cu), for tiles of `width` query rows.
struct AttendLaunch {
  AttendPlan P;
  CUtensorMap tm[2];
  int ndb, width, grid;
  size_t smem;
};
cudaError_t launch_kv_attend_group(const SharedArgs& A, const AttendLaunch& L, sv_dtype dt, int dev,
                                  cudaStream_t st);
cudaError_t at_launch(const AttendArgs& A, sv_dtype dt, int width, int dev, AttendLaunch* L);

}  // namespace sv
