// sv_kv_attend.cu -- attention of a round's new tokens over the key/value cache (sm_103a).
//
// For one row, key/value head and tile of R <= 128 query rows (tokens x query heads of the
// group, flattened) and key tiles of 128 tokens:
//     S = Q K^T  [R x 128],   P = 2^(S - m),   O += P V  [R x dim].
// Both products run on the fifth-generation tensor cores with the cache's own e4m3 bytes as
// the second operand, straight from TMA: nothing of the cache is converted. The first
// operand is carried as a sum of 8-bit terms, multiplied one after the other into the same
// float32 accumulator. A query row, scaled by a power of two to the e4m3 range, is the sum of
// an e4m3 term (4 bits) and one (bf16) or two (fp16) e5m2 terms for the rest: after rounding to
// 4 bits the rest of bf16's 8 has 3, which e5m2 holds, and e5m2's smallest number is 2^-16 where
// e4m3's is 2^-9 (2^-18 of the largest component). That is exact down to 2^-13 of the largest
// component, and off by up to 2^-21 (bf16) or 2^-24 (fp16) of that one below. A weight is rounded
// to fp16 and split into three e5m2 terms (e5m2 is fp16's upper byte, so a split is integer
// arithmetic). Weights go from registers to tensor memory and are multiplied from there.
//
// A thread owns a query row (a lane of the accumulator) and some of the tile's tokens, so
// that the softmax needs no exchange but one vote between the four threads of a row. (With
// tokens on the lanes instead, weights went through shared memory and sums across lanes: 472
// instead of 292 us for trees of 16 nodes, both as first built.) Sixteen tokens share a page:
// its key scale is a factor of their scores; its value scale is folded into their weights
// (its logarithm added to the scores, so that no weight exceeds the reference) and taken out
// of their sum again. The reference m of a row only moves when
// a score passes it by 2^4 (the accumulators are then rescaled), or with the first keys the
// row sees.
//
// The product has 128 rows whatever R is. Few rows are therefore repeated, 128 / W times
// for W = 32 or 64 >= R: each copy of a row takes its own W tokens of a tile (the weights
// of the others stay zero), so that all lanes have work and a tile's softmax costs R / 128
// of a full one; the copies' outputs are added at the end.
//
// A persistent CTA per SM takes an equal share of all (row, head, query tile, key tile)
// units in order; a query tile that crosses from one CTA to the next leaves partial
// results (output, m, sum) in the workspace, which a second kernel joins on all SMs.
//
// Warps, coupled by mbarriers: one copies K tiles page by page by tensor-map TMA (128-byte
// swizzle) into a ring, another V tiles into a second (and looks through those whose weights
// are cut, and plans the next query tile while this one is in work); one issues the scores'
// products and one the output's; sixteen form the weights, four on each quarter of a row
// copy's tokens.
//
// What bounds it. Up to dim 128 a key tile is 32 KB, 1,400 cycles of an SM's share of the
// memory rate, and 20 products of 64 cycles; its softmax is a chain of waits, loads,
// a vote, powers, splits and stores of about 1,600 cycles for 32 rows, 1,800 for 64 and 2,600
// for 128, where the integer instructions of the split alone fill half of it. Measured in CUDA
// graphs (a call from Python takes 2 to 11 us more) on 64 rows with 8 key/value heads of 128:
// single tokens of 8 queries a head, 4,100 tokens cached in the mean, 122 us (4.4 TB/s, 65 %
// of a copy); blocks of 9 tokens of 4 queries, 137 us; trees of up to 16 nodes of 8 queries,
// 149 us (560 TFLOP/s of the formula's, 2.5 times as many of 8-bit products). A query tile
// costs 3,000 to 8,000 cycles beside its key tiles, and a launch 11,000 to 18,000 before the
// first (counting, page table, queries, each a trip to memory), which is most of the 13 us of
// one row's single token.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <cmath>

#include "sv_device.cuh"
#include "sv_kv.cuh"

namespace sv {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // sv_markov.cu

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

// Row b of the batch.
struct AtRow {
  int len, n;    // cached and new tokens; n = 0 when the row's data is wrong
  int rows;      // query rows of a head
  int nrt, rr;   // query tiles, rows of each (the last may have fewer)
  bool bad;
};

__device__ __forceinline__ AtRow at_row(const AttendArgs& A, int b) {
  AtRow r;
  r.len = kv_ld(A.C.len + b);
  r.n = A.n_new ? kv_ld(A.n_new + b) : A.T;
  r.bad = r.n < 0 || r.n > A.T || r.len < 0 ||
          (long long)r.len + r.n > (long long)A.C.max_pages << A.C.lgp;
  if (r.bad) r.n = 0;
  r.rows = r.n * A.group;
  r.nrt = (r.rows + KV_ROWS - 1) / KV_ROWS;
  r.rr = r.nrt ? (r.rows + r.nrt - 1) / r.nrt : 0;
  return r;
}

// Query tile rt of a row: rows r0 .. r1 - 1, and the key tiles that any of them sees:
// `ns` at the row's start (sinks), then `lo` to `hi` - 1.
struct AtTile {
  int r0, r1;
  int end;            // keys below end are visible to some query
  int pos_lo, pos_hi; // bounds of the queries' positions
  int ns, lo, hi;
  __device__ __forceinline__ int tiles() const { return ns + hi - lo; }
  __device__ __forceinline__ int key_tile(int i) const { return i < ns ? i : lo + i - ns; }
};

__device__ __forceinline__ AtTile at_tile(const AttendArgs& A, const AtRow& r, int rt) {
  AtTile t;
  t.r0 = rt * r.rr;
  t.r1 = min(t.r0 + r.rr, r.rows);
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
  return t;
}

// Work is counted in key tiles, with KV_EXTRA more for each query tile: what its queries'
// conversion and its results cost. Its order is rows, query tiles, heads.

// Units of row b's query tile rt for one head (0: none).
__device__ __forceinline__ int at_units(const AttendArgs& A, int b, int rt) {
  const AtRow r = at_row(A, b);
  return rt < r.nrt ? KV_EXTRA + at_tile(A, r, rt).tiles() : 0;
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
  __device__ __forceinline__ void start(const AttendArgs& A, int b0, int rt0, int rem, int from,
                                        int to) {
    at = from;
    end = to;
    b = b0;
    rt = rt0;
    row = at_row(A, b);
    tile = at_tile(A, row, rt);
    const int per = KV_EXTRA + tile.tiles();
    h = rem / per;
    base = from - (rem - h * per);
    settle();
  }
  // For the warps that walk, before the first query tile.
  __device__ __forceinline__ void first(const AttendArgs& A, const uint32_t* rows) {
    if (live() && i1 <= i0) next(A, rows);
  }
  __device__ __forceinline__ bool live() const { return at < end; }
  // A whole warp; `rows` has a bit for each row that has queries.
  __device__ __noinline__ void next(const AttendArgs& A, const uint32_t* rows) {
    do {
      base += KV_EXTRA + tile.tiles();
      at = base;
      if (at >= end) return;
      if (++h == A.C.heads) {
        h = 0;
        if (++rt == row.nrt) {
          rt = 0;
          b = at_next_row(rows, A.C.batch, b);  // (it exists: units are left)
          row = at_row(A, b);
        }
        tile = at_tile(A, row, rt);
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
  int ns, lo;
  int bad;          // the row's tree is wrong
  int u0;           // unit of its first key tile
  __device__ __forceinline__ int key_tile(int i) const { return i < ns ? i : lo + i - ns; }
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
// slot `id`. Rows are next to each other: their threads store, and the join reads, whole
// sectors. (Rows one after the other made the stores of 128 x 256 floats 9,000 cycles.)
__device__ __forceinline__ size_t at_part(int id, int r, int c, int dim) {
  return ((size_t)id * (dim / 4) + c / 4) * KV_ROWS + r;
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
__device__ __noinline__ bool at_wait_on(uint64_t* bar, uint32_t parity, volatile int* abort,
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
__device__ __noinline__ void at_fetch(const AttendArgs& A, int ndb, const AtItem* it,
                                      unsigned char* Q) {
  const int hw = (threadIdx.x - AT_SM0) >> 4, l16 = threadIdx.x & 15;
#pragma unroll 1
  for (int row = hw; row < it->R; row += 2 * AT_SM_WARPS) {
    const int t = (it->r0 + row) / A.group, gh = it->r0 + row - t * A.group;
    const uint16_t* src = static_cast<const uint16_t*>(A.q) + it->b * A.q_row + t * A.q_tok +
                          (size_t)(it->h * A.group + gh) * A.C.dim;
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
__device__ __noinline__ void at_check(unsigned char* v, int ndb, int end, uint32_t* nans) {
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
__device__ __noinline__ void at_land(uint64_t* full, int n, int g) {
  const long long t0 = clock64();
  for (int j = max(0, g - n); j < g; ++j)
    while (!mbar_test(&full[j % n], (j / n) & 1) && clock64() - t0 < WAIT_CYCLES / 4) {
    }
}

// (The three are template parameters because the loops' registers and instruction fetches
// matter: with the vector's width a variable, single tokens took 127 us instead of 120 and
// trees 173 instead of 166, as they were then.) W: rows of a copy (32, 64 or 128 >= the query
// rows of a tile). BF16: type of the queries and outputs (else fp16). NDB: 128-byte blocks of a
// token's vector.
template <int W, bool BF16, int NDB>
__global__ void __launch_bounds__(AT_THREADS, 1)
    kv_attend_kernel(const __grid_constant__ AttendArgs A, const __grid_constant__ AttendPlan P,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV) {
  constexpr int COPIES = 128 / W;
  constexpr int NC = W / AT_PARTS;     // tokens of a thread
  constexpr int GC = NC < 16 ? NC : 16;  // taken at a time
  // Tensor memory: the output's accumulator, then three of scores (two above dim 128). A
  // tile's weights (32 columns a term) replace its scores.
  constexpr int ndb = NDB, nsb = ndb == 1 ? 3 : 2;
  constexpr uint32_t scol = 128 * ndb;
  extern __shared__ unsigned char dsm_raw[];
  __shared__ uint64_t kfull[AT_MAX_RING], kempty[AT_MAX_RING];
  __shared__ uint64_t vfull[AT_MAX_RING], vempty[AT_MAX_RING], tinfo[AT_INFO];
  __shared__ uint64_t sfull[3], pfull[3], pvdone[3], vchk[AT_MAX_RING], qfull, dfull[2], dempty[2], drain[2];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ AtWalk s_walk;
  __shared__ int s_total, s_sum[AT_THREADS / 32];
  __shared__ uint32_t s_rows[AT_LIVE];  // rows that have queries, a bit each
  // Per key tile and page of it: row of the pool (-1: none); key scale, log2 and inverse of
  // the value scale.
  __shared__ int s_y[AT_INFO][8];
  __shared__ float4 s_sc[AT_INFO][8];
  // Item k's description and rows, at k & 1: factor of the score, position of the query,
  // block nodes it sees (trees), its row of the output.
  __shared__ AtItem s_item[2];
  __shared__ float s_c[2][W];
  __shared__ int s_pos[2][W];
  __shared__ unsigned long long s_see[2][W];
  __shared__ long long s_out[2][W];
  __shared__ int s_par[SV_MAX_TREE], s_tpos[SV_MAX_TREE];  // a tree: parents, positions
  __shared__ unsigned long long s_tsee[SV_MAX_TREE];       // and what a node sees
  __shared__ float s_top[AT_PARTS][128], s_l[AT_PARTS][128];  // largest scores, sums
  __shared__ float2 s_stat[128];     // reference and sum of a row copy
  // Tokens of a cut tile with a NaN value, an entry per cut tile (no more of them than tiles
  // in V's ring are checked and not yet multiplied).
  __shared__ uint32_t s_vnan[AT_MAX_RING][AT_KEYS / 32];

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

  if (tid < AT_INFO) {
    mbar_init(&tinfo[tid], 1);
    if (tid < AT_MAX_RING) {
      mbar_init(&kfull[tid], 2);
      mbar_init(&kempty[tid], 1);
      mbar_init(&vfull[tid], 1);
      mbar_init(&vempty[tid], 1);
      mbar_init(&vchk[tid], 1);
    }
    if (tid < 3) {
      mbar_init(&sfull[tid], 2);
      mbar_init(&pfull[tid], AT_SM_WARPS);
      mbar_init(&pvdone[tid], 1);
    }
    if (tid < 2) {
      mbar_init(&dfull[tid], 1);
      mbar_init(&dempty[tid], AT_SM_WARPS);
      mbar_init(&drain[tid], 1);
    }
    if (tid == 0) {
      mbar_init(&qfull, AT_SM_WARPS);
      s_abort = 0;
    }
    fence_mbar_init();
  }
  if (w == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&s_tmem)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  kv_enter();
  // This CTA's share: the units of all rows' query tiles, cut into equal parts. Query tiles
  // are counted by the threads in turn; the second pass finds the one where the share begins.
  const int nrt = (A.T * A.group + KV_ROWS - 1) / KV_ROWS, pairs = C.batch * nrt;
  auto units_of = [&](int p) -> int {
    if (p >= pairs) return 0;
    const int b = nrt == 1 ? p : p / nrt;
    return at_units(A, b, p - b * nrt) * C.heads;
  };
  int mine = 0, sum = 0;
#pragma unroll 1
  for (int p = tid; p - lane < pairs; p += AT_THREADS) {
    const int c = units_of(p);
    if (p == tid) mine = c;
    sum += c;
    if (nrt == 1) {  // (p is the row)
      const uint32_t has = __ballot_sync(0xffffffffu, c != 0);
      if (lane == 0) s_rows[p / 32] = has;
    }
  }
  if (nrt > 1)
#pragma unroll 1
    for (int b = tid; b - lane < C.batch; b += AT_THREADS) {
      const uint32_t has = __ballot_sync(0xffffffffu, b < C.batch && at_row(A, b).rows > 0);
      if (lane == 0) s_rows[b / 32] = has;
    }
  auto block_sum = [&](int x, int* before) {  // sum; *before: of lower threads
    int v = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += t;
    }
    if (lane == 31) s_sum[w] = v;
    __syncthreads();
    int all = 0, pre = 0;
    for (int i = 0; i < AT_THREADS / 32; ++i) {
      if (i < w) pre += s_sum[i];
      all += s_sum[i];
    }
    *before = pre + v - x;
    return all;
  };
  int before;
  const int total = block_sum(sum, &before);
  const int ctas = min(static_cast<int>(gridDim.x), total), cta = blockIdx.x;
  const int from = cta < ctas ? at_share(cta, total, ctas) : 0;
  const int to = cta < ctas ? at_share(cta + 1, total, ctas) : 0;
  if (tid == 0) {
    s_total = total;
    if (from >= to) s_walk.at = s_walk.end = 0;
  }
  if (from < to) {
    int base = 0;
#pragma unroll 1
    for (int p0 = 0;; p0 += AT_THREADS) {
      const int c = p0 == 0 ? mine : units_of(p0 + tid);
      int all = total;
      if (pairs > AT_THREADS) {  // (otherwise `before` is right already)
        __syncthreads();
        all = block_sum(c, &before);
      }
      if (from >= base + before && from < base + before + c) {
        // (One thread for all: its row's data and this code are at hand, which saves the
        // copies 3,000 cycles before their first page.)
        const int b = (p0 + tid) / nrt;
        AtWalk walk;
        walk.start(A, b, p0 + tid - b * nrt, from - base - before, from, to);
        s_walk = walk;
      }
      base += all;
      if (base > from) break;
    }
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tmem = s_tmem;

  int copied = 0;  // tiles whose copies this warp has issued
  if (w == 0) {
    // ---- K copies. Pages are looked up for several tiles at a time, a page per lane and a
    // chunk ahead of their use; their data go to the other warps through a ring of entries,
    // one per tile, written before the tile's barrier is armed. (An entry is used again 32
    // tiles later, and K is never more than its ring and three steps ahead of the rest.)
    fence_async_global();  // (what earlier kernels stored, before copies read it)
    AtWalk walk = s_walk;
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
      page = used ? kv_page(C, walk.b, key) : -1;
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
            s_y[e][sub] = y;
            s_sc[e][sub] = make_float4(ks, log2f(vs), 1.f / vs, 0.f);
          }
          __syncwarp();
        }
        if (lane == 0) {  // (the second of kfull's arrivals: the tile's data are there)
          mbar_arrive(&kfull[q]);
          mbar_arrive(&tinfo[g & (AT_INFO - 1)]);
        }
        ++g;
        if (++q == P.nk) {
          q = 0;
          ++ph;
        }
        if (t == 0) look();
      }
    }
    copied = g;
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
    AtWalk walk = s_walk;
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
          it.ns = walk.tile.ns;
          it.lo = walk.tile.lo;
          it.u0 = walk.base + KV_EXTRA;
        }
        bool badtree = false;
        if (A.parent) {
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
        if (A.parent && !badtree) {  // what a node of the tree sees, and its position
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
          const int t = (walk.tile.r0 + r) / A.group, gh = walk.tile.r0 + r - t * A.group;
          const bool tree = A.parent && !badtree;
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
    const int queries = C.batch * A.T, spread = static_cast<int>(gridDim.x) * AT_SM_WARPS;
    const int first = static_cast<int>(gridDim.x) * (w - 4) + static_cast<int>(blockIdx.x);
    for (int u0 = first; u0 < queries; u0 += 32 * spread) {
      const long long u = u0 + (long long)lane * spread;
      int fill = 0;
      if (u < queries) {
        const int b = static_cast<int>(u) / A.T, t = static_cast<int>(u) - b * A.T;
        const AtRow rw = at_row(A, b);
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
      if (!dead && s_item[k & 1].m > 0) at_fetch(A, ndb, &s_item[k & 1], Qs);
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
      const unsigned long long see = real ? s_see[kb][r] : 0;
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
            uint32_t sees = at_below(A.parent ? len - k0 : pos - k0 + 1);
            if (A.window) sees &= ~at_below(max(pos - k0 + 1, 0) - A.window) | at_below(A.sinks - k0);
            if (A.parent) {
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
      const bool whole = m == it.tiles;
      const int slot_id = 2 * blockIdx.x + (it.i0 == 0 ? 1 : 0);
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
          A.S.stat[(size_t)slot_id * KV_ROWS + r] = make_float2(ref, sum);
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
              float4* to = reinterpret_cast<float4*>(A.S.part) + at_part(slot_id, r, c, C.dim);
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                to[e / 4 * KV_ROWS] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
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
                reinterpret_cast<float4*>(A.S.part)[at_part(slot_id, rr, c + d, C.dim)] = y;
            }
          __syncwarp();
          at_bar(5, AT_SM_THREADS);
        }
      }
      tm_fence_before();
      if (!whole && it.i0 == 0) {  // the first of the CTAs that hold this query tile
        opened = true;
        if (st == 0) {
          const int all = s_total, n = min(static_cast<int>(gridDim.x), all);
          A.S.open[blockIdx.x] =
              KvOpen{it.b, it.h, it.r0, it.R, at_owner(it.u0 + it.tiles - 1, all, n)};
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

// Joins the partial results of the query tile that begins in CTA blockIdx.x and goes on in
// others: a thread takes four components of a row over its CTAs, with the loads of four of
// them in flight and a running reference. It reads what the CTAs left in L2: 2 to 3 us for
// 30 MB. (A join by the last of the CTAs themselves held up its SM for up to 27 us: 128 rows
// of 256 components are 128 KB a CTA.)
// Blocks of a query tile: 2, 4, 8 and 16 took 161, 153, 149 and 149 us for the trees above.
constexpr int JOIN_THREADS = 256, JOIN_BLOCKS = 8;
__global__ void __launch_bounds__(JOIN_THREADS)
    kv_attend_join_kernel(const __grid_constant__ AttendArgs A, int bf16) {
  kv_enter();
  const int first = blockIdx.x;
  const KvOpen it = A.S.open[first];
  // (Eight rows and four of their vectors to a warp: whole sectors on both sides.)
  const int vec = A.C.dim / 4, n = (it.R + 7) / 8 * 8 * vec;
  constexpr int K = 4;
  for (int e = blockIdx.y * JOIN_THREADS + threadIdx.x; e < n; e += JOIN_BLOCKS * JOIN_THREADS) {
    const int r = e / (8 * vec) * 8 + e % 8, dv = e / 8 % vec;
    if (r >= it.R) continue;
    float ref = -INFINITY, sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = first; k0 <= it.last; k0 += K) {
      float2 s2[K];
      float4 y[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int kk = min(k0 + k, it.last);
        const int id = 2 * kk + (kk == first ? 1 : 0);
        s2[k] = __ldcg(A.S.stat + (size_t)id * KV_ROWS + r);
        y[k] = __ldcg(reinterpret_cast<const float4*>(A.S.part) + at_part(id, r, 4 * dv, A.C.dim));
      }
      float top = ref;
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (s2[k].y != 0.f) top = fmaxf(top, s2[k].x);
      const float f0 = sum == 0.f ? 0.f : exp2f(ref - top);
      ref = top;
      sum *= f0;
      o.x *= f0;
      o.y *= f0;
      o.z *= f0;
      o.w *= f0;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (s2[k].y == 0.f || k0 + k > it.last) continue;
        const float f = exp2f(s2[k].x - top);
        sum = fmaf(s2[k].y, f, sum);
        o.x = fmaf(y[k].x, f, o.x);
        o.y = fmaf(y[k].y, f, o.y);
        o.z = fmaf(y[k].z, f, o.z);
        o.w = fmaf(y[k].w, f, o.w);
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int t = (it.r0 + r) / A.group, gh = it.r0 + r - t * A.group;
    const long long row = ((long long)it.b * A.T + t) * A.q_heads + it.h * A.group + gh;
    at_store4(A.out, row * A.C.dim + dv * 4,
              make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv), bf16);
    if (dv == 0 && A.lse)
      A.lse[row] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
  }
}

// Shared memory of a CTA, and what the kernels' static arrays take of it (at most).
constexpr size_t AT_SMEM = 232448, AT_STATIC = 20480;

cudaError_t launch_kv_attend(const AttendArgs& A, sv_dtype dt, cudaStream_t st) {
  typedef void (*Kernel)(const AttendArgs, const AttendPlan, const CUtensorMap, const CUtensorMap);
#define SV_ROW(bf16, ndb) \
  { kv_attend_kernel<32, bf16, ndb>, kv_attend_kernel<64, bf16, ndb>, kv_attend_kernel<128, bf16, ndb> }
  static const Kernel kernels[2][2][3] = {{SV_ROW(false, 1), SV_ROW(false, 2)},
                                          {SV_ROW(true, 1), SV_ROW(true, 2)}};
#undef SV_ROW
  int dev = 0, sms = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  static OncePerDevice sized;  // (the attribute belongs to the device that is current)
  e = static_cast<cudaError_t>(sized.run(dev, [] {
    cudaError_t attr = cudaSuccess;
    for (int i = 0; i < 12 && attr == cudaSuccess; ++i)
      attr = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernels[i / 6][i / 3 % 2][i % 3]),
                                  cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)(AT_SMEM - AT_STATIC));
    return static_cast<int>(attr);
  }));
  if (e != cudaSuccess) return e;
  const KvCache& C = A.C;
  AttendPlan P;
  const bool bf16 = dt == SV_BF16;
  const int ndb = C.dim > 128 ? 2 : 1;
  const long long rows = (long long)A.T * A.group;
  // The narrowest copy that holds the rows: 8 rows a head took 121 us with copies of 32, 127
  // with 64 and 160 with 128 (64 rows of single tokens); 36 rows 137 with 64 and 169 with 128.
  const int width = rows <= 32 ? 32 : (rows <= 64 ? 64 : 128);
  const size_t tile = (size_t)ndb * AT_BLK;
  // At least 32 components of 128 row copies, or 16 of them, which leaves room for one more
  // tile of 256 bytes a token.
  P.join = width == 128 ? 0 : 128 * (ndb == 1 ? 40 : 20);
  const size_t fixed = 1024 + (bf16 ? AT_QTERMS<true> : AT_QTERMS<false>) * tile + 4 * P.join;
  const int ring = (int)((AT_SMEM - AT_STATIC - fixed) / tile);
  P.nk = ring / 2 < AT_MAX_RING ? ring / 2 : AT_MAX_RING;
  P.nv = ring - ring / 2 < AT_MAX_RING ? ring - ring / 2 : AT_MAX_RING;
  const size_t smem = fixed + (P.nk + P.nv) * tile;
  // The pools of one layer as matrices [pages * heads * page tokens][dim bytes], in boxes of
  // one page x 128 bytes (128-byte swizzle, zeros past dim).
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  CUtensorMap tm[2];
  const size_t layer = (size_t)C.pages * C.heads * C.page * C.dim;
  for (int kv = 0; kv < 2; ++kv) {
    const cuuint64_t gdim[2] = {(cuuint64_t)C.dim, (cuuint64_t)C.pages * C.heads * C.page};
    const cuuint64_t gstride[1] = {(cuuint64_t)C.dim};
    const cuuint32_t box[2] = {128, (cuuint32_t)C.page};
    const cuuint32_t estr[2] = {1, 1};
    if (enc(&tm[kv], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, (kv ? C.v : C.k) + A.layer * layer, gdim,
            gstride, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
    return e;
  const int grid = sms < KV_MAX_CTAS ? sms : KV_MAX_CTAS;
  const Kernel kernel = kernels[bf16][ndb - 1][width == 32 ? 0 : (width == 64 ? 1 : 2)];
  if ((e = kv_launch(kernel, dim3(grid), AT_THREADS, smem, st, A, P, tm[0], tm[1])) != cudaSuccess)
    return e;
  return kv_launch(kv_attend_join_kernel, dim3(grid, JOIN_BLOCKS), JOIN_THREADS, 0, st, A, bf16 ? 1 : 0);
}

}  // namespace sv
