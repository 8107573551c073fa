// sv_kv_attend.cu -- attention of a round's new tokens over the key/value cache (sm_103a).
//
// For one row, key/value head and tile of R <= 128 query rows (tokens x query heads of the
// group, flattened) the scores are a product over the cached keys, in tiles of 128 tokens:
//     S^T = K Q^T  [128 tokens x R],   P^T = 2^(S^T - m),   O^T += V^T P^T  [dim x R].
// Both products run on the fifth-generation tensor cores with the cache's own e4m3 bytes as
// the first operand, straight from TMA: nothing of the cache is converted. The other
// operand is carried as a sum of 8-bit terms, multiplied one after the other into the same
// float32 accumulator: a query row, scaled by a power of two to the e4m3 range, is exactly
// the sum of two (bf16) or three (fp16) e4m3 terms down to 2^-18 of its largest component;
// a weight is rounded to fp16 and split into three e5m2 terms of at least 9 bits in all
// (e5m2 is fp16's upper byte, so a split is integer arithmetic).
// Tokens lie on the accumulator's lanes, so that a thread owns one token: the page's
// scales are a factor of the thread, and a small R costs little (N is R, M stays 128).
//
// The key scale multiplies the scores, the value scale is folded into the weights (its
// logarithm added to the score, so that no weight exceeds the reference); the sum of the
// softmax takes it out again. The reference m of a query row only moves when a score
// passes it by 2^4 (the accumulators are then rescaled), or with the first keys a row sees:
// most tiles need no exchange between threads but one vote.
//
// A persistent CTA per SM takes an equal share of all (row, head, query tile, key tile)
// units in order; a query tile that crosses from one CTA to the next leaves partial
// results (output, m, sum) in the workspace, and the last of its CTAs to arrive joins them.
// Warps coupled by mbarriers: one copies K and V tiles page by page by tensor-map TMA
// (128-byte swizzle) into a ring; one issues the scores' products and one the output's; one
// plans the next query tile; sixteen form the weights, four to a group, the groups taking
// eight query rows each in turn.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <mutex>

#include "sv_kv.cuh"

namespace sv {

constexpr int AT_KEYS = 128;     // tokens per key tile
constexpr int AT_GROUPS = 4;     // groups of four warps that form the weights
constexpr int AT_SM_WARPS = 4 * AT_GROUPS;
constexpr int AT_THREADS = 32 * (4 + AT_SM_WARPS);  // and copies, scores, planning, outputs
constexpr int AT_SM0 = 128;      // first of their threads
constexpr int AT_SM_THREADS = 32 * AT_SM_WARPS;
constexpr int AT_BLK = AT_KEYS * 128;  // 128 tokens x 128 bytes
constexpr int AT_MAX_STAGES = 6;
constexpr int AT_PTERMS = 3;
// Weights are kept as 2^(x - m + 11): up to 2^15 before the reference must move (below
// e5m2's 57344). Their terms end at 2^-16, e5m2's smallest, so a weight has its 9 bits down
// to 2^-19 of the reference and counts down to 2^-28. A larger shift would leave less room
// for later maxima and move references in more tiles.
constexpr float AT_SHIFT = 11.f, AT_LIMIT = 15.f;

// Instruction descriptors of kind::f8f6f4 (float32 accumulator, M = 128), without N.
// Scores: A and B e4m3, K-major. Output: A e4m3 and B e5m2, both MN-major.
constexpr uint32_t AT_IDESC_S = (1u << 4) | (8u << 24);
constexpr uint32_t AT_IDESC_O = (1u << 4) | (1u << 10) | (1u << 15) | (1u << 16) | (8u << 24);

// Descriptors are given as their low words (address and the unused leading offset) with the
// constant high words of the operand's layout.
__device__ __forceinline__ void umma_f8(uint32_t d, uint32_t alo, uint32_t ahi, uint32_t blo,
                                        uint32_t bhi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %2};\n\t"
      "mov.b64 b, {%3, %4};\n\tsetp.ne.u32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t}" ::"r"(d),
      "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(accumulate)
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
// Two float32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// Eight consecutive float32 columns of this thread's lane; complete after tm_wait_ld.
__device__ __forceinline__ void tm_ld8(uint32_t addr, float* v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                 "=f"(v[6]), "=f"(v[7])
               : "r"(addr));
}
__device__ __forceinline__ void tm_st8(uint32_t addr, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
                   addr),
               "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]),
               "f"(v[7])
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

// Shared-memory matrix descriptor of a swizzled operand whose 8-row groups (K-major: rows;
// MN-major: steps of K) are `group` bytes apart; rows of 128, 64 or 32 bytes (mode 2, 4, 6).
// One swizzle atom covers the other dimension, so the leading offset is not used.
__device__ __forceinline__ uint32_t at_desc_lo(uint32_t addr) {
  return ((addr >> 4) & 0x3fffu) | (1u << 16);
}
__host__ __device__ constexpr uint32_t at_desc_hi(uint32_t group, uint32_t mode) {
  return (group >> 4) | (1u << 14) | (mode << 29);
}

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
__device__ __forceinline__ bool at_try(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity), "r"(2000u)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
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
  int rt;      // most query rows of a tile
  int width;   // columns of an accumulator: 32, 64 or 128
  int stages;  // K + V tiles in the ring
  int ndb;     // 128-byte blocks of a token's vector
  int qterms;  // e4m3 terms of a query
  int bf16;
};

// Row b of the batch.
struct AtRow {
  int len, n;    // cached and new tokens; n = 0 when the row's data is wrong
  int rows;      // query rows of a head
  int nrt, rr;   // query tiles, rows of each (the last may have fewer)
  bool bad;
};

__device__ __forceinline__ AtRow at_row(const AttendArgs& A, const AttendPlan& P, int b) {
  AtRow r;
  r.len = __ldg(A.C.len + b);
  r.n = A.n_new ? __ldg(A.n_new + b) : A.T;
  r.bad = r.n < 0 || r.n > A.T || r.len < 0 ||
          (long long)r.len + r.n > (long long)A.C.max_pages << A.C.lgp;
  if (r.bad) r.n = 0;
  r.rows = r.n * A.group;
  r.nrt = (r.rows + P.rt - 1) / P.rt;
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
  const int t0 = t.r0 / A.group, t1 = (t.r1 - 1) / A.group;
  t.pos_lo = A.parent ? r.len : r.len + t0;
  t.pos_hi = A.parent ? r.len + r.n - 1 : r.len + t1;
  t.end = t.pos_hi + 1;
  t.hi = (t.end + AT_KEYS - 1) / AT_KEYS;
  t.lo = 0;
  t.ns = 0;
  if (A.window) {
    t.lo = max(0, t.pos_lo - A.window + 1) / AT_KEYS;
    t.ns = min((min(A.sinks, t.end) + AT_KEYS - 1) / AT_KEYS, t.lo);
  }
  return t;
}

// Work is counted in key tiles, with AT_EXTRA more for each query tile: what its queries'
// conversion and its results cost.
constexpr int AT_EXTRA = 2;

__device__ __forceinline__ long long at_head_units(const AttendArgs& A, const AtRow& r) {
  long long c = 0;
  for (int rt = 0; rt < r.nrt; ++rt) c += AT_EXTRA + at_tile(A, r, rt).tiles();
  return c;
}

// The units of this CTA, one query tile after the other: key tiles i0 .. i1 - 1 of the
// current one. Every role walks the same sequence.
struct AtWalk {
  int b, h, rt;
  AtRow row;
  AtTile tile;
  int i0, i1;
  long long base, at, end;  // first unit of the query tile, of the share in it, share's end

  // The share of the current query tile; false when it has no key tile.
  __device__ __forceinline__ bool settle() {
    const long long stop = min(end, base + AT_EXTRA + tile.tiles());
    i0 = max(0, static_cast<int>(at - base) - AT_EXTRA);
    i1 = max(0, static_cast<int>(stop - base) - AT_EXTRA);
    return i1 > i0;
  }
  // From row b0, unit `rem` of it.
  __device__ void start(const AttendArgs& A, const AttendPlan& P, int b0, long long rem,
                        long long from, long long to) {
    b = b0;
    at = from;
    end = to;
    if (at >= end) return;
    row = at_row(A, P, b);
    const long long per = at_head_units(A, row);
    h = static_cast<int>(rem / per);
    rem -= h * per;
    rt = 0;
    tile = at_tile(A, row, 0);
    while (rem >= AT_EXTRA + tile.tiles()) {
      rem -= AT_EXTRA + tile.tiles();
      tile = at_tile(A, row, ++rt);
    }
    base = from - rem;
    if (!settle()) next(A, P);
  }
  __device__ __forceinline__ bool live() const { return at < end; }
  __device__ void next(const AttendArgs& A, const AttendPlan& P) {
    do {
      base += AT_EXTRA + tile.tiles();
      at = base;
      if (at >= end) return;
      if (++rt == row.nrt) {
        rt = 0;
        if (++h == A.C.heads) {
          h = 0;
          do {  // (a row with queries exists: units are left)
            row = at_row(A, P, ++b);
          } while (row.rows == 0);
        }
      }
      tile = at_tile(A, row, rt);
    } while (!settle());
  }
};

// A query tile's share as the product and weight warps read it from shared memory.
struct AtItem {
  int b, h, len, n;
  int r0, R;        // query rows r0 .. r0 + R - 1 of the head
  int i0, m;        // key tiles i0 .. i0 + m - 1 (m = 0: no more work)
  int tiles;        // of the query tile
  int end, pos_hi;  // as AtTile
  int ns, lo;
  long long u0;     // unit of its first key tile
  __device__ __forceinline__ int key_tile(int i) const { return i < ns ? i : lo + i - ns; }
};

// Sums of C values over the 32 lanes (C a power of two up to 32): lane c (mod C) gets
// column c's, by halving the columns a lane is responsible for at each exchange.
template <int C>
__device__ __forceinline__ float at_lane_sums(float* v, int lane) {
#pragma unroll
  for (int s = C / 2; s >= 1; s >>= 1) {
    const bool up = (lane & s) != 0;
#pragma unroll
    for (int i = 0; i < s; ++i) {
      const float keep = up ? v[i + s] : v[i], give = up ? v[i] : v[i + s];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, s);
    }
  }
  float x = v[0];
#pragma unroll
  for (int s = C; s < 32; s <<= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
  return x;
}

__device__ __forceinline__ void at_store(void* out, long long at, float y, int bf16) {
  if (bf16)
    static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(y);
  else
    static_cast<__half*>(out)[at] = __float2half_rn(y);
}

// A float as an integer of the same order, and back.
__device__ __forceinline__ int at_order(float x) {
  const int i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float at_unorder(int i) {
  return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}

// After a wait gave up, products already issued must end before the accumulators are freed.
__device__ __forceinline__ void at_drain(uint64_t* bar, bool abort) {
  if (!abort) return;
  umma_commit(bar);
  const long long t0 = clock64();
  while (!mbar_test(bar, 0))
    if (clock64() - t0 > WAIT_CYCLES / 8) break;
}

// W: columns of an accumulator (query rows), bytes of a token's weights.
template <int W>
__global__ void __launch_bounds__(AT_THREADS, 1)
    kv_attend_kernel(const AttendArgs A, const AttendPlan P,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV) {
  constexpr int SLOTS = W / 8 / AT_GROUPS;  // eights of columns of a thread, at most
  constexpr uint32_t PMODE = W == 128 ? 2 : (W == 64 ? 4 : 6);
  constexpr int PBLK = AT_KEYS * W;
  constexpr uint32_t HI128 = at_desc_hi(1024, 2), HIP = at_desc_hi(8 * W, PMODE);
  extern __shared__ unsigned char dsm_raw[];
  __shared__ uint64_t kfull[AT_MAX_STAGES], kempty[AT_MAX_STAGES];
  __shared__ uint64_t vfull[AT_MAX_STAGES], vempty[AT_MAX_STAGES];
  __shared__ uint64_t sfull[2], sempty[2], pfull, pvdone, qfull, drain[2];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ int s_b0, s_last;
  __shared__ int s_vnan[2][AT_KEYS];
  __shared__ AtItem s_item[2];  // of item k at k & 1
  __shared__ long long s_rem, s_sum[AT_THREADS / 32];
  // Per stage and page of the tile: key scale, log2 and inverse of the value scale.
  __shared__ float s_ks[AT_MAX_STAGES][8], s_lv[AT_MAX_STAGES][8], s_iv[AT_MAX_STAGES][8];
  __shared__ __align__(16) float s_c[W];    // per column: factor of the score
  __shared__ __align__(16) float s_nm[W];   // and 11 - reference
  __shared__ __align__(16) float2 s_mv[W];  // a reference's move and the factor it brings
  __shared__ float s_inv[W];                // inverse sum
  __shared__ int s_mx[4][W];
  __shared__ float s_l[4][W];
  __shared__ int s_pos[W];                  // position of the column's query
  __shared__ unsigned long long s_see[W];   // block nodes it sees (trees)
  __shared__ long long s_out[W];            // its row of the output, -1: none
  __shared__ int s_par[SV_MAX_TREE];

  unsigned char* dsm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(dsm_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const KvCache& C = A.C;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int ndb = P.ndb, NT = P.stages;
  unsigned char* Qs = dsm;                                       // [terms][ndb][W][128]
  unsigned char* Ps = Qs + (size_t)P.qterms * ndb * W * 128;     // [terms][128 tokens][W]
  unsigned char* ring = Ps + AT_PTERMS * PBLK;                   // [stages][K, V][ndb][128][128]
  const int slot = ndb * AT_BLK;
  auto kbuf = [&](int q) { return ring + (size_t)q * 2 * slot; };
  auto vbuf = [&](int q) { return ring + (size_t)q * 2 * slot + slot; };

  // Bounded wait: false (and a report) when it runs out or another one has.
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_test(bar, parity)) return true;
    const long long t0 = clock64();
    while (!at_try(bar, parity)) {
      if (s_abort) return false;
      if (clock64() - t0 > WAIT_CYCLES) {
        s_abort = 1;
        kv_report(A.S.hdr, ST_TIMEOUT);
        return false;
      }
    }
    return true;
  };

  if (tid == 0) {
    for (int q = 0; q < NT; ++q) {
      mbar_init(&kfull[q], 1);
      mbar_init(&kempty[q], 1);
      mbar_init(&vfull[q], 1);
      mbar_init(&vempty[q], 1);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(&sfull[q], 1);
      mbar_init(&sempty[q], AT_SM_WARPS);
    }
    mbar_init(&pfull, AT_SM_WARPS);
    mbar_init(&qfull, AT_SM_WARPS);
    mbar_init(&pvdone, 1);
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    s_abort = 0;
    fence_mbar_init();
  }
  if (w == 1) {
    const uint32_t need = (2 + ndb) * W, cols = need <= 128 ? 128 : (need <= 256 ? 256 : 512);
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&s_tmem)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // This CTA's share: the units of all rows, cut into equal parts. Rows are counted by the
  // threads in turn; the second pass finds the row where the share begins.
  long long total = 0, mine0 = 0;
  for (int b = tid; b < C.batch; b += AT_THREADS) {
    const AtRow r = at_row(A, P, b);
    const long long c = at_head_units(A, r) * C.heads;
    if (b == tid) mine0 = c;
    total += c;
  }
  auto block_sum = [&](long long x, long long* before) {  // sum; *before: of lower threads
    long long v = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += t;
    }
    if (lane == 31) s_sum[w] = v;
    __syncthreads();
    long long sum = 0, pre = 0;
    for (int i = 0; i < AT_THREADS / 32; ++i) {
      if (i < w) pre += s_sum[i];
      sum += s_sum[i];
    }
    __syncthreads();
    *before = pre + v - x;
    return sum;
  };
  long long before;
  total = block_sum(total, &before);
  const long long ctas = min((long long)gridDim.x, total);
  const long long cta = blockIdx.x;
  const long long from = cta < ctas ? cta * total / ctas : 0;
  const long long to = cta < ctas ? (cta + 1) * total / ctas : 0;
  if (from < to) {
    long long base = 0;
    for (int b0 = 0; b0 < C.batch; b0 += AT_THREADS) {
      const int b = b0 + tid;
      const long long c =
          b >= C.batch ? 0 : (b0 == 0 ? mine0 : at_head_units(A, at_row(A, P, b)) * C.heads);
      const long long sum = block_sum(c, &before);
      if (from >= base + before && from < base + before + c) {
        s_b0 = b;
        s_rem = from - base - before;
      }
      base += sum;
      if (base > from) break;
    }
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tmem = s_tmem;
  if (w == 0) {
    AtWalk walk;
    walk.start(A, P, s_b0, s_rem, from, to);
    // ---- Copies: pages of one or more tiles are looked up at a time, a page per lane and
    // a step ahead of their use.
    const int ppt = AT_KEYS >> C.lgp;  // pages per tile
    const int tpc = 32 / ppt;          // tiles per step
    const size_t layer0 = (size_t)A.layer * C.pages;
    int b = 0, h = 0, n = 0, page = -1;  // the step in hand: row, head, tiles; its page
    bool used = false;
    float ks = 1.f, vs = 1.f;
    int nb = 0, nh = 0, nn = 0, npage = -1;  // the step ahead
    bool nused = false;
    int i = walk.live() ? walk.i0 : 0;
    auto look = [&]() {  // the next step's pages
      nn = 0;
      if (!walk.live()) return;
      nb = walk.b;
      nh = walk.h;
      nn = min(tpc, walk.i1 - i);
      const int mt = lane / ppt;
      const int key = (mt < nn ? walk.tile.key_tile(i + mt) : 0) * AT_KEYS +
                      ((lane - mt * ppt) << C.lgp);
      nused = mt < nn && key < walk.tile.end;
      npage = nused ? kv_page(C, nb, key) : -1;
      i += nn;
      if (i == walk.i1) {
        walk.next(A, P);
        i = walk.live() ? walk.i0 : 0;
      }
    };
    auto scales = [&](int pg, bool use, int head, float* k, float* v) {
      *k = *v = 1.f;
      if (!use) return;
      if (pg >= 0) {
        *k = __ldg(C.ks + (layer0 + pg) * C.heads + head);
        *v = __ldg(C.vs + (layer0 + pg) * C.heads + head);
      }
      // A page out of range, or scales outside theirs: the scores become NaN.
      constexpr float LO = 5.421010862427522e-20f, HI = 18446744073709551616.f;  // 2^-64, 2^64
      if (pg < 0 || !(*k >= LO && *k <= HI && *v >= LO && *v <= HI)) {
        *k = NAN;
        *v = 1.f;
        kv_report(A.S.hdr, ST_DEVICE_INPUT);
      }
    };
    look();
    bool ok = true;
    int g = 0, q = 0, ph = 0;  // tile, its stage, the stage's pass
    float nks, nvs;
    scales(npage, nused, nh, &nks, &nvs);
    while (ok && nn) {
      b = nb; h = nh; n = nn; page = npage; used = nused; ks = nks; vs = nvs;
      look();
      for (int t = 0; t < n; ++t, ++g) {
        const bool mine = lane >= t * ppt && lane < (t + 1) * ppt;
        const int sub = lane - t * ppt;
        const uint32_t count = __popc(__ballot_sync(0xffffffffu, mine && page >= 0));
        const uint32_t bytes = (count << C.lgp) * 128u * ndb;
        for (int kv = 0; kv < 2; ++kv) {
          uint64_t* full = kv ? &vfull[q] : &kfull[q];
          uint64_t* empty = kv ? &vempty[q] : &kempty[q];
          bool go = true;
          if (ph > 0) go = wait(empty, (ph - 1) & 1);
          if (!__all_sync(0xffffffffu, go)) {
            ok = false;
            break;
          }
          if (kv == 1 && mine) {
            s_ks[q][sub] = ks;
            s_lv[q][sub] = log2f(vs);
            s_iv[q][sub] = 1.f / vs;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(full, bytes);
          __syncwarp();
          if (mine && page >= 0) {
            unsigned char* dst = (kv ? vbuf(q) : kbuf(q)) + ((size_t)sub << C.lgp) * 128;
            const int y = (page * C.heads + h) << C.lgp;
            for (int db = 0; db < ndb; ++db)
              at_tma(dst + db * AT_BLK, kv ? &tmV : &tmK, db * 128, y, full);
          }
        }
        if (!ok) break;
        if (t == 0) scales(npage, nused, nh, &nks, &nvs);
        if (++q == NT) {
          q = 0;
          ++ph;
        }
      }
    }
    if (!ok) {
      // After a wait gave up: let the copies already issued land before the CTA exits. (A
      // stage's barrier whose last pass was consumed answers at once.)
      for (int j = max(0, g - NT); j <= g; ++j) {
        const long long t0 = clock64();
        const uint32_t par = static_cast<uint32_t>((j / NT) & 1);
        while (!(mbar_test(&kfull[j % NT], par) && (j == g || mbar_test(&vfull[j % NT], par))))
          if (clock64() - t0 > WAIT_CYCLES / 8) break;
      }
    }
  } else if (w == 1) {
    // ---- Scores: S^T of a tile into one of two accumulators.
    if (at_elect()) {
      const int ksteps = (C.dim + 31) / 32;
      const uint32_t qd = at_desc_lo(smem_addr(Qs)), ring0 = at_desc_lo(smem_addr(ring));
      const uint32_t rstep = static_cast<uint32_t>(2 * slot) >> 4;
      bool ok = true;
      int g = 0, q = 0, ph = 0;
      for (int item = 0; ok; ++item) {
        if (!wait(&qfull, item & 1)) break;
        const int R = s_item[item & 1].R, m = s_item[item & 1].m;
        if (m == 0) break;
        const uint32_t ids = AT_IDESC_S | (static_cast<uint32_t>((R + 15) >> 4) << 18);
        for (int i = 0; i < m; ++i, ++g) {
          if (!wait(&kfull[q], ph & 1) || (g >= 2 && !wait(&sempty[g & 1], ((g >> 1) - 1) & 1))) {
            ok = false;
            break;
          }
          tm_fence_after();
          const uint32_t d = tmem + (g & 1) * W, ka = ring0 + q * rstep;
          uint32_t acc = 0;
          for (int t = 0; t < P.qterms; ++t)
            for (int db = 0; db < ndb; ++db) {
              const uint32_t al = ka + db * (AT_BLK >> 4), bl = qd + (t * ndb + db) * (W * 8);
              const int kn = ksteps - 4 * db;
              if (kn >= 4) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  umma_f8(d, al + 2 * k, HI128, bl + 2 * k, HI128, ids, k ? 1u : acc);
              } else {
                for (int k = 0; k < kn; ++k)
                  umma_f8(d, al + 2 * k, HI128, bl + 2 * k, HI128, ids, k ? 1u : acc);
              }
              acc = 1;
            }
          umma_commit(&sfull[g & 1]);
          umma_commit(&kempty[q]);
          if (++q == NT) {
            q = 0;
            ++ph;
          }
        }
      }
      at_drain(&drain[0], s_abort);
    }
  } else if (w == 3) {
    // ---- Outputs: O^T += V^T P^T of a tile, while the next tile's scores multiply and its
    // weights form.
    if (at_elect()) {
      const uint32_t pd = at_desc_lo(smem_addr(Ps)), ring0 = at_desc_lo(smem_addr(ring)) + (slot >> 4);
      const uint32_t rstep = static_cast<uint32_t>(2 * slot) >> 4;
      bool ok = true;
      int g = 0, q = 0, ph = 0;
      for (int item = 0; ok; ++item) {
        if (!wait(&qfull, item & 1)) break;
        const int R = s_item[item & 1].R, m = s_item[item & 1].m;
        if (m == 0) break;
        const uint32_t ido = AT_IDESC_O | (static_cast<uint32_t>((R + 15) >> 4) << 18);
        for (int i = 0; i < m; ++i, ++g) {
          if (!wait(&vfull[q], ph & 1) || !wait(&pfull, g & 1)) {
            ok = false;
            break;
          }
          tm_fence_after();
          for (int db = 0; db < ndb; ++db) {
            const uint32_t d = tmem + (2 + db) * W, va = ring0 + q * rstep + db * (AT_BLK >> 4);
            const uint32_t acc = i > 0;
#pragma unroll
            for (int t = 0; t < AT_PTERMS; ++t)
#pragma unroll
              for (int k = 0; k < AT_KEYS / 32; ++k)
                umma_f8(d, va + k * (4096 >> 4), HI128, pd + ((t * PBLK + k * 32 * W) >> 4), HIP, ido,
                        t + k ? 1u : acc);
          }
          umma_commit(&pvdone);
          umma_commit(&vempty[q]);
          if (++q == NT) {
            q = 0;
            ++ph;
          }
        }
      }
      at_drain(&drain[1], s_abort);
    }
  } else if (w == 2) {
    // ---- Planning: item k + 1 while item k is in work.
    AtWalk walk;
    walk.start(A, P, s_b0, s_rem, from, to);
    for (int k = 0;; ++k) {
      const bool live = walk.live();
      if (lane == 0) {
        AtItem& o = s_item[k & 1];
        o.m = live ? walk.i1 - walk.i0 : 0;
        o.b = walk.b;
        o.h = walk.h;
        o.len = walk.row.len;
        o.n = walk.row.n;
        o.r0 = walk.tile.r0;
        o.R = walk.tile.r1 - walk.tile.r0;
        o.i0 = walk.i0;
        o.tiles = walk.tile.tiles();
        o.end = walk.tile.end;
        o.pos_hi = walk.tile.pos_hi;
        o.ns = walk.tile.ns;
        o.lo = walk.tile.lo;
        o.u0 = walk.base + AT_EXTRA;
      }
      __syncwarp();
      at_bar(6, AT_SM_THREADS + 32);  // item k is there, item k - 1 done with
      if (!live) break;
      walk.next(A, P);
    }
  } else {
    // ---- Weights and results.
    const int sw = w - 4, quad = w & 3, grp = sw >> 2;  // lanes 32 quad ..; eights of columns
    const int st = tid - AT_SM0;
    const int tok = quad * 32 + lane;  // token of a tile; component of the output
    const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    // Queries without a token and rows with wrong data: zeros or NaN.
    for (long long u0 = (long long)blockIdx.x * AT_SM_WARPS + sw; u0 * 32 < (long long)C.batch * A.T;
         u0 += (long long)gridDim.x * AT_SM_WARPS) {
      const long long u = u0 * 32 + lane;
      int fill = 0;
      if (u < (long long)C.batch * A.T) {
        const int b = static_cast<int>(u / A.T), t = static_cast<int>(u - (long long)b * A.T);
        const AtRow r = at_row(A, P, b);
        fill = r.bad ? 2 : (t >= r.n ? 1 : 0);
        if (r.bad && t == 0) kv_report(A.S.hdr, ST_DEVICE_INPUT);
      }
      unsigned todo = __ballot_sync(0xffffffffu, fill != 0);
      while (todo) {
        const int j = __ffs(todo) - 1;
        todo &= todo - 1;
        const bool nan = __shfl_sync(0xffffffffu, fill, j) == 2;
        const long long row = (u0 * 32 + j) * A.q_heads;
        const uint32_t x = nan ? 0x7fff7fffu : 0u;  // NaN in bf16 and fp16
        uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(A.out) + row * C.dim);
        for (int e = lane; e < A.q_heads * C.dim / 8; e += 32) o[e] = make_uint4(x, x, x, x);
        if (A.lse)
          for (int e = lane; e < A.q_heads; e += 32) A.lse[row + e] = nan ? NAN : -INFINITY;
      }
    }
    bool dead = false;  // a wait gave up: skip the work, keep meeting the other warps
    int g = 0, q = 0, ph = 0;
    for (int item = 0;; ++item) {
      // Every warp is done with the last query tile.
      at_bar(6, AT_SM_THREADS + 32);
      const AtItem& it = s_item[item & 1];
      const int R = it.R, m = it.m, len = it.len, N = (R + 15) & ~15;
      if (m == 0) {
        if (lane == 0) mbar_arrive(&qfull);  // the product warp sees it too
        break;
      }
      // Columns of this thread: eights grp, grp + 4, ...; `mine` of them have a row.
      const int mine = max(0, (((R + 7) >> 3) - grp + AT_GROUPS - 1) / AT_GROUPS);
      auto col0 = [&](int slot) { return (grp + AT_GROUPS * slot) * 8; };
      // -- The queries, and what the columns stand for.
      bool badtree = false;
      if (A.parent) {
        if (st < it.n) {
          const int p = __ldg(A.parent + (size_t)it.b * A.T + st);
          badtree = st > 0 && (p < 0 || p >= st);
          s_par[st] = p;
        }
        badtree = at_vote(5, AT_SM_THREADS, badtree);
        if (badtree && st == 0) kv_report(A.S.hdr, ST_DEVICE_INPUT);
      }
      if (st < N) {
        int pos = -1;
        unsigned long long see = badtree ? ~0ull : 0ull;  // (a bad tree's scores are NaN)
        long long out = -1;
        if (st < R) {
          const int t = (it.r0 + st) / A.group, gh = it.r0 + st - t * A.group;
          pos = len + t;
          out = ((long long)it.b * A.T + t) * A.q_heads + it.h * A.group + gh;
          if (A.parent && !badtree) {
            int up = 0;
            for (int i = t;; i = s_par[i]) {
              if (!A.window || up < A.window || len + i < A.sinks) see |= 1ull << i;
              if (i == 0) break;
              ++up;
            }
            pos = len + up;
          }
        }
        s_pos[st] = pos;
        s_see[st] = see;
        s_out[st] = out;
      }
      for (int col = sw * 2 + (lane >> 4); col < N; col += 2 * AT_SM_WARPS) {
        const int l16 = lane & 15;
        float f[2][8];
        float a = 0.f;
        const uint16_t* src = nullptr;
        if (col < R) {
          const int t = (it.r0 + col) / A.group, gh = it.r0 + col - t * A.group;
          src = static_cast<const uint16_t*>(A.q) + it.b * A.q_row + t * A.q_tok +
                (size_t)(it.h * A.group + gh) * C.dim;
        }
#pragma unroll
        for (int db = 0; db < 2; ++db) {
          const int d = db * 128 + l16 * 8;
          uint4 x = make_uint4(0, 0, 0, 0);
          if (src && d < C.dim) x = __ldg(reinterpret_cast<const uint4*>(src + d));
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (P.bf16) {
              f[db][2 * e] = bf_lo(xw[e]);
              f[db][2 * e + 1] = bf_hi(xw[e]);
            } else {
              const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&xw[e]));
              f[db][2 * e] = y.x;
              f[db][2 * e + 1] = y.y;
            }
            a = fmaxf(a, fmaxf(fabsf(f[db][2 * e]), fabsf(f[db][2 * e + 1])));
          }
        }
#pragma unroll
        for (int s = 8; s; s >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, s));
        const float sc = kv_scale(a), inv = 1.f / sc;
        if (l16 == 0) {
          // (An infinite component makes the scores NaN, as the saturating terms would
          // not; a column without a row keeps weight 0 under any reference.)
          const bool nan = badtree || a == INFINITY;
          s_c[col] = col >= R ? 0.f : (nan ? NAN : sc * A.scale);
          s_nm[col] = col >= R ? -3.0e38f : 0.f;
        }
#pragma unroll
        for (int db = 0; db < 2; ++db) {
          if (db >= ndb) break;
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = f[db][e] * inv;
          unsigned char* dst = Qs + (size_t)db * W * 128 + col * 128 +
                               (((l16 >> 1) ^ (col & 7)) << 4) + (l16 & 1) * 8;
          for (int t = 0; t < P.qterms; ++t) {
            uint2 o;
            o.x = e4m3x4(y[0], y[1], y[2], y[3]);
            o.y = e4m3x4(y[4], y[5], y[6], y[7]);
            *reinterpret_cast<uint2*>(dst + (size_t)t * ndb * W * 128) = o;
            const uint32_t ow[2] = {o.x, o.y};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 lo = e4m3_to_f2(ow[e] & 0xffffu), hi = e4m3_to_f2(ow[e] >> 16);
              y[4 * e] -= lo.x;
              y[4 * e + 1] -= lo.y;
              y[4 * e + 2] -= hi.x;
              y[4 * e + 3] -= hi.y;
            }
          }
        }
      }
      fence_async();
      at_bar(5, AT_SM_THREADS);
      if (lane == 0) mbar_arrive(&qfull);
      float l[8 * SLOTS];
#pragma unroll
      for (int c = 0; c < 8 * SLOTS; ++c) l[c] = 0.f;
      // Thread j of a group keeps the state of its column j: has its query seen a key?
      const int j = st & 127, jcol = col0(j >> 3) + (j & 7);
      const bool jreal = j < 8 * SLOTS && jcol < R;
      bool unseen = jreal, any_unseen = mine > 0;

      // -- Key tiles.
      for (int i = 0; i < m; ++i, ++g) {
        const int key0 = it.key_tile(it.i0 + i) * AT_KEYS, key = key0 + tok;
        // (The page scales are written before V's barrier is armed.)
        if (!dead && !(wait(&vfull[q], ph & 1) && wait(&sfull[g & 1], (g >> 1) & 1))) dead = true;
        tm_fence_after();
        const int sub = tok >> C.lgp;
        const float ks = s_ks[q][sub], lv = s_lv[q][sub], iv = s_iv[q][sub];
        const uint32_t sa = tl + (g & 1) * W;
        // Is there a key of the tile that some query does not see? Then also look after the
        // values that weight 0 would not hide: tokens past the end (whatever the page
        // holds) are zeroed, and a NaN is zeroed where it stands and made the weight of the
        // queries that do see it.
        const bool cut = key0 + AT_KEYS > len ||
                         (A.window && key0 < it.pos_hi - A.window + 1 && key0 + AT_KEYS > A.sinks);
        bool vnan = false;
        if (cut) {
          // A group looks at two of a token's eight 16-byte chunks, turned so that the lanes
          // of a warp spread over the banks.
          if (grp == 0) s_vnan[g & 1][tok] = 0;
          at_bar(5, AT_SM_THREADS);
          for (int db = 0; db < ndb && !dead; ++db) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint4* p = reinterpret_cast<uint4*>(vbuf(q) + db * AT_BLK + tok * 128) +
                         ((2 * grp + e + tok) & 7);
              if (key >= it.end) {
                *p = make_uint4(0, 0, 0, 0);
                continue;
              }
              uint4 y = *p;
              const uint4 z = make_uint4(
                  __vcmpeq4(y.x & 0x7f7f7f7fu, 0x7f7f7f7fu), __vcmpeq4(y.y & 0x7f7f7f7fu, 0x7f7f7f7fu),
                  __vcmpeq4(y.z & 0x7f7f7f7fu, 0x7f7f7f7fu), __vcmpeq4(y.w & 0x7f7f7f7fu, 0x7f7f7f7fu));
              if (z.x | z.y | z.z | z.w) {
                s_vnan[g & 1][tok] = 1;
                *p = make_uint4(y.x & ~z.x, y.y & ~z.y, y.z & ~z.z, y.w & ~z.w);
              }
            }
          }
          at_bar(5, AT_SM_THREADS);
          vnan = s_vnan[g & 1][tok] != 0;
        }
        // Columns of slots s0 .. s0 + XS - 1, as the accumulator has them, and as logarithms of
        // their weights. All of a thread's columns stay in registers when they are few; else
        // (W = 128) each use takes them from the accumulator again, which costs less than
        // registers that spill.
        constexpr int XS = SLOTS < 2 ? SLOTS : 2;
        float x[8 * XS];
        auto fetch = [&](int s0) {
#pragma unroll
          for (int s = 0; s < XS; ++s)
            if (s0 + s < mine) tm_ld8(sa + col0(s0 + s), x + 8 * s);
          tm_wait_ld<8 * XS>(x);
#pragma unroll
          for (int s = 0; s < XS; ++s) {
            if (s0 + s >= mine) continue;
            const int c0 = col0(s0 + s);
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
              const float4 cf = *reinterpret_cast<const float4*>(&s_c[c0 + e]);
              const float4 nm = *reinterpret_cast<const float4*>(&s_nm[c0 + e]);
              float* y = x + 8 * s + e;
              const float2 ks2 = make_float2(ks, ks), lv2 = make_float2(lv, lv);
              const float2 u = fma2(make_float2(y[0], y[1]), mul2(make_float2(cf.x, cf.y), ks2),
                                    add2(make_float2(nm.x, nm.y), lv2));
              const float2 v = fma2(make_float2(y[2], y[3]), mul2(make_float2(cf.z, cf.w), ks2),
                                    add2(make_float2(nm.z, nm.w), lv2));
              y[0] = u.x;
              y[1] = u.y;
              y[2] = v.x;
              y[3] = v.y;
            }
            if (cut) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int pos = s_pos[c0 + e];
                bool see = !A.window || pos - key < A.window || key < A.sinks;
                if (key >= len) {
                  const int o = key - len;
                  see = A.parent ? o < it.n && ((s_see[c0 + e] >> (o & 63)) & 1) != 0
                                 : see && key <= pos;
                }
                x[8 * s + e] = !see ? -INFINITY : (vnan ? NAN : x[8 * s + e]);
              }
            }
          }
        };
        float top = -INFINITY;
#pragma unroll
        for (int s0 = 0; s0 < SLOTS; s0 += XS) {
          if (s0 >= mine) continue;
          fetch(s0);
#pragma unroll
          for (int e = 0; e < 8 * XS; ++e)
            if (s0 + e / 8 < mine) top = fmaxf(top, x[e]);
        }
        if (mine && at_vote(1 + grp, 128, any_unseen || top > AT_LIMIT)) {
          // Move references to the tile's largest scores: maximum over the lanes, then over
          // the four warps; the outputs and sums so far shrink by the difference.
#pragma unroll
          for (int s0 = 0; s0 < SLOTS; s0 += XS) {
            if (s0 >= mine) continue;
            if (SLOTS > XS) fetch(s0);
#pragma unroll
            for (int e = 0; e < 8 * XS; ++e) {
              if (s0 + e / 8 >= mine) continue;
              const int o = __reduce_max_sync(0xffffffffu, at_order(x[e]));
              if (lane == (e & 7)) s_mx[quad][col0(s0 + e / 8) + (e & 7)] = o;
            }
          }
          at_bar(1 + grp, 128);
          if (jreal) {
            int o = max(s_mx[0][jcol], s_mx[1][jcol]);
            o = max(o, max(s_mx[2][jcol], s_mx[3][jcol]));
            const float d = at_unorder(o);  // over the reference - 11
            float move = 0.f, fac = 1.f;
            if (unseen) {  // nothing to shrink: the reference goes wherever the scores are
              if (d > -INFINITY) move = d - AT_SHIFT;
              unseen = d == -INFINITY;
            } else if (d > AT_SHIFT) {
              move = d - AT_SHIFT;
              fac = exp2f(-move);
            }
            s_mv[jcol] = make_float2(move, fac);
            s_nm[jcol] -= move;
          } else if (j < 8 * SLOTS) {
            s_mv[jcol] = make_float2(0.f, 1.f);
          }
          any_unseen = at_vote(1 + grp, 128, unseen);
          if (i > 0 && !dead && !wait(&pvdone, (g - 1) & 1)) dead = true;
          tm_fence_after();
#pragma unroll
          for (int s = 0; s < SLOTS; ++s) {
            if (s >= mine) continue;
            float fac[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 mv = s_mv[col0(s) + e];
              if (SLOTS == XS) x[8 * (s % XS) + e] -= mv.x;
              fac[e] = mv.y;
              l[8 * s + e] *= mv.y;
            }
            if (i == 0) continue;
            for (int db = 0; db < ndb; ++db) {
              const uint32_t oa = tl + (2 + db) * W + col0(s);
              float o[8];
              tm_ld8(oa, o);
              tm_wait_ld<8>(o);
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] *= fac[e];
              tm_st8(oa, o);
            }
          }
          tm_wait_st();
          tm_fence_before();
        }
        // Weights: 2^x, summed with the value scale taken out, rounded to fp16 and split.
        // A term is the upper byte of the remainder rounded to it (halves away from zero);
        // what is left of an fp16 number after that is exact.
        if (i > 0 && !dead && !wait(&pvdone, (g - 1) & 1)) dead = true;
        unsigned char* prow = Ps + tok * W;
        const int swz = W == 128 ? (tok & 7) : (W == 64 ? (tok >> 1) & 3 : (tok >> 2) & 1);
#pragma unroll
        for (int s0 = 0; s0 < SLOTS; s0 += XS) {
          if (s0 >= mine) continue;
          if (SLOTS > XS) fetch(s0);
#pragma unroll
          for (int s = 0; s < XS; ++s) {
            if (s0 + s >= mine) continue;
            uint32_t t[AT_PTERMS][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int c = 8 * s + 2 * e, k2 = 8 * (s0 + s) + 2 * e;
              const float2 p = make_float2(ex2(x[c]), ex2(x[c + 1]));
              const float2 sum = fma2(p, make_float2(iv, iv), make_float2(l[k2], l[k2 + 1]));
              l[k2] = sum.x;
              l[k2 + 1] = sum.y;
              __half2 r = __floats2half2_rn(p.x, p.y);
#pragma unroll
              for (int k = 0; k < AT_PTERMS; ++k) {
                t[k][e] = *reinterpret_cast<const uint32_t*>(&r) + 0x00800080u;
                const uint32_t hi = t[k][e] & 0xff00ff00u;
                r = __hsub2(r, *reinterpret_cast<const __half2*>(&hi));
              }
            }
            const int c0 = col0(s0 + s);
            unsigned char* dst = prow + (((c0 >> 4) ^ swz) << 4) + (c0 & 8);
#pragma unroll
            for (int k = 0; k < AT_PTERMS; ++k)
              *reinterpret_cast<uint2*>(dst + k * PBLK) =
                  make_uint2(__byte_perm(t[k][0], t[k][1], 0x7531),
                             __byte_perm(t[k][2], t[k][3], 0x7531));
          }
        }
        tm_fence_before();
        fence_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sempty[g & 1]);
          mbar_arrive(&pfull);
        }
        if (++q == NT) {
          q = 0;
          ++ph;
        }
      }

      // -- The query tile's sums and outputs: the result when this CTA saw all its keys,
      // else partial results.
      if (!dead && !wait(&pvdone, (g - 1) & 1)) dead = true;
      tm_fence_after();
      const bool whole = m == it.tiles;
      const int slot_id = 2 * static_cast<int>(cta) + (it.i0 == 0 ? 1 : 0);
      if (mine) {
        constexpr int LC = 8 * SLOTS;
        const float lsum = at_lane_sums<LC>(l, lane);
        if (lane < LC) s_l[quad][col0(lane >> 3) + (lane & 7)] = lsum;
        at_bar(1 + grp, 128);
        if (jreal) {
          const float sum = s_l[0][jcol] + s_l[1][jcol] + s_l[2][jcol] + s_l[3][jcol];
          const float ref = -s_nm[jcol];
          s_inv[jcol] = sum == 0.f ? 0.f : 1.f / sum;
          if (!whole)
            A.S.stat[(size_t)slot_id * KV_ROWS + jcol] = make_float2(ref, sum);
          else if (A.lse)
            A.lse[s_out[jcol]] =
                sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
        }
        at_bar(1 + grp, 128);
        for (int db = 0; db < ndb; ++db) {
          const int d = db * 128 + tok;
#pragma unroll
          for (int s = 0; s < SLOTS; ++s) {
            if (s >= mine) continue;
            const int c0 = col0(s);
            float o[8];
            tm_ld8(tl + (2 + db) * W + c0, o);
            tm_wait_ld<8>(o);
            if (d >= C.dim) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if (c0 + e >= R) continue;
              if (whole) {
                const float inv = s_inv[c0 + e];
                at_store(A.out, s_out[c0 + e] * C.dim + d, inv == 0.f ? 0.f : o[e] * inv, P.bf16);
              } else {
                A.S.part[((size_t)slot_id * KV_ROWS + c0 + e) * C.dim + d] = o[e];
              }
            }
          }
        }
      }
      tm_fence_before();
      if (!whole) {
        // The CTAs that hold this query tile: the first of them keeps the ticket.
        const int first = static_cast<int>(((it.u0 + 1) * ctas - 1) / total);
        const int last = static_cast<int>(((it.u0 + it.tiles) * ctas - 1) / total);
        __threadfence();
        at_bar(5, AT_SM_THREADS);
        if (st == 0) {
          const bool end = atomicAdd(A.S.ticket + first, 1u) == static_cast<uint32_t>(last - first);
          if (end) A.S.ticket[first] = 0;
          s_last = end;
        }
        at_bar(5, AT_SM_THREADS);
        if (s_last) {
          __threadfence();
          const int vec = C.dim / 4;
          for (int e = st; e < R * vec; e += AT_SM_THREADS) {
            const int r = e / vec, dv = e - r * vec;
            auto slot_of = [&](int k) { return (size_t)(2 * k + (k == first ? 1 : 0)) * KV_ROWS + r; };
            float top = -INFINITY;
            for (int k = first; k <= last; ++k) {
              const float2 s2 = __ldcg(A.S.stat + slot_of(k));
              if (s2.y != 0.f) top = fmaxf(top, s2.x);
            }
            float sum = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = first; k <= last; ++k) {
              const float2 s2 = __ldcg(A.S.stat + slot_of(k));
              if (s2.y == 0.f) continue;
              const float f = exp2f(s2.x - top);
              const float4 y =
                  __ldcg(reinterpret_cast<const float4*>(A.S.part + slot_of(k) * C.dim) + dv);
              sum = fmaf(s2.y, f, sum);
              o.x = fmaf(y.x, f, o.x);
              o.y = fmaf(y.y, f, o.y);
              o.z = fmaf(y.z, f, o.z);
              o.w = fmaf(y.w, f, o.w);
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const long long at = s_out[r] * C.dim + dv * 4;
            at_store(A.out, at, o.x * inv, P.bf16);
            at_store(A.out, at + 1, o.y * inv, P.bf16);
            at_store(A.out, at + 2, o.z * inv, P.bf16);
            at_store(A.out, at + 3, o.w * inv, P.bf16);
            if (dv == 0 && A.lse)
              A.lse[s_out[r]] =
                  sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
          }
        }
      }
    }
  }

  tm_fence_before();
  __syncthreads();
  if (w == 1) {
    __syncwarp();
    tm_fence_after();
    const uint32_t need = (2 + ndb) * W, cols = need <= 128 ? 128 : (need <= 256 ? 256 : 512);
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols)
                 : "memory");
  }
}

// The driver's tensor-map encoder, looked up once through the runtime.
static PFN_cuTensorMapEncodeTiled_v12000 at_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    (void)cudaGetLastError();
  });
  return fn;
}

// Shared memory that a kernel may use beside its static arrays (227 KB a CTA).
constexpr size_t AT_SMEM = 232448 - 12288;

cudaError_t launch_kv_attend(const AttendArgs& A, sv_dtype dt, cudaStream_t st) {
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  std::call_once(once, [] {
    const void* ks[3] = {reinterpret_cast<const void*>(kv_attend_kernel<32>),
                         reinterpret_cast<const void*>(kv_attend_kernel<64>),
                         reinterpret_cast<const void*>(kv_attend_kernel<128>)};
    for (int i = 0; i < 3 && attr == cudaSuccess; ++i)
      attr = cudaFuncSetAttribute(ks[i], cudaFuncAttributeMaxDynamicSharedMemorySize, (int)AT_SMEM);
  });
  if (attr != cudaSuccess) return attr;
  const KvCache& C = A.C;
  AttendPlan P;
  P.bf16 = dt == SV_BF16;
  P.qterms = P.bf16 ? 2 : 3;
  P.ndb = C.dim > 128 ? 2 : 1;
  // Above dim 128 the ring's tiles take 64 KB, which leaves room for the queries and weights
  // of 64 rows.
  P.rt = P.ndb == 2 ? 64 : KV_ROWS;
  const long long rows = (long long)A.T * A.group;
  P.width = rows <= 32 ? 32 : (rows <= 64 || P.rt == 64 ? 64 : 128);
  const size_t fixed = 1024 + (size_t)P.qterms * P.ndb * P.width * 128 +
                       (size_t)AT_PTERMS * AT_KEYS * P.width;
  const size_t stage = (size_t)2 * P.ndb * AT_BLK;
  P.stages = (int)((AT_SMEM - fixed) / stage);
  if (P.stages > AT_MAX_STAGES) P.stages = AT_MAX_STAGES;
  const size_t smem = fixed + P.stages * stage;
  // The pools of one layer as matrices [pages * heads * page tokens][dim bytes], in boxes of
  // one page x 128 bytes (128-byte swizzle, zeros past dim).
  PFN_cuTensorMapEncodeTiled_v12000 enc = at_encoder();
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
  int dev = 0, sms = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
    return e;
  const int grid = sms < KV_MAX_CTAS ? sms : KV_MAX_CTAS;
  if (P.width == 32)
    kv_attend_kernel<32><<<grid, AT_THREADS, smem, st>>>(A, P, tm[0], tm[1]);
  else if (P.width == 64)
    kv_attend_kernel<64><<<grid, AT_THREADS, smem, st>>>(A, P, tm[0], tm[1]);
  else
    kv_attend_kernel<128><<<grid, AT_THREADS, smem, st>>>(A, P, tm[0], tm[1]);
  return cudaGetLastError();
}

}  // namespace sv
