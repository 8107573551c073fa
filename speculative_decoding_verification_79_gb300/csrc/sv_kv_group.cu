// sv_kv_group.cu -- attention of large groups of rows to their common tokens (sm_103a).
//
// With 128 queries a key tile the products and weights bound it, not its copy. So the values are
// multiplied as fp16, which holds every e4m3 number exactly: a weight of 11 bits is then one
// operand instead of the three e5m2 terms that 8-bit products need, its product takes two thirds
// of the time (512 cycles instead of 768), and it needs no splitting. Four warps convert V tiles.
// Scores are the same 8-bit products as in sv_kv_attend.cuh (two or three terms of a query), and so
// are the reference that moves late, the value scales' place in the weights, and the partial results.
//
// A step, a key tile, is a chain: scores (520 cycles of products, 1,000 until they are seen),
// weights, outputs (510, 840), and only then the accumulator's next scores, whose place the weights
// had. Three accumulators of scores beside one of outputs keep three steps going. (Two query tiles of
// 128 with two accumulators each, which convert a V tile for both, took 4,400 to 5,800 cycles for a
// key tile of the two, however its warps were divided: a chain is 3,500.)
//
// Bound by that chain: once it runs, a step takes 1,580 cycles (bf16) or 1,730 (fp16, three terms).
// Products keep the tensor cores for 1,030 and 1,290 of them; the weights take 1,200 from scores seen
// to weights stored (their instructions 830 if all warps' were spread evenly), and then wait some
// 400 for the next scores, whose products waited for the outputs of three steps before. Tensor memory
// has no room for a fourth accumulator. 64 rows of 8 queries a head behind 8,100 common tokens (8
// heads, 14 steps a CTA): 30 us. 8 rows of 35 queries a head behind 120,001 (4 heads, 74 steps): 94
// us, 0.73 PFLOP/s. With its start, queries and results that is 2,400 cycles a step.
//
// All of a group's queries see all of its common tokens (no window), so no key is masked, and a NaN
// in the cache reaches all of them by itself: 0 times NaN is NaN.
#include "sv_kv_attend.cuh"

namespace sv {

constexpr int GR_BLK = AT_KEYS * 128 * 2;  // 128 tokens x 128 values of 16 bits
// Weights are kept as 2^(x - m + 4): up to 2^15 before the reference must move, which 11 binades make
// rare (with the 4 that e5m2 terms leave, a quarter of the steps formed their weights twice). fp16
// holds all 11 bits of a weight down to 2^-18 of the reference's, and 2^-28 of it below.
constexpr float GR_SHIFT = 4.f;
constexpr uint32_t AT_IDESC_W = (1u << 4) | (1u << 16) | (8u << 24);  // fp16, B MN-major, M = 128

struct GroupShared : AtCommon<AT_GROUPS> {
  float c[2][KV_ROWS];                       // factor of a query's scores
  // Largest scores and sums by part of a row's tokens; 4 - reference.
  float top[AT_PARTS][KV_ROWS], l[AT_PARTS][KV_ROWS], nm[KV_ROWS];
};
// Warps: copies of K, scores, copies of V, outputs; then those that form weights, and those that
// convert values.
constexpr int GR_WARPS = GR_WEIGHTS + GR_CONVERT;
constexpr int GR_THREADS = 128 + 32 * GR_WARPS;
template <bool BF16>
constexpr int GR_KRING = BF16 ? 4 : 3;       // tiles in shared memory
constexpr int GR_VRING = 3, GR_WRING = 2;

__device__ __forceinline__ void umma_ts16(uint32_t d, uint32_t a, uint32_t blo, uint32_t bmid, uint32_t hi,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\tsetp.ne.u32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(blo | bmid), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tm_st16u(uint32_t addr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tm_ld32(uint32_t addr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
        "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]),
        "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(addr));
}
// Has the barrier's phase completed? Suspends the thread for up to 20 us: a wait that comes back more
// often takes its SM's issue slots from the warps that work (the CTA issued twice the instructions).
__device__ __forceinline__ bool gr_try(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}
static __device__ __noinline__ bool gr_wait_on(uint64_t* bar, uint32_t parity, volatile int* abort,
                                               const AttendArgs& A) {
  long long t0 = 0;
  while (!gr_try(bar, parity)) {
    if (*abort) return false;
    if (at_expired(&t0, A.wait_limit)) {
      *abort = 1;
      kv_report(A.S.hdr, ST_TIMEOUT);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ uint32_t gr_half2(uint32_t w) {  // two e4m3 (the low 16 bits) as fp16
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w)));
  return h;
}

static __device__ __noinline__ void gr_fetch(const SharedArgs& A, const AtItem* it, unsigned char* Q) {
  const int hw = (threadIdx.x - AT_SM0) >> 4, l16 = threadIdx.x & 15;
#pragma unroll 1
  for (int row = hw; row < it->R; row += 2 * GR_WARPS) {
    const AtQuery q = at_query<AT_GROUPS>(A, it->b, it->r0 + row);
    const uint16_t* src = static_cast<const uint16_t*>(A.q) + q.b * A.q_row + q.t * A.q_tok +
                          (size_t)(it->h * A.group + q.gh) * A.C.dim;
    if (l16 * 8 < A.C.dim)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(Q + at_raw(0, row, l16))),
                   "l"(src + l16 * 8)
                   : "memory");
  }
}
// As at_convert, without copies of rows.
template <bool BF16>
__device__ __noinline__ void gr_convert(const SharedArgs& A, const AtItem* it, unsigned char* Q, float* cs) {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  const int hw = (threadIdx.x - AT_SM0) >> 4, l16 = threadIdx.x & 15;
  const uint32_t half = 0xffffu << (threadIdx.x & 16);  // (the other half may have no row)
#pragma unroll 1
  for (int row = hw; row < it->R; row += 2 * GR_WARPS) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (l16 * 8 < A.C.dim) x = *reinterpret_cast<const uint4*>(Q + at_raw(0, row, l16));
    const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
    float y[8], a = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&xw[e]));
      y[2 * e] = BF16 ? bf_lo(xw[e]) : h.x;
      y[2 * e + 1] = BF16 ? bf_hi(xw[e]) : h.y;
      a = fmaxf(a, fmaxf(fabsf(y[2 * e]), fabsf(y[2 * e + 1])));
    }
    __syncwarp(half);  // the row is in registers: its place is free
#pragma unroll
    for (int s = 8; s; s >>= 1) a = fmaxf(a, __shfl_xor_sync(half, a, s));
    const float sc = kv_scale(a);
    const float inv = __uint_as_float((254u << 23) - __float_as_uint(sc));
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] *= inv;
    unsigned char* dst = Q + row * 128 + (((l16 >> 1) ^ (row & 7)) << 4) + (l16 & 1) * 8;
#pragma unroll
    for (int t = 0; t < AT_QTERMS<BF16>; ++t) {
      uint2 o;
      o.x = t ? e5m2x4(y[0], y[1], y[2], y[3]) : e4m3x4(y[0], y[1], y[2], y[3]);
      o.y = t ? e5m2x4(y[4], y[5], y[6], y[7]) : e4m3x4(y[4], y[5], y[6], y[7]);
      *reinterpret_cast<uint2*>(dst + (size_t)t * AT_BLK) = o;
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
    if (l16 == 0) cs[row] = a == INFINITY ? NAN : sc * A.scale;
  }
  __syncwarp();
  fence_async();
}

// Groups of eight tokens of a V tile (128 tokens x 128 bytes, 128-byte swizzle) as fp16: two blocks of
// 64 components, each 128 tokens x 128 bytes in the same swizzle. `warp` of GR_CONVERT; a lane takes
// 16 components of one token of each group. Tokens t and t ^ 5 are neighbours, which leaves no two of
// eight lanes in one bank, neither in the load nor in the stores.
__device__ __forceinline__ void gr_values(uint32_t V, uint32_t W, int warp) {
  const int lane = threadIdx.x & 31, c = lane & 3, k = lane >> 2, t = (k >> 1) ^ (k & 1 ? 5 : 0);
  const int block = warp & 1;
  const uint32_t from = V + t * 128 + (((c + 4 * block) ^ t) << 4), to = W + block * AT_BLK + t * 128;
  const uint32_t to0 = to + (((2 * c) ^ t) << 4), to1 = to + (((2 * c + 1) ^ t) << 4);
  auto put = [](uint32_t at, uint32_t a, uint32_t b) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(gr_half2(a)), "r"(gr_half2(a >> 16)),
                 "r"(gr_half2(b)), "r"(gr_half2(b >> 16))
                 : "memory");
  };
  constexpr int N = AT_KEYS / 8 / (GR_CONVERT / 2);  // groups of a warp
  uint4 x[N];
#pragma unroll
  for (int i = 0; i < N; ++i)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x[i].x), "=r"(x[i].y), "=r"(x[i].z), "=r"(x[i].w)
                 : "r"(from + ((warp >> 1) + i * (GR_CONVERT / 2)) * 1024)
                 : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t g = ((warp >> 1) + i * (GR_CONVERT / 2)) * 1024;
    put(to0 + g, x[i].x, x[i].y);
    put(to1 + g, x[i].z, x[i].w);
  }
}

// A row's outputs, n columns from oa on in steps of 64, times fac.
static __device__ __noinline__ void gr_shrink(uint32_t oa, int n, float fac) {
#pragma unroll 1
  for (int c = 0; c < n; c += 64) {
    float o[16];
    tm_ld16(oa + c, o);
    tm_wait_ld<16>(o);
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] *= fac;
    tm_st16(oa + c, o);
  }
}

// A thread's 32 weights of a step, in order: 2^(x - move) of the scores x = score * factor + nm, in
// fp16; their sum with the value scales taken out; the largest x.
struct Weighed {
  uint32_t v[16];
  float sum, top;
};
template <bool MOVED>
__device__ __forceinline__ void gr_weigh(Weighed& r, uint32_t sa, const float4* sc, int lgp, int key, float cs,
                                         float nm, float move) {
  float y[32];
  tm_ld32(sa, y);
  const float4 f0 = sc[key >> lgp], f1 = sc[(key + 16) >> lgp];
  const float2 a[2] = {make_float2(f0.x * cs, f0.x * cs), make_float2(f1.x * cs, f1.x * cs)};
  const float2 d[2] = {make_float2(f0.y + nm, f0.y + nm), make_float2(f1.y + nm, f1.y + nm)};
  tm_wait_ld<32>(y);
  float top[4];
  float2 sum[4];
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    float2 x = __ffma2_rn(make_float2(y[e], y[e + 1]), a[e / 16], d[e / 16]);
    top[e / 2 & 3] = e < 8 ? fmaxf(x.x, x.y) : max3(top[e / 2 & 3], x.x, x.y);
    if (MOVED) x = make_float2(x.x - move, x.y - move);
    const float2 p = make_float2(ex2(x.x), ex2(x.y));
    const int k = (e / 2 & 1) | e / 16 * 2;
    sum[k] = (e & 15) < 4 ? p : __fadd2_rn(sum[k], p);
    r.v[e / 2] = at_pack(p.x, p.y, 0);
  }
  r.top = fmaxf(max3(top[0], top[1], top[2]), top[3]);
  const float2 t0 = __fadd2_rn(sum[0], sum[1]), t1 = __fadd2_rn(sum[2], sum[3]);
  r.sum = fmaf(t0.x + t0.y, f0.z, (t1.x + t1.y) * f1.z);
}

template <bool BF16>
__global__ void __launch_bounds__(GR_THREADS, 1)
    kv_attend_group_kernel(const __grid_constant__ SharedArgs A, const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV) {
  constexpr int TERMS = AT_QTERMS<BF16>, NW = GR_WRING, NS = 3;
  // Tensor memory: the outputs' accumulator, three of scores. A step's weights (64 columns, 16 of each
  // 32) replace its scores.
  constexpr uint32_t scol = 128;
  extern __shared__ unsigned char dsm_raw[];
  __shared__ GroupShared sh;
  const KvCache& C = A.C;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  unsigned char* dsm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(dsm_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned char* Qs = dsm;                             // [terms][128][128]
  unsigned char* Ks = Qs + TERMS * AT_BLK;             // [GR_KRING<BF16>][128][128]
  unsigned char* Vs = Ks + GR_KRING<BF16> * AT_BLK;          // [GR_VRING][128][128]
  unsigned char* Ws = Vs + GR_VRING * AT_BLK;          // [NW][2][128][128]
  volatile int& s_abort = *const_cast<volatile int*>(&sh.abort);
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return gr_try(bar, parity) || gr_wait_on(bar, parity, &s_abort, A);
  };
  // A CTA starts as an SM's CTA of the launch for rows ends: it needs nothing of that one but that it
  // is over before this one is. (Waiting for all of it first: 64 chats behind one prompt 92.3 us
  // instead of 83.8, 8 samples of a document of 120,001 tokens 134 instead of 122.6. This launch first,
  // the rows' behind it: 90 us instead of 84 for the chats, and 75 instead of 67 for 64 rows of 64
  // queries without a group, as they were then, since the rows' CTAs find no room to be set up early.)
  kv_enter_behind(A.ready);
  AtCount count = {0, 0};
  int before = 0, total = 0;
  if (at_large(A, (long long)kv_ld(A.H.head + 1) * A.T * A.group)) {
    count = at_count<AT_GROUPS, GR_THREADS>(A, sh.rows);
    total = at_block_sum<GR_THREADS>(count.sum, sh.sum, &before);
  }
  if (total == 0) {  // (before anything is set up)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  at_setup<GR_WARPS>(sh);
  const int cta = blockIdx.x, most_ctas = gridDim.x;
  const uint32_t* const s_rows = sh.rows;
  at_begin<AT_GROUPS, GR_THREADS>(A, sh, count, total, before, cta, most_ctas);
  const uint32_t tmem = sh.tmem;

  int copied = 0;  // tiles whose copies this warp has issued
  if (w == 0) {
    copied = at_copy_keys<AT_GROUPS, 1>(A, GR_KRING<BF16>, tmK, sh, s_rows, Ks, &tmV);
  } else if (w == 1) {
    // ---- Scores of a step. (Steps are key tiles, numbered through all items.)
    if (at_elect()) {
      const int ksteps = (C.dim + 31) / 32;
      const uint32_t qd = at_desc_lo(smem_addr(Qs)), ring0 = at_desc_lo(smem_addr(Ks));
      constexpr uint32_t ids = AT_IDESC_S | ((AT_KEYS / 8) << 17);
      bool ok = true;
      int g = 0, q = 0, ph = 0, sb = 0, sph = 0;
      for (int item = 0; ok; ++item) {
        if (!wait(&sh.qfull, item & 1)) break;
        const int m = sh.item[item & 1].m;
        if (m == 0) break;
        for (int i = 0; i < m; ++i, ++g) {
          // An accumulator is free once the weights that replaced its scores are multiplied.
          if ((sph > 0 && !wait(&sh.pvdone[sb], (sph - 1) & 1)) || !wait(&sh.kfull[q], ph & 1)) {
            ok = false;
            break;
          }
          tm_fence_after();
          const uint32_t d = tmem + scol + sb * 128, bl = ring0 + q * (AT_BLK >> 4);
          for (int t = 0; t < TERMS; ++t) {
            const uint32_t id = t ? ids | AT_IDESC_E5M2_A : ids, al = qd + t * (AT_BLK >> 4);
            for (int k = 0; k < ksteps; ++k)
              umma_ss(d, al + 2 * k, bl + 2 * k, AT_HI, id, t + k ? 1u : 0u);
          }
          // (Two arrivals: the products' end, and what this thread has seen of the tile's data.)
          umma_commit(&sh.sfull[sb]);
          mbar_arrive(&sh.sfull[sb]);
          umma_commit(&sh.kempty[q]);
          if (++sb == NS) {
            sb = 0;
            ++sph;
          }
          if (++q == GR_KRING<BF16>) {
            q = 0;
            ++ph;
          }
        }
      }
      at_drain(&sh.drain[0], s_abort);
    }
  } else if (w == 2) {
    // ---- V copies, and before an item's the description that the other warps go by.
    fence_async_global();
    AtWalk<AT_GROUPS> walk = sh.walk;
    walk.first(A, s_rows);
    const int ppt = AT_KEYS >> C.lgp;
    bool ok = true;
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
    };
    int g = 0;  // tiles copied
    for (int k = 0;; ++k) {
      const int kb = k & 1;
      // (Item k's place is free once item k - 2 is done with.)
      if (k >= 2 && !warp_wait(&sh.dempty[kb], ((k >> 1) - 1) & 1)) break;
      const bool live = walk.live();
      AtItem& it = sh.item[kb];
      if (lane == 0) {
        it.m = live ? walk.i1 - walk.i0 : 0;
        if (live) {
          it.b = walk.b;
          it.h = walk.h;
          it.r0 = walk.tile.r0;
          it.R = walk.tile.r1 - walk.tile.r0;
          it.i0 = walk.i0;
          it.tiles = walk.tile.tiles();
          it.u0 = walk.base + KV_EXTRA;
          it.no = at_tile_no(A, AT_GROUPS, walk.b, walk.rt, walk.h);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.dfull[kb]);
      if (!live) break;
      for (int i = walk.i0; i < walk.i1; ++i, ++g) {
        const int q = g % GR_VRING, ph = g / GR_VRING;
        if ((ph > 0 && !warp_wait(&sh.vempty[q], (ph - 1) & 1)) ||
            !warp_wait(&sh.tinfo[g & (AT_INFO - 1)], (g / AT_INFO) & 1)) {
          ok = false;
          break;
        }
        const int y = lane < ppt ? sh.y[g & (AT_INFO - 1)][lane] : -1;
        const uint32_t pages = __popc(__ballot_sync(0xffffffffu, y >= 0));
        if (lane == 0) mbar_arrive_expect_tx(&sh.vfull[q], (pages << C.lgp) * 128u);
        __syncwarp();
        if (y >= 0) at_tma(Vs + q * AT_BLK + ((size_t)lane << C.lgp) * 128, &tmV, 0, y, &sh.vfull[q]);
      }
      if (!ok) break;
      walk.next(A, s_rows);
    }
    copied = g;
  } else if (w == 3) {
    // ---- Outputs: O += P V of a step.
    if (at_elect()) {
      const uint32_t ring0 = at_desc_lo(smem_addr(Ws)) & 0xffffu;
      const uint32_t idw = AT_IDESC_W | (static_cast<uint32_t>(C.dim) >> 3 << 17);
      bool ok = true;
      int g = 0, sb = 0, sph = 0;
      for (int item = 0; ok; ++item) {
        if (!wait(&sh.qfull, item & 1)) break;
        const int m = sh.item[item & 1].m;
        if (m == 0) break;
        for (int i = 0; i < m; ++i, ++g) {
          const int wb = g % NW;
          if (!wait(&sh.wfull[wb], (g / NW) & 1) || !wait(&sh.hfull[sb], sph & 1)) {
            ok = false;
            break;
          }
          mbar_arrive(&sh.vempty[g % GR_VRING]);  // (the tile is converted)
          tm_fence_after();
          // (Blocks of 64 components are 128 tokens apart: the descriptor's leading offset.)
          const uint32_t pa = tmem + scol + sb * 128, wd = ring0 + wb * (GR_BLK >> 4);
#pragma unroll
          for (int k = 0; k < AT_KEYS / 16; ++k)
            umma_ts16(tmem, pa + k / 2 * 32 + k % 2 * 8, wd + k * (2048 >> 4), (AT_BLK >> 4) << 16, AT_HI,
                      idw, i > 0 || k > 0 ? 1u : 0u);
          umma_commit(&sh.pvdone[sb]);
          umma_commit(&sh.wempty[wb]);
          if (++sb == NS) {
            sb = 0;
            ++sph;
          }
        }
      }
      at_drain(&sh.drain[1], s_abort);
    }
  } else {
    // ---- Weights and results (the first 16 warps), and conversion of values (the last four).
    const int st = tid - AT_SM0, quad = w & 3, part = (w - 4) >> 2;  // (part 4 converts)
    const int row = quad * 32 + lane;  // lane of the accumulators
    const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    bool dead = false;  // a wait gave up: skip the work, keep meeting the other warps
    // (Lanes take up a wait's answer together; see at_body.)
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
    };
    auto fetch = [&](int k) {
      if (!dead && !warp_wait(&sh.dfull[k & 1], (k >> 1) & 1)) dead = true;
      if (!dead && sh.item[k & 1].m > 0) gr_fetch(A, &sh.item[k & 1], Qs);
    };
    auto convert = [&](int k) {
      if (!dead && sh.item[k & 1].m > 0) gr_convert<BF16>(A, &sh.item[k & 1], Qs, sh.c[k & 1]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.qfull);
    };
    fetch(0);
    convert(0);
    int g = 0, sb = 0, sph = 0;  // key tiles; accumulator of a step's scores, and its pass
    // Is the step before done?
    auto done = [&]() {
      const int b = sb ? sb - 1 : NS - 1;
      return warp_wait(&sh.pvdone[b], (sb ? sph : sph - 1) & 1);
    };
    for (int item = 0;; ++item) {
      const int kb = item & 1;
      if (!dead && !warp_wait(&sh.qfull, item & 1)) dead = true;
      if (at_vote(5, 32 * GR_WARPS, dead)) break;
      const AtItem& it = sh.item[kb];
      const int m = it.m, rows = it.R;
      if (m == 0) break;
      const bool real = row < rows, live = quad * 32 < rows;
      if (part == AT_PARTS) {
#pragma unroll 1
        for (int i = 0; i < m; ++i, ++g) {
          // A tile's values, once the products that read the buffer before are done.
          const int q = g % GR_VRING, wb = g % NW;
          if (!dead && ((g >= NW && !warp_wait(&sh.wempty[wb], (g / NW - 1) & 1)) ||
                        !warp_wait(&sh.vfull[q], (g / GR_VRING) & 1)))
            dead = true;
          if (!dead) gr_values(smem_addr(Vs) + q * AT_BLK, smem_addr(Ws) + wb * GR_BLK, w - 4 - GR_WEIGHTS);
          fence_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.wfull[wb]);
        }
      } else {
        const float cs = real ? sh.c[kb][row] : 0.f;
        float l = 0.f, nm = 0.f;  // sum of the weights; 4 - reference
        bool unseen = real;       // no key yet
#pragma unroll 1
        for (int i = 0; i < m; ++i, ++g) {
          const uint32_t sa = tl + scol + sb * 128 + part * 32;
          if (!dead && !warp_wait(&sh.sfull[sb], sph & 1)) dead = true;
          tm_fence_after();
          if (live) {
            // Weights at the reference so far; they count when no score has passed it by 2^11.
            const float4* sc = sh.sc[g & (AT_INFO - 1)];
            Weighed x;
            gr_weigh<false>(x, sa, sc, C.lgp, part * 32, cs, nm, 0.f);
            if (__builtin_expect(at_vote(1 + quad, 128, unseen || (real && x.top > AT_LIMIT)), 0)) {
              // Move references to the step's largest scores (see at_body) and form the weights
              // again, from the same scores, so that the largest is at 4 exactly.
              sh.top[part][row] = x.top;
              at_bar(1 + quad, 128);
              const float d = fmaxf(fmaxf(sh.top[0][row], sh.top[1][row]),
                                    fmaxf(sh.top[2][row], sh.top[3][row]));  // over the reference - 4
              float move = 0.f, fac = 1.f;
              if (unseen) {
                if (d > -INFINITY) {
                  move = d - GR_SHIFT;
                  unseen = false;
                }
              } else if (real && d > GR_SHIFT) {
                move = d - GR_SHIFT;
                fac = exp2f(-move);
              }
              l *= fac;
              __syncwarp();
              if (i > 0 && !dead && !done()) dead = true;
              tm_fence_after();
              gr_shrink(tl + part * 16, i > 0 ? C.dim - part * 16 : 0, fac);
              // (Into registers of their own: sharing x's cost the other path a move for each.)
              Weighed z;
              gr_weigh<true>(z, sa, sc, C.lgp, part * 32, cs, nm, move);
              nm -= move;
              l += z.sum;
              tm_st16u(sa, z.v);
            } else {
              l += x.sum;
              tm_st16u(sa, x.v);
            }
            tm_wait_st();
          }
          tm_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.hfull[sb]);
          if (++sb == NS) {
            sb = 0;
            ++sph;
          }
        }
        sh.l[part][row] = l;
        if (part == 0) sh.nm[row] = nm;
      }

      // -- The query tile's sums and outputs, always partial results. The last scores are done (the
      // weight warps have seen them), so the next queries go in first.
      at_bar(5, 32 * GR_WARPS);
      fetch(item + 1);
      convert(item + 1);
      if (part < AT_PARTS) {
        if (!dead && !done()) dead = true;
        tm_fence_after();
        if (live) {
          const int id = it.no + cta;
          if (real && part == 0)
            A.stat[(size_t)id * KV_ROWS + row] = make_float2(-sh.nm[row], sh.l[0][row] + sh.l[1][row] + (sh.l[2][row] + sh.l[3][row]));
          float4* const parts = reinterpret_cast<float4*>(A.part);
          __syncwarp();
#pragma unroll 1
          for (int c = part * 16; c < C.dim; c += 64) {
            float o[16];
            tm_ld16(tl + c, o);
            tm_wait_ld<16>(o);
            if (real) {
              float4* to = parts + at_part(id, row, c, C.dim);
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                to[e / 4 * KV_ROWS] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
            __syncwarp();
          }
        }
        tm_fence_before();
      }
      if (it.i0 == 0 && st == 0) {
        const int all = sh.total, n = min(most_ctas, all);
        A.span[it.no] = KvSpan{cta, at_owner(it.u0 + it.tiles - 1, all, n)};
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.dempty[kb]);
    }
  }

  tm_fence_before();
  __syncthreads();
  // After a wait gave up, what is on its way to shared memory lands before the CTA exits.
  if (s_abort) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (w == 0) at_land(sh.kfull, GR_KRING<BF16>, copied);
    if (w == 2) at_land(sh.vfull, GR_VRING, copied);
  }
  if (w == 1) {
    __syncwarp();
    tm_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Its shared memory beside static arrays.
template <bool BF16>
constexpr size_t GR_SMEM = 1024 + (AT_QTERMS<BF16> + GR_KRING<BF16> + GR_VRING) * (size_t)AT_BLK +
                           GR_WRING * (size_t)GR_BLK;
static_assert(GR_SMEM<true> + sizeof(GroupShared) <= AT_SMEM && GR_SMEM<false> + sizeof(GroupShared) <= AT_SMEM,
              "a CTA's shared memory");

cudaError_t launch_kv_attend_group(const SharedArgs& A, const AttendLaunch& L, sv_dtype dt, int dev, cudaStream_t st) {
  static OncePerDevice sized;  // (the attribute belongs to the device that is current)
  cudaError_t e = static_cast<cudaError_t>(sized.run(dev, [] {
    cudaError_t attr = cudaFuncSetAttribute(reinterpret_cast<const void*>(kv_attend_group_kernel<true>),
                                            cudaFuncAttributeMaxDynamicSharedMemorySize, (int)GR_SMEM<true>);
    if (attr == cudaSuccess)
      attr = cudaFuncSetAttribute(reinterpret_cast<const void*>(kv_attend_group_kernel<false>),
                                  cudaFuncAttributeMaxDynamicSharedMemorySize, (int)GR_SMEM<false>);
    return static_cast<int>(attr);
  }));
  if (e != cudaSuccess) return e;
  const bool bf16 = dt == SV_BF16;
  return kv_launch(bf16 ? kv_attend_group_kernel<true> : kv_attend_group_kernel<false>, dim3(L.grid), GR_THREADS,
                   bf16 ? GR_SMEM<true> : GR_SMEM<false>, st, A, L.tm[0], L.tm[1]);
}

}  // namespace sv
