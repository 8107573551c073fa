// sv_kv_shared.cu -- attention of rows that share pages (sm_103a): which rows share how much, the
// launch, and the join of the parts. The kernel is in sv_kv_shared.cuh.
#include "sv_kv_shared.cuh"

namespace sv {

namespace {

constexpr int SH_THREADS = 1024;
constexpr int SH_MOST = 4096;  // rows, at most (SV_MAX_B)
static_assert(SV_MAX_B <= SH_MOST, "a CTA sorts all rows");

// How many tokens every row of a group has in common: whole tiles of 128 on pages that are the same
// in all of them, and no more than any row holds. A warp compares a row, the i-th in `order`, with
// its group's lowest, and writes that one's pages down: they are the group's from then on, whatever
// becomes of the row.
__device__ __forceinline__ void share_pages(const KvCache& C, const KvShare& H, int i) {
  const int lane = threadIdx.x & 31;
  const int b = kv_ld(H.order + i), g = kv_ld(H.row + b).x, lead = kv_ld(H.group + g).w;
  const int len = max(0, kv_ld(C.len + b));
  const int pages = min(min(kv_ld(C.np + b), C.max_pages), len >> C.lgp);
  const int32_t *mine = C.table + (size_t)b * C.max_pages, *its = C.table + (size_t)lead * C.max_pages;
  int32_t* const kept = H.pages + (size_t)g * C.max_pages;
  int common = max(pages, 0);
  for (int j0 = 0; j0 < common; j0 += 128) {
    unsigned differ[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = j0 + 32 * k + lane;
      bool d = j >= common;
      if (!d) {
        const int p = kv_ld(mine + j);
        d = p < 0 || p >= C.pages || p != kv_ld(its + j);
        if (b == lead) kept[j] = p;
      }
      differ[k] = __ballot_sync(0xffffffffu, d);
    }
#pragma unroll
    for (int k = 3; k >= 0; --k)
      if (differ[k]) common = min(common, j0 + 32 * k + __ffs(differ[k]) - 1);
  }
  if (lane == 0)
    atomicMin(&H.group[g].z, static_cast<int>(((long long)common << C.lgp) & ~127LL));
}
__device__ __forceinline__ void share_row(const KvShare& H, int b) {
  const int g = kv_ld(H.row + b).x;
  if (g >= 0) H.row[b].z = __ldcg(&H.group[g].z);
}

// Rows by group. One CTA sorts (group's key, row), lowest rows first, and numbers the runs of two
// or more: rows of those go to `order`, all others are alone. The key is group[b] or, without it,
// the page of the row's first token. For a few rows, two to a warp, it does the rest as well: with
// the two launches behind it a round of 34 rows took 274.6 us instead of 273.
constexpr int SH_ONE = 64;
__global__ void __launch_bounds__(SH_THREADS)
    kv_share_group_kernel(const KvCache C, const KvScratch S, const KvShare H, const int32_t* group) {
  kv_enter();
  __shared__ unsigned long long s_key[SH_MOST];
  __shared__ int s_scan[64], s_first[SH_MOST / 2 + 1], s_most;
  constexpr unsigned long long ALONE = 1ull << 48, NONE = ~0ull;
  const int tid = threadIdx.x;
  int n = 2;
  while (n < C.batch) n *= 2;
  if (tid == 0) s_most = 0;
  for (int b = tid; b < n; b += SH_THREADS) {
    unsigned long long key = NONE;
    if (b < C.batch) {
      key = ALONE | b;
      if (group) {
        const int g = kv_ld(group + b);
        if (g < -1 || g >= C.batch)
          kv_report(S.hdr, ST_DEVICE_INPUT);
        else if (g >= 0)
          key = (unsigned long long)g << 12 | b;
      } else {
        const int p = kv_page(C, b, 0);
        if (p >= 0) key = (unsigned long long)p << 12 | b;
      }
      H.bad[b] = 0;
    }
    s_key[b] = key;
  }
  for (int size = 2; size <= n; size *= 2)
    for (int d = size / 2; d; d /= 2) {
      __syncthreads();
      for (int i = tid; i < n / 2; i += SH_THREADS) {
        const int lo = i / d * 2 * d + i % d, hi = lo + d;
        const bool up = (lo & size) == 0;
        const unsigned long long x = s_key[lo], y = s_key[hi];
        if ((x > y) == up) {
          s_key[lo] = y;
          s_key[hi] = x;
        }
      }
    }
  __syncthreads();
  // Four neighbours a thread: rows in groups before each (low half) and groups before (high).
  auto same = [&](int i) {  // are entries i - 1 and i of one group?
    return i > 0 && i < C.batch && s_key[i] < ALONE && s_key[i] >> 12 == s_key[i - 1] >> 12;
  };
  int in[4], c = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = 4 * tid + k;
    const bool with = same(i), head = !with && same(i + 1);
    in[k] = head ? 2 : (with ? 1 : 0);
    c += (in[k] ? 1 : 0) + (in[k] == 2 ? 1 << 16 : 0);
  }
  int all;
  int at = block_scan(c, s_scan, &all);
  const int groups = all >> 16, rows = all & 0xffff, at0 = at;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (in[k] == 2) s_first[at >> 16] = at & 0xffff;
    at += (in[k] ? 1 : 0) + (in[k] == 2 ? 1 << 16 : 0);
  }
  if (tid == 0) s_first[groups] = rows;
  __syncthreads();
  at = at0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = 4 * tid + k;
    if (i >= C.batch) break;
    const int b = static_cast<int>(s_key[i] & 0xfff);
    if (!in[k]) {
      H.row[b] = make_int4(-1, 1, 0, 0);
      continue;
    }
    const int g = (at >> 16) - (in[k] == 2 ? 0 : 1), first = s_first[g], size = s_first[g + 1] - first;
    H.row[b] = make_int4(g, size, 0, (at & 0xffff) - first);
    H.order[at & 0xffff] = b;
    if (in[k] == 2) {
      H.group[g] = make_int4(first, size, 0x7fffffff, b);
      atomicMax(&s_most, size);
    }
    at += 1 + (in[k] == 2 ? 1 << 16 : 0);
  }
  __syncthreads();
  if (tid == 0) {
    H.head[0] = groups;
    H.head[1] = s_most;
    H.head[2] = rows;
  }
  if (C.batch > SH_ONE) return;
  __syncthreads();
  for (int i = tid / 32; i < rows; i += SH_THREADS / 32) share_pages(C, H, i);
  __syncthreads();
  if (tid < C.batch) share_row(H, tid);
}

__global__ void __launch_bounds__(256) kv_share_pages_kernel(const KvCache C, const KvShare H) {
  kv_enter();
  const int i = blockIdx.x * 8 + threadIdx.x / 32;
  if (i < kv_ld(H.head + 2)) share_pages(C, H, i);
}

__global__ void __launch_bounds__(256) kv_share_rows_kernel(const KvCache C, const KvShare H) {
  kv_enter();
  const int b = blockIdx.x * 256 + threadIdx.x;
  if (b < C.batch) share_row(H, b);
}


// Joins the parts of every query tile of a row: its own keys' and, where it is in a group, those
// of the common ones, in the order of the CTAs that made them. (A query tile with one part has its
// result already.)
constexpr int SJ_THREADS = 256;
// (When a wait gave up, a query tile may have no span of this call: what is there is kept in range.)
__device__ __forceinline__ KvSpan join_span(const KvSpan* p) {
  const KvSpan s = kv_ld(p);
  return KvSpan{min(max(s.first, 0), KV_MAX_CTAS - 1), min(s.last, KV_MAX_CTAS - 1)};
}

// A warp: 64 components of eight query rows of a query tile and head, four lanes a row, four parts'
// loads in flight and a running reference. (Rows next to each other: whole sectors.) Query tiles of
// rows alone are in parts only where two CTAs' shares meet: the first warps take those from the
// CTAs' records, the others those of rows in groups. (Looking at every query tile and head
// instead took a call for 64 rows of 64 queries on 740 tokens 81 us instead of 75, as it was then;
// all sums first, then the parts two at a time, 8 samples of a document of 120,001 tokens, whose
// query tiles have some fourteen parts, 140 us instead of 126.)
__global__ void __launch_bounds__(SJ_THREADS, 2)
    kv_shared_join_kernel(const __grid_constant__ SharedArgs A, int ctas, int bf16) {
  kv_enter();
  constexpr int U = 4, K = 4;
  const int vec = A.C.dim / 4, pieces = (vec + 4 * U - 1) / (4 * U), heads = A.C.heads;
  const int eights = A.own_rows / 8, lane = threadIdx.x & 31;
  const long long met = (long long)ctas * eights;  // items of CTAs' shares that meet
  const long long at = (long long)blockIdx.x * (SJ_THREADS / 32) + threadIdx.x / 32;
  const long long item = at / pieces;
  const int piece = static_cast<int>(at - item * pieces), chunk = static_cast<int>(item % eights);
  int b, h, r0, R, no, owns;      // (no: the first of `owns` slots of the row's own)
  int id = 0, gr = 0, count = 0;  // of the group's: row gr of `count` slots from id on
  const int r = 8 * chunk + (lane & 7);
  bool bad = false;
  if (item < met) {
    const KvOpen it = A.S.open[item / eights];
    if (8 * chunk >= it.R) return;
    b = it.b;
    h = it.h;
    r0 = it.r0;
    R = it.R;
    no = it.slot;
    owns = it.last + 1;
  } else {
    if (kv_ld(A.H.head) == 0) return;
    const long long tile = (item - met) / eights, bt = tile / heads;
    h = static_cast<int>(tile - bt * heads);
    b = static_cast<int>(bt / A.tiles);
    if (b >= A.C.batch) return;
    const int rt = static_cast<int>(bt - (long long)b * A.tiles);
    const AtRow row = at_row<AT_OWN>(A, b);
    if (!row.skip) return;
    bad = kv_ld(A.H.bad + b) != 0;
    // (Of a row that is NaN all queries, new tokens or not: 128 to a query tile.)
    r0 = rt * (bad ? KV_ROWS : row.rr);
    R = min(r0 + (bad ? KV_ROWS : row.rr), bad ? A.T * A.group : row.rows) - r0;
    if ((rt >= row.nrt && !bad) || 8 * chunk >= R) return;
    no = owns = 0;
    if (!bad) {
      no = at_tile_no(A, AT_OWN, b, rt, h);
      const KvSpan own = join_span(A.own_span + no);
      no += own.first;
      owns = own.last - own.first + 1;
      const int4 mine = kv_ld(A.H.row + b);
      const AtRow group = at_row<AT_GROUPS>(A, mine.x);
      const int i = mine.w * A.T * A.group + r0 + min(r, R - 1), grt = i / group.rr;
      gr = i - grt * group.rr;
      if (!A.window || at_tile<AT_GROUPS>(A, group, mine.x, grt).tiles() > 0) {
        id = at_tile_no(A, AT_GROUPS, mine.x, grt, h);
        const KvSpan span = join_span(A.span + id);
        count = span.last - span.first + 1;
        id += span.first;
      }
    }
  }
  if (r >= R) return;
  const int slots = count + owns;
  auto slot = [&](int k, const float2** stat, const float4** part, int* rows) {
    const bool mine = k >= count;
    const int at = mine ? no + k - count : id + k, rr = mine ? r : gr;
    *rows = mine ? A.own_rows : KV_ROWS;
    *stat = (mine ? A.own_stat : A.stat) + (size_t)at * *rows + rr;
    *part = reinterpret_cast<const float4*>(mine ? A.own_part : A.part) +
            at_part(at, rr, 0, A.C.dim, *rows);
  };
  const int v0 = 4 * U * piece + (lane >> 3);
  float ref = -INFINITY, sum = 0.f;
  float4 o[U];
#pragma unroll
  for (int u = 0; u < U; ++u) o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < slots; k0 += K) {
    float2 x[K];
    float4 y[K][U];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      x[k] = make_float2(0.f, 0.f);
      if (k0 + k >= slots) continue;
      const float2* stat;
      const float4* part;
      int rows;
      slot(k0 + k, &stat, &part, &rows);
      x[k] = __ldcg(stat);
#pragma unroll
      for (int u = 0; u < U; ++u) y[k][u] = __ldcg(part + (size_t)min(v0 + 4 * u, vec - 1) * rows);
    }
    float top = ref;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (x[k].y != 0.f) top = fmaxf(top, x[k].x);
    const float f0 = sum == 0.f ? 0.f : exp2f(ref - top);
    ref = top;
    sum *= f0;
#pragma unroll
    for (int u = 0; u < U; ++u) o[u] = make_float4(o[u].x * f0, o[u].y * f0, o[u].z * f0, o[u].w * f0);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (x[k].y == 0.f) continue;
      const float f = exp2f(x[k].x - top);
      sum = fmaf(x[k].y, f, sum);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        o[u].x = fmaf(y[k][u].x, f, o[u].x);
        o[u].y = fmaf(y[k][u].y, f, o[u].y);
        o[u].z = fmaf(y[k][u].z, f, o[u].z);
        o[u].w = fmaf(y[k][u].w, f, o[u].w);
      }
    }
  }
  float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (bad) inv = sum = NAN;
  const int i = r0 + r, t = i / A.group, gh = i - t * A.group;
  const long long out = ((long long)b * A.T + t) * A.q_heads + h * A.group + gh;
  if (piece == 0 && lane < 8 && A.lse)
    A.lse[out] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (v0 + 4 * u < vec)
      at_store4(A.out, out * A.C.dim + (v0 + 4 * u) * 4,
                make_float4(o[u].x * inv, o[u].y * inv, o[u].z * inv, o[u].w * inv), bf16);
}

}  // namespace

size_t kv_share_layout(const KvCache& C, int T, int group, unsigned char* base, SharedArgs* A) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    unsigned char* const at = base + off;
    off = align_up(off + bytes, 256);
    return at;
  };
  const size_t B = (size_t)C.batch;
  A->H.head = reinterpret_cast<int32_t*>(take(4 * KV_SHARE_HEAD));
  A->H.row = reinterpret_cast<int4*>(take(16 * B));
  A->H.group = reinterpret_cast<int4*>(take(16 * (B / 2 + 1)));
  A->H.order = reinterpret_cast<int32_t*>(take(4 * B));
  A->H.bad = reinterpret_cast<int32_t*>(take(4 * B));
  A->H.ready = reinterpret_cast<uint32_t*>(take(4 * KV_MAX_CTAS));
  A->H.pages = reinterpret_cast<int32_t*>(take(4 * (B / 2) * C.max_pages));
  const size_t rows = (size_t)T * group;
  A->tiles = static_cast<int>((rows + KV_ROWS - 1) / KV_ROWS);
  A->own_rows = rows < KV_ROWS ? static_cast<int>((rows + 7) / 8 * 8) : KV_ROWS;
  // Slots: a query tile has one more than CTAs' shares end in it.
  const size_t own_tiles = B * A->tiles * C.heads, tiles = (B * rows / KV_ROWS + B / 2 + 1) * C.heads;
  A->own_span = reinterpret_cast<KvSpan*>(take(sizeof(KvSpan) * own_tiles));
  A->span = reinterpret_cast<KvSpan*>(take(sizeof(KvSpan) * tiles));
  A->own_stat = reinterpret_cast<float2*>(take(8 * (own_tiles + KV_MAX_CTAS) * A->own_rows));
  A->stat = reinterpret_cast<float2*>(take(8 * (tiles + KV_MAX_CTAS) * KV_ROWS));
  A->own_part = reinterpret_cast<float*>(take(4 * (own_tiles + KV_MAX_CTAS) * A->own_rows * C.dim));
  A->part = reinterpret_cast<float*>(take(4 * (tiles + KV_MAX_CTAS) * KV_ROWS * C.dim));
  return off;
}

cudaError_t launch_kv_share(const KvCache& C, const KvScratch& S, const KvShare& H,
                            const int32_t* group, cudaStream_t st) {
  cudaError_t e = kv_launch(kv_share_group_kernel, dim3(1), SH_THREADS, 0, st, C, S, H, group);
  if (C.batch <= SH_ONE) return e;
  if (e == cudaSuccess)
    e = kv_launch(kv_share_pages_kernel, dim3((C.batch + 7) / 8), 256, 0, st, C, H);
  if (e == cudaSuccess)
    e = kv_launch(kv_share_rows_kernel, dim3((C.batch + 255) / 256), 256, 0, st, C, H);
  return e;
}

cudaError_t launch_kv_attend_shared(SharedArgs& A, sv_dtype dt, cudaStream_t st) {
  at_rule(&A);
  static const SharedKernel* const kernels[2][2] = {{shared_kernels_f16_1, shared_kernels_f16_2},
                                                    {shared_kernels_bf16_1, shared_kernels_bf16_2}};
  int dev = 0;
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
  AttendLaunch L;
  if ((e = at_launch(A, dt, at_width((long long)A.T * A.group), dev, &L)) != cudaSuccess) return e;
  const SharedKernel kernel = kernels[dt == SV_BF16][L.ndb - 1][L.width == 32 ? 0 : (L.width == 64 ? 1 : 2)];
  // (No group has more rows than the batch.)
  const bool groups = A.large && at_width((long long)A.C.batch * A.T * A.group) == 128;
  A.ready = groups ? A.H.ready : nullptr;
  if ((e = kv_launch(kernel, dim3(L.grid), AT_THREADS, L.smem, st, A, L.P, L.tm[0], L.tm[1])) != cudaSuccess)
    return e;
  if (groups && (e = launch_kv_attend_group(A, L, dt, dev, st)) != cudaSuccess) return e;
  const long long eights = ((long long)A.C.batch * A.tiles * A.C.heads + L.grid) * (A.own_rows / 8);
  const long long warps = eights * ((A.C.dim / 4 + 15) / 16);
  const long long blocks = (warps + SJ_THREADS / 32 - 1) / (SJ_THREADS / 32);
  return kv_launch(kv_shared_join_kernel, dim3(static_cast<unsigned>(blocks)), SJ_THREADS, 0, st, A,
                   static_cast<int>(L.grid), dt == SV_BF16 ? 1 : 0);
}

}  // namespace sv
