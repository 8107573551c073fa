// sv_kv_pages.cu -- the page calls of the key/value cache (sm_103a): reserve, fork, commit.
//
// Pages are handed out lowest free id first and in row order, so that results do not
// depend on scheduling: a free page is one whose refs entry is 0, and one CTA finds the
// first `want` of them by counting zeros block by block with prefix sums (4,096 entries a
// step, and no further than needed). Reserve for 64 rows is that one launch: 5 us, nearly
// all of it the trips to memory one after the other.
#include "sv_kv.cuh"

namespace sv {

constexpr int PG_THREADS = 1024;

// Exclusive prefix sum of x over the block's PG_THREADS threads; *total gets the sum.
// Two barriers; `sh` holds 64 values.
template <typename I>
__device__ I block_scan(I x, I* sh, I* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  I v = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const I t = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += t;
  }
  if (lane == 31) sh[w] = v;
  __syncthreads();
  if (w == 0) {
    I s = sh[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const I t = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += t;
    }
    sh[32 + lane] = s;  // inclusive
  }
  __syncthreads();
  *total = sh[63];
  return v - x + (w ? sh[32 + w - 1] : 0);
}

// The first `want` free pages (refs 0) in ascending order, to list[0 ..]; returns how many
// there are (at most `want`). Whole block.
__device__ int find_free(const KvCache& C, int want, int32_t* list, int* sh) {
  int found = 0;
  for (int base = 0; base < C.pages && found < want; base += 4 * PG_THREADS) {
    const int p0 = base + 4 * static_cast<int>(threadIdx.x);
    int z[4], c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[i] = p0 + i < C.pages && __ldcg(C.refs + p0 + i) == 0;
      c += z[i];
    }
    int total;
    int r = found + block_scan(c, sh, &total);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (z[i] && r < want) list[r++] = p0 + i;
    found += total;
    __syncthreads();  // sh is used again
  }
  __syncthreads();  // the list is complete
  return found < want ? found : want;
}

__global__ void __launch_bounds__(PG_THREADS, 1)
    kv_reserve_kernel(const KvCache C, const KvScratch S, const int32_t* n_new,
                      int32_t* ok) {
  kv_enter();
  __shared__ int sh[64];
  __shared__ long long shl[64];
  extern __shared__ int end[];  // [batch] pages needed by rows 0 .. b, cut at pages + 1
  const int tid = threadIdx.x;
  // Pages that row b needs in all, or -1 when its data is wrong. (A negative n_pages is below
  // that -1: compare the two only for h >= 0.)
  auto holds = [&](int b) -> long long {
    const int n = kv_ld(n_new + b), len = C.len[b], np = S.np[b];
    const long long h = ((long long)len + n + C.page - 1) >> C.lgp;
    return n < 0 || len < 0 || np < 0 || np > C.max_pages || h > C.max_pages ? -1 : h;
  };
  long long all = 0;
  for (int base = 0; base < C.batch; base += PG_THREADS) {
    const int b = base + tid;
    long long need = 0;
    if (b < C.batch) {
      S.np[b] = C.np[b];  // as it was: the row's own entry changes below
      const long long h = holds(b);
      if (h < 0) kv_report(S.hdr, ST_DEVICE_INPUT);
      need = h >= 0 && h > S.np[b] ? h - S.np[b] : 0;
    }
    long long total;
    const long long e = all + block_scan(need, shl, &total) + need;
    if (b < C.batch) end[b] = static_cast<int>(e > C.pages ? C.pages + 1LL : e);
    all += total;
    __syncthreads();  // shl is used again, end is read below
  }
  const long long most = (long long)C.batch * C.max_pages;
  const int cap = static_cast<int>(most < C.pages ? most : C.pages);
  const int got = find_free(C, all < cap ? static_cast<int>(all) : cap, S.list, sh);
  // Row b is served when end[b] <= got. Fresh page r goes to the row whose range of ranks
  // holds r.
  for (int r = tid; r < got; r += PG_THREADS) {
    int lo = 0, hi = C.batch - 1;  // the first row with end > r
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (end[mid] > r)
        hi = mid;
      else
        lo = mid + 1;
    }
    if (end[lo] > got || end[lo] <= r) continue;
    const int p = S.list[r], b0 = lo ? end[lo - 1] : 0;
    C.table[(size_t)lo * C.max_pages + S.np[lo] + (r - b0)] = p;
    C.refs[p] = 1;
  }
  for (int b = tid; b < C.batch; b += PG_THREADS) {
    const long long h = holds(b);
    const bool needs = h >= 0 && h > S.np[b], served = h >= 0 && (!needs || end[b] <= got);
    if (needs && served) C.np[b] = static_cast<int>(h);
    if (needs && !served) kv_report(S.hdr, ST_NO_PAGES);
    if (ok) ok[b] = served ? 1 : 0;
  }
}

// ---------------------------------------------------------------------------
// Fork, in three launches: (1) a CTA per old row counts its takers, snapshots the row and
// changes its pages' refs; (2) one CTA hands fresh pages to the copies; (3) CTAs per new
// row write its table and copy its partial page. The counts and the hand-out are a few us
// each; the copies are bound by memory: 48 partial pages of 32 layers and 8 heads (K and V,
// on average half full, 92 MB of traffic) in 43 us cold.
// ---------------------------------------------------------------------------

// src of row b, with one outside [-1, batch) read as b.
__device__ __forceinline__ int fork_src(const KvCache& C, const int32_t* src, int b) {
  const int s = kv_ld(src + b);
  return s >= -1 && s < C.batch ? s : b;
}

__global__ void __launch_bounds__(128)
    kv_fork_count_kernel(const KvCache C, const KvScratch S, const int32_t* src) {
  kv_enter();
  __shared__ int s_m, s_first;
  const int i = blockIdx.x, tid = threadIdx.x;
  if (tid == 0) {
    s_m = 0;
    s_first = C.batch;
  }
  __syncthreads();
  int m = 0, first = C.batch;
  for (int b = tid; b < C.batch; b += blockDim.x)
    if (fork_src(C, src, b) == i) {
      ++m;
      first = min(first, b);
    }
  if (m) {
    atomicAdd(&s_m, m);
    atomicMin(&s_first, first);
  }
  __syncthreads();
  m = s_m;
  const int np = min(max(C.np[i], 0), C.max_pages);
  // A length past the pages held is cut to them.
  const int len = max(0, static_cast<int>(min((long long)C.len[i], (long long)np << C.lgp)));
  const int full = len >> C.lgp;
  if (tid == 0) {
    const int raw = kv_ld(src + i);
    if (raw < -1 || raw >= C.batch || np != C.np[i] || len != C.len[i])
      kv_report(S.hdr, ST_DEVICE_INPUT);
    S.keeper[i] = m == 0 ? -1 : (fork_src(C, src, i) == i ? i : s_first);
    S.np[i] = np;
    S.len[i] = len;
  }
  for (int j = tid; j < np; j += blockDim.x) {
    const int p = C.table[(size_t)i * C.max_pages + j];
    S.table[(size_t)i * C.max_pages + j] = p;
    const int delta = j < full ? m - 1 : (m > 0 ? 0 : -1);
    if (delta == 0) continue;
    if (p >= 0 && p < C.pages)
      atomicAdd(C.refs + p, delta);
    else
      kv_report(S.hdr, ST_DEVICE_INPUT);
  }
}

__global__ void __launch_bounds__(PG_THREADS, 1)
    kv_fork_alloc_kernel(const KvCache C, const KvScratch S, const int32_t* src,
                         int32_t* ok) {
  kv_enter();
  __shared__ int sh[64];
  const int tid = threadIdx.x;
  int all = 0;
  for (int base = 0; base < C.batch; base += PG_THREADS) {
    const int b = base + tid;
    int need = 0;
    if (b < C.batch) {
      const int s = fork_src(C, src, b);
      need = s >= 0 && S.keeper[s] != b && (S.len[s] & (C.page - 1)) != 0;
    }
    int total;
    const int at = block_scan(need, sh, &total);
    if (b < C.batch) S.fresh[b] = need ? all + at : -1;
    all += total;
    __syncthreads();
  }
  const int cap = C.batch < C.pages ? C.batch : C.pages;
  const int got = find_free(C, all < cap ? all : cap, S.list, sh);
  for (int b = tid; b < C.batch; b += PG_THREADS) {
    const int raw = kv_ld(src + b);
    bool good = raw >= -1 && raw < C.batch;
    const int r = S.fresh[b];
    if (r >= 0) {
      if (r < got) {
        const int p = S.list[r];
        S.fresh[b] = p;
        C.refs[p] = 1;
      } else {
        S.fresh[b] = -2;  // not covered
        kv_report(S.hdr, ST_NO_PAGES);
        good = false;
      }
    }
    if (ok) ok[b] = good ? 1 : 0;
  }
}

// grid (x: shares of the (layer, head) pairs, y: new rows)
__global__ void __launch_bounds__(128)
    kv_fork_write_kernel(const KvCache C, const KvScratch S, const int32_t* src) {
  kv_enter();
  const int b = blockIdx.y, tid = threadIdx.x;
  const int s = fork_src(C, src, b);
  if (s == b) return;  // the row itself: nothing of it changes (it keeps its partial page)
  const int keep = s >= 0 && S.keeper[s] == b;
  const int len = s >= 0 ? S.len[s] : 0, full = len >> C.lgp, tail = len & (C.page - 1);
  const int fresh = s >= 0 && !keep ? S.fresh[b] : -1;
  if (blockIdx.x == 0) {
    const int np = s < 0 ? 0 : (keep ? S.np[s] : full + (fresh >= 0 ? 1 : 0));
    for (int j = tid; j < C.max_pages; j += blockDim.x) {
      int p = -1;
      if (j < np) p = (!keep && j == full) ? fresh : S.table[(size_t)s * C.max_pages + j];
      C.table[(size_t)b * C.max_pages + j] = p;
    }
    if (tid == 0) {
      C.np[b] = np;
      C.len[b] = fresh == -2 ? full << C.lgp : len;
    }
  }
  if (fresh < 0) return;
  const int from = S.table[(size_t)s * C.max_pages + full];
  if (from < 0 || from >= C.pages) {
    if (tid == 0) kv_report(S.hdr, ST_DEVICE_INPUT);
    return;
  }
  const int nv = tail * C.dim / 16;
  for (int u = blockIdx.x; u < C.layers * C.heads; u += gridDim.x) {
    const int layer = u / C.heads, h = u - layer * C.heads;
    const size_t a = kv_block(C, layer, from, h), d = kv_block(C, layer, fresh, h);
    for (int i = tid; i < nv; i += blockDim.x) {
      const uint4 x = reinterpret_cast<const uint4*>(C.k + a)[i];
      const uint4 y = reinterpret_cast<const uint4*>(C.v + a)[i];
      reinterpret_cast<uint4*>(C.k + d)[i] = x;
      reinterpret_cast<uint4*>(C.v + d)[i] = y;
    }
    if (tid == 0) {
      C.ks[kv_sidx(C, layer, fresh, h)] = C.ks[kv_sidx(C, layer, from, h)];
      C.vs[kv_sidx(C, layer, fresh, h)] = C.vs[kv_sidx(C, layer, from, h)];
    }
  }
}

// ---------------------------------------------------------------------------
// Commit, in two launches: (1) CTAs per row move the kept tokens of their (layer, head)
// pairs; (2) a CTA per row moves len and releases the pages past it. (1) reads a pair's kept
// tokens before it writes any, through shared memory, since a path's sources and targets
// overlap; a block of 16 is 2 KB, so that its time is the chain of table, scales and tokens:
// 12 us for 64 rows of 8 layers and heads, 38 CTAs a row. A chain moves nothing.
// ---------------------------------------------------------------------------
constexpr int CM_THREADS = 128;

// Does row b's commit hold together (counts, length, path, pages)? One warp; every lane gets the
// answer. *moves: is there a token that changes place?
__device__ bool commit_ok(const KvCache& C, int b, int acc, const int32_t* path, int N,
                          bool* moves) {
  const int lane = threadIdx.x & 31;
  bool good = acc >= -1 && acc < N;
  const int len = C.len[b], np = C.np[b];
  good = good && np >= 0 && np <= C.max_pages && len >= 0 && len <= (long long)np << C.lgp;
  bool mv = false;
  if (good && path) {
    bool bad = false;
    for (int i = lane; i < acc; i += 32) {
      const int x = kv_ld(path + (size_t)b * N + i);
      const int prev = i ? kv_ld(path + (size_t)b * N + i - 1) : 0;
      bad = bad || x <= prev || x >= N;
      mv = mv || x != i + 1;
    }
    good = !__any_sync(0xffffffffu, bad);
    mv = __any_sync(0xffffffffu, mv);
  }
  if (good && acc >= 0) {
    const int last = path && acc > 0 ? kv_ld(path + (size_t)b * N + acc - 1) : acc;
    good = (long long)len + last < (1LL << 31) - 1;
    // The row holds the block's pages, and alone those that tokens move to. A lane a page.
    bool bad = false;
    if (good)
      for (int j = (len >> C.lgp) + lane; j <= (len + last) >> C.lgp; j += 32) {
        const int p = kv_page(C, b, j << C.lgp);
        bad = bad || p < 0 || (mv && j <= (len + acc) >> C.lgp && kv_ld(C.refs + p) != 1);
      }
    good = good && !__any_sync(0xffffffffu, bad);
  }
  *moves = mv && good;
  return good;
}

// grid (x: shares of the (layer, head) pairs, y: rows)
__global__ void __launch_bounds__(CM_THREADS)
    kv_commit_move_kernel(const KvCache C, const KvScratch S, const int32_t* accepted,
                          const int32_t* path, int N) {
  kv_enter();
  const int b = blockIdx.y, tid = threadIdx.x;
  __shared__ int s_moves;
  __shared__ int s_src[SV_MAX_TREE], s_dst[SV_MAX_TREE];      // page of each kept token
  __shared__ int s_slot[SV_MAX_TREE], s_dslot[SV_MAX_TREE];   // and its slot there
  __shared__ float s_ss[SV_MAX_TREE], s_ds[SV_MAX_TREE];      // source and new scale
  extern __shared__ __align__(16) uint4 buf[];                // kept tokens of one block
  const int acc = kv_ld(accepted + b);
  if (tid < 32) {
    bool moves;
    const bool good = commit_ok(C, b, acc, path, N, &moves);
    if (tid == 0) {
      s_moves = moves;
      if (blockIdx.x == 0) {
        S.flag[b] = good ? 1 : 0;
        if (!good) kv_report(S.hdr, ST_DEVICE_INPUT);
      }
    }
  }
  __syncthreads();
  if (!s_moves) return;
  const int len = C.len[b], n = acc + 1;
  if (tid < n) {
    const int from = len + (tid ? kv_ld(path + (size_t)b * N + tid - 1) : 0), to = len + tid;
    s_src[tid] = kv_page(C, b, from);
    s_slot[tid] = from & (C.page - 1);
    s_dst[tid] = kv_page(C, b, to);
    s_dslot[tid] = to & (C.page - 1);
  }
  __syncthreads();
  const int vpt = C.dim / 16;  // 16-byte vectors per token
  for (int u = blockIdx.x; u < 2 * C.layers * C.heads; u += gridDim.x) {
    const int kv = u & 1, layer = (u >> 1) / C.heads, h = (u >> 1) - layer * C.heads;
    uint8_t* pool = kv ? C.v : C.k;
    float* scale = kv ? C.vs : C.ks;
    if (tid < n) s_ss[tid] = scale[kv_sidx(C, layer, s_src[tid], h)];
    for (int i = tid; i < n * vpt; i += CM_THREADS) {
      const int t = i / vpt, c = i - t * vpt;
      buf[i] = reinterpret_cast<const uint4*>(pool + kv_block(C, layer, s_src[t], h) +
                                              (size_t)s_slot[t] * C.dim)[c];
    }
    __syncthreads();
    // The new scale of each token's page: the largest source scale among its tokens, older
    // ones (of the first page) included.
    if (tid < n) {
      const float own = scale[kv_sidx(C, layer, s_dst[tid], h)];
      float s = s_dst[tid] == s_dst[0] && (len & (C.page - 1)) ? own : 0.f;
      for (int t = 0; t < n; ++t)
        if (s_dst[t] == s_dst[tid]) s = fmaxf(s, s_ss[t]);
      s_ds[tid] = s;
    }
    __syncthreads();
    // Older tokens of the first page, when its scale grows.
    const int off = len & (C.page - 1);
    const float old = scale[kv_sidx(C, layer, s_dst[0], h)];
    if (off && s_ds[0] != old) {
      uint4* p = reinterpret_cast<uint4*>(pool + kv_block(C, layer, s_dst[0], h));
      for (int i = tid; i < off * vpt; i += CM_THREADS) {
        uint4 x = p[i];
        uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = kv_rescale4(w[j], old, s_ds[0]);
        p[i] = x;
      }
    }
    for (int i = tid; i < n * vpt; i += CM_THREADS) {
      const int t = i / vpt, c = i - t * vpt;
      uint4 x = buf[i];
      if (s_ss[t] != s_ds[t]) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = kv_rescale4(w[j], s_ss[t], s_ds[t]);
      }
      reinterpret_cast<uint4*>(pool + kv_block(C, layer, s_dst[t], h) +
                               (size_t)s_dslot[t] * C.dim)[c] = x;
    }
    __syncthreads();  // every thread has read the old scale
    if (tid < n) scale[kv_sidx(C, layer, s_dst[tid], h)] = s_ds[tid];
    __syncthreads();  // buf and the shared scales are used again
  }
}

__global__ void __launch_bounds__(CM_THREADS)
    kv_commit_release_kernel(const KvCache C, const KvScratch S,
                             const int32_t* accepted) {
  kv_enter();
  const int b = blockIdx.x, tid = threadIdx.x;
  __shared__ int s_len, s_np;
  if (tid == 0) {
    s_len = C.len[b] + kv_ld(accepted + b) + 1;
    s_np = C.np[b];  // (in range when the flag is set)
  }
  __syncthreads();
  if (!S.flag[b]) return;
  const int np = s_np, used = min(np, (s_len + C.page - 1) >> C.lgp);
  for (int j = used + tid; j < np; j += CM_THREADS) {
    int32_t* e = C.table + (size_t)b * C.max_pages + j;
    const int p = *e;
    if (p >= 0 && p < C.pages)
      atomicSub(C.refs + p, 1);
    else
      kv_report(S.hdr, ST_DEVICE_INPUT);
    *e = -1;
  }
  if (tid == 0) {
    C.len[b] = s_len;
    C.np[b] = used;
  }
}

// ---------------------------------------------------------------------------

cudaError_t launch_kv_reserve(const KvCache& C, const KvScratch& S, const int32_t* n_new,
                              int32_t* ok, cudaStream_t st) {
  return kv_launch(kv_reserve_kernel, dim3(1), PG_THREADS, 4 * (size_t)C.batch, st, C, S, n_new, ok);
}

// Shares of the (layer, head) pairs per row: enough CTAs to fill the GPU a few times over.
static int shares(const KvCache& C, int pairs) {
  const int want = (152 * 16 + C.batch - 1) / C.batch;
  return want < pairs ? want : pairs;
}

cudaError_t launch_kv_fork(const KvCache& C, const KvScratch& S, const int32_t* src, int32_t* ok,
                           cudaStream_t st) {
  cudaError_t e = kv_launch(kv_fork_count_kernel, dim3(C.batch), 128, 0, st, C, S, src);
  if (e != cudaSuccess) return e;
  e = kv_launch(kv_fork_alloc_kernel, dim3(1), PG_THREADS, 0, st, C, S, src, ok);
  if (e != cudaSuccess) return e;
  const dim3 grid(shares(C, C.layers * C.heads), C.batch);
  return kv_launch(kv_fork_write_kernel, grid, 128, 0, st, C, S, src);
}

cudaError_t launch_kv_commit(const KvCache& C, const KvScratch& S, const int32_t* acc,
                             const int32_t* path, int N, cudaStream_t st) {
  // A chain moves nothing: one CTA per row checks it.
  const dim3 grid(path ? shares(C, 2 * C.layers * C.heads) : 1, C.batch);
  const size_t smem = path ? (size_t)N * C.dim : 0;
  const cudaError_t e = kv_launch(kv_commit_move_kernel, grid, CM_THREADS, smem, st, C, S, acc, path, N);
  if (e != cudaSuccess) return e;
  return kv_launch(kv_commit_release_kernel, dim3(C.batch), CM_THREADS, 0, st, C, S, acc);
}

}  // namespace sv
