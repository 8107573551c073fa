// sv_kv_rope.cu -- appending rotated keys, and values, to the key/value cache, and rotating the
// queries, in one launch (sm_103a).
//
// A block takes the keys (or the values) of one page of one row, head after head: loads a head's
// new tokens, rotates them in float32, reduces the largest |x| over the block for the page's scale
// and rounds once, to e4m3. A thread has the same pairs of the same tokens in every head, so that
// their cosines and sines stay in its registers, and the next head's loads are under way while a
// head's largest value is found. Blocks behind those of keys and values rotate the queries
// (rope_row). Bound by memory.
#include "sv_rope.cuh"

namespace sv {

constexpr int AR_THREADS = 256;
constexpr int AR_VALUES = 32;  // of a page and head that a thread keeps in registers

template <int P>
__device__ __forceinline__ void put_e4m3(uint8_t* p, const float* f, float inv) {
  if constexpr (P == 8)
    *reinterpret_cast<uint2*>(p) =
        make_uint2(e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                   e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
  else if constexpr (P == 4)
    *reinterpret_cast<uint32_t*>(p) = e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
  else
    *p = static_cast<uint8_t>(e4m3x4(f[0] * inv, 0.f, 0.f, 0.f));
}

// Position of a row's new token t: in a chain or, with depths, in a draft tree.
struct RowPos {
  long long len;
  const int* depth;
  __device__ __forceinline__ long long operator()(int t) const { return len + (depth ? depth[t] : t); }
};

// Part of a page that a block fills: the new tokens t0 .. t0 + count - 1 of a row.
struct PagePart {
  int t0, count, units;
  long long row;  // of the source, in elements
};

// Values of unit i (token by token) of head h, rotated when ROT; returns the token in the part.
template <typename E, int P, bool INTER, bool ROT>
__device__ __forceinline__ int load_unit(const AppendRopeArgs& A, const KvSrc& src, const PagePart& g,
                                         int i, int h, RowPos pos, float* f,
                                         RopeUnit<P, INTER>* unit) {
  const int t = i / g.units, u = i - t * g.units;
  *unit = RopeUnit<P, INTER>(u, ROT ? A.R.rot : 0);
  const E* x = static_cast<const E*>(src.p) + g.row + (long long)(g.t0 + t) * src.tok +
               (size_t)h * A.C.dim;
  RopeVec<E, P> a, b;
  a.load(x + unit->lo);
  b.load(x + unit->hi);
  a.get(f);
  b.get(f + P);
  if (ROT && unit->turns) {
    float2 cs[P];
    rope_turns<P>(A.R, pos(g.t0 + t), u, cs);
    rope_apply<P, INTER>(f, cs);
  }
  return t;
}

// The new values of a head at a scale that is no power of two, which another quantiser gave the
// page. (On a path of its own, which reads the values again: it leaves the registers to the rest.)
template <typename E, int P, bool INTER, bool ROT>
__device__ __noinline__ void append_any(const AppendRopeArgs& A, const KvSrc& src, const PagePart& g,
                                        int h, RowPos pos, uint8_t* out, float s) {
  for (int i = threadIdx.x; i < g.count * g.units; i += AR_THREADS) {
    float x[2 * P];
    RopeUnit<P, INTER> unit(0, 0);
    const int t = load_unit<E, P, INTER, ROT>(A, src, g, i, h, pos, x, &unit);
#pragma unroll
    for (int e = 0; e < 2 * P; ++e) x[e] = kv_quotient(x[e], 1.f, s);
    put_e4m3<P>(out + (size_t)t * A.C.dim + unit.lo, x, 1.f);
    put_e4m3<P>(out + (size_t)t * A.C.dim + unit.hi, x + P, 1.f);
  }
}

// Keys or values of heads h0 .. h1 - 1 in one page, the row's j-th. ROT: they are rotated.
template <typename E, int P, bool INTER, bool ROT>
__device__ __forceinline__ void append_page(const AppendRopeArgs& A, const KvSrc& src, uint8_t* pool,
                                            float* scales, int b, int j, int h0, int h1, int len,
                                            int n, int page, RowPos pos) {
  __shared__ float s_max[2][AR_THREADS / 32];
  const KvCache& C = A.C;
  const int tid = threadIdx.x, lo = max(len, j << C.lgp), hi = min(len + n, (j + 1) << C.lgp);
  const PagePart g{lo - len, hi - lo, C.dim / (2 * P), b * src.row};
  const int nu = g.count * g.units, off = lo - (j << C.lgp), rot = ROT ? A.R.rot : 0;
  constexpr int K = AR_VALUES / (2 * P);
  const E* const base = static_cast<const E*>(src.p) + g.row + (long long)g.t0 * src.tok;
  float2 cs[ROT ? K : 1][P];
  RopeVec<E, P> raw[K][2];
  auto fetch = [&](int h) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = tid + k * AR_THREADS;
      if (i >= nu) break;
      const int t = i / g.units;
      const RopeUnit<P, INTER> unit(i - t * g.units, rot);
      const E* x = base + (long long)t * src.tok + (size_t)h * C.dim;
      raw[k][0].load(x + unit.lo);
      raw[k][1].load(x + unit.hi);
    }
  };
  fetch(h0);
  if constexpr (ROT) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = tid + k * AR_THREADS, t = i / g.units, u = i - t * g.units;
      if (i < nu && 2 * P * u < rot) rope_turns<P>(A.R, pos(g.t0 + t), u, cs[k]);
    }
  }
  for (int h = h0; h < h1; ++h) {
    float* const scale = scales + kv_sidx(C, A.layer, page, h);
    const float old = off ? kv_ld(scale) : 0.f;
    float f[K][2 * P], a = 0.f;
    bool odd = false;  // a value outside the scales' range
    auto see = [&](const float* x) {
#pragma unroll
      for (int e = 0; e < 2 * P; ++e) {
        const float y = fabsf(x[e]);
        if (y <= KV_XMAX)
          a = fmaxf(a, y);
        else
          odd = true;
      }
    };
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = tid + k * AR_THREADS;
      if (i >= nu) break;
      raw[k][0].get(f[k]);
      raw[k][1].get(f[k] + P);
      if (ROT && 2 * P * (i % g.units) < rot) rope_apply<P, INTER>(f[k], cs[ROT ? k : 0]);
      see(f[k]);
    }
    if (h + 1 < h1) fetch(h + 1);
    // (Values past the registers' share are loaded, and rotated, again for the second step.)
    for (int i = tid + K * AR_THREADS; i < nu; i += AR_THREADS) {
      float x[2 * P];
      RopeUnit<P, INTER> unit(0, 0);
      load_unit<E, P, INTER, ROT>(A, src, g, i, h, pos, x, &unit);
      see(x);
    }
    if (odd) kv_report(A.S.hdr, ST_DEVICE_INPUT);
#pragma unroll
    for (int d = 16; d; d >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
    float* const mx = s_max[(h - h0) & 1];
    if ((tid & 31) == 0) mx[tid >> 5] = a;
    __syncthreads();  // (every thread has read the old scale; the other half of s_max is free)
#pragma unroll
    for (int w = 0; w < AR_THREADS / 32; ++w) a = fmaxf(a, mx[w]);
    const float s = fmaxf(kv_scale(a), old);
    uint8_t* const dst = pool + kv_block(C, A.layer, page, h);
    if (off && s != old)  // older tokens of the page, at its new scale
      for (int i = tid; i < off * C.dim / 16; i += AR_THREADS) {
        uint4 x = reinterpret_cast<uint4*>(dst)[i];
        uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = kv_rescale4(w[q], old, s);
        reinterpret_cast<uint4*>(dst)[i] = x;
      }
    if (tid == 0) *scale = s;
    uint8_t* const out = dst + (size_t)off * C.dim;
    if (!kv_pow2(s)) {
      append_any<E, P, INTER, ROT>(A, src, g, h, pos, out, s);
      continue;
    }
    const float inv = 1.f / s;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = tid + k * AR_THREADS;
      if (i >= nu) break;
      const int t = i / g.units;
      const RopeUnit<P, INTER> unit(i - t * g.units, rot);
      put_e4m3<P>(out + (size_t)t * C.dim + unit.lo, f[k], inv);
      put_e4m3<P>(out + (size_t)t * C.dim + unit.hi, f[k] + P, inv);
    }
    for (int i = tid + K * AR_THREADS; i < nu; i += AR_THREADS) {
      float x[2 * P];
      RopeUnit<P, INTER> unit(0, 0);
      const int t = load_unit<E, P, INTER, ROT>(A, src, g, i, h, pos, x, &unit);
      put_e4m3<P>(out + (size_t)t * C.dim + unit.lo, x, inv);
      put_e4m3<P>(out + (size_t)t * C.dim + unit.hi, x + P, inv);
    }
  }
}

// grid (x: blocks of keys, of values, of queries; y: rows)
template <typename E, int P, bool INTER>
__global__ void __launch_bounds__(AR_THREADS, sizeof(E) == 2 ? 2 : 1)
    kv_append_rope_kernel(const __grid_constant__ AppendRopeArgs A) {
  kv_enter();
  __shared__ int s_par[SV_MAX_TREE], s_depth[SV_MAX_TREE];
  const KvCache& C = A.C;
  const int b = blockIdx.y, T = A.T, tid = threadIdx.x, kv_blocks = A.pages * A.chunks;
  const int n = A.n_new ? kv_ld(A.n_new + b) : T, len = kv_ld(C.len + b);
  bool bad = n < 0 || n > T || len < 0;
  const bool values = static_cast<int>(blockIdx.x) >= kv_blocks;
  const bool queries = static_cast<int>(blockIdx.x) >= 2 * kv_blocks;
  if (A.parent && !bad)  // (values need no positions, but a row whose tree is wrong stays as it is)
    bad = !rope_depths(A.parent + (size_t)b * T, n, s_par, s_depth);
  const RowPos pos{len, A.parent ? s_depth : nullptr};
  if (bad && blockIdx.x == 0 && tid == 0) kv_report(A.S.hdr, ST_DEVICE_INPUT);
  if (queries) {
    RopeRow w = A.q;
    w.x = static_cast<const E*>(A.q.x) + b * A.q_row;
    w.out = static_cast<E*>(A.q.out) + b * A.q_out_row;
    w.n = n;
    w.bad = bad;
    rope_row<E, P, INTER>(A.R, w, (blockIdx.x - 2 * kv_blocks) * AR_THREADS + tid,
                          A.q_blocks * AR_THREADS, pos);
    return;
  }
  if (bad || n == 0) return;
  const int i = blockIdx.x - (values ? kv_blocks : 0);
  const int chunk = i / A.pages, j = (len >> C.lgp) + i - chunk * A.pages;
  // Every page that the row writes is its own.
  const bool sane = kv_append_fits(C, len, n, T);
  const bool fine = A.checked ? kv_ld(A.S.flag + b) != 0 : sane && kv_append_holds(C, b, len, n);
  if (!__syncthreads_and(fine ? 1 : 0)) {
    if (tid == 0 && blockIdx.x == 0 && !A.checked) kv_report(A.S.hdr, ST_DEVICE_INPUT);
    return;
  }
  if ((long long)j << C.lgp >= (long long)len + n) return;
  const int page = kv_page(C, b, j << C.lgp), h0 = chunk * A.per, h1 = min(h0 + A.per, C.heads);
  if (values)
    append_page<E, 8, false, false>(A, A.v, C.v, C.vs, b, j, h0, h1, len, n, page, pos);
  else
    append_page<E, P, INTER, true>(A, A.k, C.k, C.ks, b, j, h0, h1, len, n, page, pos);
}

template <typename E>
static cudaError_t launch_type(const AppendRopeArgs& A, bool inter, dim3 grid, cudaStream_t st) {
  const int P = rope_pairs(A.R.rot);
  auto* kernel = P == 8   ? (inter ? kv_append_rope_kernel<E, 8, true> : kv_append_rope_kernel<E, 8, false>)
                 : P == 4 ? (inter ? kv_append_rope_kernel<E, 4, true> : kv_append_rope_kernel<E, 4, false>)
                          : (inter ? kv_append_rope_kernel<E, 1, true> : kv_append_rope_kernel<E, 1, false>);
  return kv_launch(kernel, grid, AR_THREADS, 0, st, A);
}

cudaError_t launch_kv_append_rope(AppendRopeArgs& A, bool inter, sv_dtype dt, cudaStream_t st) {
  const KvCache& C = A.C;
  // A row's tokens start anywhere in a page, so T of them touch at most this many.
  A.pages = (A.T + C.page - 2) / C.page + 1;
  // Heads of a block: all of them, which computes cosines once, or fewer while the blocks are
  // not four to an SM.
  const long long blocks = 2LL * A.pages * C.batch;
  const long long want = (4 * 152 + blocks - 1) / blocks;
  const int cut = static_cast<int>(want < C.heads ? want : C.heads);
  A.per = (C.heads + cut - 1) / cut;
  A.chunks = (C.heads + A.per - 1) / A.per;
  A.q_blocks = 0;
  if (A.q.heads) {
    const int units = (A.q.same ? A.R.rot : A.q.dim) / (2 * rope_pairs(A.R.rot));
    rope_cut(C.batch, A.T, A.q.heads, units, AR_THREADS, &A.q.shares, &A.q_blocks);
  }
  A.checked = A.pages > KV_APPEND_CHECK;
  if (A.checked) {
    const cudaError_t e = launch_kv_append_check(C, A.S, A.T, A.n_new, st);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid(2 * A.pages * A.chunks + A.q_blocks, C.batch);
  return dt == SV_F32    ? launch_type<float>(A, inter, grid, st)
         : dt == SV_BF16 ? launch_type<__nv_bfloat16>(A, inter, grid, st)
                         : launch_type<__half>(A, inter, grid, st);
}

}  // namespace sv
