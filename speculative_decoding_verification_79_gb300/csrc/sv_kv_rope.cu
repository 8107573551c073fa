// sv_kv_rope.cu -- appending rotated keys, and values, to the key/value cache, and rotating the
// queries, in one launch (sm_103a).
//
// A block takes the keys (or the values) of one page of one row, head after head: loads a head's
// new tokens, rotates them in float32, reduces the largest |x| over the block for the page's scale
// and rounds once, to e4m3. A thread has the same pairs of the same token in every head, so that
// their cosines and sines stay in its registers, and the next head's loads are under way while a
// head's largest value is found. Blocks behind those of keys and values rotate the queries
// (rope_row). Bound by memory: 8 prompts of 4,093 tokens with 8 heads and 32 query heads of 128
// take 128 us, 738 MB at 5.8 TB/s (the queries alone 80). A few tokens of many rows take the trips
// to memory one after the other (lengths, table, counts of holders, old scale, beside the tokens
// themselves): 64 rows 5.1 us for a token, 9.5 us for trees of 16.
//
// What decides is that the loop over heads has no call in it and fits 64 registers, so that an SM
// holds 1,024 threads: with calls for the rare cases inside it (another quantiser's scale, the
// rescaling of older tokens, divisions) it spilt on every head, and those prompts took 232 us. So
// the loop leaves a page's rare cases to append_rest, behind it. (Which was given what it needs by
// the loop's block, kept in registers meanwhile: 135 us; with the block's maximum found by shuffles
// and a loop: 141.)
//
// It fits for 16-bit values with rot a multiple of 16. Others spill, and a page of more than 16,384
// values (128 tokens of 192 or 256 components) goes to append_rest whole, which reads it twice and
// computes cosines for each head again. Those prompts with keys and queries, and keys and values alone
// (beside sv_kv_append, which does not rotate), us:
//   dim 128, rot 128, pages of 64 / 128, bf16      128, 58 (43) / 141, 69 (45)
//   the same, pages of 64, float32                 231, 73 (61); 160 to 184 bytes of spill loads
//   dim 80, rot 40, bf16                           103, 43 (33); 40 to 64 (4 pairs a thread)
//   dim 80, rot 20, bf16                           272, 129 (33); 270 to 370 (single pairs)
//   dim 192, pages of 64 / 128, bf16               240, 109 (62) / 367, 258 (68)
//   dim 256, pages of 64 / 128, bf16               279, 125 (80) / 445, 308 (93)
//   dim 256, pages of 128, float32                 659, 363 (167)
#include "sv_rope.cuh"

namespace sv {

// Threads of a block: one for 16 values of the new tokens of a page, in whole warps, as far as that
// goes. (The queries in a launch of their own: those prompts 149 us instead of 140, as it was then,
// trees 15.2 instead of 10.8. Twice or four times as many blocks, of fewer heads each: 153 and 167
// us, the cosines being computed again. At least 32, 64, 128 and 256 threads: 7.1, 6.7, 7.8 and 8.7
// us for a token of 64 rows with 64 query heads, appended and read.)
constexpr int AR_LEAST = 64, AR_MOST = 1024;
constexpr int AR_VALUES = 16;  // of a page and head that a thread keeps in registers
constexpr int AR_PER = 32;     // heads of a block

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

// The largest |x| that the scales' range holds; `odd` when another one is there.
template <int P>
__device__ __forceinline__ float append_seen(const float* x, bool* odd) {
  float a = 0.f;
#pragma unroll
  for (int e = 0; e < 2 * P; ++e) {
    const float y = fabsf(x[e]);
    if (y <= KV_XMAX)
      a = fmaxf(a, y);
    else
      *odd = true;
  }
  return a;
}

// The scale of a page and head from the largest |x| of each thread's values (whole block). `mx`:
// shared memory that no thread reads any more.
__device__ __forceinline__ float append_scale(float a, float old, float* scale, uint32_t* mx) {
  const int tid = threadIdx.x, lane = tid & 31;
  // (Numbers from 0 on are in the order of their bits.)
  const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(a));
  if (lane == 0) mx[tid >> 5] = most;
  __syncthreads();  // (and every thread has read the old scale)
  const uint32_t x = lane < static_cast<int>(blockDim.x) / 32 ? mx[lane] : 0;
  a = __uint_as_float(__reduce_max_sync(0xffffffffu, x));
  const float s = fmaxf(kv_scale(a), old);
  if (tid == 0) *scale = s;
  return s;
}

// Is s a power of two whose reciprocal is a normal number too? (Any other scale is of another
// quantiser.)
__device__ __forceinline__ bool append_plain(float s) {
  const uint32_t u = __float_as_uint(s);
  return (u & 0x807fffffu) == 0 && u >= 0x00800000u && u <= 0x7e800000u;
}

// A block's part of a row: keys (ROT) or values of heads h0 .. h1 - 1 in one page, the row's j-th,
// of which the first `off` tokens are older.
template <int P, bool ROT>
struct AppendPart {
  KvSrc src;
  uint8_t* pool;
  float* scales;
  int b, j, h0, h1, len, n, off;
  PagePart g;
  __device__ __forceinline__ explicit AppendPart(const AppendRopeArgs& A) {
    const KvCache& C = A.C;
    b = blockIdx.y;
    n = A.n_new ? kv_ld(A.n_new + b) : A.T;
    len = kv_ld(C.len + b);
    const int i = blockIdx.x - (ROT ? 0 : A.pages * A.chunks), chunk = i / A.pages;
    j = (len >> C.lgp) + i - chunk * A.pages;
    h0 = chunk * A.per;
    h1 = min(h0 + A.per, C.heads);
    src = ROT ? A.k : A.v;
    pool = ROT ? C.k : C.v;
    scales = ROT ? C.ks : C.vs;
    const int lo = max(len, j << C.lgp), hi = min(len + n, (j + 1) << C.lgp);
    g = PagePart{lo - len, hi - lo, C.dim / (2 * P), b * src.row};
    off = lo - (j << C.lgp);
  }
};

// What the registers' path leaves, head by head: a page's older tokens, brought from scale `old` to
// the page's new one; the new tokens when that is no plain power of two; and, in a page whose new
// tokens exceed the block's registers (`large`), its scale and tokens in two passes over the values.
// (It finds out by itself what part the block has, so that nothing for it is kept in registers.)
template <typename E, int P, bool INTER, bool ROT>
__device__ __noinline__ void append_rest(const AppendRopeArgs& A, const int* depth, const float* s_old,
                                         uint32_t* s_max, bool large) {
  const AppendPart<P, ROT> W(A);
  const RowPos pos{W.len, depth};
  const int nu = W.g.count * W.g.units, step = static_cast<int>(blockDim.x);
  const int page = kv_page(A.C, W.b, W.j << A.C.lgp);
  for (int h = W.h0; h < W.h1; ++h) {
    uint8_t* dst = W.pool + kv_block(A.C, A.layer, page, h);
    float* const scale = W.scales + kv_sidx(A.C, A.layer, page, h);
    float old = s_old[h - W.h0];
    float s;
    if (large) {
      old = W.off ? kv_ld(scale) : 0.f;
      float a = 0.f;
      bool odd = false;
      for (int i = threadIdx.x; i < nu; i += step) {
        float x[2 * P];
        RopeUnit<P, INTER> unit(0, 0);
        load_unit<E, P, INTER, ROT>(A, W.src, W.g, i, h, pos, x, &unit);
        a = fmaxf(a, append_seen<P>(x, &odd));
      }
      if (odd) kv_report(A.S.hdr, ST_DEVICE_INPUT);
      s = append_scale(a, old, scale, s_max + (h & 1) * 32);
    } else {
      s = kv_ld(scale);
    }
    if (W.off && s != old)
      for (int i = threadIdx.x; i < W.off * A.C.dim / 16; i += step) {
        uint4 x = reinterpret_cast<uint4*>(dst)[i];
        uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = kv_rescale4(w[q], old, s);
        reinterpret_cast<uint4*>(dst)[i] = x;
      }
    if (!large && append_plain(s)) continue;
    dst += (size_t)W.off * A.C.dim;
    const bool pow2 = kv_pow2(s);
    const float inv = pow2 ? 1.f / s : 1.f;
    for (int i = threadIdx.x; i < nu; i += step) {
      float x[2 * P];
      RopeUnit<P, INTER> unit(0, 0);
      const int t = load_unit<E, P, INTER, ROT>(A, W.src, W.g, i, h, pos, x, &unit);
      if (!pow2) {
#pragma unroll
        for (int e = 0; e < 2 * P; ++e) x[e] = kv_quotient(x[e], 1.f, s);
      }
      put_e4m3<P>(dst + (size_t)t * A.C.dim + unit.lo, x, inv);
      put_e4m3<P>(dst + (size_t)t * A.C.dim + unit.hi, x + P, inv);
    }
  }
}

// Keys (ROT) or values.
template <typename E, int P, bool INTER, bool ROT>
__device__ __forceinline__ void append_page(const AppendRopeArgs& A, const int* depth) {
  __shared__ uint32_t s_max[2][32];
  __shared__ float s_old[AR_PER];
  const KvCache& C = A.C;
  const AppendPart<P, ROT> W(A);
  const PagePart& g = W.g;
  const KvSrc& src = W.src;
  const int tid = threadIdx.x, nu = g.count * g.units, off = W.off, h0 = W.h0, h1 = W.h1;
  const int rot = ROT ? A.R.rot : 0;
  constexpr int K = AR_VALUES / (2 * P);
  const E* const base = static_cast<const E*>(src.p) + g.row + (long long)g.t0 * src.tok;
  // Of this thread's units: the token, where its two vectors begin, and whether it is rotated.
  const E* from[K];
  int to[K], gap[K];
  bool turns[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int i = tid + k * static_cast<int>(blockDim.x), t = i / g.units;
    const RopeUnit<P, INTER> unit(i - t * g.units, rot);
    from[k] = base + (long long)t * src.tok + (size_t)h0 * C.dim + unit.lo;
    to[k] = i < nu ? t * C.dim + unit.lo : -1;
    gap[k] = unit.hi - unit.lo;
    turns[k] = ROT && unit.turns;
  }
  float2 cs[ROT ? K : 1][P];
  RopeVec<E, P> raw[K][2];
  auto fetch = [&]() {  // the next head's
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (to[k] < 0) break;
      raw[k][0].load(from[k]);
      raw[k][1].load(from[k] + gap[k]);
      from[k] += C.dim;
    }
  };
  const bool large = nu > K * static_cast<int>(blockDim.x);
  if (!large) fetch();
  // (The tokens are on their way while the row's pages are looked up: is every one that it writes its
  // own?)
  const int page = kv_page(C, W.b, W.j << C.lgp);
  const bool fine =
      A.checked ? kv_ld(A.S.flag + W.b) != 0 : kv_append_holds(C, W.b, W.len, W.n);
  if (!__syncthreads_and(fine ? 1 : 0)) {
    if (tid == 0 && blockIdx.x == 0 && !A.checked) kv_report(A.S.hdr, ST_DEVICE_INPUT);
    return;
  }
  if (nu <= 0) return;
  if (large) {
    append_rest<E, P, INTER, ROT>(A, depth, s_old, s_max[0], true);
    return;
  }
  if constexpr (ROT) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = tid + k * static_cast<int>(blockDim.x), t = i / g.units;
      if (i < nu && turns[k]) rope_turns<P>(A.R, RowPos{W.len, depth}(g.t0 + t), i - t * g.units, cs[k]);
    }
  }
  bool more = false;  // a scale has changed, or is no plain power of two
  float* scale = W.scales + kv_sidx(C, A.layer, page, h0);
  uint8_t* out = W.pool + kv_block(C, A.layer, page, h0) + (size_t)off * C.dim;
  const int block = C.page * C.dim;
  for (int h = h0; h < h1; ++h, ++scale, out += block) {
    const float old = off ? kv_ld(scale) : 0.f;
    float f[K][2 * P], a = 0.f;
    uint32_t most = 0;  // of |x|, whose order as numbers is that of their bits, NaN above all
    bool odd = false;  // a value outside the scales' range
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (to[k] < 0) break;
      raw[k][0].get(f[k]);
      raw[k][1].get(f[k] + P);
      if (turns[k]) rope_apply<P, INTER>(f[k], cs[ROT ? k : 0]);
#pragma unroll
      for (int e = 0; e < 2 * P; e += 2)
        most = __vimax3_u32(most, __float_as_uint(fabsf(f[k][e])), __float_as_uint(fabsf(f[k][e + 1])));
    }
    if (h + 1 < h1) fetch();
    if (most <= __float_as_uint(KV_XMAX)) {
      a = __uint_as_float(most);
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (to[k] >= 0) a = fmaxf(a, append_seen<P>(f[k], &odd));
    }
    if (odd) kv_report(A.S.hdr, ST_DEVICE_INPUT);
    if (tid == 0) s_old[h - h0] = old;
    const float s = append_scale(a, old, scale, s_max[h & 1]);
    more = more || (off && s != old) || !append_plain(s);
    if (!append_plain(s)) continue;
    const float inv = __uint_as_float(0x7f000000u - __float_as_uint(s));  // 1 / s
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (to[k] < 0) break;
      put_e4m3<P>(out + to[k], f[k], inv);
      put_e4m3<P>(out + to[k] + gap[k], f[k] + P, inv);
    }
  }
  if (more) {  // (the same in every thread)
    __syncthreads();
    append_rest<E, P, INTER, ROT>(A, depth, s_old, s_max[0], false);
  }
}

// grid (x: blocks of keys, of values, of queries; y: rows)
template <typename E, int P, bool INTER>
__global__ void __launch_bounds__(AR_MOST)
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
    rope_row<E, P, INTER, 2>(A.R, w, (blockIdx.x - 2 * kv_blocks) * blockDim.x + tid,
                             A.q_blocks * blockDim.x, pos);
    return;
  }
  if (bad || n == 0) return;
  if (!kv_append_fits(C, len, n, T)) {
    if (tid == 0 && blockIdx.x == 0 && !A.checked) kv_report(A.S.hdr, ST_DEVICE_INPUT);
    return;
  }
  const int* const depth = A.parent ? s_depth : nullptr;
  if (values)
    append_page<E, 8, false, false>(A, depth);
  else
    append_page<E, P, INTER, true>(A, depth);
}

template <typename E>
static cudaError_t launch_type(const AppendRopeArgs& A, bool inter, dim3 grid, int threads,
                               cudaStream_t st) {
  const int P = rope_pairs(A.R.rot);
  auto* kernel = P == 8   ? (inter ? kv_append_rope_kernel<E, 8, true> : kv_append_rope_kernel<E, 8, false>)
                 : P == 4 ? (inter ? kv_append_rope_kernel<E, 4, true> : kv_append_rope_kernel<E, 4, false>)
                          : (inter ? kv_append_rope_kernel<E, 1, true> : kv_append_rope_kernel<E, 1, false>);
  return kv_launch(kernel, grid, threads, 0, st, A);
}

cudaError_t launch_kv_append_rope(AppendRopeArgs& A, bool inter, sv_dtype dt, cudaStream_t st) {
  const KvCache& C = A.C;
  // A row's tokens start anywhere in a page, so T of them touch at most this many.
  A.pages = (A.T + C.page - 2) / C.page + 1;
  const int tokens = A.T < C.page ? A.T : C.page;
  int threads = (tokens * C.dim / AR_VALUES + 31) / 32 * 32;
  threads = threads < AR_LEAST ? AR_LEAST : (threads > AR_MOST ? AR_MOST : threads);
  // Heads of a block: all of them, which computes cosines once, or fewer while the blocks do not
  // fill the SMs.
  const long long blocks = 2LL * A.pages * C.batch;
  const long long want = (152LL * AR_MOST / threads + blocks - 1) / blocks;
  const long long least = (C.heads + AR_PER - 1) / AR_PER;
  const int cut = static_cast<int>(want < least ? least : (want < C.heads ? want : C.heads));
  A.per = (C.heads + cut - 1) / cut;
  A.chunks = (C.heads + A.per - 1) / A.per;
  A.q_blocks = 0;
  if (A.q.heads) {
    const int units = (A.q.same ? A.R.rot : A.q.dim) / (2 * rope_pairs(A.R.rot));
    rope_cut(C.batch, A.T, A.q.heads, units, threads, AR_MOST, &A.q.shares, &A.q_blocks);
  }
  A.checked = A.pages > KV_APPEND_CHECK;
  if (A.checked) {
    const cudaError_t e = launch_kv_append_check(C, A.S, A.T, A.n_new, st);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid(2 * A.pages * A.chunks + A.q_blocks, C.batch);
  return dt == SV_F32    ? launch_type<float>(A, inter, grid, threads, st)
         : dt == SV_BF16 ? launch_type<__nv_bfloat16>(A, inter, grid, threads, st)
                         : launch_type<__half>(A, inter, grid, threads, st);
}

}  // namespace sv
