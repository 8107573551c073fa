// sv_rope.cuh -- rotary positions: angles, vectors of pairs, and the rotation of a row's tokens,
// shared by the kernels that rotate (sv_rope.cu, sv_kv_rope.cu).
//
// Angles are kept in turns, as fractions of 2^64: a position is a whole number, so position times
// frequency modulo a turn is one 64-bit product that wraps, exact for any position and off by
// no more than position * 2^-65 for the frequency's own rounding. (In float32 the product is off by
// 2^-7 radians at position 131,072; in float64 it needs instructions that this GPU has few of.)
// The upper 32 bits go to sincospi as float32 half turns; what that cut off turns the result a bit
// further (sin(a + e) = sin a + e cos a), which keeps keys that lie next to a rounding border of
// e4m3 on their side of it as often as correctly rounded cosines do. A component is off by 2^-21
// of its pair's length at most, before its own rounding.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sv_kv.cuh"

namespace sv {

// sv_rope_spec as kernels see it; the gain is that of the cosine, sgain that of the sine (negative
// for the inverse).
struct Rope {
  const int64_t* freq;
  int rot;
  float gain, sgain;
};

// Pairs of a thread, by the rotated size: 8, whose halves are 16-byte vectors of 16-bit values when
// the second half begins at a multiple of 8 components; else 4 or 1, as its alignment allows. (The
// components that stay as they are go the same way. 8 x 4,093 tokens of 32 heads of 80 in bf16: 52 us,
// 6.4 TB/s, with rot 40; 99 us, 3.4 TB/s, with rot 20, in float32 111 us at 6.1. 8 heads of 512: 80 us
// with rot 32, 136 with rot 30.)
inline int rope_pairs(int rot) { return rot % 16 == 0 ? 8 : (rot % 8 == 0 ? 4 : 1); }

__device__ __forceinline__ float2 rope_turn(const Rope& R, long long pos, int64_t freq) {
  const unsigned long long a =
      static_cast<unsigned long long>(pos) * static_cast<unsigned long long>(freq);
  const int turn = static_cast<int>(a >> 32);
  const float cut = __int2float_rz(turn);
  const float e = static_cast<float>(turn - static_cast<int>(cut)) * (3.14159265f * 0x1p-31f);
  float s, c;
  sincospif(cut * 0x1p-31f, &s, &c);
  return make_float2(fmaf(-s, e, c) * R.gain, fmaf(c, e, s) * R.sgain);
}

template <typename E>
__device__ __forceinline__ float2 rope_two(uint32_t w);
template <>
__device__ __forceinline__ float2 rope_two<__nv_bfloat16>(uint32_t w) {
  return make_float2(bf_lo(w), bf_hi(w));
}
template <>
__device__ __forceinline__ float2 rope_two<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename E>
__device__ __forceinline__ uint32_t rope_pack(float a, float b);
template <>
__device__ __forceinline__ uint32_t rope_pack<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 y = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&y);
}
template <>
__device__ __forceinline__ uint32_t rope_pack<__half>(float a, float b) {
  const __half2 y = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&y);
}

// P consecutive elements (their address is a multiple of their size, up to 16 bytes).
template <typename E, int P>
struct RopeVec {
  static constexpr int B = P * static_cast<int>(sizeof(E)), W = B < 4 ? 1 : B / 4;
  uint32_t w[W];
  __device__ __forceinline__ void load(const E* p) {
    if constexpr (B >= 16) {
#pragma unroll
      for (int i = 0; i < B / 16; ++i) {
        const uint4 x = kv_ld(reinterpret_cast<const uint4*>(p) + i);
        w[4 * i] = x.x;
        w[4 * i + 1] = x.y;
        w[4 * i + 2] = x.z;
        w[4 * i + 3] = x.w;
      }
    } else if constexpr (B == 8) {
      const uint2 x = kv_ld(reinterpret_cast<const uint2*>(p));
      w[0] = x.x;
      w[1] = x.y;
    } else if constexpr (B == 4) {
      w[0] = kv_ld(reinterpret_cast<const uint32_t*>(p));
    } else {
      w[0] = kv_ld(reinterpret_cast<const uint16_t*>(p));
    }
  }
  __device__ __forceinline__ void store(E* p) const {
    if constexpr (B >= 16) {
#pragma unroll
      for (int i = 0; i < B / 16; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else if constexpr (B == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else if constexpr (B == 4) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else {
      *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
    }
  }
  __device__ __forceinline__ void get(float* f) const {
    if constexpr (sizeof(E) == 4) {
#pragma unroll
      for (int i = 0; i < P; ++i) f[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float2 y = rope_two<E>(w[i]);
        f[2 * i] = y.x;
        if (2 * i + 1 < P) f[2 * i + 1] = y.y;
      }
    }
  }
  __device__ __forceinline__ void set(const float* f) {
    if constexpr (sizeof(E) == 4) {
#pragma unroll
      for (int i = 0; i < P; ++i) w[i] = __float_as_uint(f[i]);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = rope_pack<E>(f[2 * i], 2 * i + 1 < P ? f[2 * i + 1] : 0.f);
    }
  }
  __device__ __forceinline__ void fill(uint32_t x) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = x;
  }
};

// A head's vector is dim / 2P units. The first rot / 2P have P pairs each: in halves, the vectors
// at u P and rot / 2 + u P; interleaved, the two next to each other at 2 u P. The others are 2 P
// components that stay as they are.
template <int P, bool INTER>
struct RopeUnit {
  int lo, hi;  // where the two vectors begin
  bool turns;
  __device__ __forceinline__ RopeUnit(int u, int rot) {
    turns = 2 * P * u < rot;
    const bool halves = !INTER && turns;
    lo = halves ? P * u : 2 * P * u;
    hi = halves ? rot / 2 + P * u : lo + P;
  }
};

// The unit's 2 P values f (the vector at lo, then that at hi), rotated in place.
template <int P, bool INTER>
__device__ __forceinline__ void rope_apply(float* f, const float2* cs) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int a = INTER ? 2 * i : i, b = INTER ? 2 * i + 1 : P + i;
    const float x = f[a], y = f[b];
    f[a] = fmaf(x, cs[i].x, -(y * cs[i].y));
    f[b] = fmaf(y, cs[i].x, x * cs[i].y);
  }
}

template <int P>
__device__ __forceinline__ void rope_turns(const Rope& R, long long pos, int u, float2* cs) {
#pragma unroll
  for (int i = 0; i < P; ++i) cs[i] = rope_turn(R, pos, kv_ld(R.freq + P * u + i));
}

// Depths of a row's n tokens under the parent links of a draft tree, to depth[0 .. n - 1] (shared
// memory, SV_MAX_TREE entries each); false when a link is wrong. Whole block.
__device__ __forceinline__ bool rope_depths(const int32_t* parent, int n, int* par, int* depth) {
  bool bad = false;
  for (int t = threadIdx.x; t < n; t += blockDim.x) {
    const int p = t ? kv_ld(parent + t) : 0;
    bad = bad || (t && (p < 0 || p >= t));
    par[t] = p;
  }
  if (__syncthreads_or(bad)) return false;
  for (int t = threadIdx.x; t < n; t += blockDim.x) {
    int d = 0;
    for (int i = t; i > 0; i = par[i]) ++d;
    depth[t] = d;
  }
  __syncthreads();
  return true;
}

// A row's tokens: rotated to out, which may be x itself (`same`). `pos` gives a token's position.
// Items are (token, share of the heads, unit); a thread takes its unit of every `shares`-th head,
// with one set of cosines and sines. Of tokens from n on, zeros are written unless in place; NaN
// everywhere when the row is bad.
struct RopeRow {
  const void* x;
  void* out;
  long long x_tok, out_tok;  // elements between tokens
  int T, n, heads, dim, shares;
  bool same, bad;
};
template <typename E, int P, bool INTER, int K, typename Pos>
__device__ __forceinline__ void rope_row(const Rope& R, const RopeRow& w, int first, int step, Pos pos) {
  const int units = (w.same && !w.bad ? R.rot : w.dim) / (2 * P);
  const int live = w.bad ? w.T : (w.same ? w.n : w.T);
  const long long items = (long long)live * w.shares * units;
  for (long long i = first; i < items; i += step) {
    const int t = static_cast<int>(i / (w.shares * units)), r = static_cast<int>(i - (long long)t * (w.shares * units));
    const int share = r / units, u = r - share * units;
    const RopeUnit<P, INTER> unit(u, R.rot);
    const E* x = static_cast<const E*>(w.x) + t * w.x_tok;
    E* out = static_cast<E*>(w.out) + t * w.out_tok;
    if (w.bad || t >= w.n) {
      RopeVec<E, P> y;
      y.fill(w.bad ? (sizeof(E) == 4 ? 0x7fffffffu : 0x7fff7fffu) : 0u);
      for (int h = share; h < w.heads; h += w.shares) {
        y.store(out + (size_t)h * w.dim + unit.lo);
        y.store(out + (size_t)h * w.dim + unit.hi);
      }
      continue;
    }
    float2 cs[P];
    if (unit.turns) rope_turns<P>(R, pos(t), u, cs);
    // (K heads' loads are in flight.)
    for (int h0 = share; h0 < w.heads; h0 += K * w.shares) {
      RopeVec<E, P> a[K], b[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int h = h0 + k * w.shares;
        if (h < w.heads) {
          a[k].load(x + (size_t)h * w.dim + unit.lo);
          b[k].load(x + (size_t)h * w.dim + unit.hi);
        }
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int h = h0 + k * w.shares;
        if (h >= w.heads) break;
        if (unit.turns) {
          float f[2 * P];
          a[k].get(f);
          b[k].get(f + P);
          rope_apply<P, INTER>(f, cs);
          a[k].set(f);
          b[k].set(f + P);
        }
        a[k].store(out + (size_t)h * w.dim + unit.lo);
        b[k].store(out + (size_t)h * w.dim + unit.hi);
      }
    }
  }
}

// How a call's rows are cut: shares of the heads, and blocks of a row. A thread takes up to 8
// heads, so that their loads hide each other and cosines are computed once for them; fewer while
// the threads of all rows do not fill the GPU's 152 SMs (with `resident` threads each).
inline void rope_cut(int rows, int T, int heads, int units, int threads, int resident, int* shares,
                     int* blocks) {
  const long long all = (long long)rows * T * units * heads;
  long long per = (all + 152LL * resident - 1) / (152LL * resident);
  per = per < 1 ? 1 : (per > 8 ? 8 : per);
  *shares = static_cast<int>((heads + per - 1) / per);
  const long long items = (long long)T * units * *shares;
  const long long most = (items + threads - 1) / threads;
  *blocks = static_cast<int>(most < 65535 ? most : 65535);
}

struct RopeArgs {
  Rope R;
  RopeRow row;                     // of row 0; n and bad are the kernel's
  long long x_row, out_row;        // elements between rows
  const int32_t *pos, *start, *parent, *n_new;
  WsHeader* hdr;
};

struct AppendRopeArgs {
  KvCache C;
  KvScratch S;
  Rope R;
  int layer, T;
  KvSrc k, v;
  const int32_t *n_new, *parent;
  RopeRow q;                       // of row 0; heads 0: no queries
  long long q_row, q_out_row;
  int checked;                     // the rows' pages were checked by a launch before
  int pages, chunks, per, q_blocks;  // of a row: pages touched, chunks of `per` heads, query blocks
};

cudaError_t launch_rope(const RopeArgs& A, bool interleaved, sv_dtype dt, int rows, cudaStream_t st);
cudaError_t launch_kv_append_rope(AppendRopeArgs& A, bool interleaved, sv_dtype dt, cudaStream_t st);

}  // namespace sv
