// sv_kv_store.cu -- writing and reading the key/value cache (sm_103a).
//
// Append: a CTA takes one page and head of one row; half of its threads the keys, half the
// values. Two steps: the largest |x| of the page's new tokens gives the scale, then each
// value is rounded to e4m3 at that scale, sixteen to a 16-byte store. The values stay in
// registers between the steps, so that they are read once. Bound by memory: 8 prompts of
// 4,093 tokens (8 heads of 128, bf16, pages of 64) are 201 MB; 39 to 42 us, 4.8 to 5.1 TB/s. With four CTAs an SM
// (64 registers; three took 45 us). A block of 9 tokens of 64 rows is a chain of memory
// trips (length, page table, values), 6 us; page, old scale and values are fetched together.
//
// Read: a thread per 16 values, nothing shared; 67 MB of cache to 134 MB of bf16 in 40 us,
// 5.1 TB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sv_kv.cuh"

namespace sv {

constexpr int AP_THREADS = 256;
constexpr int AP_HALF = AP_THREADS / 2;
// With more pages to a row than this, its pages are checked by a launch before. On pages of 16,
// 8 heads of 128: 2,056 tokens (130 pages) take 11.6 us with it and 9.6 without, 4,093 of eight
// rows (257) 75 and 77, 16,384 of one row 41 and 52, 65,535 155 and 331.
constexpr int AP_CHECK = 256;
constexpr int AP_CACHE = 4;  // vectors of 16 values that a thread keeps between the steps

template <typename E>
struct Vec16;  // sixteen consecutive elements
template <>
struct Vec16<float> {
  float4 x[4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = kv_ld(reinterpret_cast<const float4*>(p) + i);
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[4 * i] = x[i].x;
      f[4 * i + 1] = x[i].y;
      f[4 * i + 2] = x[i].z;
      f[4 * i + 3] = x[i].w;
    }
  }
};
template <>
struct Vec16<__nv_bfloat16> {
  uint4 x[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    x[0] = kv_ld(reinterpret_cast<const uint4*>(p));
    x[1] = kv_ld(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[8 * i + 2 * j] = bf_lo(w[j]);
        f[8 * i + 2 * j + 1] = bf_hi(w[j]);
      }
    }
  }
};
template <>
struct Vec16<__half> {
  uint4 x[2];
  __device__ __forceinline__ void load(const __half* p) {
    x[0] = kv_ld(reinterpret_cast<const uint4*>(p));
    x[1] = kv_ld(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        f[8 * i + 2 * j] = t.x;
        f[8 * i + 2 * j + 1] = t.y;
      }
    }
  }
};

// Sixteen values at scale s (inv = 1 / s, exact for a power of two).
__device__ __forceinline__ uint4 quantise16(const float* f, float inv) {
  uint4 o;
  o.x = e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
  o.y = e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
  o.z = e4m3x4(f[8] * inv, f[9] * inv, f[10] * inv, f[11] * inv);
  o.w = e4m3x4(f[12] * inv, f[13] * inv, f[14] * inv, f[15] * inv);
  return o;
}

// May row b's n new tokens be written: is their number right, and does the row hold the pages
// that they touch, alone? This thread's part of the answer (all threads' must be true).
__device__ __forceinline__ bool append_fits(const KvCache& C, int len, int n, int T) {
  return n > 0 && n <= T && len >= 0 && ((long long)len + n - 1) >> C.lgp < C.max_pages;
}
__device__ __forceinline__ bool append_holds(const KvCache& C, int b, int len, int n) {
  bool fine = true;
  const int j0 = len >> C.lgp, j1 = (len + n - 1) >> C.lgp;
  for (int j = j0 + static_cast<int>(threadIdx.x); j <= j1; j += AP_THREADS) {
    const int p = kv_page(C, b, j << C.lgp);
    fine = fine && p >= 0 && kv_ld(C.refs + p) == 1;
  }
  return fine;
}

// The same for every row, a CTA each, to flag: a launch before those of long appends, whose CTAs
// would each look at all of a row's pages.
__global__ void __launch_bounds__(AP_THREADS)
    kv_append_check_kernel(const KvCache C, const KvScratch S, int T, const int32_t* n_new) {
  kv_enter();
  const int b = blockIdx.x;
  const int n = n_new ? kv_ld(n_new + b) : T, len = kv_ld(C.len + b);
  const bool fine = n == 0 || (append_fits(C, len, n, T) && append_holds(C, b, len, n));
  const int all = __syncthreads_and(fine ? 1 : 0);
  if (threadIdx.x == 0) {
    S.flag[b] = all;
    if (!all) kv_report(S.hdr, ST_DEVICE_INPUT);
  }
}

// The new values of a page (vectors of 16, vpt of them a token) at a scale that is no power of
// two, which another quantiser gave the page.
template <typename E>
__device__ __noinline__ void append_any(const E* base, long long tok, int vpt, int nv, uint4* out,
                                        float s) {
  for (int i = threadIdx.x % AP_HALF; i < nv; i += AP_HALF) {
    const int t = i / vpt;
    Vec16<E> x;
    x.load(base + t * tok + (i - t * vpt) * 16);
    float f[16];
    x.get(f);
#pragma unroll
    for (int e = 0; e < 16; ++e) f[e] = kv_quotient(f[e], 1.f, s);
    out[i] = quantise16(f, 1.f);
  }
}

// grid (x: pages the new tokens can touch, y: heads, z: rows)
template <typename E>
__global__ void __launch_bounds__(AP_THREADS, sizeof(E) == 2 ? 4 : 2)
    kv_append_kernel(const KvCache C, const KvScratch S, int layer, const KvSrc ksrc,
                     const KvSrc vsrc, int T, const int32_t* n_new, int checked) {
  kv_enter();
  __shared__ float s_max[AP_THREADS / 32];
  const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
  const int n = n_new ? kv_ld(n_new + b) : T;
  if (n == 0) return;
  const int len = kv_ld(C.len + b);
  const bool sane = append_fits(C, len, n, T);
  const int half = tid / AP_HALF, t0 = tid - half * AP_HALF;
  const KvSrc src = half ? vsrc : ksrc;
  const int j0 = sane ? len >> C.lgp : 0, j = j0 + blockIdx.x;
  const bool in = sane && j < C.max_pages;
  const int lo = in ? max(len, j << C.lgp) : 0, hi = in ? min(len + n, (j + 1) << C.lgp) : 0;
  const int vpt = C.dim / 16, nv = max(0, hi - lo) * vpt, off = lo - (j << C.lgp);
  const E* base = static_cast<const E*>(src.p) + b * src.row + (lo - len) * src.tok +
                  (size_t)h * C.dim;
  auto at = [&](int i) {
    const int t = i / vpt, c = i - t * vpt;
    return base + t * src.tok + c * 16;
  };
  // The values are on their way while the row's pages are looked up.
  Vec16<E> keep[AP_CACHE];
#pragma unroll
  for (int r = 0; r < AP_CACHE; ++r) {
    const int i = t0 + r * AP_HALF;
    if (i < nv) keep[r].load(at(i));
  }
  // So are this page's scales, when it holds older tokens.
  const int p = hi > lo ? kv_page(C, b, j << C.lgp) : -1;
  float* scale = (half ? C.vs : C.ks) + kv_sidx(C, layer, max(p, 0), h);
  const float old = off && p >= 0 ? kv_ld(scale) : 0.f;
  // Every page that the row writes is its own.
  const bool fine = checked ? kv_ld(S.flag + b) != 0 : sane && append_holds(C, b, len, n);
  if (!__syncthreads_and(fine ? 1 : 0)) {
    if (tid == 0 && h == 0 && blockIdx.x == 0 && !checked) kv_report(S.hdr, ST_DEVICE_INPUT);
    return;
  }
  if (hi <= lo) return;
  uint8_t* dst = (half ? C.v : C.k) + kv_block(C, layer, p, h);
  float a = 0.f;
  bool odd = false;  // a value outside the scales' range
  auto see = [&](const Vec16<E>& x) {
    float f[16];
    x.get(f);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float y = fabsf(f[e]);
      if (y <= KV_XMAX)
        a = fmaxf(a, y);
      else
        odd = true;
    }
  };
#pragma unroll
  for (int r = 0; r < AP_CACHE; ++r)
    if (t0 + r * AP_HALF < nv) see(keep[r]);
  for (int i = t0 + AP_CACHE * AP_HALF; i < nv; i += AP_HALF) {
    Vec16<E> x;
    x.load(at(i));
    see(x);
  }
  if (odd) kv_report(S.hdr, ST_DEVICE_INPUT);
#pragma unroll
  for (int d = 16; d; d >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
  if ((tid & 31) == 0) s_max[tid >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < AP_HALF / 32; ++w) a = fmaxf(a, s_max[half * (AP_HALF / 32) + w]);
  float s = kv_scale(a);
  if (off) {
    s = fmaxf(s, old);
    if (s != old && kv_pow2(old) && kv_pow2(s)) {  // older tokens of the page, at its new scale
      for (int i = t0; i < off * vpt; i += AP_HALF) {
        uint4 x = reinterpret_cast<uint4*>(dst)[i];
        uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = kv_rescale4(w[q], old, s);
        reinterpret_cast<uint4*>(dst)[i] = x;
      }
    }
  }
  uint4* out = reinterpret_cast<uint4*>(dst + (size_t)off * C.dim);
  if (t0 == 0) *scale = s;
  // (On a path of its own, which reads the values again: it leaves the registers to the rest.)
  if (off && !(kv_pow2(old) && kv_pow2(s))) {
    append_any<E>(base, src.tok, vpt, nv, out, s);
    if (s != old)
      for (int i = t0; i < off * vpt; i += AP_HALF) {
        uint4 x = reinterpret_cast<uint4*>(dst)[i];
        uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = kv_rescale4(w[q], old, s);
        reinterpret_cast<uint4*>(dst)[i] = x;
      }
    return;
  }
  const float inv = 1.f / s;
#pragma unroll
  for (int r = 0; r < AP_CACHE; ++r) {
    const int i = t0 + r * AP_HALF;
    if (i < nv) {
      float f[16];
      keep[r].get(f);
      out[i] = quantise16(f, inv);
    }
  }
  for (int i = t0 + AP_CACHE * AP_HALF; i < nv; i += AP_HALF) {
    Vec16<E> x;
    x.load(at(i));
    float f[16];
    x.get(f);
    out[i] = quantise16(f, inv);
  }
}

// One thread per 16 values; grid (x: vectors of one row and layer, y: rows, z: layers).
template <bool BF16>
__global__ void __launch_bounds__(256)
    kv_read_kernel(const KvCache C, int layer0, const int32_t* start,
                   const int32_t* count, int T, void* ko, void* vo) {
  kv_enter();
  const int b = blockIdx.y, layer = layer0 + blockIdx.z;
  const int vpt = C.dim / 16;
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  const int t = i / (C.heads * vpt);
  if (t >= T) return;
  const int r = i - t * (C.heads * vpt), h = r / vpt, c = r - h * vpt;
  const int n = count ? kv_ld(count + b) : T;
  const long long pos = (long long)kv_ld(start + b) + t;
  const int p = t < n && pos >= 0 && pos < 0x7fffffffLL ? kv_page(C, b, (int)pos) : -1;
  uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  float s[2] = {0.f, 0.f};
  if (p >= 0) {
    const size_t o = kv_block(C, layer, p, h) + (size_t)(pos & (C.page - 1)) * C.dim + c * 16;
    x[0] = *reinterpret_cast<const uint4*>(C.k + o);
    x[1] = *reinterpret_cast<const uint4*>(C.v + o);
    s[0] = C.ks[kv_sidx(C, layer, p, h)];
    s[1] = C.vs[kv_sidx(C, layer, p, h)];
  }
  const size_t to = (((size_t)blockIdx.z * C.batch + b) * T * C.heads * vpt + i) * 16;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const uint32_t w[4] = {x[kv].x, x[kv].y, x[kv].z, x[kv].w};
    float f[16];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 lo = e4m3_to_f2(w[q] & 0xffffu), hi = e4m3_to_f2(w[q] >> 16);
      f[4 * q] = lo.x * s[kv];
      f[4 * q + 1] = lo.y * s[kv];
      f[4 * q + 2] = hi.x * s[kv];
      f[4 * q + 3] = hi.y * s[kv];
    }
    if (BF16) {
      uint32_t o[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const __nv_bfloat162 y = __floats2bfloat162_rn(f[2 * q], f[2 * q + 1]);
        o[q] = *reinterpret_cast<const uint32_t*>(&y);
      }
      uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(kv ? vo : ko) + to);
      __stcs(d, make_uint4(o[0], o[1], o[2], o[3]));
      __stcs(d + 1, make_uint4(o[4], o[5], o[6], o[7]));
    } else {
      float4* d = reinterpret_cast<float4*>(static_cast<float*>(kv ? vo : ko) + to);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        __stcs(d + q, make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]));
    }
  }
}

cudaError_t launch_kv_append(const KvCache& C, const KvScratch& S, int layer, KvSrc k, KvSrc v,
                             sv_dtype dt, int T, const int32_t* n_new, cudaStream_t st) {
  // A row's tokens start anywhere in a page, so T of them touch at most this many.
  const dim3 grid((T + C.page - 2) / C.page + 1, C.heads, C.batch);
  const auto kernel = dt == SV_F32    ? kv_append_kernel<float>
                      : dt == SV_BF16 ? kv_append_kernel<__nv_bfloat16>
                                      : kv_append_kernel<__half>;
  const int checked = static_cast<int>(grid.x) > AP_CHECK;
  if (checked) {
    const cudaError_t e =
        kv_launch(kv_append_check_kernel, dim3(C.batch), AP_THREADS, 0, st, C, S, T, n_new);
    if (e != cudaSuccess) return e;
  }
  return kv_launch(kernel, grid, AP_THREADS, 0, st, C, S, layer, k, v, T, n_new, checked);
}

cudaError_t launch_kv_read(const KvCache& C, const KvScratch&, int layer, int n_layers,
                           const int32_t* start, const int32_t* count, int T, void* ko, void* vo,
                           sv_dtype dt, cudaStream_t st) {
  const long long vecs = (long long)T * C.heads * (C.dim / 16);
  const auto kernel = dt == SV_BF16 ? kv_read_kernel<true> : kv_read_kernel<false>;
  constexpr int MOST = 65535;  // layers of a launch (the grid's third dimension)
  for (int l = 0; l < n_layers; l += MOST) {
    const int n = n_layers - l < MOST ? n_layers - l : MOST;
    const size_t at = (size_t)l * C.batch * vecs * 16 * (dt == SV_BF16 ? 2 : 4);
    const dim3 grid(static_cast<unsigned>((vecs + 255) / 256), C.batch, n);
    const cudaError_t e = kv_launch(kernel, grid, 256, 0, st, C, layer + l, start, count, T,
                                    static_cast<void*>(static_cast<char*>(ko) + at),
                                    static_cast<void*>(static_cast<char*>(vo) + at));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace sv
