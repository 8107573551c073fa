// sv_kv.cuh -- the paged 8-bit key/value cache: kernel arguments, workspace layout, row
// checks and e4m3 helpers shared by its kernels (sv_kv_*.cu).
#pragma once
#include <cuda_fp8.h>

#include "sv_common.cuh"

namespace sv {

// The cache as kernels see it (see sv_kv_cache in specverify.h).
struct KvCache {
  uint8_t *k, *v;    // [layers, pages, heads, page, dim] e4m3
  float *ks, *vs;    // [layers, pages, heads]
  int32_t *table;    // [batch, max_pages]
  int32_t *np, *len; // [batch]
  int32_t* refs;     // [pages]
  int layers, pages, page, heads, dim, batch, max_pages;
  int lgp;           // log2(page)
};

// Status bit of the cache calls, beside those of every workspace header.
constexpr uint32_t ST_NO_PAGES = 4u;

// Workspace: header, then the snapshot that sv_kv_fork reads while it rewrites rows, the
// list of fresh pages, a flag per row, and the attention's partial results.
constexpr int KV_MAX_CTAS = 160;  // persistent CTAs of the attention kernel
constexpr int KV_ROWS = 128;      // most query rows of its tile
// Work of a query tile beside its key tiles, in key tiles: 3, 4, 5, 6 and 7 took 132, 121, 121,
// 121 and 123 us for single tokens of 64 rows, and 161, 152, 150, 149 and 152 for trees of 16
// nodes.
constexpr int KV_EXTRA = 6;

// A query tile of the attention that begins in one CTA and goes on in others, up to `last`:
// rows r0 .. r0 + R - 1 of (row b, head h). R = 0: the CTA has none.
struct KvOpen {
  int b, h, r0, R, last;
  int slot;  // (rows that share pages: of the first of its parts, and last counts from there)
};

struct KvWs {
  size_t open;    // KvOpen [KV_MAX_CTAS]
  size_t table;   // int32 [batch * max_pages]
  size_t np, len, keeper, fresh, flag;  // int32 [batch] each
  size_t list;    // int32 [min(pages, batch * max_pages)]
  size_t part;    // float [2 * KV_MAX_CTAS][KV_ROWS * dim]
  size_t stat;    // float2 [2 * KV_MAX_CTAS][KV_ROWS]
  size_t total;
};

inline KvWs kv_ws(const KvCache& C) {
  KvWs W;
  size_t off = sizeof(WsHeader);
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  const size_t B = (size_t)C.batch, P = B * (size_t)C.max_pages;
  W.open = take(sizeof(KvOpen) * KV_MAX_CTAS);
  W.table = take(4 * P);
  W.np = take(4 * B);
  W.len = take(4 * B);
  W.keeper = take(4 * B);
  W.fresh = take(4 * B);
  W.flag = take(4 * B);
  W.list = take(4 * (P < (size_t)C.pages ? P : (size_t)C.pages));
  W.part = take(4 * (size_t)2 * KV_MAX_CTAS * KV_ROWS * C.dim);
  W.stat = take(8 * (size_t)2 * KV_MAX_CTAS * KV_ROWS);
  W.total = off;
  return W;
}

struct KvScratch {  // the same, as pointers
  WsHeader* hdr;
  KvOpen* open;
  int32_t *table, *np, *len, *keeper, *fresh, *flag, *list;
  float* part;
  float2* stat;
};

// Largest |x| that the scales 2^-64 .. 2^64 cover, and the bounds of a scale.
constexpr float KV_XMAX = 448.f * 18446744073709551616.f;

// Smallest power of two s = 2^e, e >= SV_KV_MIN_EXP, with a <= 448 s, for 0 <= a <=
// KV_XMAX: 448 = 1.75 * 2^8, so with a = f * 2^x, 1 <= f < 2, e = x - 8, plus one when
// f > 1.75. Exact, from the bits.
__device__ __forceinline__ float kv_scale(float a) {
  const uint32_t u = __float_as_uint(a);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = e < SV_KV_MIN_EXP ? SV_KV_MIN_EXP : e;
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Four floats to e4m3, nearest, ties to even, saturating (NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// The same for e5m2.
__device__ __forceinline__ uint32_t e5m2x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Two e4m3 (the low 16 bits) as floats, exactly.
__device__ __forceinline__ float2 e4m3_to_f2(uint16_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(w));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The same for e5m2, which is the upper byte of fp16.
__device__ __forceinline__ float2 e5m2_to_f2(uint16_t w) {
  const uint32_t h = __byte_perm(w, 0, 0x1404);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Is the positive scale s a power of two?
__device__ __forceinline__ bool kv_pow2(float s) {
  return (__float_as_uint(s) & 0x7fffffu) == 0;
}

// x * m / s so that rounding it to e4m3 rounds the exact value: x of 24 bits with m = 1, or an
// e4m3 x with a scale m. The product is exact in double; the quotient's 53 bits tell values of
// at most 28 by 24 bits from the points halfway between e4m3 numbers (5 bits), and so does its
// cut to float with the rest marked in the lowest bit. (A quotient rounded to float may fall
// on such a point.) For scales that another quantiser wrote: a power of two needs none of it.
static __device__ __noinline__ float kv_quotient(float x, float m, float s) {
  const double y = static_cast<double>(x) * m / s;
  const float f = __double2float_rz(y);
  return static_cast<double>(f) == y ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// Four e4m3 values at scale `from` (the bytes of w), at scale `to`.
__device__ __forceinline__ uint32_t kv_rescale4(uint32_t w, float from, float to) {
  const float2 lo = e4m3_to_f2(w & 0xffffu), hi = e4m3_to_f2(w >> 16);
  float f[4] = {lo.x, lo.y, hi.x, hi.y};
  if (kv_pow2(from) && kv_pow2(to)) {
    const float r = from / to;
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] *= r;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = kv_quotient(f[i], from, to);
  }
  return e4m3x4(f[0], f[1], f[2], f[3]);
}

// A load of data that an earlier kernel of the stream may have written. Not a read-only load:
// those may be moved above the wait of kv_enter, and the data still changes while a kernel
// that was brought up early is resident.
template <typename V>
__device__ __forceinline__ V kv_ld(const V* p) {
  return *p;
}

// The page that holds position pos of row b, or -1 when the row does not hold one in
// range (0 <= pos < 2^31).
__device__ __forceinline__ int kv_page(const KvCache& C, int b, int pos) {
  const int j = pos >> C.lgp;
  if (pos < 0 || j >= C.max_pages || j >= kv_ld(C.np + b)) return -1;
  const int p = kv_ld(C.table + (size_t)b * C.max_pages + j);
  return p >= 0 && p < C.pages ? p : -1;
}

__device__ __forceinline__ void kv_report(WsHeader* hdr, uint32_t bits) {
  atomicOr(&hdr->status, bits);
}

// Byte offset of (layer, page, head)'s block of page x dim values, and its scale's index.
__device__ __forceinline__ size_t kv_block(const KvCache& C, int layer, int p, int h) {
  return (((size_t)layer * C.pages + p) * C.heads + h) * ((size_t)C.page * C.dim);
}
__device__ __forceinline__ size_t kv_sidx(const KvCache& C, int layer, int p, int h) {
  return ((size_t)layer * C.pages + p) * C.heads + h;
}

// May row b's n new tokens be written: is their number right, and does the row hold the pages
// that they touch, alone? This thread's part of the answer (all threads' must be true).
__device__ __forceinline__ bool kv_append_fits(const KvCache& C, int len, int n, int T) {
  return n > 0 && n <= T && len >= 0 && ((long long)len + n - 1) >> C.lgp < C.max_pages;
}
__device__ __forceinline__ bool kv_append_holds(const KvCache& C, int b, int len, int n) {
  bool fine = true;
  const int j0 = len >> C.lgp, j1 = (len + n - 1) >> C.lgp;
  for (int j = j0 + static_cast<int>(threadIdx.x); j <= j1; j += static_cast<int>(blockDim.x)) {
    const int p = kv_page(C, b, j << C.lgp);
    fine = fine && p >= 0 && kv_ld(C.refs + p) == 1;
  }
  return fine;
}

// With more pages to a row than this, its pages are checked by a launch before. On pages of 16,
// 8 heads of 128: 2,056 tokens (130 pages) take 11.6 us with it and 9.6 without, 4,093 of eight
// rows (257) 75 and 77, 16,384 of one row 41 and 52, 65,535 155 and 331.
constexpr int KV_APPEND_CHECK = 256;

// Source of a call's new keys or values: elements between rows and between tokens.
struct KvSrc {
  const void* p;
  long long row, tok;
};

struct AttendArgs {
  KvCache C;
  KvScratch S;
  int layer;
  const void* q;
  long long q_row, q_tok;
  int T, q_heads, group;
  const int32_t *n_new, *parent;
  float scale;  // scale * log2(e)
  int window, sinks;
  long long wait_limit;  // bound, in clock cycles, on waits inside a CTA
  void* out;
  float* lse;
};

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

// Every kernel of the cache is launched with programmatic stream serialization: it may be
// brought up while the kernel before it in the stream ends, and first waits for that one's
// completion (kv_enter), so that its results and all earlier ones are there. It lets the
// next one be brought up at once.
__device__ __forceinline__ void kv_enter() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... P>
cudaError_t kv_launch(void (*kernel)(P...), dim3 grid, int block, size_t smem, cudaStream_t st,
                      P... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The bound on waits that calls are given now, in clock cycles (sv_set_wait_limit; sv_api.cu).
long long wait_limit();

// Every check that a cache and its workspace need, and their kernel form (sv_kv_api.cu).
sv_status kv_open(const sv_kv_cache* c, void* ws_d, size_t ws_bytes, KvCache* C, KvScratch* S);
// A strided [batch, T, heads, dim] source of `width` elements a token: 16-byte aligned base and
// strides, tokens that do not overlap.
bool kv_src_ok(const void* p, int64_t row, int64_t tok, size_t eb, int64_t width);

cudaError_t launch_kv_reserve(const KvCache& C, const KvScratch& S, const int32_t* n_new,
                              int32_t* ok, cudaStream_t st);
cudaError_t launch_kv_fork(const KvCache& C, const KvScratch& S, const int32_t* src, int32_t* ok,
                           cudaStream_t st);
cudaError_t launch_kv_commit(const KvCache& C, const KvScratch& S, const int32_t* acc,
                             const int32_t* path, int N, cudaStream_t st);
cudaError_t launch_kv_append_check(const KvCache& C, const KvScratch& S, int T,
                                   const int32_t* n_new, cudaStream_t st);
cudaError_t launch_kv_append(const KvCache& C, const KvScratch& S, int layer, KvSrc k, KvSrc v,
                             sv_dtype dt, int T, const int32_t* n_new, cudaStream_t st);
cudaError_t launch_kv_read(const KvCache& C, const KvScratch& S, int layer, int n_layers,
                           const int32_t* start, const int32_t* count, int T, void* ko, void* vo,
                           sv_dtype dt, cudaStream_t st);
cudaError_t launch_kv_attend(const AttendArgs& A, sv_dtype dt, cudaStream_t st);

}  // namespace sv
