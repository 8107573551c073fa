// sv_kv_attend.cu -- attention of a round's new tokens over the key/value cache (sm_103a).
//
// A CTA takes one query (row, token, head): its warps take keys in turn, a lane holds
// dim / 32 of the vector, and each warp keeps the running maximum and sum of the softmax
// and its output; the warps' results are joined at the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "sv_kv.cuh"

namespace sv {

constexpr int AT_WARPS = 4;
constexpr int AT_E = SV_KV_MAX_DIM / 32;

// grid (x: query heads, y: tokens, z: rows)
template <typename Q>
__global__ void __launch_bounds__(32 * AT_WARPS) kv_attend_kernel(const AttendArgs A) {
  const KvCache& C = A.C;
  const int hq = blockIdx.x, t = blockIdx.y, b = blockIdx.z, h = hq / A.group;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  __shared__ unsigned long long s_see;
  __shared__ int s_pos, s_bad;
  __shared__ float s_m[AT_WARPS], s_l[AT_WARPS], s_o[AT_WARPS][SV_KV_MAX_DIM];
  const int n = A.n_new ? __ldg(A.n_new + b) : A.T, len = __ldg(C.len + b);
  if (tid == 0) {
    bool bad = n < 0 || n > A.T || len < 0 || ((long long)len + n) > (long long)C.max_pages << C.lgp;
    unsigned long long see = 0;
    int depth = t;
    if (!bad && A.parent) {
      const int32_t* par = A.parent + (size_t)b * A.T;
      for (int i = 1; i < n; ++i) bad = bad || __ldg(par + i) < 0 || __ldg(par + i) >= i;
      depth = 0;
      if (!bad && t < n)
        for (int i = t;; i = __ldg(par + i)) {
          // `depth` steps above t: visible inside the window, or as a sink.
          if (!A.window || depth < A.window || len + i < A.sinks) see |= 1ull << i;
          if (i == 0) break;
          ++depth;
        }
    }
    s_see = see;
    s_pos = bad ? 0 : len + depth;
    s_bad = bad;
  }
  __syncthreads();
  const size_t row = ((size_t)b * A.T + t) * A.q_heads + hq;
  Q* out = static_cast<Q*>(A.out) + row * C.dim;
  bool bad = s_bad;
  float m = -INFINITY, l = 0.f, o[AT_E], q[AT_E];
#pragma unroll
  for (int e = 0; e < AT_E; ++e) o[e] = 0.f;
  if (!bad && t < n) {
    const Q* src = static_cast<const Q*>(A.q) + b * A.q_row + t * A.q_tok + (size_t)hq * C.dim;
#pragma unroll
    for (int e = 0; e < AT_E; ++e)
      q[e] = lane + 32 * e < C.dim ? static_cast<float>(src[lane + 32 * e]) : 0.f;
    for (int j = w; j < len + n; j += AT_WARPS) {
      if (j < len ? (A.window && s_pos - j >= A.window && j >= A.sinks)
                  : (A.parent ? !((s_see >> (j - len)) & 1)
                              : (j - len > t || (A.window && s_pos - j >= A.window && j >= A.sinks))))
        continue;
      const int p = kv_page(C, b, j);
      if (p < 0) {
        bad = true;
        break;
      }
      const size_t at = kv_block(C, A.layer, p, h) + (size_t)(j & (C.page - 1)) * C.dim;
      float s = 0.f, v[AT_E];
#pragma unroll
      for (int e = 0; e < AT_E; ++e) {
        const int d = lane + 32 * e;
        v[e] = 0.f;
        if (d < C.dim) {
          s += q[e] * e4m3_to_f2(C.k[at + d]).x;
          v[e] = e4m3_to_f2(C.v[at + d]).x;
        }
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      s *= C.ks[kv_sidx(C, A.layer, p, h)] * A.scale;
      const float mn = fmaxf(m, s), f = exp2f(m - mn), x = exp2f(s - mn);
      const float xv = x * C.vs[kv_sidx(C, A.layer, p, h)];
      l = l * f + x;
      m = mn;
#pragma unroll
      for (int e = 0; e < AT_E; ++e) o[e] = o[e] * f + xv * v[e];
    }
  }
  if (lane == 0) {
    s_m[w] = m;
    s_l[w] = l;
  }
#pragma unroll
  for (int e = 0; e < AT_E; ++e)
    if (lane + 32 * e < C.dim) s_o[w][lane + 32 * e] = o[e];
  bad = __syncthreads_or(bad ? 1 : 0);
  float mx = -INFINITY, sum = 0.f;
  for (int i = 0; i < AT_WARPS; ++i) mx = fmaxf(mx, s_m[i]);
  for (int i = 0; i < AT_WARPS; ++i)
    if (s_m[i] != -INFINITY) sum += s_l[i] * exp2f(s_m[i] - mx);
  for (int d = tid; d < C.dim; d += 32 * AT_WARPS) {
    float y = 0.f;
    for (int i = 0; i < AT_WARPS; ++i)
      if (s_m[i] != -INFINITY) y += s_o[i][d] * exp2f(s_m[i] - mx);
    y = bad ? NAN : (mx == -INFINITY ? 0.f : y / sum);
    out[d] = static_cast<Q>(y);
  }
  if (tid == 0) {
    if (bad) kv_report(A.S.hdr, ST_DEVICE_INPUT);
    if (A.lse)
      A.lse[row] = bad ? NAN : (mx == -INFINITY ? -INFINITY
                                                : (mx + log2f(sum)) * 0.6931471805599453f);
  }
}

cudaError_t launch_kv_attend(const AttendArgs& A, sv_dtype dt, cudaStream_t st) {
  const dim3 grid(A.q_heads, A.T, A.C.batch);
  if (dt == SV_BF16)
    kv_attend_kernel<__nv_bfloat16><<<grid, 32 * AT_WARPS, 0, st>>>(A);
  else
    kv_attend_kernel<__half><<<grid, 32 * AT_WARPS, 0, st>>>(A);
  return cudaGetLastError();
}

}  // namespace sv
