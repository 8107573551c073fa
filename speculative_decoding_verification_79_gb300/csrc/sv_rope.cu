// sv_rope.cu -- rotary positions of queries, keys and their gradients (sm_103a).
//
// A block takes tokens of one row; a thread P pairs of one token in up to 8 heads. Bound by
// memory: every value is read and written once; the 8 cosines and sines of a thread are some 300
// instructions, spread over its heads. 8 x 4,093 tokens of 32 heads of 128 in bf16: 80.4 us, 537 MB
// at 6.7 TB/s. 4 x 2,047 tokens of 12 heads of 80 in float32, interleaved: 13.1 us, 63 MB at 4.8;
// one token: 2.5 us, a launch. (Blocks of 256 threads: 80.7, 13.7 and 2.9 us. Two heads' loads in
// flight instead of four: 85 for the first; 64 registers: 87.)
#include "sv_rope.cuh"

namespace sv {

constexpr int ROPE_THREADS = 128;

template <typename E, int P, bool INTER>
__global__ void __launch_bounds__(ROPE_THREADS)
    rope_kernel(const __grid_constant__ RopeArgs A) {
  kv_enter();
  __shared__ int s_par[SV_MAX_TREE], s_depth[SV_MAX_TREE];
  const int b = blockIdx.y, T = A.row.T;
  RopeRow w = A.row;
  w.x = static_cast<const E*>(A.row.x) + b * A.x_row;
  w.out = static_cast<E*>(A.row.out) + b * A.out_row;
  w.n = A.n_new ? kv_ld(A.n_new + b) : T;
  w.bad = w.n < 0 || w.n > T;
  if (A.parent && !w.bad)
    w.bad = !rope_depths(A.parent + (size_t)b * T, w.n, s_par, s_depth);
  if (w.bad && blockIdx.x == 0 && threadIdx.x == 0) kv_report(A.hdr, ST_DEVICE_INPUT);
  const long long start = A.start ? kv_ld(A.start + b) : 0;
  rope_row<E, P, INTER, 4>(A.R, w, blockIdx.x * ROPE_THREADS + threadIdx.x, gridDim.x * ROPE_THREADS,
                        [&](int t) -> long long {
                          if (A.pos) return kv_ld(A.pos + (size_t)b * T + t);
                          return start + (A.parent ? s_depth[t] : t);
                        });
}

template <typename E>
static cudaError_t launch_type(const RopeArgs& A, bool inter, dim3 grid, cudaStream_t st) {
  const int P = rope_pairs(A.R.rot);
  auto* kernel = P == 8   ? (inter ? rope_kernel<E, 8, true> : rope_kernel<E, 8, false>)
                 : P == 4 ? (inter ? rope_kernel<E, 4, true> : rope_kernel<E, 4, false>)
                          : (inter ? rope_kernel<E, 1, true> : rope_kernel<E, 1, false>);
  return kv_launch(kernel, grid, ROPE_THREADS, 0, st, A);
}

cudaError_t launch_rope(const RopeArgs& A0, bool inter, sv_dtype dt, int rows, cudaStream_t st) {
  RopeArgs A = A0;
  int blocks;
  const int units = (A.row.same ? A.R.rot : A.row.dim) / (2 * rope_pairs(A.R.rot));
  rope_cut(rows, A.row.T, A.row.heads, units, ROPE_THREADS, 2048, &A.row.shares, &blocks);
  const dim3 grid(blocks, rows);
  return dt == SV_F32    ? launch_type<float>(A, inter, grid, st)
         : dt == SV_BF16 ? launch_type<__nv_bfloat16>(A, inter, grid, st)
                         : launch_type<__half>(A, inter, grid, st);
}

}  // namespace sv
