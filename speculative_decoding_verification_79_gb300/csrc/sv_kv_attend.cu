// sv_kv_attend.cu -- attention of a round's new tokens over the key/value cache (sm_103a).
//
// For one row, key/value head and tile of R <= 128 query rows (tokens x query heads of the
// group, flattened) and key tiles of 128 tokens:
//     S = Q K^T  [R x 128],   P = 2^(S - m),   O += P V  [R x dim].
// Both products run on the fifth-generation tensor cores with the cache's own e4m3 bytes as
// the second operand, straight from TMA: nothing of the cache is converted. The first
// operand is carried as a sum of 8-bit terms, multiplied one after the other into the same
// float32 accumulator. A query row, scaled by a power of two to the e4m3 range, is the sum of
// an e4m3 term (4 bits) and one (bf16) or two (fp16) e5m2 terms for the rest: after rounding to
// 4 bits the rest of bf16's 8 has 3, which e5m2 holds, and e5m2's smallest number is 2^-16 where
// e4m3's is 2^-9 (2^-18 of the largest component). That is exact down to 2^-13 of the largest
// component, and off by up to 2^-21 (bf16) or 2^-24 (fp16) of that one below. A weight is rounded
// to fp16 and split into three e5m2 terms (e5m2 is fp16's upper byte, so a split is integer
// arithmetic). Weights go from registers to tensor memory and are multiplied from there.
//
// A thread owns a query row (a lane of the accumulator) and some of the tile's tokens, so
// that the softmax needs no exchange but one vote between the four threads of a row. (With
// tokens on the lanes instead, weights went through shared memory and sums across lanes: 472
// instead of 292 us for trees of 16 nodes, both as first built.) Sixteen tokens share a page:
// its key scale is a factor of their scores; its value scale is folded into their weights
// (its logarithm added to the scores, so that no weight exceeds the reference) and taken out
// of their sum again. The reference m of a row only moves when
// a score passes it by 2^4 (the accumulators are then rescaled), or with the first keys the
// row sees.
//
// The product has 128 rows whatever R is. Few rows are therefore repeated, 128 / W times
// for W = 32 or 64 >= R: each copy of a row takes its own W tokens of a tile (the weights
// of the others stay zero), so that all lanes have work and a tile's softmax costs R / 128
// of a full one; the copies' outputs are added at the end.
//
// A persistent CTA per SM takes an equal share of all (row, head, query tile, key tile)
// units in order; a query tile that crosses from one CTA to the next leaves partial
// results (output, m, sum) in the workspace, which a second kernel joins on all SMs.
//
// Warps, coupled by mbarriers: one copies K tiles page by page by tensor-map TMA (128-byte
// swizzle) into a ring, another V tiles into a second (and looks through those whose weights
// are cut, and plans the next query tile while this one is in work); one issues the scores'
// products and one the output's; sixteen form the weights, four on each quarter of a row
// copy's tokens.
//
// What bounds it. Up to dim 128 a key tile is 32 KB, 1,400 cycles of an SM's share of the
// memory rate, and 20 products of 64 cycles; its softmax is a chain of waits, loads,
// a vote, powers, splits and stores of about 1,600 cycles for 32 rows, 1,800 for 64 and 2,600
// for 128, where the integer instructions of the split alone fill half of it. Measured in CUDA
// graphs (a call from Python takes 2 to 11 us more) on 64 rows with 8 key/value heads of 128:
// single tokens of 8 queries a head, 4,100 tokens cached in the mean, 122 us (4.4 TB/s, 65 %
// of a copy); blocks of 9 tokens of 4 queries, 137 us; trees of up to 16 nodes of 8 queries,
// 149 us (560 TFLOP/s of the formula's, 2.5 times as many of 8-bit products). A query tile
// costs 3,000 to 8,000 cycles beside its key tiles, and a launch 11,000 to 18,000 before the
// first (counting, page table, queries, each a trip to memory), which is most of the 13 us of
// one row's single token.
#include "sv_kv_attend.cuh"

namespace sv {

template <int W, bool BF16, int NDB>
__global__ void __launch_bounds__(AT_THREADS, 1)
    kv_attend_kernel(const __grid_constant__ AttendArgs A, const __grid_constant__ AttendPlan P,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV) {
  extern __shared__ unsigned char dsm_raw[];
  __shared__ AtShared<AT_ROWS, W> sh;
  at_setup(sh);
  kv_enter();
  const AtCount count = at_count<AT_ROWS>(A, sh.rows);
  int before;
  const int total = at_block_sum(count.sum, sh.sum, &before);
  at_body<AT_ROWS, W, BF16, NDB>(A, P, tmK, tmV, sh, sh.rows, dsm_raw, count, total, before, blockIdx.x,
                                 gridDim.x);
}

// Joins the partial results of the query tile that begins in CTA blockIdx.x and goes on in
// others: a thread takes four components of a row over its CTAs, with the loads of four of
// them in flight and a running reference. It reads what the CTAs left in L2: 2 to 3 us for
// 30 MB. (A join by the last of the CTAs themselves held up its SM for up to 27 us: 128 rows
// of 256 components are 128 KB a CTA.)
// Blocks of a query tile: 2, 4, 8 and 16 took 161, 153, 149 and 149 us for the trees above.
constexpr int JOIN_THREADS = 256, JOIN_BLOCKS = 8;
__global__ void __launch_bounds__(JOIN_THREADS)
    kv_attend_join_kernel(const __grid_constant__ AttendArgs A, int bf16) {
  kv_enter();
  const int first = blockIdx.x;
  const KvOpen it = A.S.open[first];
  // (Eight rows and four of their vectors to a warp: whole sectors on both sides.)
  const int vec = A.C.dim / 4, n = (it.R + 7) / 8 * 8 * vec;
  constexpr int K = 4;
  for (int e = blockIdx.y * JOIN_THREADS + threadIdx.x; e < n; e += JOIN_BLOCKS * JOIN_THREADS) {
    const int r = e / (8 * vec) * 8 + e % 8, dv = e / 8 % vec;
    if (r >= it.R) continue;
    float ref = -INFINITY, sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = first; k0 <= it.last; k0 += K) {
      float2 s2[K];
      float4 y[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int kk = min(k0 + k, it.last);
        const int id = 2 * kk + (kk == first ? 1 : 0);
        s2[k] = __ldcg(A.S.stat + (size_t)id * KV_ROWS + r);
        y[k] = __ldcg(reinterpret_cast<const float4*>(A.S.part) + at_part(id, r, 4 * dv, A.C.dim));
      }
      float top = ref;
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (s2[k].y != 0.f) top = fmaxf(top, s2[k].x);
      const float f0 = sum == 0.f ? 0.f : exp2f(ref - top);
      ref = top;
      sum *= f0;
      o.x *= f0;
      o.y *= f0;
      o.z *= f0;
      o.w *= f0;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (s2[k].y == 0.f || k0 + k > it.last) continue;
        const float f = exp2f(s2[k].x - top);
        sum = fmaf(s2[k].y, f, sum);
        o.x = fmaf(y[k].x, f, o.x);
        o.y = fmaf(y[k].y, f, o.y);
        o.z = fmaf(y[k].z, f, o.z);
        o.w = fmaf(y[k].w, f, o.w);
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int t = (it.r0 + r) / A.group, gh = it.r0 + r - t * A.group;
    const long long row = ((long long)it.b * A.T + t) * A.q_heads + it.h * A.group + gh;
    at_store4(A.out, row * A.C.dim + dv * 4,
              make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv), bf16);
    if (dv == 0 && A.lse)
      A.lse[row] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
  }
}

cudaError_t at_launch(const AttendArgs& A, sv_dtype dt, int width, int dev, AttendLaunch* L) {
  const KvCache& C = A.C;
  const bool bf16 = dt == SV_BF16;
  const int ndb = C.dim > 128 ? 2 : 1;
  const size_t tile = (size_t)ndb * AT_BLK;
  // At least 32 components of 128 row copies, or 16 of them, which leaves room for one more
  // tile of 256 bytes a token.
  L->P.join = width == 128 ? 0 : 128 * (ndb == 1 ? 40 : 20);
  const size_t fixed = 1024 + (bf16 ? AT_QTERMS<true> : AT_QTERMS<false>) * tile + 4 * L->P.join;
  const int ring = (int)((AT_SMEM - AT_STATIC - fixed) / tile);
  L->P.nk = ring / 2 < AT_MAX_RING ? ring / 2 : AT_MAX_RING;
  L->P.nv = ring - ring / 2 < AT_MAX_RING ? ring - ring / 2 : AT_MAX_RING;
  L->smem = fixed + (L->P.nk + L->P.nv) * tile;
  // The pools of one layer as matrices [pages * heads * page tokens][dim bytes], in boxes of
  // one page x 128 bytes (128-byte swizzle, zeros past dim).
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  const size_t layer = (size_t)C.pages * C.heads * C.page * C.dim;
  for (int kv = 0; kv < 2; ++kv) {
    const cuuint64_t gdim[2] = {(cuuint64_t)C.dim, (cuuint64_t)C.pages * C.heads * C.page};
    const cuuint64_t gstride[1] = {(cuuint64_t)C.dim};
    const cuuint32_t box[2] = {128, (cuuint32_t)C.page};
    const cuuint32_t estr[2] = {1, 1};
    if (enc(&L->tm[kv], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, (kv ? C.v : C.k) + A.layer * layer, gdim,
            gstride, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  int sms = 0;
  const cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  L->grid = sms < KV_MAX_CTAS ? sms : KV_MAX_CTAS;
  L->ndb = ndb;
  L->width = width;
  return e;
}

cudaError_t launch_kv_attend(const AttendArgs& A, sv_dtype dt, cudaStream_t st) {
  typedef void (*Kernel)(const AttendArgs, const AttendPlan, const CUtensorMap, const CUtensorMap);
#define SV_ROW(bf16, ndb) \
  { kv_attend_kernel<32, bf16, ndb>, kv_attend_kernel<64, bf16, ndb>, kv_attend_kernel<128, bf16, ndb> }
  static const Kernel kernels[2][2][3] = {{SV_ROW(false, 1), SV_ROW(false, 2)},
                                          {SV_ROW(true, 1), SV_ROW(true, 2)}};
#undef SV_ROW
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
  // The narrowest copy that holds the rows: 8 rows a head took 121 us with copies of 32, 127
  // with 64 and 160 with 128 (64 rows of single tokens); 36 rows 137 with 64 and 169 with 128.
  const int width = at_width((long long)A.T * A.group);
  AttendLaunch L;
  if ((e = at_launch(A, dt, width, dev, &L)) != cudaSuccess) return e;
  const bool bf16 = dt == SV_BF16;
  const Kernel kernel = kernels[bf16][L.ndb - 1][width == 32 ? 0 : (width == 64 ? 1 : 2)];
  if ((e = kv_launch(kernel, dim3(L.grid), AT_THREADS, L.smem, st, A, L.P, L.tm[0], L.tm[1])) != cudaSuccess)
    return e;
  return kv_launch(kv_attend_join_kernel, dim3(L.grid, JOIN_BLOCKS), JOIN_THREADS, 0, st, A, bf16 ? 1 : 0);
}

}  // namespace sv
