// sv_kv_api.cu -- the C-ABI boundary of the key/value cache: argument checks, workspace
// layout, launches. Declarations and contracts are in include/specverify.h.
#include <cmath>

#include "sv_kv.cuh"

using namespace sv;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The sizes of a cache (no pointers); false when unsupported.
bool kv_sizes(const sv_kv_cache* c, KvCache* C) {
  if (!c) return false;
  int lgp = 0;
  while (lgp < 8 && (1 << lgp) != c->page) ++lgp;
  if (lgp < 4 || lgp > 7) return false;
  if (c->layers < 1 || c->pages < 1 || c->max_pages < 1 || c->heads < 1 ||
      c->heads > SV_KV_MAX_HEADS || c->dim < 16 || c->dim > SV_KV_MAX_DIM || c->dim % 16 != 0 ||
      c->batch < 1 || c->batch > SV_MAX_B)
    return false;
  const long long lim = 1LL << 31;
  if ((long long)c->pages * c->heads >= lim / c->page ||
      (long long)c->max_pages >= lim / c->page)
    return false;
  C->layers = c->layers;
  C->pages = c->pages;
  C->page = c->page;
  C->heads = c->heads;
  C->dim = c->dim;
  C->batch = c->batch;
  C->max_pages = c->max_pages;
  C->lgp = lgp;
  return true;
}

// Every check that a cache and its workspace need, and their kernel form.
sv_status kv_open(const sv_kv_cache* c, void* ws_d, size_t ws_bytes, KvCache* C, KvScratch* S) {
  if (!c) return SV_ERR_ARG;
  if (!kv_sizes(c, C)) return SV_ERR_SHAPE;
  const KvWs W = kv_ws(*C);
  if (!ws_d || !aligned(ws_d, 256) || ws_bytes < W.total) return SV_ERR_WORKSPACE;
  if (!c->k_d || !c->v_d || !c->k_scale_d || !c->v_scale_d || !c->table_d || !c->n_pages_d ||
      !c->len_d || !c->refs_d)
    return SV_ERR_ARG;
  if (!aligned(c->k_d, 16) || !aligned(c->v_d, 16) || !aligned(c->k_scale_d, 4) ||
      !aligned(c->v_scale_d, 4) || !aligned(c->table_d, 4) || !aligned(c->n_pages_d, 4) ||
      !aligned(c->len_d, 4) || !aligned(c->refs_d, 4))
    return SV_ERR_ARG;
  C->k = static_cast<uint8_t*>(c->k_d);
  C->v = static_cast<uint8_t*>(c->v_d);
  C->ks = c->k_scale_d;
  C->vs = c->v_scale_d;
  C->table = c->table_d;
  C->np = c->n_pages_d;
  C->len = c->len_d;
  C->refs = c->refs_d;
  unsigned char* ws = static_cast<unsigned char*>(ws_d);
  S->hdr = reinterpret_cast<WsHeader*>(ws);
  S->open = reinterpret_cast<KvOpen*>(ws + W.open);
  S->table = reinterpret_cast<int32_t*>(ws + W.table);
  S->np = reinterpret_cast<int32_t*>(ws + W.np);
  S->len = reinterpret_cast<int32_t*>(ws + W.len);
  S->keeper = reinterpret_cast<int32_t*>(ws + W.keeper);
  S->fresh = reinterpret_cast<int32_t*>(ws + W.fresh);
  S->flag = reinterpret_cast<int32_t*>(ws + W.flag);
  S->list = reinterpret_cast<int32_t*>(ws + W.list);
  S->part = reinterpret_cast<float*>(ws + W.part);
  S->stat = reinterpret_cast<float2*>(ws + W.stat);
  return SV_OK;
}

sv_status done(cudaError_t e) { return e == cudaSuccess ? SV_OK : SV_ERR_CUDA; }

size_t elem_bytes(sv_dtype dt) { return dt == SV_F32 ? 4 : 2; }

// A strided [batch, T, heads, dim] source: 16-byte aligned base and strides, tokens that do
// not overlap.
bool src_ok(const void* p, int64_t row, int64_t tok, size_t eb, int64_t width) {
  return p && aligned(p, 16) && row >= 0 && tok >= width && (row * (int64_t)eb) % 16 == 0 &&
         (tok * (int64_t)eb) % 16 == 0;
}

}  // namespace

extern "C" {

size_t sv_kv_workspace_bytes(const sv_kv_cache* cache) {
  KvCache C;
  return kv_sizes(cache, &C) ? kv_ws(C).total : 0;
}

sv_status sv_kv_reserve(const sv_kv_cache* cache, const int32_t* n_new_d, int32_t* ok_d,
                        void* ws_d, size_t ws_bytes, void* stream) {
  KvCache C;
  KvScratch S;
  const sv_status st = kv_open(cache, ws_d, ws_bytes, &C, &S);
  if (st != SV_OK) return st;
  if (!n_new_d || !aligned(n_new_d, 4) || (ok_d && !aligned(ok_d, 4))) return SV_ERR_ARG;
  return done(launch_kv_reserve(C, S, n_new_d, ok_d, static_cast<cudaStream_t>(stream)));
}

sv_status sv_kv_append(const sv_kv_cache* cache, int layer, const void* k_src_d,
                       const void* v_src_d, sv_dtype dtype, int64_t k_row, int64_t k_tok,
                       int64_t v_row, int64_t v_tok, int T, const int32_t* n_new_d, void* ws_d,
                       size_t ws_bytes, void* stream) {
  if (dtype != SV_F32 && dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_DTYPE;
  KvCache C;
  KvScratch S;
  const sv_status st = kv_open(cache, ws_d, ws_bytes, &C, &S);
  if (st != SV_OK) return st;
  if (T < 0 || T > SV_KV_MAX_T) return SV_ERR_SHAPE;
  if (layer < 0 || layer >= C.layers) return SV_ERR_ARG;
  if (T == 0) return SV_OK;
  const int64_t width = (int64_t)C.heads * C.dim;
  const size_t eb = elem_bytes(dtype);
  if (!src_ok(k_src_d, k_row, k_tok, eb, width) || !src_ok(v_src_d, v_row, v_tok, eb, width) ||
      (n_new_d && !aligned(n_new_d, 4)))
    return SV_ERR_ARG;
  return done(launch_kv_append(C, S, layer, KvSrc{k_src_d, k_row, k_tok},
                               KvSrc{v_src_d, v_row, v_tok}, dtype, T, n_new_d,
                               static_cast<cudaStream_t>(stream)));
}

sv_status sv_kv_read(const sv_kv_cache* cache, int layer, int n_layers, const int32_t* start_d,
                     const int32_t* count_d, int T, void* k_out_d, void* v_out_d,
                     sv_dtype dtype, void* ws_d, size_t ws_bytes, void* stream) {
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  KvCache C;
  KvScratch S;
  const sv_status st = kv_open(cache, ws_d, ws_bytes, &C, &S);
  if (st != SV_OK) return st;
  if (T < 0 || T > SV_KV_MAX_T) return SV_ERR_SHAPE;
  if (layer < 0 || n_layers < 0 || n_layers > C.layers - layer) return SV_ERR_ARG;
  if (T == 0 || n_layers == 0) return SV_OK;
  if (!start_d || !aligned(start_d, 4) || (count_d && !aligned(count_d, 4)) || !k_out_d ||
      !v_out_d || !aligned(k_out_d, 16) || !aligned(v_out_d, 16))
    return SV_ERR_ARG;
  return done(launch_kv_read(C, S, layer, n_layers, start_d, count_d, T, k_out_d, v_out_d, dtype,
                             static_cast<cudaStream_t>(stream)));
}

sv_status sv_kv_attend(const sv_kv_cache* cache, int layer, const void* q_d, sv_dtype dtype,
                       int64_t q_row, int64_t q_tok, int T, int q_heads,
                       const int32_t* n_new_d, const int32_t* parent_d, float scale, int window,
                       int sinks, void* out_d, float* lse_d, void* ws_d, size_t ws_bytes,
                       void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_DTYPE;
  KvCache C;
  KvScratch S;
  const sv_status st = kv_open(cache, ws_d, ws_bytes, &C, &S);
  if (st != SV_OK) return st;
  if (T < 0 || T > SV_KV_MAX_T || (parent_d && T > SV_MAX_TREE)) return SV_ERR_SHAPE;
  if (q_heads < C.heads || q_heads % C.heads != 0 || q_heads / C.heads > KV_ROWS)
    return SV_ERR_SHAPE;
  // Key tiles of 128 tokens, and what a query tile of 128 rows costs beside them, in 31 bits.
  const long long qtiles = ((long long)T * (q_heads / C.heads) + KV_ROWS - 1) / KV_ROWS;
  const long long ktiles = ((long long)C.max_pages * C.page + 127) / 128 + KV_EXTRA;
  if (qtiles * C.batch * C.heads >= (1LL << 31) / ktiles) return SV_ERR_SHAPE;
  if ((long long)C.max_pages * C.page > (1LL << 31) - 256) return SV_ERR_SHAPE;
  const float scale2 = static_cast<float>((double)scale * 1.4426950408889634);
  if (layer < 0 || layer >= C.layers || !std::isfinite(scale2) || window < 0 || sinks < 0)
    return SV_ERR_ARG;
  if (T == 0) return SV_OK;
  if (!src_ok(q_d, q_row, q_tok, 2, (int64_t)q_heads * C.dim) || !out_d || !aligned(out_d, 16) ||
      (lse_d && !aligned(lse_d, 4)) || (n_new_d && !aligned(n_new_d, 4)) ||
      (parent_d && !aligned(parent_d, 4)))
    return SV_ERR_ARG;
  AttendArgs A;
  A.C = C;
  A.S = S;
  A.layer = layer;
  A.q = q_d;
  A.q_row = q_row;
  A.q_tok = q_tok;
  A.T = T;
  A.q_heads = q_heads;
  A.group = q_heads / C.heads;
  A.n_new = n_new_d;
  A.parent = parent_d;
  A.scale = scale2;
  A.window = window;
  A.sinks = sinks;
  A.wait_limit = wait_limit();
  A.out = out_d;
  A.lse = lse_d;
  return done(launch_kv_attend(A, dtype, static_cast<cudaStream_t>(stream)));
}

sv_status sv_kv_commit(const sv_kv_cache* cache, const int32_t* accepted_d, const int32_t* path_d,
                       int N, void* ws_d, size_t ws_bytes, void* stream) {
  KvCache C;
  KvScratch S;
  const sv_status st = kv_open(cache, ws_d, ws_bytes, &C, &S);
  if (st != SV_OK) return st;
  if (N < 1 || N > SV_KV_MAX_T || (path_d && N > SV_MAX_TREE)) return SV_ERR_SHAPE;
  if (!accepted_d || !aligned(accepted_d, 4) || (path_d && !aligned(path_d, 4)))
    return SV_ERR_ARG;
  return done(launch_kv_commit(C, S, accepted_d, path_d, N, static_cast<cudaStream_t>(stream)));
}

sv_status sv_kv_fork(const sv_kv_cache* cache, const int32_t* src_d, int32_t* ok_d, void* ws_d,
                     size_t ws_bytes, void* stream) {
  KvCache C;
  KvScratch S;
  const sv_status st = kv_open(cache, ws_d, ws_bytes, &C, &S);
  if (st != SV_OK) return st;
  if (!src_d || !aligned(src_d, 4) || (ok_d && !aligned(ok_d, 4))) return SV_ERR_ARG;
  return done(launch_kv_fork(C, S, src_d, ok_d, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
