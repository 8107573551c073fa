// sv_rope_api.cu -- the C-ABI boundary of the rotary calls: frequencies, argument checks,
// launches. Declarations and contracts are in include/specverify.h.
#include <cmath>

#include "sv_rope.cuh"

using namespace sv;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr double TWO_PI = 6.283185307179586476925;

// Frequencies are rounded once, to 2^-64 of a turn, from sums of two doubles (some 100 bits): a
// double's own 2^-56 of a turn would be 2^-25 of one at position 2^31. (Not long double, which has
// other sizes on other machines.)
struct Two {
  double hi, lo;
};
Two two_sum(double a, double b) {
  const double s = a + b, t = s - a;
  return Two{s, (a - (s - t)) + (b - t)};
}
Two operator+(Two a, Two b) {
  const Two s = two_sum(a.hi, b.hi);
  return two_sum(s.hi, s.lo + (a.lo + b.lo));
}
Two operator*(Two a, Two b) {
  const double p = a.hi * b.hi;
  return two_sum(p, std::fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}
Two operator/(Two a, Two b) {
  const double q = a.hi / b.hi;
  const Two r = a + Two{-q, 0.0} * b;
  return two_sum(q, r.hi / b.hi);
}
Two one(double x) { return Two{x, 0.0}; }
// e^x for |x| <= 710, x / 2^20 by its series (ten terms: 10^-35) and the square of that 20 times.
Two exp_two(Two x) {
  const Two r{std::ldexp(x.hi, -20), std::ldexp(x.lo, -20)};
  Two y = one(1.0);
  for (int k = 10; k; --k) y = one(1.0) + r * y / one(k);
  for (int k = 0; k < 20; ++k) y = y * y;
  return y;
}
// ln x of 1 < x: a step of Newton's method on e^y = x from the double.
Two log_two(double x) {
  const double y = std::log(x);
  return one(y) + (one(x) * exp_two(one(-y)) + one(-1.0));
}

// Turns per position of an angle (radians) as a fraction of 2^64. (Whole turns make none.)
int64_t fixed(Two angle) {
  const Two turns = angle * Two{0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};  // 1 / 2 pi
  const double whole = turns.hi - std::nearbyint(turns.hi), rest = turns.lo - std::nearbyint(turns.lo);
  // Both in units of 2^-64, rounded together; what passes 2^32 is carried.
  const double up = std::floor(std::ldexp(whole, 32));
  const double low = std::nearbyint(std::ldexp(std::ldexp(whole, 32) - up, 32) + std::ldexp(rest, 64));
  const double carry = std::floor(std::ldexp(low, -32));
  return static_cast<int64_t>((static_cast<uint64_t>(static_cast<int64_t>(up + carry)) << 32) +
                              static_cast<uint64_t>(low - std::ldexp(carry, 32)));
}

bool spec_ok(const sv_rope_spec* r, int dim) {
  return r && r->freq_d && aligned(r->freq_d, 8) && r->rot >= 2 && r->rot % 2 == 0 &&
         r->rot <= dim && std::isfinite(r->gain);
}

Rope rope_of(const sv_rope_spec* r, bool inverse) {
  return Rope{r->freq_d, r->rot, r->gain, inverse ? -r->gain : r->gain};
}

// A rotation's result: x itself, or strided like a source, its tokens apart.
bool out_ok(const void* x, int64_t x_row, int64_t x_tok, const void* out, int64_t row, int64_t tok,
            size_t eb, int64_t width, int batch, int T) {
  if (!kv_src_ok(out, row, tok, eb, width)) return false;
  if (out == x && (row != x_row || tok != x_tok)) return false;
  // Rows one after the other, or tokens of all rows side by side.
  return batch == 1 || row >= (int64_t)(T - 1) * tok + width ||
         (row >= width && (T == 1 || tok >= (int64_t)(batch - 1) * row + width));
}

size_t elem_bytes(sv_dtype dt) { return dt == SV_F32 ? 4 : 2; }

sv_status done(cudaError_t e) { return e == cudaSuccess ? SV_OK : SV_ERR_CUDA; }

}  // namespace

extern "C" {

sv_status sv_rope_fixed(const double* angle, int n, int64_t* freq_out) {
  if (n < 0 || n > SV_ROPE_MAX_DIM / 2) return SV_ERR_SHAPE;
  if (n && (!angle || !freq_out)) return SV_ERR_ARG;
  for (int i = 0; i < n; ++i)
    if (!std::isfinite(angle[i])) return SV_ERR_ARG;
  for (int i = 0; i < n; ++i) freq_out[i] = fixed(one(angle[i]));
  return SV_OK;
}

sv_status sv_rope_freqs(int rot, double base, sv_rope_scaling scaling, double stretch,
                        double original, double low, double high, int64_t* freq_out) {
  if (rot < 2 || rot > SV_ROPE_MAX_DIM || rot % 2 != 0) return SV_ERR_SHAPE;
  const bool blend = scaling == SV_ROPE_TURNS || scaling == SV_ROPE_INDEX;
  if (scaling != SV_ROPE_PLAIN && scaling != SV_ROPE_LINEAR && !blend) return SV_ERR_ARG;
  if (!freq_out || !(base > 1.0) || !std::isfinite(base) || !(stretch > 0.0) ||
      !std::isfinite(stretch))
    return SV_ERR_ARG;
  if (blend && (!(original > 0.0) || !std::isfinite(original) || !(low > 0.0) || !(high > low) ||
                !std::isfinite(high)))
    return SV_ERR_ARG;
  auto index = [&](double turns) {  // of the pair that makes so many turns
    return rot * std::log(original / (TWO_PI * turns)) / (2.0 * std::log(base));
  };
  double i0 = 0.0, i1 = 1.0;
  if (scaling == SV_ROPE_INDEX) {
    i0 = std::fmax(std::floor(index(high)), 0.0);
    i1 = std::fmin(std::ceil(index(low)), rot - 1.0);
  }
  const Two ln = log_two(base);
  for (int i = 0; i < rot / 2; ++i) {
    const Two f = exp_two(one(-2.0 * i) / one(rot) * ln);
    Two w = one(scaling == SV_ROPE_PLAIN ? 1.0 : 0.0);
    if (scaling == SV_ROPE_TURNS)
      w = (one(original) * f * Two{0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57} + one(-low)) /
          two_sum(high, -low);
    if (scaling == SV_ROPE_INDEX) w = one(1.0) + one(i0 - i) / one(std::fmax(i1 - i0, 1e-3));
    if (!(w.hi > 0.0)) w = one(0.0);
    if (w.hi > 1.0 || (w.hi == 1.0 && w.lo > 0.0)) w = one(1.0);
    freq_out[i] = fixed(f * (w + (one(1.0) + Two{-w.hi, -w.lo}) / one(stretch)));
  }
  return SV_OK;
}

sv_status sv_rope(const sv_rope_spec* rope, const void* x_d, sv_dtype dtype, int64_t x_row,
                  int64_t x_tok, int batch, int T, int heads, int dim, const int32_t* pos_d,
                  const int32_t* start_d, const int32_t* parent_d, const int32_t* n_new_d,
                  int inverse, void* out_d, int64_t out_row, int64_t out_tok, void* ws_d,
                  size_t ws_bytes, void* stream) {
  if (dtype != SV_F32 && dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_DTYPE;
  if (batch < 0 || batch > SV_MAX_B || T < 0 || T > SV_KV_MAX_T || heads < 1 ||
      heads > SV_KV_MAX_HEADS || dim < 16 || dim > SV_ROPE_MAX_DIM || dim % 16 != 0 ||
      (parent_d && T > SV_MAX_TREE))
    return SV_ERR_SHAPE;
  if (!spec_ok(rope, dim) || (pos_d && (start_d || parent_d))) return SV_ERR_ARG;
  if (!ws_d || ws_bytes < sizeof(WsHeader) || !aligned(ws_d, 256)) return SV_ERR_WORKSPACE;
  if (batch == 0 || T == 0) return SV_OK;
  const size_t eb = elem_bytes(dtype);
  const int64_t width = (int64_t)heads * dim;
  if (!kv_src_ok(x_d, x_row, x_tok, eb, width) ||
      !out_ok(x_d, x_row, x_tok, out_d, out_row, out_tok, eb, width, batch, T) ||
      !aligned(pos_d, 4) || !aligned(start_d, 4) || !aligned(parent_d, 4) || !aligned(n_new_d, 4))
    return SV_ERR_ARG;
  RopeArgs A;
  A.R = rope_of(rope, inverse != 0);
  A.row = RopeRow{x_d, out_d, x_tok, out_tok, T, T, heads, dim, 1, out_d == x_d, false};
  A.x_row = x_row;
  A.out_row = out_row;
  A.pos = pos_d;
  A.start = start_d;
  A.parent = parent_d;
  A.n_new = n_new_d;
  A.hdr = static_cast<WsHeader*>(ws_d);
  return done(launch_rope(A, rope->interleaved != 0, dtype, batch, static_cast<cudaStream_t>(stream)));
}

sv_status sv_kv_append_rope(const sv_kv_cache* cache, int layer, const void* k_src_d,
                            const void* v_src_d, sv_dtype dtype, int64_t k_row, int64_t k_tok,
                            int64_t v_row, int64_t v_tok, int T, const int32_t* n_new_d,
                            const int32_t* parent_d, const sv_rope_spec* rope, const void* q_d,
                            int64_t q_row, int64_t q_tok, int q_heads, void* q_out_d,
                            int64_t q_out_row, int64_t q_out_tok, void* ws_d, size_t ws_bytes,
                            void* stream) {
  if (dtype != SV_F32 && dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_DTYPE;
  AppendRopeArgs A;
  const sv_status st = kv_open(cache, ws_d, ws_bytes, &A.C, &A.S);
  if (st != SV_OK) return st;
  if (T < 0 || T > SV_KV_MAX_T || (parent_d && T > SV_MAX_TREE) || q_heads < 0 ||
      q_heads > SV_KV_MAX_HEADS * 128)
    return SV_ERR_SHAPE;
  if (layer < 0 || layer >= A.C.layers || !spec_ok(rope, A.C.dim) || (q_d != nullptr) != (q_heads > 0))
    return SV_ERR_ARG;
  if (T == 0) return SV_OK;
  const int64_t width = (int64_t)A.C.heads * A.C.dim, q_width = (int64_t)q_heads * A.C.dim;
  const size_t eb = elem_bytes(dtype);
  if (!kv_src_ok(k_src_d, k_row, k_tok, eb, width) || !kv_src_ok(v_src_d, v_row, v_tok, eb, width) ||
      !aligned(n_new_d, 4) || !aligned(parent_d, 4))
    return SV_ERR_ARG;
  if (q_heads && (!kv_src_ok(q_d, q_row, q_tok, eb, q_width) ||
                  !out_ok(q_d, q_row, q_tok, q_out_d, q_out_row, q_out_tok, eb, q_width, A.C.batch, T)))
    return SV_ERR_ARG;
  A.R = rope_of(rope, false);
  A.layer = layer;
  A.T = T;
  A.k = KvSrc{k_src_d, k_row, k_tok};
  A.v = KvSrc{v_src_d, v_row, v_tok};
  A.n_new = n_new_d;
  A.parent = parent_d;
  A.q = RopeRow{q_d, q_out_d, q_tok, q_out_tok, T, T, q_heads, A.C.dim, 1, q_out_d == q_d, false};
  A.q_row = q_row;
  A.q_out_row = q_out_row;
  return done(launch_kv_append_rope(A, rope->interleaved != 0, dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
