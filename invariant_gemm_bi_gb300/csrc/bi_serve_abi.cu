// bi_serve_abi.cu -- C ABI of the serving operations around the paged
// key-value cache: argument validation (all of it before any launch) and
// operand layouts.
#include <cmath>
#include <cstring>
#include <string>

#include "bi_check.h"
#include "bi_launch.h"
#include "bi_serve.h"

using namespace bi;

// ---------------------------------------------------------------------------
// Page planning
// ---------------------------------------------------------------------------
extern "C" bi_status bi_paged_plan(const bi_tensor* context_lens, const bi_tensor* new_lens,
                                   const bi_tensor* page_table, const bi_tensor* free_pages, int32_t page_size,
                                   const bi_tensor* seq_lens, const bi_tensor* token_offsets,
                                   const bi_tensor* positions, const bi_tensor* slots, const bi_tensor* totals,
                                   bi_stream stream) {
  Check c;
  c.tensor(page_table, "page_table", 2, true);
  c.that(!c.ok() || page_table->dtype == BI_I32, BI_ERR_UNSUPPORTED_DTYPE, "page_table: int32 is needed");
  c.that(page_size >= 1, BI_ERR_INVALID_ARG, "page_size must be positive");
  c.tensor(free_pages, "free_pages", 1, true);
  c.that(!c.ok() || free_pages->dtype == BI_I32, BI_ERR_UNSUPPORTED_DTYPE, "free_pages: int32 is needed");
  c.tensor(positions, "positions", 1, true);
  if (!c.ok()) return abi_finish(c.st, c.why);
  const int64_t B = page_table->shape[0], T = positions->shape[0];
  c.that(B <= kMaxRequests, BI_ERR_INVALID_ARG, "too many requests");
  c.vec(context_lens, "context_lens", B, BI_I32);
  c.vec(new_lens, "new_lens", B, BI_I32);
  c.vec(seq_lens, "seq_lens", B, BI_I32);
  c.vec(token_offsets, "token_offsets", B + 1, BI_I32);
  c.vec(positions, "positions", T, BI_I32);
  c.vec(slots, "slots", T, BI_I64);
  c.vec(totals, "totals", 2, BI_I32);
  c.distinct(page_table, "page_table");
  if (!c.ok()) return abi_finish(c.st, c.why);
  const bi_tensor* out[6] = {page_table, seq_lens, token_offsets, positions, slots, totals};
  const bi_tensor* in[3] = {context_lens, new_lens, free_pages};
  for (int i = 0; i < 6; ++i) {
    for (int j = 0; j < 3; ++j) c.apart(out[i], in[j], "bi_paged_plan");
    for (int j = 0; j < i; ++j) c.apart(out[i], out[j], "bi_paged_plan");
  }
  if (!c.ok()) return abi_finish(c.st, c.why);
  PlanParams p;
  p.ctx = static_cast<const int32_t*>(context_lens->ptr);
  p.add = static_cast<const int32_t*>(new_lens->ptr);
  p.pool = static_cast<const int32_t*>(free_pages->ptr);
  p.table = static_cast<int32_t*>(page_table->ptr);
  p.ld_table = stride_or(page_table, 0, page_table->shape[1]);
  p.seq_lens = static_cast<int32_t*>(seq_lens->ptr);
  p.offsets = static_cast<int32_t*>(token_offsets->ptr);
  p.positions = static_cast<int32_t*>(positions->ptr);
  p.slots = static_cast<int64_t*>(slots->ptr);
  p.totals = static_cast<int32_t*>(totals->ptr);
  p.B = (int32_t)B, p.W = (int32_t)page_table->shape[1], p.F = (int32_t)free_pages->shape[0];
  p.T = (int32_t)T, p.ps = page_size;
  c.st = launch_plan(p, (cudaStream_t)stream, &c.why);
  return abi_finish(c.st, c.why);
}

// ---------------------------------------------------------------------------
// Rotary positions and cache writes
// ---------------------------------------------------------------------------
namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

constexpr double kMaxFrequency = 9007199254740992.0;  // 2^53

// A number of 256 bits, the last one 2^-192; w[3] is the whole part.
struct Fixed {
  uint64_t w[4];
};
bool at_least(const Fixed& a, const Fixed& b) {
  for (int i = 3; i >= 0; --i)
    if (a.w[i] != b.w[i]) return a.w[i] > b.w[i];
  return true;
}
void subtract(Fixed& a, const Fixed& b) {
  uint64_t borrow = 0;
  for (int i = 0; i < 4; ++i) {
    const uint64_t x = a.w[i] - b.w[i], y = x - borrow;
    borrow = (a.w[i] < b.w[i]) | (x < borrow);
    a.w[i] = y;
  }
}
Fixed shifted(const Fixed& a, int n) {  // left, by 0 .. 255
  Fixed r = {};
  for (int i = 3; i >= n / 64; --i) {
    const int k = i - n / 64;
    r.w[i] = a.w[k] << n % 64;
    if (n % 64 && k > 0) r.w[i] |= a.w[k - 1] >> (64 - n % 64);
  }
  return r;
}

// 2^64 * (f / (2 pi) mod 1), rounded to nearest, 0 <= f < 2^53: binary long
// division by 2 pi, since a quotient in doubles would be off by up to 2^-56 of
// a turn for f near 1 -- 2^8 of the phase's units, and a millionth of a radian
// at positions around 2^33.  (2 pi's bits past 2^-192 move the quotient by
// 2^-139 at most.)
uint64_t turns_of(double f) {
  if (f < 1.0842021724855044e-19 /* 2^-63 */) return 0;  // below 2^-65 of a turn
  const Fixed turn = {{0x48127044533e63a0ull, 0x2633145c06e0e689ull, 0x487ed5110b4611a6ull, 6}};  // 2 pi
  int e;
  const double m = std::frexp(f, &e);  // f = m 2^e, -62 <= e <= 53
  Fixed rest = shifted({{(uint64_t)std::ldexp(m, 53), 0, 0, 0}}, 192 + e - 53);
  for (int k = 51; k >= 0; --k) {  // whole turns
    const Fixed d = shifted(turn, k);
    if (at_least(rest, d)) subtract(rest, d);
  }
  uint64_t q = 0;
  for (int k = 0; k <= 64; ++k) {  // 64 bits of the fraction, and the one that rounds them
    rest = shifted(rest, 1);
    const bool bit = at_least(rest, turn);
    if (bit) subtract(rest, turn);
    q = k < 64 ? q << 1 | bit : q + bit;
  }
  return q;
}

bi_status rope_config_ok(const bi_rope_config* cfg, std::string* why) {
  if (cfg->rotary_dim < 2 || cfg->rotary_dim > 2 * BI_ROPE_MAX_PAIRS || cfg->rotary_dim % 2 != 0 ||
      (cfg->interleaved != 0 && cfg->interleaved != 1) || !std::isfinite(cfg->magnitude)) {
    *why = "the rotary configuration is inconsistent (bi_rope_init fills one)";
    return BI_ERR_INVALID_ARG;
  }
  return BI_OK;
}

void positions_into(RopeParams* p, const bi_tensor* positions) {
  p->positions = positions->ptr;
  p->pos64 = positions->dtype == BI_I64;
}

void config_into(RopeParams* p, const bi_rope_config* cfg) {
  memcpy(p->phase, cfg->phase, sizeof(p->phase));
  p->magnitude = cfg->magnitude;
  p->half = cfg->rotary_dim / 2;
  p->interleaved = cfg->interleaved;
}

// The 16-byte units need whole octets of pairs and whole double octets of tail.
bool units_fit(const RopeParams& p) { return p.half % 8 == 0 && (p.D - 2 * p.half) % 16 == 0; }

bi_status run_rope(RopeParams& p, int64_t T, bi_stream stream, std::string* why) {
  if ((double)T * p.D * std::max(1, p.hq + 2 * p.hkv) > 5e11) {  // grids stay below 2^31 blocks
    *why = "too many elements";
    return BI_ERR_INVALID_ARG;
  }
  p.T = (int32_t)T;
  return launch_rope(p, (cudaStream_t)stream, why);
}

}  // namespace

extern "C" bi_status bi_rope_init_frequencies(bi_rope_config* out, int32_t rotary_dim, int32_t interleaved,
                                              const double* frequencies, double magnitude) {
  if (!out || !frequencies) return abi_finish(BI_ERR_INVALID_ARG, "null argument");
  bi_rope_config cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.rotary_dim = rotary_dim;
  cfg.interleaved = interleaved != 0;
  cfg.magnitude = (float)magnitude;
  std::string why;
  const bi_status st = rope_config_ok(&cfg, &why);
  if (st != BI_OK)
    return abi_finish(st, "rotary_dim must be even and within [2, 256], the magnitude finite");
  for (int i = 0; i < rotary_dim / 2; ++i) {
    if (!(std::fabs(frequencies[i]) < kMaxFrequency))
      return abi_finish(BI_ERR_INVALID_ARG, "a frequency is not finite, or 2^53 or more");
    const uint64_t turns = turns_of(std::fabs(frequencies[i]));
    cfg.phase[i] = frequencies[i] < 0.0 ? 0 - turns : turns;
  }
  *out = cfg;
  return abi_finish(BI_OK, "");
}

extern "C" bi_status bi_rope_init(bi_rope_config* out, int32_t rotary_dim, int32_t interleaved, double base,
                                  const bi_rope_scaling* scaling, double magnitude) {
  if (!out) return abi_finish(BI_ERR_INVALID_ARG, "null argument");
  if (rotary_dim < 2 || rotary_dim > 2 * BI_ROPE_MAX_PAIRS || rotary_dim % 2 != 0)
    return abi_finish(BI_ERR_INVALID_ARG, "rotary_dim must be even and within [2, 256]");
  if (!(base > 1.0) || !std::isfinite(base)) return abi_finish(BI_ERR_INVALID_ARG, "base must be finite and > 1");
  const int kind = scaling ? scaling->kind : BI_ROPE_PLAIN;
  if (kind < BI_ROPE_PLAIN || kind > BI_ROPE_RAMP_INDEX)
    return abi_finish(BI_ERR_INVALID_ARG, "unknown rotary scaling");
  const double R = rotary_dim;
  if (kind != BI_ROPE_PLAIN) {
    if (!(scaling->factor > 0.0) || !std::isfinite(scaling->factor))
      return abi_finish(BI_ERR_INVALID_ARG, "the scaling factor must be finite and > 0");
    if (kind == BI_ROPE_BASE && rotary_dim <= 2)
      return abi_finish(BI_ERR_INVALID_ARG, "scaling the base needs rotary_dim > 2");
    if (kind >= BI_ROPE_RAMP_TURNS &&
        (!(scaling->original_length > 0.0) || !std::isfinite(scaling->original_length) || !(scaling->low > 0.0) ||
         !(scaling->high > scaling->low) || !std::isfinite(scaling->high)))
      return abi_finish(BI_ERR_INVALID_ARG, "a ramp needs original_length > 0 and 0 < low < high");
  }
  if (kind == BI_ROPE_BASE) base *= std::pow(scaling->factor, R / (R - 2.0));
  double i_high = 0.0, i_low = 0.0;
  if (kind == BI_ROPE_RAMP_INDEX) {
    auto idx = [&](double r) { return R * std::log(scaling->original_length / (kTwoPi * r)) / (2.0 * std::log(base)); };
    i_high = std::max(std::floor(idx(scaling->high)), 0.0);
    i_low = std::min(std::ceil(idx(scaling->low)), R - 1.0);
  }
  double f[BI_ROPE_MAX_PAIRS];
  for (int i = 0; i < rotary_dim / 2; ++i) {
    f[i] = std::pow(base, -2.0 * i / R);
    if (kind == BI_ROPE_LINEAR) f[i] /= scaling->factor;
    if (kind >= BI_ROPE_RAMP_TURNS) {
      double g;
      if (kind == BI_ROPE_RAMP_TURNS) {
        const double r = scaling->original_length * f[i] / kTwoPi;
        g = (r - scaling->low) / (scaling->high - scaling->low);
      } else {
        g = 1.0 - (i - i_high) / std::max(i_low - i_high, 1e-3);  // a step where the two indices meet
      }
      g = std::min(1.0, std::max(0.0, g));
      f[i] *= g + (1.0 - g) / scaling->factor;
    }
  }
  return bi_rope_init_frequencies(out, rotary_dim, interleaved, f, magnitude);
}

extern "C" bi_status bi_rope(const bi_rope_config* config, const bi_tensor* x, const bi_tensor* positions,
                             int32_t transpose, const bi_tensor* y, bi_stream stream) {
  Check c;
  c.that(config != nullptr, BI_ERR_INVALID_ARG, "null rotary configuration");
  if (c.ok()) c.st = rope_config_ok(config, &c.why);
  c.tensor(x, "x", 3, false);
  c.tensor(y, "y", 3, false);
  c.tensor(positions, "positions", 1, true);
  if (!c.ok()) return abi_finish(c.st, c.why);
  const int64_t T = x->shape[0], H = x->shape[1], D = x->shape[2];
  c.that(y->shape[0] == T && y->shape[1] == H && y->shape[2] == D, BI_ERR_SHAPE_MISMATCH, "y must have x's shape");
  c.that(positions->shape[0] == T, BI_ERR_SHAPE_MISMATCH, "positions must be [T]");
  c.that(D >= config->rotary_dim && D <= 1024, BI_ERR_INVALID_ARG, "the head dimension must be within [rotary_dim, 1024]");
  if (!c.ok()) return abi_finish(c.st, c.why);
  c.distinct(y, "y");
  c.that(H <= kMaxHeads, BI_ERR_INVALID_ARG, "too many heads");
  if (!same_view(x, y)) c.apart(y, x, "bi_rope");
  c.apart(y, positions, "bi_rope");
  if (!c.ok() || T == 0 || H == 0) return abi_finish(c.st, c.why);
  RopeParams p;
  memset(&p, 0, sizeof(p));
  config_into(&p, config);
  positions_into(&p, positions);
  p.transpose = transpose != 0;
  p.q = {x->ptr, stride_or(x, 0, 0), stride_or(x, 1, 0)};
  p.q_out = y->ptr, p.qo_t = stride_or(y, 0, 0), p.qo_h = stride_or(y, 1, 0);
  p.hq = (int32_t)H, p.D = (int32_t)D, p.ps = 1;
  p.q_kind = kind_of(x->dtype), p.qo_kind = kind_of(y->dtype);
  p.vec = units_fit(p) && rows_on_16(x) && rows_on_16(y);
  c.st = run_rope(p, T, stream, &c.why);
  return abi_finish(c.st, c.why);
}

namespace {

// The caches of a layer: two tensors [P, page_size, Hkv, D] of one type, and for
// caches in 8 bits their scales [P, page_size, Hkv].
struct Caches {
  const bi_tensor *k, *v, *k_scales, *v_scales;
  bool scaled;

  void check(Check& c) const {
    const Check::Kind kind = scaled ? Check::kE4m3 : Check::kFloat;
    c.operand(k, "k_cache", 4, kind, true);
    c.operand(v, "v_cache", 4, kind, true);
    if (scaled) {
      c.operand(k_scales, "k_scales", 3, Check::kScale, false);
      c.operand(v_scales, "v_scales", 3, Check::kScale, false);
    }
    if (!c.ok()) return;
    for (int i = 0; i < 4; ++i)
      c.that(v->shape[i] == k->shape[i], BI_ERR_SHAPE_MISMATCH, "v_cache must have k_cache's shape");
    for (int i = 0; scaled && i < 3; ++i)
      c.that(k_scales->shape[i] == k->shape[i] && v_scales->shape[i] == k->shape[i], BI_ERR_SHAPE_MISMATCH,
             "k_scales and v_scales must be [P, page_size, Hkv] as the caches");
    c.that(v->dtype == k->dtype, BI_ERR_UNSUPPORTED_DTYPE, "k_cache and v_cache must have one type");
  }
  static PageView view(const bi_tensor* t) {
    return {t->ptr, stride_or(t, 0, 0), stride_or(t, 1, 0), stride_or(t, 2, 0)};
  }
};

bi_status store_impl(const bi_rope_config* config, const bi_tensor* positions, const bi_tensor* slots,
                     const bi_tensor* q, const bi_tensor* q_out, const bi_tensor* k, const bi_tensor* v,
                     const Caches& to, const char* name, bi_stream stream) {
  const bi_tensor *k_cache = to.k, *v_cache = to.v;
  Check c;
  if (config) {
    c.st = rope_config_ok(config, &c.why);
    c.tensor(positions, "positions", 1, true);
  } else {
    c.that(!q && !q_out && !positions, BI_ERR_INVALID_ARG,
           "without a rotary configuration q, q_out and positions must be absent");
  }
  c.that(!q == !q_out, BI_ERR_INVALID_ARG, "q and q_out are given together or not at all");
  c.tensor(k, "k", 3, false);
  c.tensor(v, "v", 3, false);
  to.check(c);
  if (q) {
    c.tensor(q, "q", 3, false);
    c.tensor(q_out, "q_out", 3, false);
  }
  if (!c.ok()) return abi_finish(c.st, c.why);
  const int64_t T = k->shape[0], H = k->shape[1], D = k->shape[2], P = k_cache->shape[0], ps = k_cache->shape[1];
  c.vec(slots, "slots", T, BI_I64);
  if (config) {
    c.that(positions->shape[0] == T, BI_ERR_SHAPE_MISMATCH, "positions must be [T]");
    c.that(D >= config->rotary_dim, BI_ERR_INVALID_ARG, "the head dimension is below rotary_dim");
  }
  c.that(D >= 1 && D <= 1024, BI_ERR_INVALID_ARG, "the head dimension must be within [1, 1024]");
  c.that(v->shape[0] == T && v->shape[1] == H && v->shape[2] == D, BI_ERR_SHAPE_MISMATCH, "v must have k's shape");
  c.that(v->dtype == k->dtype, BI_ERR_UNSUPPORTED_DTYPE, "k and v must have one type");
  c.that(k_cache->shape[2] == H && k_cache->shape[3] == D, BI_ERR_SHAPE_MISMATCH,
         "the caches must be [P, page_size, Hkv, D] with k's Hkv and D");
  c.that(ps >= 1 && P * ps <= INT32_MAX, BI_ERR_INVALID_ARG, "page_size must be positive and P * page_size < 2^31");
  if (q) {
    c.that(q->shape[0] == T && q->shape[2] == D, BI_ERR_SHAPE_MISMATCH, "q must be [T, Hq, D] with k's T and D");
    for (int i = 0; i < 3; ++i)
      c.that(q_out->shape[i] == q->shape[i], BI_ERR_SHAPE_MISMATCH, "q_out must have q's shape");
  }
  if (!c.ok()) return abi_finish(c.st, c.why);
  const bi_tensor* in[5] = {k, v, slots, positions, q};
  const bi_tensor* out[5] = {k_cache, v_cache, q_out, to.k_scales, to.v_scales};
  const char* names[5] = {"k_cache", "v_cache", "q_out", "k_scales", "v_scales"};
  for (int i = 0; i < 5; ++i) {
    if (!out[i]) continue;
    c.distinct(out[i], names[i]);
    for (int j = 0; j < 5; ++j)
      if (in[j] && !(i == 2 && j == 4 && same_view(q, q_out))) c.apart(out[i], in[j], name);
    for (int j = 0; j < i; ++j) c.apart(out[i], out[j], name);
  }
  const int64_t Hq = q ? q->shape[1] : 0;
  c.that(Hq + 2 * H <= kMaxHeads, BI_ERR_INVALID_ARG, "too many heads");
  if (!c.ok() || T == 0 || Hq + H == 0) return abi_finish(c.st, c.why);
  RopeParams p;
  memset(&p, 0, sizeof(p));
  if (config) {
    config_into(&p, config);
    positions_into(&p, positions);
  }
  if (q) {
    p.q = {q->ptr, stride_or(q, 0, 0), stride_or(q, 1, 0)};
    p.q_out = q_out->ptr, p.qo_t = stride_or(q_out, 0, 0), p.qo_h = stride_or(q_out, 1, 0);
    p.q_kind = kind_of(q->dtype), p.qo_kind = kind_of(q_out->dtype);
  }
  p.k = {k->ptr, stride_or(k, 0, 0), stride_or(k, 1, 0)};
  p.v = {v->ptr, stride_or(v, 0, 0), stride_or(v, 1, 0)};
  p.kc = Caches::view(k_cache), p.vc = Caches::view(v_cache);
  if (to.scaled) p.ks = Caches::view(to.k_scales), p.vs = Caches::view(to.v_scales);
  p.slots = static_cast<const int64_t*>(slots->ptr);
  p.num_slots = P * ps;
  p.hq = (int32_t)Hq, p.hkv = (int32_t)H, p.D = (int32_t)D, p.ps = (int32_t)ps;
  p.kv_kind = kind_of(k->dtype), p.c_kind = kind_of(k_cache->dtype);
  p.vec = units_fit(p) && rows_on_16(k) && rows_on_16(v) && rows_on_16(k_cache) && rows_on_16(v_cache) &&
          (!q || (rows_on_16(q) && rows_on_16(q_out)));
  // a scale is found by the lanes that hold a head: a whole, aligned group of one warp's
  if (to.scaled) p.vec = p.vec && D <= 512 && (D & (D - 1)) == 0;
  c.st = run_rope(p, T, stream, &c.why);
  return abi_finish(c.st, c.why);
}

}  // namespace

extern "C" bi_status bi_paged_store(const bi_rope_config* config, const bi_tensor* positions,
                                    const bi_tensor* slots, const bi_tensor* q, const bi_tensor* q_out,
                                    const bi_tensor* k, const bi_tensor* v, const bi_tensor* k_cache,
                                    const bi_tensor* v_cache, bi_stream stream) {
  return store_impl(config, positions, slots, q, q_out, k, v, {k_cache, v_cache, nullptr, nullptr, false},
                    "bi_paged_store", stream);
}

extern "C" bi_status bi_paged_store_quantized(const bi_rope_config* config, const bi_tensor* positions,
                                              const bi_tensor* slots, const bi_tensor* q, const bi_tensor* q_out,
                                              const bi_tensor* k, const bi_tensor* v, const bi_tensor* k_cache,
                                              const bi_tensor* k_scales, const bi_tensor* v_cache,
                                              const bi_tensor* v_scales, bi_stream stream) {
  return store_impl(config, positions, slots, q, q_out, k, v, {k_cache, v_cache, k_scales, v_scales, true},
                    "bi_paged_store_quantized", stream);
}

extern "C" bi_status bi_paged_load_quantized(const bi_tensor* slots, const bi_tensor* k_cache,
                                             const bi_tensor* k_scales, const bi_tensor* v_cache,
                                             const bi_tensor* v_scales, const bi_tensor* k, const bi_tensor* v,
                                             bi_stream stream) {
  const Caches from = {k_cache, v_cache, k_scales, v_scales, true};
  Check c;
  from.check(c);
  c.tensor(k, "k", 3, false);
  c.tensor(v, "v", 3, false);
  if (!c.ok()) return abi_finish(c.st, c.why);
  const int64_t T = k->shape[0], H = k->shape[1], D = k->shape[2], P = k_cache->shape[0], ps = k_cache->shape[1];
  c.vec(slots, "slots", T, BI_I64);
  c.that(D >= 1 && D <= 1024, BI_ERR_INVALID_ARG, "the head dimension must be within [1, 1024]");
  c.that(v->shape[0] == T && v->shape[1] == H && v->shape[2] == D, BI_ERR_SHAPE_MISMATCH, "v must have k's shape");
  c.that(v->dtype == k->dtype, BI_ERR_UNSUPPORTED_DTYPE, "k and v must have one type");
  c.that(k_cache->shape[2] == H && k_cache->shape[3] == D, BI_ERR_SHAPE_MISMATCH,
         "the caches must be [P, page_size, Hkv, D] with k's Hkv and D");
  c.that(ps >= 1 && P * ps <= INT32_MAX, BI_ERR_INVALID_ARG, "page_size must be positive and P * page_size < 2^31");
  // a token's heads of k and v, and its units of 16 elements, are counted in 32 bits
  c.that(2 * H <= kMaxHeads && H * ((D + 15) / 16) <= INT32_MAX, BI_ERR_INVALID_ARG, "too many heads");
  c.that((double)T * H * D <= 5e11, BI_ERR_INVALID_ARG, "too many elements");
  if (!c.ok()) return abi_finish(c.st, c.why);
  const bi_tensor* in[5] = {slots, k_cache, k_scales, v_cache, v_scales};
  c.distinct(k, "k");
  c.distinct(v, "v");
  for (int j = 0; j < 5; ++j) {
    c.apart(k, in[j], "bi_paged_load_quantized");
    c.apart(v, in[j], "bi_paged_load_quantized");
  }
  c.apart(k, v, "bi_paged_load_quantized");
  if (!c.ok() || T == 0 || H == 0) return abi_finish(c.st, c.why);
  LoadParams p;
  memset(&p, 0, sizeof(p));
  p.kc = Caches::view(k_cache), p.vc = Caches::view(v_cache);
  p.ks = Caches::view(k_scales), p.vs = Caches::view(v_scales);
  p.k = k->ptr, p.k_t = stride_or(k, 0, 0), p.k_h = stride_or(k, 1, 0);
  p.v = v->ptr, p.v_t = stride_or(v, 0, 0), p.v_h = stride_or(v, 1, 0);
  p.slots = static_cast<const int64_t*>(slots->ptr);
  p.num_slots = P * ps;
  p.T = (int32_t)T, p.H = (int32_t)H, p.D = (int32_t)D, p.ps = (int32_t)ps, p.kind = kind_of(k->dtype);
  p.vec = D % 16 == 0 && rows_on_16(k) && rows_on_16(v) && rows_on_16(k_cache) && rows_on_16(v_cache);
  c.st = launch_paged_load(p, (cudaStream_t)stream, &c.why);
  return abi_finish(c.st, c.why);
}

// ---------------------------------------------------------------------------
// Attention over the paged cache
// ---------------------------------------------------------------------------
extern "C" int64_t bi_paged_attention_workspace_bytes(int64_t B, int64_t Hq, int64_t D, int64_t max_len) {
  if (B <= 0 || Hq <= 0 || max_len <= 0 || B > INT32_MAX || Hq > INT32_MAX || !attention_head_dim_ok(D)) return 0;
  const int64_t n = paged_max_splits(max_len, false);
  if (n <= 1) return 0;
  const int64_t rows = B * Hq;  // below 2^62
  return rows > INT64_MAX / (n * (D + 2) * 4) ? INT64_MAX : rows * n * (D + 2) * 4;
}

namespace {

bi_status attention_impl(const bi_tensor* q, const Caches& caches, const bi_tensor* page_table,
                         const bi_tensor* seq_lens, float scale, const bi_tensor* o, void* workspace,
                         int64_t workspace_bytes, const char* name, bi_stream stream) {
  const bi_tensor *k_cache = caches.k, *v_cache = caches.v;
  Check c;
  c.tensor(q, "q", 3, false);
  caches.check(c);
  c.tensor(page_table, "page_table", 2, true);
  c.tensor(o, "o", 3, false);
  if (!c.ok()) return abi_finish(c.st, c.why);
  const int64_t B = q->shape[0], Hq = q->shape[1], D = q->shape[2];
  const int64_t P = k_cache->shape[0], ps = k_cache->shape[1], Hkv = k_cache->shape[2], W = page_table->shape[1];
  c.that(page_table->dtype == BI_I32, BI_ERR_UNSUPPORTED_DTYPE, "page_table: int32 is needed");
  c.that(page_table->shape[0] == B, BI_ERR_SHAPE_MISMATCH, "page_table must be [B, W] with q's B");
  c.vec(seq_lens, "seq_lens", B, BI_I32);
  c.that(k_cache->shape[3] == D, BI_ERR_SHAPE_MISMATCH, "the caches must be [P, page_size, Hkv, D] with q's D");
  c.that(o->shape[0] == B && o->shape[1] == Hq && o->shape[2] == D, BI_ERR_SHAPE_MISMATCH, "o must have q's shape");
  c.that(q->dtype == BI_BF16 || q->dtype == BI_F16, BI_ERR_UNSUPPORTED_DTYPE, "q must be bf16 or fp16");
  c.that(caches.scaled || k_cache->dtype == q->dtype, BI_ERR_UNSUPPORTED_DTYPE, "the caches must have q's type");
  c.that(attention_head_dim_ok(D), BI_ERR_INVALID_ARG, "head dimension must be 64, 128 or 256");
  const float score_log2 = (float)((double)scale * 1.4426950408889634);
  c.that(std::isfinite(score_log2), BI_ERR_INVALID_ARG, "scale and scale * log2(e) must be finite");
  c.that(ps >= 1, BI_ERR_INVALID_ARG, "page_size must be positive");
  c.that(Hkv >= 1 ? Hq % Hkv == 0 : Hq == 0, BI_ERR_SHAPE_MISMATCH, "Hkv must divide Hq");
  c.that(P * ps <= INT32_MAX, BI_ERR_INVALID_ARG, "P * page_size must be below 2^31");
  c.that(W * ps <= (int64_t)1 << 30, BI_ERR_INVALID_ARG, "W * page_size must be at most 2^30");
  c.that(workspace_bytes >= 0, BI_ERR_INVALID_ARG, "negative workspace size");
  if (!c.ok()) return abi_finish(c.st, c.why);
  const bi_tensor* ts[4] = {q, k_cache, v_cache, o};
  for (int i = 0; i < 4; ++i)
    c.that(Check::empty(ts[i]) || rows_on_16(ts[i]), BI_ERR_UNSUPPORTED_LAYOUT,
           "base pointers and strides of q, the caches and o must be multiples of 16 bytes");
  const bi_tensor* in[7] = {q, k_cache, v_cache, page_table, seq_lens, caches.k_scales, caches.v_scales};
  c.distinct(o, "o");
  for (int i = 0; i < 7; ++i) c.apart(o, in[i], name);
  if (!c.ok() || B == 0 || Hq == 0) return abi_finish(c.st, c.why);
  const int64_t cap = W * ps, need = bi_paged_attention_workspace_bytes(B, Hq, D, cap);
  c.that(B * Hq * (D / 64) <= INT32_MAX && B <= kMaxRequests, BI_ERR_INVALID_ARG, "too many requests");
  c.that(!workspace || on(workspace, 16), BI_ERR_UNSUPPORTED_LAYOUT, "the workspace must be 16-byte aligned");
  if (!c.ok()) return abi_finish(c.st, c.why);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return abi_finish(BI_ERR_INVALID_ARG, "key ranges of up to " + std::to_string(cap) + " need a workspace of " +
                                              std::to_string(need) + " bytes (bi_paged_attention_workspace_bytes)");
  if (need > 0) {
    bi_tensor ws;
    memset(&ws, 0, sizeof(ws));
    ws.ptr = workspace, ws.ndim = 1, ws.dtype = BI_F32, ws.shape[0] = need / 4, ws.stride[0] = 1;
    for (int i = 0; i < 7; ++i) c.apart(&ws, in[i], "workspace");
    c.apart(&ws, o, "workspace");
    if (!c.ok()) return abi_finish(c.st, c.why);
  }
  PagedAttnParams p;
  memset(&p, 0, sizeof(p));
  p.q = q->ptr, p.q_b = stride_or(q, 0, 0), p.q_h = stride_or(q, 1, 0);
  // (an empty cache may have no address: its keys are all absent, and a copy of
  // no bytes is given some address that is one)
  p.k = P * ps > 0 ? k_cache->ptr : q->ptr, p.v = P * ps > 0 ? v_cache->ptr : q->ptr;
  p.k_page = stride_or(k_cache, 0, 0), p.k_row = stride_or(k_cache, 1, 0), p.k_head = stride_or(k_cache, 2, 0);
  p.v_page = stride_or(v_cache, 0, 0), p.v_row = stride_or(v_cache, 1, 0), p.v_head = stride_or(v_cache, 2, 0);
  p.table = static_cast<const int32_t*>(page_table->ptr);
  p.ld_table = stride_or(page_table, 0, W);
  p.lens = static_cast<const int32_t*>(seq_lens->ptr);
  p.o = o->ptr, p.o_b = stride_or(o, 0, 0), p.o_h = stride_or(o, 1, 0);
  p.max_splits = paged_max_splits(cap, caches.scaled);
  p.ws_o = static_cast<float*>(workspace);
  p.ws_ml = p.ws_o ? p.ws_o + B * p.max_splits * Hq * D : nullptr;
  p.B = (int32_t)B, p.Hq = (int32_t)Hq, p.Hkv = (int32_t)Hkv, p.D = (int32_t)D;
  p.W = (int32_t)W, p.ps = (int32_t)ps, p.P = (int32_t)P, p.cap = (int32_t)cap;
  p.group = (int32_t)(Hq / Hkv);
  p.ps_shift = (ps & (ps - 1)) == 0 ? __builtin_ctzll((unsigned long long)ps) : -1;
  if (caches.scaled) {
    p.ks = Caches::view(caches.k_scales), p.vs = Caches::view(caches.v_scales);
    if (P * ps == 0) p.ks.ptr = p.vs.ptr = seq_lens->ptr;
  }
  p.e4m3 = caches.scaled;
  p.in_f16 = q->dtype == BI_F16;
  p.out_kind = kind_of(o->dtype);
  p.score_log2 = score_log2;
  c.st = launch_paged_attention(p, (cudaStream_t)stream, &c.why);
  return abi_finish(c.st, c.why);
}

}  // namespace

extern "C" bi_status bi_paged_attention(const bi_tensor* q, const bi_tensor* k_cache, const bi_tensor* v_cache,
                                        const bi_tensor* page_table, const bi_tensor* seq_lens, float scale,
                                        const bi_tensor* o, void* workspace, int64_t workspace_bytes,
                                        bi_stream stream) {
  return attention_impl(q, {k_cache, v_cache, nullptr, nullptr, false}, page_table, seq_lens, scale, o, workspace,
                        workspace_bytes, "bi_paged_attention", stream);
}

extern "C" bi_status bi_paged_attention_quantized(const bi_tensor* q, const bi_tensor* k_cache,
                                                  const bi_tensor* k_scales, const bi_tensor* v_cache,
                                                  const bi_tensor* v_scales, const bi_tensor* page_table,
                                                  const bi_tensor* seq_lens, float scale, const bi_tensor* o,
                                                  void* workspace, int64_t workspace_bytes, bi_stream stream) {
  return attention_impl(q, {k_cache, v_cache, k_scales, v_scales, true}, page_table, seq_lens, scale, o, workspace,
                        workspace_bytes, "bi_paged_attention_quantized", stream);
}

// ---------------------------------------------------------------------------
// Token log probabilities
// ---------------------------------------------------------------------------
extern "C" bi_status bi_token_logprobs(const bi_tensor* logits, const bi_tensor* tokens, const bi_tensor* logprobs,
                                       const bi_tensor* entropy, const bi_tensor* top_logprobs,
                                       const bi_tensor* top_ids, bi_stream stream) {
  Check c;
  c.tensor(logits, "logits", 2, false);
  c.tensor(tokens, "tokens", 1, true);
  c.tensor(logprobs, "logprobs", 1, false);
  if (entropy) c.tensor(entropy, "entropy", 1, false);
  c.that(!top_logprobs == !top_ids, BI_ERR_INVALID_ARG, "top_logprobs and top_ids are given together or not at all");
  if (top_ids) {
    c.tensor(top_logprobs, "top_logprobs", 2, false);
    c.tensor(top_ids, "top_ids", 2, true);
  }
  if (!c.ok()) return abi_finish(c.st, c.why);
  const int64_t R = logits->shape[0], N = logits->shape[1], K = top_ids ? top_ids->shape[1] : 0;
  c.that(tokens->shape[0] == R, BI_ERR_SHAPE_MISMATCH, "tokens must be [R]");
  c.that(logprobs->shape[0] == R, BI_ERR_SHAPE_MISMATCH, "logprobs must be [R]");
  c.that(logprobs->dtype == BI_F32, BI_ERR_UNSUPPORTED_DTYPE, "logprobs must be fp32");
  if (entropy) {
    c.that(entropy->shape[0] == R, BI_ERR_SHAPE_MISMATCH, "entropy must be [R]");
    c.that(entropy->dtype == BI_F32, BI_ERR_UNSUPPORTED_DTYPE, "entropy must be fp32");
  }
  if (top_ids) {
    c.that(top_ids->shape[0] == R && top_logprobs->shape[0] == R && top_logprobs->shape[1] == K,
           BI_ERR_SHAPE_MISMATCH, "top_ids and top_logprobs must be [R, K]");
    c.that(top_ids->dtype == BI_I32 && top_logprobs->dtype == BI_F32, BI_ERR_UNSUPPORTED_DTYPE,
           "top_ids must be int32 and top_logprobs fp32");
    c.that(K <= 64 && K <= N, BI_ERR_INVALID_ARG, "at most 64 alternatives, and at most N");
    for (const bi_tensor* t : {top_ids, top_logprobs})
      c.that(R <= 1 || t->stride[0] == K, BI_ERR_UNSUPPORTED_LAYOUT, "top_ids and top_logprobs must be contiguous");
  }
  c.that(N <= (1 << 24), BI_ERR_INVALID_ARG, "rows longer than 2^24 elements are not supported");
  c.that(N >= 1 || R == 0, BI_ERR_INVALID_ARG, "a row needs at least one logit");
  if (!c.ok()) return abi_finish(c.st, c.why);
  const bi_tensor* out[4] = {logprobs, entropy, top_logprobs, top_ids};
  for (int i = 0; i < 4; ++i) {
    c.apart(out[i], logits, "bi_token_logprobs");
    c.apart(out[i], tokens, "bi_token_logprobs");
    for (int j = 0; j < i; ++j) c.apart(out[i], out[j], "bi_token_logprobs");
  }
  if (!c.ok() || R == 0) return abi_finish(c.st, c.why);
  LogprobParams p;
  memset(&p, 0, sizeof(p));
  p.x = logits->ptr, p.tokens = tokens->ptr;
  p.lp = static_cast<float*>(logprobs->ptr);
  p.entropy = entropy ? static_cast<float*>(entropy->ptr) : nullptr;
  p.top_lp = K ? static_cast<float*>(top_logprobs->ptr) : nullptr;
  p.top_ids = K ? static_cast<int32_t*>(top_ids->ptr) : nullptr;
  p.R = R, p.N = N, p.ld_x = R > 1 ? logits->stride[0] : 0;
  p.K = (int32_t)K, p.tok64 = tokens->dtype == BI_I64, p.x_kind = kind_of(logits->dtype);
  c.st = launch_logprobs(p, (cudaStream_t)stream, &c.why);
  return abi_finish(c.st, c.why);
}
