// C ABI of rotary positions (include/idx_rope.h): the tables, worked out on the host, and
// the call's argument validation. As in api.cpp, validation makes no HIP call.
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "idx_rope.h"
#include "launch.h"

namespace {

constexpr int64_t kMaxInt = (int64_t(1) << 31) - 1;
constexpr int kMaxTokens = 1 << 24;  // 256 threads each: what a launch holds
constexpr double kTwoPi = 6.283185307179586476925286766559;
constexpr double kMaxFreq = 4;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// f / (2 pi) turns in units of 2^-64, modulo a turn: off by less than a unit (64 bits of
// fraction; a double's 53 would be felt at positions from 2^25 on)
bool turns_of(double f, uint64_t* out) {
  static_assert(LDBL_MANT_DIG >= 64, "the table's units");
  if (!isfinite(f) || fabs(f) > kMaxFreq) return false;
  const long double two_pi = 6.283185307179586476925286766559005768L;
  const uint64_t n = (uint64_t)rintl(ldexpl(fabsl((long double)f) / two_pi, 64));
  *out = f < 0 ? 0 - n : n;
  return true;
}

bool in_order(double lo, double hi) {
  return isfinite(lo) && isfinite(hi) && lo > 0 && hi > lo;
}

}  // namespace

extern "C" {

int idx_rope_turns(const double* inv_freq, int pairs, uint64_t* turns) {
  if (inv_freq == nullptr || turns == nullptr || pairs < 1) return IDX_ERR_INVALID_ARG;
  if (pairs > IDX_HEAD_DIM / 2) return IDX_ERR_UNSUPPORTED;
  for (int i = 0; i < pairs; ++i)
    if (!turns_of(inv_freq[i], turns + i)) return IDX_ERR_INVALID_ARG;
  return IDX_OK;
}

int idx_rope_table(double base, int rot, int kind, double stretch, double original, double lo,
                   double hi, uint64_t* turns) {
  if (turns == nullptr || rot < 2 || rot % 2 != 0 || kind < IDX_ROPE_PLAIN ||
      kind > IDX_ROPE_BY_INDEX || !isfinite(base) || !(base > 1))
    return IDX_ERR_INVALID_ARG;
  if (rot > IDX_HEAD_DIM) return IDX_ERR_UNSUPPORTED;
  if (kind != IDX_ROPE_PLAIN && !(isfinite(stretch) && stretch >= 1)) return IDX_ERR_INVALID_ARG;
  if (kind == IDX_ROPE_BASE && rot == 2) return IDX_ERR_INVALID_ARG;
  const bool blend = kind == IDX_ROPE_BY_TURNS || kind == IDX_ROPE_BY_INDEX;
  if (blend && !(isfinite(original) && original > 0 && in_order(lo, hi)))
    return IDX_ERR_INVALID_ARG;

  const int pairs = rot / 2;
  if (kind == IDX_ROPE_BASE) base *= pow(stretch, (double)rot / (rot - 2));
  if (!isfinite(base)) return IDX_ERR_INVALID_ARG;
  // the pair with n turns over the original length, as a fraction of an index
  auto index_of = [&](double n) { return pairs * log(original / (kTwoPi * n)) / log(base); };
  double from = 0, to = 0;
  if (kind == IDX_ROPE_BY_INDEX) {
    from = fmax(floor(index_of(hi)), 0);
    to = fmin(ceil(index_of(lo)), rot - 1);
    if (to <= from) to = from + 0.001;  // a step
  }
  uint64_t made[IDX_HEAD_DIM / 2];
  for (int i = 0; i < pairs; ++i) {
    double f = pow(base, -2.0 * i / rot), keep = 1;
    if (kind == IDX_ROPE_LINEAR) keep = 0;
    if (kind == IDX_ROPE_BY_TURNS) keep = (original * f / kTwoPi - lo) / (hi - lo);
    if (kind == IDX_ROPE_BY_INDEX) keep = 1 - (i - from) / (to - from);
    if (kind == IDX_ROPE_LINEAR || blend) {
      keep = fmin(fmax(keep, 0), 1);
      f *= keep + (1 - keep) / stretch;
    }
    if (!turns_of(f, made + i)) return IDX_ERR_INVALID_ARG;
  }
  for (int i = 0; i < pairs; ++i) turns[i] = made[i];
  return IDX_OK;
}

int idx_rope(const void* q, const void* k, int64_t q_stride, int64_t k_stride,
             const int32_t* tok_len, const uint64_t* turns, void* q_out, void* k_out,
             int64_t q_out_stride, int64_t k_out_stride, int n_tok, int Hq, int Hkv, int D,
             int first, int rot, float factor, uint32_t flags, idx_dtype dt, void* stream) {
  if (n_tok < 0 || Hq < 1 || Hkv < 0 || D < 1 || first < 0 || rot < 2 || rot % 2 != 0 ||
      !isfinite(factor) || (flags & ~(IDX_ROPE_ADJACENT | IDX_ROPE_INVERSE)) != 0)
    return IDX_ERR_INVALID_ARG;
  if (dt != IDX_F32 && dt != IDX_BF16) return IDX_ERR_INVALID_ARG;
  if (D != IDX_HEAD_DIM) return IDX_ERR_UNSUPPORTED;
  if ((int64_t)first + rot > D) return IDX_ERR_INVALID_ARG;
  if (rot % 16 != 0 || first % 8 != 0) return IDX_ERR_UNSUPPORTED;
  if (((int64_t)Hq + Hkv) * D > kMaxInt || n_tok >= kMaxTokens)
    return IDX_ERR_INVALID_ARG;
  if (n_tok > 0) {
    if (q == nullptr || q_out == nullptr || tok_len == nullptr || turns == nullptr)
      return IDX_ERR_INVALID_ARG;
    if ((k == nullptr || k_out == nullptr) && Hkv > 0) return IDX_ERR_INVALID_ARG;
    const int64_t strides[] = {q_stride, q_out_stride, k_stride, k_out_stride};
    for (int i = 0; i < (Hkv > 0 ? 4 : 2); ++i)
      if (strides[i] < (int64_t)(i < 2 ? Hq : Hkv) * D || strides[i] % 8 != 0)
        return IDX_ERR_INVALID_ARG;
    if ((q == q_out && q_stride != q_out_stride) ||
        (Hkv > 0 && k == k_out && k_stride != k_out_stride))
      return IDX_ERR_INVALID_ARG;
  }
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) ||
      !aligned(tok_len, 4) || !aligned(turns, 8))
    return IDX_ERR_INVALID_ARG;
  if (n_tok == 0) return IDX_OK;
  idxk::RopeArgs a{};
  a.q = q;
  a.k = k;
  a.q_out = q_out;
  a.k_out = k_out;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.q_out_stride = q_out_stride;
  a.k_out_stride = k_out_stride;
  a.tok_len = tok_len;
  a.turns = turns;
  a.n_tok = n_tok;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.first = first;
  a.rot = rot;
  a.factor = factor;
  a.adjacent = (flags & IDX_ROPE_ADJACENT) != 0;
  a.inverse = (flags & IDX_ROPE_INVERSE) != 0;
  return idxk::launch_rope(a, dt == IDX_BF16, stream) == 0 ? IDX_OK : IDX_ERR_HIP;
}

}  // extern "C"
