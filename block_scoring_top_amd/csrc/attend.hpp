// Attention over the paged 8-bit cache: what its kernels share (gfx950, wave64).
//
// The online softmax runs in base 2 over tiles of 64 tokens. A tile is four units of
// 16 tokens, each inside one page; lane group g = lane / 16 owns unit g. With keys as
// the A operand of v_mfma_f32_16x16x32_bf16 and queries as B, row m of product s is
// given token 4 s + m % 4 of unit m / 4, so that a lane's 16 scores (row 4 g + i of
// s = 0..3) are the 16 tokens of its own unit for query row n = lane % 16:
//   - the unit's page scales are one number per lane;
//   - the probabilities of eight consecutive tokens are already in the lane that needs
//     them as the B operand of the second product, whose A operand, the values of
//     those tokens at one dim, is 8 consecutive bytes of the value cache;
// so neither scores nor values cross lanes, and both caches go straight from memory
// into registers, 16 bytes a lane.
// A probability is held as 2^(x - m + kPBias), with a reference m that is moved only when
// the row's maximum has grown by kLazy or more (most tiles then leave the sums alone): it
// reaches 2^(kPBias + kLazy), which fp16 holds, and keeps 11 bits down to 2^-23 of the
// row's largest. The value scale of a unit enters with the exponential's argument, as a
// logarithm relative to the largest scale that the row has seen, and leaves the sum of
// weights once a unit. References are each row's own: rows that share products see
// different tokens, and no bit of one depends on what only another sees.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attend_args.h"
#include "common.hpp"

namespace idxk {

typedef __bf16 at_bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 at_bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 at_f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 at_f16x2 __attribute__((ext_vector_type(2)));
typedef float at_f32x2 __attribute__((ext_vector_type(2)));
typedef float at_f32x4 __attribute__((ext_vector_type(4)));

constexpr int kUnit = 16;       // tokens of a unit
constexpr int kTileTok = 64;    // tokens of a tile: one unit per lane group
constexpr float kPBias = 9.f;
constexpr float kLazy = 6.f;
constexpr float kLog2e = 1.4426950408889634f;

// four e4m3 codes -> bf16 / fp16 (both exact)
__device__ __forceinline__ void codes_bf16(uint32_t w, uint32_t (&o)[2]) {
  o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, false));
  o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, true));
}
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&o)[2]) {
  o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, false));
  o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, true));
}
__device__ __forceinline__ at_bf16x8 codes_bf16x8(uint32_t lo, uint32_t hi) {
  uint32_t a[2], b[2];
  codes_bf16(lo, a);
  codes_bf16(hi, b);
  return __builtin_bit_cast(at_bf16x8, make_uint4(a[0], a[1], b[0], b[1]));
}
__device__ __forceinline__ at_f16x8 codes_f16x8(uint32_t lo, uint32_t hi) {
  uint32_t a[2], b[2];
  codes_f16(lo, a);
  codes_f16(hi, b);
  return __builtin_bit_cast(at_f16x8, make_uint4(a[0], a[1], b[0], b[1]));
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  at_f32x2 f = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, at_f16x2));
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  at_f32x2 f = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, at_bf16x2));
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// over the four lane groups of one query row
__device__ __forceinline__ float groups_max(float v) {
  v = fmaxf(v, __uint_as_float(lane_xor<16>(__float_as_uint(v))));
  return fmaxf(v, __uint_as_float(lane_xor<32>(__float_as_uint(v))));
}
__device__ __forceinline__ float groups_sum(float v) {
  v += __uint_as_float(lane_xor<16>(__float_as_uint(v)));
  return v + __uint_as_float(lane_xor<32>(__float_as_uint(v)));
}

// What happens to a score beside its scale (a capped one may be biased too).
constexpr int kPlain = 0, kBiased = 1, kCapped = 2, kCappedFar = 3;

// The constants of capped scores, cap * tanh(x / cap) in base-2 units, by
// tanh y = 1 - 2 / (1 + e^(2y)): y large gives 1, y small -1, no overflow. It is off by up
// to 2^-21 of the cap, which is a bound of the score's own error for caps up to kNearCap.
// Above it (kCappedFar: the score is small beside the cap) |y| < 1/4 takes the series
// y (1 - z/3 + 2 z^2/15 - 17 z^3/315 + 62 z^4/2835), z = y^2, whose next term is 2^-26.8:
// off by 2^-19 of the score, as the formula is from 1/4 on. Five instructions a score
// against sixteen: 1024 tokens of 128 selected pages 87 us against 93, two prompts of 8192
// tokens 1.58 ms against 1.85.
constexpr float kNearCap = 64.f;
struct Cap {
  float in, out;  // exponent of a unit-scaled product; cap in base-2 units
  float inv;
  __device__ __forceinline__ explicit Cap(float cap)
      : in(cap > 0.f ? 2.f * kLog2e / cap : 0.f), out(cap * kLog2e),
        inv(cap > 0.f ? 1.f / cap : 0.f) {}
};

// The capped or biased score of a token: ksc holds the page's key scale, the call's
// scale and, for uncapped scores, log2(e); bias = -slope * distance.
template <int KIND>
__device__ __forceinline__ float score2(float dot, float ksc, const Cap& cap, float bias) {
  if constexpr (KIND == kCapped) {
    const float r = __builtin_amdgcn_rcpf(1.f + exp2_fast(dot * (ksc * cap.in)));
    return __builtin_fmaf(-2.f * cap.out, r, cap.out) + bias;
  }
  if constexpr (KIND == kCappedFar) {
    const float x = dot * ksc, y = x * cap.inv, z = y * y;
    const float r = __builtin_amdgcn_rcpf(1.f + exp2_fast(y * (2.f * kLog2e)));
    float p = __builtin_fmaf(z, 62.f / 2835.f, -17.f / 315.f);
    p = __builtin_fmaf(z, __builtin_fmaf(z, p, 2.f / 15.f), -1.f / 3.f);
    const float near = __builtin_fmaf(x * z, p, x) * kLog2e;
    return (z < 0.0625f ? near : __builtin_fmaf(-2.f * cap.out, r, cap.out)) + bias;
  }
  return __builtin_fmaf(dot, ksc, bias);
}

// the running softmax of NT tiles of 16 query rows
template <int NT>
struct AttnState {
  at_f32x4 o[NT][8];  // dims 16 dt + 4 g + i of query row n
  float m[NT], l[NT];  // m: all groups alike; l: this group's units alone
  // largest value scale seen, and its logarithm: o is in its units (rows of different
  // visible lengths: each lane's row has its own, and NT is 1)
  float vref, lref;
};

template <int NT>
__device__ __forceinline__ void attn_init(AttnState<NT>& st) {
  st.vref = 0.f;
  st.lref = 0.f;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    st.m[j] = -__builtin_inff();
    st.l[j] = 0.f;
#pragma unroll
    for (int dt = 0; dt < 8; ++dt) st.o[j][dt] = at_f32x4{0.f, 0.f, 0.f, 0.f};
  }
}

// Query rows of a lane as the B operand: chunk (c, half) holds dims
// 64 c + 16 g + 8 half .. + 7 of query row n. A negative call scale turns the queries'
// signs, so that scores keep their order under the (positive) scale of a unit.
__device__ __forceinline__ void load_query(const uint16_t* row, int g, bool negative,
                                           at_bf16x8 (&q)[4]) {
  const uint32_t sign = negative ? 0x80008000u : 0u;
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint4 x = *reinterpret_cast<const uint4*>(row + 64 * c + 16 * g + 8 * half);
      q[2 * c + half] = __builtin_bit_cast(
          at_bf16x8, make_uint4(x.x ^ sign, x.y ^ sign, x.z ^ sign, x.w ^ sign));
    }
}

// zeroes the codes of the tokens from `have` on (whatever they hold, NaN included,
// they would meet a probability of zero)
__device__ __forceinline__ uint4 keep_tokens(uint4 v, int have) {
  auto word = [&](uint32_t w, int first) -> uint32_t {
    const int n = have - first;
    return n >= 4 ? w : n <= 0 ? 0u : w & (0xFFFFFFFFu >> (32 - 8 * n));
  };
  return make_uint4(word(v.x, 0), word(v.y, 4), word(v.z, 8), word(v.w, 12));
}

// Whether a code is NaN: low seven bits all set.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// In a tile that some rows see only in part, a NaN value code must reach the rows that
// see its token and no others, though all rows share the product (0 x NaN = NaN).
// Replaces NaN codes by zero and puts NaN into the sums of the rows that see them: the
// product of "code is NaN" with "row sees token" is positive exactly there.
template <int NT>
__device__ __forceinline__ void attn_nan_values(AttnState<NT>& st, uint4 (&v)[8], int pos,
                                                int have, const int (&len)[NT]) {
  uint32_t bad = 0;
#pragma unroll
  for (int dt = 0; dt < 8; ++dt)
    bad |= nan_codes(v[dt].x) | nan_codes(v[dt].y) | nan_codes(v[dt].z) | nan_codes(v[dt].w);
  if (!__any(bad != 0)) return;
  uint4 sees[NT][2];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    uint32_t w[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      auto one = [&](int tok) { return tok < have && pos + tok < len[j] ? 0x3C00u : 0u; };
      w[t] = one(2 * t) | (one(2 * t + 1) << 16);
    }
    sees[j][0] = make_uint4(w[0], w[1], w[2], w[3]);
    sees[j][1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
#pragma unroll
  for (int dt = 0; dt < 8; ++dt) {
    uint32_t w[4] = {v[dt].x, v[dt].y, v[dt].z, v[dt].w}, is[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t n = nan_codes(w[e]) >> 7;  // 1 in each NaN byte
      is[e] = n * 0x38u;                        // e4m3 1.0 there
      w[e] &= ~(n * 0xFFu);
    }
    v[dt] = make_uint4(w[0], w[1], w[2], w[3]);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      at_f32x4 hit = {0.f, 0.f, 0.f, 0.f};
      hit = __builtin_amdgcn_mfma_f32_16x16x32_f16(
          codes_f16x8(is[0], is[1]), __builtin_bit_cast(at_f16x8, sees[j][0]), hit, 0, 0, 0);
      hit = __builtin_amdgcn_mfma_f32_16x16x32_f16(
          codes_f16x8(is[2], is[3]), __builtin_bit_cast(at_f16x8, sees[j][1]), hit, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (hit[i] > 0.f) st.o[j][dt][i] = __builtin_nanf("");
    }
    __builtin_amdgcn_sched_barrier(0);  // a rare path: no registers for it
  }
}

// One tile. k: this lane's key bytes, k[s][c] = dims 64 c + 16 g .. + 15 of token
// 4 s + m % 4 of unit m / 4; v[dt]: the 16 tokens of unit g at dim 16 dt + n.
// ksc: the score scale of unit g; vs: its value scale, 0 if it holds no token; pos:
// position of its first token; have: how many of its tokens exist; len: visible length
// of each of the lane's query rows; any: whether a token of the tile is masked for any
// row (uniform over the wave). MIXED: the rows' visible lengths differ (then NT is 1).
template <int NT, int KIND, bool MIXED>
__device__ __forceinline__ void attn_tile(AttnState<NT>& st, const at_bf16x8 (&q)[NT][4],
                                          const uint4 (&k)[4][2], uint4 (&v)[8], float ksc,
                                          float vs, int pos, int have, const int (&len)[NT],
                                          const float (&slope2)[NT], const Cap& cap, bool any) {
  static_assert(!MIXED || NT == 1, "one reference of the value scales a lane");
  if (MIXED && pos >= len[0]) vs = 0.f;  // none of the unit for this row
  const float vtop = groups_max(vs);
  if (vtop > st.vref) {
    const float f = st.vref / vtop;
    st.vref = vtop;
    st.lref = __log2f(vtop);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int dt = 0; dt < 8; ++dt) st.o[j][dt] *= f;
  }
  // (below 2^-60 of the largest, fp16 holds nothing of it)
  const float lv = vs == st.vref ? 0.f : fmaxf(__log2f(vs) - st.lref, -60.f);
  const float unlv = exp2_fast(-lv);
  at_f32x4 x[NT][4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
#pragma unroll
    for (int j = 0; j < NT; ++j) x[j][s] = at_f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const at_bf16x8 k0 = codes_bf16x8(k[s][c].x, k[s][c].y);
      const at_bf16x8 k1 = codes_bf16x8(k[s][c].z, k[s][c].w);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        x[j][s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, q[j][2 * c], x[j][s], 0, 0, 0);
        x[j][s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, q[j][2 * c + 1], x[j][s], 0, 0, 0);
      }
    }
  }
  uint4 p[NT][2];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    float top = -__builtin_inff();
    const float bias = KIND == kPlain ? 0.f : -slope2[j] * (float)(len[j] - 1 - pos);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tok = 4 * s + i;
        float y = x[j][s][i];
        if constexpr (KIND != kPlain)
          y = score2<KIND>(y, ksc, cap, __builtin_fmaf((float)tok, slope2[j], bias));
        if (any) y = (tok < have && pos + tok < len[j]) ? y : -__builtin_inff();
        x[j][s][i] = y;
        top = fmaxf(top, y);
      }
    // uncapped scores are scaled by ksc > 0 from here on (not 0, for masked ones)
    const float sc = KIND != kPlain ? 1.f : fmaxf(ksc, 0x1p-126f);
    top = groups_max(top * sc);
    if (__any(top > st.m[j] + kLazy)) {
      const float m = top > st.m[j] + kLazy ? top : st.m[j];
      const float f = exp2_fast(st.m[j] - (m == -__builtin_inff() ? 0.f : m));
      st.m[j] = m;
      st.l[j] *= f;
#pragma unroll
      for (int dt = 0; dt < 8; ++dt) st.o[j][dt] *= f;
    }
    const float off = (st.m[j] == -__builtin_inff() ? 0.f : st.m[j]) - kPBias - lv;
    float sum[2] = {0.f, 0.f};
    uint32_t w[8];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      float e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e[i] = exp2_fast(__builtin_fmaf(x[j][s][i], sc, -off));
        sum[i & 1] += e[i];
      }
      w[2 * s] = pack_f16(e[0], e[1]);
      w[2 * s + 1] = pack_f16(e[2], e[3]);
    }
    p[j][0] = make_uint4(w[0], w[1], w[2], w[3]);
    p[j][1] = make_uint4(w[4], w[5], w[6], w[7]);
    st.l[j] = __builtin_fmaf(sum[0] + sum[1], unlv, st.l[j]);
  }
  // (values of tokens that no row sees: whatever they hold, it would meet a zero)
  if (any) {
#pragma unroll
    for (int dt = 0; dt < 8; ++dt) v[dt] = keep_tokens(v[dt], have);
    if constexpr (MIXED) attn_nan_values<NT>(st, v, pos, have, len);
  }
#pragma unroll
  for (int dt = 0; dt < 8; ++dt) {
    const at_f16x8 v0 = codes_f16x8(v[dt].x, v[dt].y);
    const at_f16x8 v1 = codes_f16x8(v[dt].z, v[dt].w);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      st.o[j][dt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
          v0, __builtin_bit_cast(at_f16x8, p[j][0]), st.o[j][dt], 0, 0, 0);
      st.o[j][dt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
          v1, __builtin_bit_cast(at_f16x8, p[j][1]), st.o[j][dt], 0, 0, 0);
    }
  }
}

// The page list of a request.
struct PageList {
  int64_t base;
  int n;  // pages
};
__device__ __forceinline__ PageList page_list(const AttnArgs& a, int b) {
  const int64_t lo = a.kv_indptr[b], hi = a.kv_indptr[b + 1];
  const int64_t n = hi - lo;
  return {lo, (int)(n < 0 ? 0 : n < a.max_pages ? n : a.max_pages)};
}
// The cache block (page, head) of a list slot, or -1.
__device__ __forceinline__ int block_of(const AttnArgs& a, const PageList& p, int slot, int h) {
  if (slot < 0 || slot >= p.n) return -1;
  const int64_t at = p.base + slot;
  if (at < 0 || at >= a.n_indices) return -1;
  const int page = a.kv_indices[at];
  if (page < 0 || page >= a.n_pages) return -1;
  return page * a.Hkv + h;
}

__device__ __forceinline__ float slope_of(const AttnArgs& a, int hq) {
  return a.slopes == nullptr ? 0.f : a.slopes[hq] * kLog2e;
}

// Row tiles of packed tokens: `per` rows (token, head of the group) of one request each.
// Request b's first is floor(rows before it / per) + b: floor(y / T) - floor(x / T) + 1
// tiles hold any x..y rows, so tiles never span requests.
__device__ __forceinline__ int64_t first_tile(const AttnArgs& a, int b, int G, int per) {
  const int64_t p = min(max(a.tok_indptr[b], 0), a.R);
  return p * G / per + b;
}
struct RowTile {
  int b, t0;           // request and its first token row
  int64_t row0, rows;  // first row of the tile, rows of the request (0 <= row0 < rows, or
                       // the tile holds none)
};
// (Every request is looked at by a thread of the workgroup at once: a search by halves is
// a chain of loads, 77.5 us against 75.9 for 47 short prompts.) found: a word of LDS.
template <int NT>
__device__ __forceinline__ RowTile row_tile(const AttnArgs& a, int64_t tile, int G, int per,
                                            int* found) {
  if (threadIdx.x == 0) *found = -1;
  __syncthreads();
  for (int i = threadIdx.x; i < a.B; i += NT)
    if (first_tile(a, i, G, per) <= tile && tile < first_tile(a, i + 1, G, per)) *found = i;
  __syncthreads();
  const int b = *found;
  if (b < 0) return {0, 0, 0, 0};
  const int t0 = min(max(a.tok_indptr[b], 0), a.R);
  const int t1 = min(max(a.tok_indptr[b + 1], 0), a.R);
  return {b, t0, (tile - first_tile(a, b, G, per)) * per, (int64_t)(t1 - t0) * G};
}

}  // namespace idxk
