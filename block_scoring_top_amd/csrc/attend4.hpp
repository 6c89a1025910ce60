// Attention over the paged 4-bit cache: its tile of 64 tokens, for the rows' kernel of
// attend_rows.hpp (the layout of units, products and lanes is that of attend.hpp).
//
// With lane = (n, g), n = lane % 16, g = lane / 16:
//   - keys: product s takes token 4 s + n % 4 of unit n / 4; a lane's 16 bytes of it are
//     the 32 dims of block g, so that one scale goes with them, and step t of the four
//     products over the dims takes dims 32 g + 8 t .. of every block (queries are loaded in
//     that order). The conversion to bf16 takes the scale along: exact, and no scale is left
//     to apply to a score;
//   - values: eight bytes are the 16 tokens of unit g at one dim; codes are exact in fp16.
//     Their scales, a byte for each token and 32 dims, go to the probabilities: once for
//     each of the four groups of 32 dims, as packed fp16 products with
//     S = 2^(scale - the unit's largest scale), exact, and the unit's largest enters with
//     the exponential's argument. The 16 lanes of a group make the factors of four tokens and
//     32 dims each, and hand them to each other in LDS.
// The reference of a row's sums is the running maximum of score + log2(the unit's largest
// value scale): what it bounds is the products of weight and value, not the weights, so
// that one token with large values and no weight costs the others no bits. Both the sums
// and the sum of weights are held in units of it. Weights reach 2^60 then, in fp32, and the
// reference moves by up to 2^120 more than the scores do, which no single exponential holds: the
// sum of weights moves in two (scaled_down), and the exponentials of a unit far below the
// reference take along more than its scale (far_scale).
#pragma once

#include "attend.hpp"

namespace idxk {

typedef uint16_t at_u16x2 __attribute__((ext_vector_type(2)));

constexpr uint32_t kNanScale = 255;

// The exponent that a unit's exponentials take along, and the sum of weights gives back: its
// largest scale's, lv, or, where its best product of weight and scale, 2^best, lies 2^kFar or
// more below the reference, as much more as brings it there. The probabilities of such a unit
// are zeros in fp16 either way; its weights may count all the same, with scales up to 2^120
// apart, and keep the bits of those down to 2^-35 of the unit's largest (exponentials below
// 2^-126 are zeros). At most the largest scale's 60: what is below the reference then still has a
// weight of 2^-100 of the row's largest or less.
// (The largest scales, 2^60, lie 2^kFar above those of kLowTop: units from there on need none of
// this.)
constexpr float kFar = 100.f;
constexpr uint32_t kLowTop = 127 - 40;
__device__ __forceinline__ float far_scale(float lv, float best, float m) {
  return fminf(fmaxf(lv, floorf(m - kFar - (best - lv))), 60.f);
}

// eight codes times the scale -> bf16, exact
__device__ __forceinline__ at_bf16x8 codes4_bf16(uint32_t w, float scale) {
  auto two = [](auto r) { return __builtin_bit_cast(uint32_t, r); };
  return __builtin_bit_cast(
      at_bf16x8, make_uint4(two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)),
                            two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)),
                            two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)),
                            two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3))));
}
// eight codes times 1 or 2 -> fp16, exact
__device__ __forceinline__ at_f16x8 codes4_f16(uint32_t w, float scale = 1.f) {
  auto two = [](auto r) { return __builtin_bit_cast(uint32_t, r); };
  return __builtin_bit_cast(
      at_f16x8, make_uint4(two(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 0)),
                           two(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 1)),
                           two(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 2)),
                           two(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 3))));
}

// the bytes of 255
__device__ __forceinline__ uint32_t nan_scales(uint32_t w) {
  return nan_codes(w) & w;
}
// the largest of four bytes, NaN scales left out
__device__ __forceinline__ uint32_t top_byte(uint32_t w) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = (w >> (8 * i)) & 255u;
    m = max(m, b == kNanScale ? 0u : b);
  }
  return m;
}
// over the 16 lanes of a group
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  v = max(v, dpp_u32<kDppQuadXor1>(v));
  v = max(v, dpp_u32<kDppQuadXor2>(v));
  v = max(v, dpp_u32<kDppRowHalfMirror>(v));
  return max(v, dpp_u32<kDppRowMirror>(v));
}
// the bytes of the tokens from `have` on of a word of four become 0
__device__ __forceinline__ uint32_t keep_bytes(uint32_t w, int have) {
  return have >= 4 ? w : have <= 0 ? 0u : w & (0xFFFFFFFFu >> (32 - 8 * have));
}

// bytes of two words, the larger of each place
__device__ __forceinline__ uint32_t max_u16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(at_u16x2, a),
                                                                __builtin_bit_cast(at_u16x2, b)));
}
// Two scales (bytes 2 i, 2 i + 1 of w) as fp16 relative to the scale byte floor + 25:
// 2^(byte - floor - 25), down to the least subnormal, 2^-24; zero from 2^-25 on. Bytes are at
// most floor + 25, or, with CLAMP, larger ones (of tokens that a row does not see, or NaN) give
// something finite. (Bit patterns are in the order of the values: e = byte - floor above 10 has
// the exponent e - 10, the others are 2^(e - 1) units of 2^-24.)
constexpr uint32_t kBelow = 25;
template <int I, bool CLAMP = false>
__device__ __forceinline__ uint32_t two_scales(uint32_t w, uint32_t floor2) {
  const uint32_t b = __builtin_amdgcn_perm(0u, w, I == 0 ? 0x0C010C00u : 0x0C030C02u);
  at_u16x2 e = __builtin_elementwise_sub_sat(__builtin_bit_cast(at_u16x2, b),
                                             __builtin_bit_cast(at_u16x2, floor2));
  if constexpr (CLAMP) e = __builtin_elementwise_min(e, at_u16x2{40, 40});
  const at_u16x2 normal = __builtin_elementwise_sub_sat(e, at_u16x2{10, 10}) << (uint16_t)10;
  const at_u16x2 small = (at_u16x2{1, 1} << __builtin_elementwise_min(e, at_u16x2{10, 10})) >>
                         (uint16_t)1;
  return max_u16(__builtin_bit_cast(uint32_t, normal), __builtin_bit_cast(uint32_t, small));
}
constexpr uint32_t kEvenBytes = 0x00FF00FFu;
// A group's 16 lanes hold, each, a byte for four tokens, of four blocks of 32 dims (lane i:
// block i / 4, tokens 4 (i % 4) ..): the largest of each token, NaN left out, in every lane of
// its place.
__device__ __forceinline__ uint32_t token_tops(uint32_t w) {
  w &= ~((nan_scales(w) >> 7) * 255u);
  uint32_t even = w & kEvenBytes, odd = (w >> 8) & kEvenBytes;
  even = max_u16(even, dpp_u32<kDppRowRor1 + 3>(even));
  odd = max_u16(odd, dpp_u32<kDppRowRor1 + 3>(odd));
  even = max_u16(even, dpp_u32<kDppRowRor1 + 7>(even));
  odd = max_u16(odd, dpp_u32<kDppRowRor1 + 7>(odd));
  return even | (odd << 8);
}
// the largest of 16 tokens' bytes, of the first `have`
__device__ __forceinline__ uint32_t seen_top(uint4 tops, int have) {
  const uint32_t w[4] = {keep_bytes(tops.x, have), keep_bytes(tops.y, have - 4),
                         keep_bytes(tops.z, have - 8), keep_bytes(tops.w, have - 12)};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = max_u16(m, max_u16(w[i] & kEvenBytes, (w[i] >> 8) & kEvenBytes));
  return max(m & 0xFFFFu, m >> 16);
}
// which of the four blocks of dims hold a NaN scale of the first `have` tokens
__device__ __forceinline__ uint32_t seen_nans(const uint4 (&bytes)[4], int have) {
  uint32_t bad = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 w = bytes[i];
    if ((nan_scales(keep_bytes(w.x, have)) | nan_scales(keep_bytes(w.y, have - 4)) |
         nan_scales(keep_bytes(w.z, have - 8)) | nan_scales(keep_bytes(w.w, have - 12))) != 0)
      bad |= 1u << i;
  }
  return bad;
}
__device__ __forceinline__ uint32_t mul_f16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(at_f16x2, a) *
                                          __builtin_bit_cast(at_f16x2, b));
}

// the four bytes' largest, and over the 16 lanes of a group
__device__ __forceinline__ uint32_t group_top(uint32_t w) {
  return group_max(max(max(w & 255u, (w >> 8) & 255u), max((w >> 16) & 255u, w >> 24)));
}

// Between one lane's store to LDS and another's load, in one wave: LDS takes a wave's
// accesses in order, the compiler has to as well.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

struct Cache4 {
  // The rows' operands stay in LDS: 16 registers fewer, and with them four waves a SIMD
  // where nothing spills for it (4 rows of 4096 to 131072 tokens 73.7 us with three, 71.0 with
  // four; 128 rows of 256 selected pages, two workgroups a CU, 57.5 and 57.2).
  static constexpr bool kRowsInLds = true;
  template <int NT, int KIND, bool PACKED>
  static constexpr int kWaves = NT == 1 && !PACKED && KIND == kPlain ? 4 : NT == 1 ? 3 : 2;
  // A unit's value scales, and those as fp16 factors: written by the 16 lanes of its group, a
  // word of four tokens each, read by all of them.
  struct Scratch {
    uint4 bytes[4][4];    // [unit][32 dims], a byte a token
    uint32_t tops[4][4];  // [unit], a byte a token: its largest
    uint2 factor[4][16];  // [unit][32 dims, four tokens]
  };
  struct Tile {
    uint4 k[4];       // token 4 s + n % 4 of unit n / 4, dims 32 g ..
    uint32_t ks[4];   // their scales
    uint2 v[8];       // the 16 tokens of unit g at dim 32 (i / 2) + 2 n + i % 2
    uint32_t vs;      // four tokens' value scales: dims 32 (n / 4) .., tokens 4 (n % 4) ..

    __device__ __forceinline__ void load(const AttnArgs& a, int kblk, int ksub, int vblk, int vsub,
                                         int n, int g) {
      const int64_t kb = max(kblk, 0), vb = max(vblk, 0);
      const int64_t row = kb * a.page_size + ksub * kUnit + (n & 3);
      const uint8_t* kp = a.k_cache + row * (kHeadDim / 2) + 16 * g;
      const uint8_t* sp = a.k_exp + row * 4 + g;
      vs = *reinterpret_cast<const uint32_t*>(a.v_exp +
                                              (vb * 4 + (n >> 2)) * (int64_t)a.page_size +
                                              vsub * kUnit + 4 * (n & 3));
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        k[s] = *reinterpret_cast<const uint4*>(kp + s * (4 * kHeadDim / 2));
        ks[s] = sp[16 * s];
      }
      const int half = a.page_size / 2;
      const uint8_t* vp =
          a.v_cache + vb * (kHeadDim * (int64_t)half) + 2 * n * half + vsub * (kUnit / 2);
      if (a.page_size == kUnit) {  // two dims are 16 bytes
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 x = *reinterpret_cast<const uint4*>(vp + i * 32 * (kUnit / 2));
          v[2 * i] = make_uint2(x.x, x.y);
          v[2 * i + 1] = make_uint2(x.z, x.w);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] = *reinterpret_cast<const uint2*>(vp + ((i >> 1) * 32 + (i & 1)) * half);
      }
    }

    template <int NT, int KIND, bool MIXED>
    __device__ __forceinline__ void add(AttnState<NT>& st, const uint4 (&q)[4 * NT][kWave], int vblk,
                                        float call_scale, int pos, int have, const int (&len)[NT],
                                        const float (&slope2)[NT], const Cap& cap, bool any,
                                        Scratch& lds) {
      static_assert(!MIXED || NT == 1, "one visible length a lane");
      const int lane = lane_id(), n = lane & 15, g = lane >> 4;
      // The unit's largest value scale, of the tokens that the row sees, and the factors
      // relative to it; NaN scales are left out (rows that see them are seen to below).
      if (any) vs = keep_bytes(vs, have - 4 * (n & 3));
      uint32_t vtop = group_top(vs);
      const bool nan = __any(vtop == kNanScale);
      if (nan) vtop = group_max(top_byte(vs));
      // rows of different lengths that see a unit in part: each takes its own
      const bool own = MIXED && any;
      wave_order();  // (behind the loads of the tile before)
      if (nan || own) reinterpret_cast<uint32_t*>(lds.bytes[g])[n] = vs;
      const int mine = min(have, len[0] - pos);
      if (own) {
        lds.tops[g][n & 3] = token_tops(vs);
        wave_order();
        vtop = seen_top(*reinterpret_cast<const uint4*>(lds.tops[g]), mine);
      }
      vtop = max(vtop, kBelow);
      const uint32_t floor2 = (vtop - kBelow) * 0x00010001u;
      if (!own)
        lds.factor[g][n] = make_uint2(two_scales<0>(vs, floor2), two_scales<1>(vs, floor2));
      wave_order();
      const float lv = (float)((int)vtop - 127);
      const float unlv = __uint_as_float((254u - vtop) << 23);

      at_f32x4 x[NT][4];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
#pragma unroll
        for (int j = 0; j < NT; ++j) x[j][s] = at_f32x4{0.f, 0.f, 0.f, 0.f};
        const float sc = __uint_as_float(ks[s] << 23);
        const uint32_t w[4] = {k[s].x, k[s].y, k[s].z, k[s].w};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const at_bf16x8 kt = codes4_bf16(w[t], sc);
#pragma unroll
          for (int j = 0; j < NT; ++j)
            x[j][s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                kt, __builtin_bit_cast(at_bf16x8, q[4 * j + t][lane]), x[j][s], 0, 0, 0);
        }
      }
      uint32_t p[NT][8];  // probabilities of token pairs, times 2^lv
      // (not 0 for masked scores)
      const float sc = KIND != kPlain ? 1.f : fmaxf(call_scale, 0x1p-126f);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if constexpr (KIND != kPlain) {
          const float bias = -slope2[j] * (float)(len[j] - 1 - pos);
#pragma unroll
          for (int t = 0; t < 16; ++t)
            x[j][t >> 2][t & 3] = score2<KIND>(x[j][t >> 2][t & 3], call_scale, cap,
                                               __builtin_fmaf((float)t, slope2[j], bias));
        }
        if (any) {
          asm volatile("");  // a branch: few tiles are masked
#pragma unroll
          for (int t = 0; t < 16; ++t)
            if (t >= min(have, len[j] - pos)) x[j][t >> 2][t & 3] = -__builtin_inff();
        }
        float unit = -__builtin_inff();  // this lane's unit's best product
#pragma unroll
        for (int t = 0; t < 16; ++t) unit = fmaxf(unit, x[j][t >> 2][t & 3]);
        unit = __builtin_fmaf(unit, sc, lv);
        const float best = groups_max(unit);
        if (__any(best > st.m[j] + kLazy)) {
          const float m = best > st.m[j] + kLazy ? best : st.m[j];
          const float d = st.m[j] - (m == -__builtin_inff() ? 0.f : m), f = exp2_fast(d);
          st.m[j] = m;
          st.l[j] = scaled_down(st.l[j], d);
#pragma unroll
          for (int dt = 0; dt < 8; ++dt) st.o[j][dt] *= f;
        }
        float take = lv, back = unlv;
        if (__any(unit < st.m[j] - kFar)) {
          asm volatile("");  // a branch: few tiles are that far
          take = far_scale(lv, unit, st.m[j]);
          back = exp2_fast(-take);
        }
        const float off = (st.m[j] == -__builtin_inff() ? 0.f : st.m[j]) - kPBias - take;
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          float e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            e[i] = exp2_fast(__builtin_fmaf(x[j][s][i], sc, -off));
            sum[i & 1] += e[i];
          }
          p[j][2 * s] = pack_f16(e[0], e[1]);
          p[j][2 * s + 1] = pack_f16(e[2], e[3]);
        }
        st.l[j] = __builtin_fmaf(sum[0] + sum[1], back, st.l[j]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t sv[8];
        if (own) {
          asm volatile("");
          const uint4 b = lds.bytes[g][i];
          const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            sv[2 * t] = two_scales<0, true>(w[t], floor2);
            sv[2 * t + 1] = two_scales<1, true>(w[t], floor2);
          }
        } else {
          const uint4* f = reinterpret_cast<const uint4*>(&lds.factor[g][4 * i]);
          const uint4 a = f[0], b = f[1];
          sv[0] = a.x, sv[1] = a.y, sv[2] = a.z, sv[3] = a.w;
          sv[4] = b.x, sv[5] = b.y, sv[6] = b.z, sv[7] = b.w;
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint32_t pv[8];
#pragma unroll
          for (int t = 0; t < 8; ++t) pv[t] = mul_f16(p[j][t], sv[t]);
          const at_f16x8 p0 = __builtin_bit_cast(at_f16x8, make_uint4(pv[0], pv[1], pv[2], pv[3]));
          const at_f16x8 p1 = __builtin_bit_cast(at_f16x8, make_uint4(pv[4], pv[5], pv[6], pv[7]));
#pragma unroll
          for (int dt = 2 * i; dt < 2 * i + 2; ++dt) {
            st.o[j][dt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes4_f16(v[dt].x), p0,
                                                                 st.o[j][dt], 0, 0, 0);
            st.o[j][dt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes4_f16(v[dt].y), p1,
                                                                 st.o[j][dt], 0, 0, 0);
          }
        }
      }
      if (nan) {
        // the groups of dims in which the row sees a NaN scale, of any unit
        uint32_t bad = seen_nans(lds.bytes[g], mine);
        bad |= lane_xor<16>(bad);
        bad |= lane_xor<32>(bad);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int dt = 0; dt < 8; ++dt)
            if ((bad >> (dt >> 1)) & 1u)
              st.o[j][dt] = at_f32x4{1.f, 1.f, 1.f, 1.f} * __builtin_nanf("");
      }
    }
  };

  // Query rows of a lane as the B operand: step t holds dims 32 g + 8 t .. + 7. A negative
  // call scale turns the queries' signs (scores keep their order under its size).
  static __device__ __forceinline__ void load_query(const uint16_t* row, int g, bool negative,
                                                    at_bf16x8 (&q)[4]) {
    const uint32_t sign = negative ? 0x80008000u : 0u;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint4 x = *reinterpret_cast<const uint4*>(row + 32 * g + 8 * t);
      q[t] = __builtin_bit_cast(at_bf16x8,
                                make_uint4(x.x ^ sign, x.y ^ sign, x.z ^ sign, x.w ^ sign));
    }
  }
  template <int NT>
  static __device__ __forceinline__ void init(AttnState<NT>& st) {
    st.vref = 1.f;  // sums are in units of the reference alone
  }
  template <int NT>
  static __device__ __forceinline__ const uint4 (&rows(
      const at_bf16x8 (&)[NT][4], const uint4 (&lds)[4 * NT][kWave]))[4 * NT][kWave] {
    return lds;
  }
  // (rows 4 g .. of the products 2 i and 2 i + 1 are the even and odd dims of eight)
  static __device__ __forceinline__ int dim_of(int dt, int g) {
    return 32 * (dt >> 1) + 8 * g + 4 * (dt & 1);
  }
  template <int NT>
  static __device__ __forceinline__ at_f32x4 sums(const AttnState<NT>& st, int j, int dt) {
    const at_f32x4 &a = st.o[j][dt & ~1], &b = st.o[j][dt | 1];
    return dt & 1 ? at_f32x4{a[2], b[2], a[3], b[3]} : at_f32x4{a[0], b[0], a[1], b[1]};
  }
};

}  // namespace idxk
