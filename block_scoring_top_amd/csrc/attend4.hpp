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
//     the exponential's argument.
// The reference of a row's sums is the running maximum of score + log2(the unit's largest
// value scale): what it bounds is the products of weight and value, not the weights, so
// that one token with large values and no weight costs the others no bits. Both the sums
// and the sum of weights are held in units of it (weights reach 2^60 then, in fp32).
#pragma once

#include "attend.hpp"

namespace idxk {

typedef uint16_t at_u16x2 __attribute__((ext_vector_type(2)));

constexpr uint32_t kNanScale = 255;

// eight codes times the scale -> bf16, exact
__device__ __forceinline__ at_bf16x8 codes4_bf16(uint32_t w, float scale) {
  auto two = [](auto r) { return __builtin_bit_cast(uint32_t, r); };
  return __builtin_bit_cast(
      at_bf16x8, make_uint4(two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)),
                            two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)),
                            two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)),
                            two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3))));
}
// eight codes -> fp16, exact
__device__ __forceinline__ at_f16x8 codes4_f16(uint32_t w) {
  auto two = [](auto r) { return __builtin_bit_cast(uint32_t, r); };
  return __builtin_bit_cast(
      at_f16x8, make_uint4(two(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.f, 0)),
                           two(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.f, 1)),
                           two(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.f, 2)),
                           two(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.f, 3))));
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

// Two scales (bytes 2 i, 2 i + 1 of w) as fp16 relative to the scale byte floor + 15:
// 2^(byte - floor - 15), zero from 2^-15 on. Bytes are at most floor + 15.
template <int I>
__device__ __forceinline__ uint32_t two_scales(uint32_t w, uint32_t floor2) {
  const uint32_t b = __builtin_amdgcn_perm(0u, w, I == 0 ? 0x0C010C00u : 0x0C030C02u);
  const at_u16x2 d = __builtin_elementwise_sub_sat(__builtin_bit_cast(at_u16x2, b),
                                                   __builtin_bit_cast(at_u16x2, floor2));
  return __builtin_bit_cast(uint32_t, d << (uint16_t)10);
}
__device__ __forceinline__ uint32_t mul_f16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(at_f16x2, a) *
                                          __builtin_bit_cast(at_f16x2, b));
}

struct Cache4 {
  struct Tile {
    uint4 k[4];       // token 4 s + n % 4 of unit n / 4, dims 32 g ..
    uint32_t ks[4];   // their scales
    uint2 v[8];       // the 16 tokens of unit g at dim 16 dt + n
    uint4 vs[4];      // the 16 tokens' scales of dims 32 i ..
    uint32_t top;     // a word of vs: together the group's lanes hold each of them once

    __device__ __forceinline__ void load(const AttnArgs& a, int kblk, int ksub, int vblk, int vsub,
                                         int n, int g) {
      const int64_t kb = max(kblk, 0), vb = max(vblk, 0);
      const int64_t row = kb * a.page_size + ksub * kUnit + (n & 3);
      const uint8_t* kp = a.k_cache + row * (kHeadDim / 2) + 16 * g;
      const uint8_t* sp = a.k_exp + row * 4 + g;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        k[s] = *reinterpret_cast<const uint4*>(kp + s * (4 * kHeadDim / 2));
        ks[s] = sp[16 * s];
      }
      const int half = a.page_size / 2;
      const uint8_t* vp =
          a.v_cache + vb * (kHeadDim * (int64_t)half) + n * half + vsub * (kUnit / 2);
#pragma unroll
      for (int dt = 0; dt < 8; ++dt)
        v[dt] = *reinterpret_cast<const uint2*>(vp + dt * 16 * half);
      const uint8_t* ep = a.v_exp + vb * (4 * (int64_t)a.page_size) + vsub * kUnit;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        vs[i] = *reinterpret_cast<const uint4*>(ep + i * a.page_size);
      top = *reinterpret_cast<const uint32_t*>(ep + (n >> 2) * a.page_size + 4 * (n & 3));
    }

    template <int NT, int KIND, bool MIXED>
    __device__ __forceinline__ void add(AttnState<NT>& st, const at_bf16x8 (&q)[NT][4], int vblk,
                                        float call_scale, int pos, int have, const int (&len)[NT],
                                        const float (&slope2)[NT], const Cap& cap, bool any) {
      static_assert(!MIXED || NT == 1, "one visible length a lane");
      // The unit's largest value scale, of the tokens that the row sees. NaN scales are
      // left out of it, and make NaN of S.
      bool nan = false;
      uint32_t vtop = 0;
      if (any) {
        const int mine = min(have, len[0] - pos);
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t* w = reinterpret_cast<uint32_t*>(&vs[i]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            w[j] = keep_bytes(w[j], mine - 4 * j);
            vtop = max(vtop, top_byte(w[j]));
            bad |= nan_scales(w[j]);
          }
        }
        nan = __any(bad != 0);
      } else {
        vtop = group_max(top_byte(top));
        nan = __any(nan_scales(top) != 0);
      }
      vtop = max(vtop, 15u);
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
            x[j][s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kt, q[j][t], x[j][s], 0, 0, 0);
        }
      }
      uint32_t p[NT][8];  // probabilities of token pairs, over 2^lv
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float best = -__builtin_inff();
        const float bias = KIND == kPlain ? 0.f : -slope2[j] * (float)(len[j] - 1 - pos);
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tok = 4 * s + i;
            float y = x[j][s][i];
            if constexpr (KIND != kPlain)
              y = score2<KIND>(y, call_scale, cap, __builtin_fmaf((float)tok, slope2[j], bias));
            if (any) y = (tok < have && pos + tok < len[j]) ? y : -__builtin_inff();
            x[j][s][i] = y;
            best = fmaxf(best, y);
          }
        // (not 0 for masked scores)
        const float sc = KIND != kPlain ? 1.f : fmaxf(call_scale, 0x1p-126f);
        best = groups_max(__builtin_fmaf(best, sc, lv));
        if (__any(best > st.m[j] + kLazy)) {
          const float m = best > st.m[j] + kLazy ? best : st.m[j];
          const float f = exp2_fast(st.m[j] - (m == -__builtin_inff() ? 0.f : m));
          st.m[j] = m;
          st.l[j] *= f;
#pragma unroll
          for (int dt = 0; dt < 8; ++dt) st.o[j][dt] *= f;
        }
        const float off = (st.m[j] == -__builtin_inff() ? 0.f : st.m[j]) - kPBias - lv;
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
        st.l[j] = __builtin_fmaf(sum[0] + sum[1], unlv, st.l[j]);
      }
      const uint32_t floor2 = (vtop - 15u) * 0x00010001u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {vs[i].x, vs[i].y, vs[i].z, vs[i].w};
        uint32_t sv[8];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          sv[2 * t] = two_scales<0>(w[t], floor2);
          sv[2 * t + 1] = two_scales<1>(w[t], floor2);
        }
        if (nan) {  // a rare path
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            const uint32_t pair = w[t >> 1] >> (16 * (t & 1));
            if ((pair & 255u) == kNanScale) sv[t] = (sv[t] & 0xFFFF0000u) | 0x7E00u;
            if (((pair >> 8) & 255u) == kNanScale) sv[t] = (sv[t] & 0xFFFFu) | 0x7E000000u;
          }
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
};

}  // namespace idxk
