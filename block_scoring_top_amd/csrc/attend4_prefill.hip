// Attention of packed prompt tokens over the paged 4-bit cache (include/idx_cache4.h,
// idx_attend4_prefill). The split of the work, the products and the layout of their operands
// in LDS are those of attend_prefill.hip: a workgroup owns kP4Rows rows (token, head of the
// KV head's group) of one request, 32 to a wave, and walks its tokens in tiles of 64, whose
// codes are converted once, on their way into LDS.
//   - Keys become bf16 with their scales, exact.
//   - Values become fp16, doubled: whole numbers, exact with factors down to fp16's least,
//     2^-24. In a tile that all rows see whole, a value takes its scale along, relative to the
//     largest of the 16 tokens' (of its unit, 2^lv), and 2^lv enters with the exponential's
//     argument and leaves the sum of weights once a unit. In one that some rows see in part
//     (the end of each row), values stay plain codes, and the scales of the tokens that a row
//     sees go to its probabilities, a group of 32 dims at a time, as in attend4.hpp: nothing
//     of a row comes from tokens that it does not see, and a NaN scale reaches just the rows
//     that see it. (Units that a wave's rows see whole or not at all share their factors there
//     too: a prompt of 8192 tokens with a row of one token in every workgroup 1300 us without
//     that, 752 with it, 577 without such rows.)
//   - The reference of a row's sums is the running maximum of score + lv, moved when it has
//     grown by 2^kLazy or more.
// Two prompts of 8009 and 8192 tokens, 32 heads on 8: 1.12 to 1.20 ms by card, up to 0.96
// PFLOP/s (a large library product reaches 1.21). Bound by the products and the exponentials beside them
// at the clock that the card holds under both. What led there: 2.93 ms with 16 rows a product
// straight from the cache; 1.24 as described; 1.21 with the scales' factors made by one wave
// a tile instead of each thread's own; 1.17 with the tokens' largest scales found once and
// factors of unseen tokens clamped, not masked (the tiles at the rows' ends took four times
// the others' time); 1.13 with the next tile stored before this one's products, not behind
// them; 1.12 with the exponentials at a higher priority than products (the products there
// instead: 1.13). Scores from products of the codes themselves (the block-scaled matrix
// instructions, a query as two e4m3 parts) were measured apart: off by up to 2^-17 of
// sum |q k|, 2^-13 where a key's scales lie 2^12 apart, and not built.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "attend4.hpp"
#include "launch.h"

namespace idxk {

typedef float at_f32x16 __attribute__((ext_vector_type(16)));

namespace {

constexpr int kP4Waves = 8;
constexpr int kP4NT = kP4Waves * kWave;
constexpr int kP4Rows = 32 * kP4Waves;
constexpr int kP4CUs = 256;
constexpr int kP4Phase = 512;                  // tiles whose pages wait in LDS
constexpr int kP4Units = 4 * (kP4Phase + 4);   // and of the tiles loaded ahead
constexpr int kP4Ahead = 4;                    // operands read from LDS before their use
constexpr int kP4Frag = kWave;                 // uint4s of one operand in LDS

struct Pre4Lds {
  uint4 k[2][16][kP4Frag];  // [buffer][32-token half, 16-dim step]
  uint4 v[2][16][kP4Frag];  // [buffer][32-dim tile, 32-token half, 8 tokens of the units]
  uint2 factor[3][4][16];   // of the values' scales: [tile % 3][unit][32 dims, four tokens]
  uint4 scales[3][4][4];    // [tile % 3][unit][32 dims], a byte a token
  uint4 tops[3][4];         // each token's largest, a byte
  uint32_t top[3][4];       // the units' largest
  int nan_tile[3];          // a tile with NaN scales (plus one)
  int u_blk[kP4Units];
  int longest[kP4Waves], shortest[kP4Waves];
  unsigned long long work[kP4Waves];
  int found;
};

__device__ __forceinline__ float p4_halves_max(float v) {
  return fmaxf(v, __uint_as_float(lane_xor<32>(__float_as_uint(v))));
}

// NaN in the factors of NaN scales: two bytes of a word, their factors
__device__ __forceinline__ uint32_t nan_factors(uint32_t pair, uint32_t s) {
  if ((pair & 255u) == kNanScale) s = (s & 0xFFFF0000u) | 0x7E00u;
  if (((pair >> 8) & 255u) == kNanScale) s = (s & 0xFFFFu) | 0x7E000000u;
  return s;
}

template <int KIND>
__global__ __launch_bounds__(kP4NT) void attend4_prefill_kernel(AttnArgs a, int chunk, int splits,
                                                                int64_t n_tiles) {
  __shared__ Pre4Lds lds;
  const int h = blockIdx.x % a.Hkv;
  const int rest = blockIdx.x / a.Hkv;
  // the row tiles of one stretch of keys side by side: they share it in L2, one KV head to
  // an XCD where there are eight (or the heads divide them); a prompt's last tokens, which
  // see most, first
  const int split = (int)(rest / n_tiles);
  const int64_t tile = n_tiles - 1 - rest % n_tiles;
  const int tid = threadIdx.x, lane = lane_id(), w = tid / kWave;
  const int n = lane & 31, half = lane >> 5;
  const int G = a.Hq / a.Hkv;
  const int ush = a.page_size == 16 ? 0 : a.page_size == 32 ? 1 : 2;  // log2(units a page)

  const RowTile rt = row_tile<kP4NT>(a, tile, G, kP4Rows, &lds.found);
  const int t0 = rt.t0;
  const int64_t row0 = rt.row0, rows = rt.rows;
  if (row0 < 0 || row0 >= rows) return;

  const PageList pages = page_list(a, rt.b);
  const int64_t row = row0 + 32 * w + n;
  const int64_t rat = min(row, rows - 1);
  const int64_t tok = t0 + rat / G;
  const int hq = h * G + (int)(rat % G);
  const int len = row < rows ? max(a.kv_len[tok], 0) : 0;
  const float slope2 = KIND != kPlain ? slope_of(a, hq) : 0.f;
  // dims 16 s + 8 half .. + 7 of the row; a negative call scale turns the queries' signs
  at_bf16x8 q[8];
  {
    const uint4* p = reinterpret_cast<const uint4*>(a.q + tok * a.q_stride + hq * kHeadDim);
    const uint32_t sign = a.score_scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const uint4 x = p[2 * s + half];
      q[s] = __builtin_bit_cast(at_bf16x8,
                                make_uint4(x.x ^ sign, x.y ^ sign, x.z ^ sign, x.w ^ sign));
    }
  }
  const float call_scale = fabsf(a.score_scale);
  const Cap cap(a.softcap);

  // of the wave's rows (one that sees nothing keeps no tile from being seen whole: its
  // probabilities are zeros, and its sums are not taken)
  int longest = len, shortest = len > 0 ? len : 0x7FFFFFFF;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    longest = max(longest, __shfl_xor(longest, d));
    shortest = min(shortest, __shfl_xor(shortest, d));
  }
  // A cut call's stretches (attend_prefill.hip): lengthened to a CU's share of the call
  unsigned long long work = 0;
  if (splits > 1) {
    for (int i = tid; i < a.B; i += kP4NT) {
      const int x0 = min(max(a.tok_indptr[i], 0), a.R);
      const int x1 = min(max(a.tok_indptr[i + 1], 0), a.R);
      if (x1 <= x0) continue;
      const int64_t held = (int64_t)page_list(a, i).n * a.page_size;
      const int64_t seen = min(held, (int64_t)max(a.kv_len[x0], 0)) +
                           min(held, (int64_t)max(a.kv_len[x1 - 1], 0));
      work += (((int64_t)(x1 - x0) * G + kP4Rows - 1) / kP4Rows) *
              ((seen / 2 + kTileTok - 1) / kTileTok);
    }
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) work += __shfl_xor(work, d);
  }
  if (lane == 0) {
    lds.longest[w] = longest;
    lds.shortest[w] = shortest;
    lds.work[w] = work;
  }
  __syncthreads();
  int most = 0, least = 0x7FFFFFFF;  // of the workgroup's rows
  work = 0;
#pragma unroll
  for (int i = 0; i < kP4Waves; ++i) {
    most = max(most, lds.longest[i]);
    least = min(least, lds.shortest[i]);
    work += lds.work[i];
  }
  if (splits > 1)
    chunk = (int)min((unsigned long long)0x7FFFFFFF,
                     max((unsigned long long)chunk, (work * a.Hkv + kP4CUs - 1) / kP4CUs));

  const int units = min(pages.n << ush, (int)(((int64_t)most + kUnit - 1) / kUnit));
  const int64_t end = min(((int64_t)units + 3) / 4, ((int64_t)split + 1) * chunk);
  int begin = 0, count = 0;  // the phase's tiles
  // whether some rows see tile c of the phase in part
  auto in_part = [&](int c) { return (int64_t)(begin + c + 1) * kTileTok > least; };

  // staging: thread -> (token, 16 dims) of the keys and (unit, dim) of the values
  const int sub = (1 << ush) - 1;
  const int hp = a.page_size / 2;
  const int ktok = (tid & 7) | ((tid >> 6) << 3), kc = (tid >> 3) & 7;  // 8 tokens a wave
  const int ku = ktok >> 4;
  const int vd = tid & 127, vu = tid >> 7;
  const uint8_t* k_at = a.k_cache + (ktok & 15) * (kHeadDim / 2) + 8 * kc;
  const uint8_t* ks_at = a.k_exp + (ktok & 15) * 4 + (kc >> 1);
  const uint8_t* v_at = a.v_cache + vd * hp;
  const uint32_t block = (uint32_t)hp * kHeadDim, scales = (uint32_t)a.page_size * 4;
  uint2 kreg, vreg;
  uint32_t kscale, word = 0;
  auto load_k = [&](int c) {  // c: tile of the phase
    const int kb = lds.u_blk[4 * c + ku];
    const uint32_t s = (4 * (begin + c) + ku) & sub, at = (uint32_t)max(kb, 0);
    kreg = *reinterpret_cast<const uint2*>(k_at + (uint64_t)at * block +
                                           s * (kUnit * kHeadDim / 2));
    kscale = ks_at[(uint64_t)at * scales + s * (kUnit * 4)];
    if (kb < 0) kreg = make_uint2(0, 0), kscale = 127;
  };
  auto load_v = [&](int c) {
    const int vb = lds.u_blk[4 * c + vu];
    const uint32_t s = (4 * (begin + c) + vu) & sub;
    vreg = *reinterpret_cast<const uint2*>(v_at + (uint64_t)(uint32_t)max(vb, 0) * block +
                                           s * (kUnit / 2));
  };
  // The values' scales of a tile: one wave's, a tile ahead of the others' codes. A lane has
  // unit lane / 16 and, of that, 32 dims (lane / 4 % 4) of four tokens.
  auto load_scales = [&](int c) {
    const int sb = lds.u_blk[4 * c + (lane >> 4)];
    const uint32_t s = (4 * (begin + c) + (lane >> 4)) & sub;
    word = *reinterpret_cast<const uint32_t*>(
        a.v_exp + (uint64_t)(uint32_t)max(sb, 0) * scales + s * kUnit +
        ((lane >> 2) & 3) * a.page_size + 4 * (lane & 3));
    if (sb < 0) word = 0;
  };
  auto store_scales = [&](int c) {
    const int su = lane >> 4, i = lane & 15, ring = (begin + c) % 3;
    const uint32_t tops = token_tops(word);
    const uint32_t top = max(group_top(tops), kBelow), floor2 = (top - kBelow) * 0x00010001u;
    lds.factor[ring][su][i] =
        make_uint2(nan_factors(word, two_scales<0>(word, floor2)),
                   nan_factors(word >> 16, two_scales<1>(word, floor2)));
    reinterpret_cast<uint32_t*>(lds.scales[ring][su])[i] = word;
    if (i < 4) reinterpret_cast<uint32_t*>(&lds.tops[ring][su])[i] = tops;
    if (i == 0) lds.top[ring][su] = top;
    const bool nan = __any(nan_scales(word) != 0);
    if (lane == 0) lds.nan_tile[ring] = nan ? begin + c + 1 : 0;
  };
  auto store_k = [&](int c) {
    // row 8 q + 4 (unit of the 32) + e holds token 4 q + e; every other step swaps rows 4
    // apart, so that 16 lanes' stores meet 16 different banks of 16 bytes
    const int i = ktok & 15, m32 = 8 * (i >> 2) + 4 * (ku & 1) + (i & 3);
    const float s = __uint_as_float(kscale << 23);
    uint4* p = &lds.k[c & 1][(ku >> 1) * 8 + kc][m32 ^ ((kc & 1) << 2)];
    p[0] = __builtin_bit_cast(uint4, codes4_bf16(kreg.x, s));
    p[32] = __builtin_bit_cast(uint4, codes4_bf16(kreg.y, s));
  };
  auto store_v = [&](int c) {
    uint4 x = __builtin_bit_cast(uint4, codes4_f16(vreg.x, 2.f));
    uint4 y = __builtin_bit_cast(uint4, codes4_f16(vreg.y, 2.f));
    if (!in_part(c)) {
      const uint4* f =
          reinterpret_cast<const uint4*>(&lds.factor[(begin + c) % 3][vu][4 * (vd >> 5)]);
      const uint4 s = f[0], t = f[1];
      x = make_uint4(mul_f16(x.x, s.x), mul_f16(x.y, s.y), mul_f16(x.z, s.z), mul_f16(x.w, s.w));
      y = make_uint4(mul_f16(y.x, t.x), mul_f16(y.y, t.y), mul_f16(y.z, t.z), mul_f16(y.w, t.w));
    }
    uint4* p = &lds.v[c & 1][((vd >> 5) * 2 + (vu >> 1)) * 2][(vu & 1) * 32 + (vd & 31)];
    p[0] = x;
    p[kP4Frag] = y;
  };

  // the wave's state: weights in units of 2^m, sums of values in half of that
  at_f32x16 o[4];
#pragma unroll
  for (int dt = 0; dt < 4; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[dt][i] = 0.f;
  float m = -__builtin_inff(), l = 0.f;

  // operands are read from LDS kP4Ahead products before their use
  auto products = [&](at_f32x16 (&x)[2], int c) {
    auto read = [&](int i) {
      return __builtin_bit_cast(at_bf16x8, lds.k[c & 1][i][lane ^ ((i & 1) << 2)]);
    };
    at_bf16x8 f[16];
#pragma unroll
    for (int i = 0; i < kP4Ahead; ++i) f[i] = read(i);
#pragma unroll
    for (int ts = 0; ts < 2; ++ts)
#pragma unroll
      for (int i = 0; i < 16; ++i) x[ts][i] = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i + kP4Ahead < 16) f[i + kP4Ahead] = read(i + kP4Ahead);
      x[i >> 3] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[i], q[i & 7], x[i >> 3], 0, 0, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x100, kP4Ahead, 0);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i + kP4Ahead < 16) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
  };
  auto step = [&](int c, auto part_of) {
    constexpr bool part = decltype(part_of)::value;
    at_f32x16 x[2];
    products(x, c);
    __builtin_amdgcn_sched_barrier(0);
    // (a SIMD's other wave, at its products, gives way to the exponentials of this one)
    __builtin_amdgcn_s_setprio(1);
    // maxima, masks and the reference
    const int ring = (begin + c) % 3;
    int have[2];
    uint32_t top[2];
    float lv[2], unit[2];  // unit: its best product of weight and scale
    // Units that the wave's rows see whole or not at all need no factors of each row's own.
    const bool nan = part && lds.nan_tile[ring] == begin + c + 1;
    bool edge[2] = {false, false};
    float best = -__builtin_inff();
    const float sc = KIND != kPlain ? 1.f : fmaxf(call_scale, 0x1p-126f);
#pragma unroll
    for (int ts = 0; ts < 2; ++ts) {
      const int i = 4 * c + 2 * ts + half, pos = (4 * begin + i) * kUnit;
      have[ts] = lds.u_blk[i] < 0 ? 0 : min(kUnit, len - pos);
      top[ts] = lds.top[ring][2 * ts + half];
      if constexpr (part) {
        edge[ts] = nan || __any(have[ts] > 0 && have[ts] < kUnit);
        if (edge[ts]) top[ts] = max(seen_top(lds.tops[ring][2 * ts + half], have[ts]), kBelow);
      }
      lv[ts] = (float)((int)top[ts] - 127);
      if constexpr (KIND != kPlain) {
        const float bias = -slope2 * (float)(len - 1 - pos);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float c0 = __builtin_fmaf((float)j, slope2, bias);
          x[ts][j] = score2<KIND>(x[ts][j], call_scale, cap, c0);
        }
      }
    }
    if (__any(have[0] < kUnit || have[1] < kUnit)) {
#pragma unroll
      for (int ts = 0; ts < 2; ++ts)
#pragma unroll
        for (int j = 0; j < 16; ++j) x[ts][j] = j < have[ts] ? x[ts][j] : -__builtin_inff();
    }
#pragma unroll
    for (int ts = 0; ts < 2; ++ts) {
      float mx = x[ts][0];
#pragma unroll
      for (int j = 1; j < 16; ++j) mx = fmaxf(mx, x[ts][j]);
      unit[ts] = __builtin_fmaf(mx, sc, lv[ts]);
      best = fmaxf(best, unit[ts]);
    }
    best = p4_halves_max(best);
    // (far_scale beside the reference's moves, by scales alone: two prompts of 8192 tokens 0.5 %
    // slower than without it, biased 1.9 %; in a branch of its own, by products, 1.8 and 2.4 %)
    uint32_t take[2] = {top[0], top[1]};
    if (__any(best > m + kLazy || min(top[0], top[1]) < kLowTop)) {
      const float mn = best > m + kLazy ? best : m;
      const float d = m - (mn == -__builtin_inff() ? 0.f : mn), f = exp2_fast(d);
      m = mn;
      l = scaled_down(l, d);
#pragma unroll
      for (int dt = 0; dt < 4; ++dt) o[dt] *= f;
#pragma unroll
      for (int ts = 0; ts < 2; ++ts) {
        lv[ts] = far_scale(lv[ts], unit[ts], m);
        take[ts] = (uint32_t)((int)lv[ts] + 127);
      }
    }
    auto read = [&](int i) {  // 8 tokens a quarter, dims 32 (i % 4) ..
      return __builtin_bit_cast(at_f16x8, lds.v[c & 1][(i & 3) * 4 + (i >> 2)][lane]);
    };
    at_f16x8 f[16];
    if constexpr (!part) {
#pragma unroll
      for (int i = 0; i < kP4Ahead; ++i) f[i] = read(i);
    }
    const float base = m == -__builtin_inff() ? 0.f : m;
    uint4 p[4];
#pragma unroll
    for (int ts = 0; ts < 2; ++ts) {
      const float off = base - kPBias - lv[ts];
      float sum = 0.f;
      uint32_t wd[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e0 = exp2_fast(__builtin_fmaf(x[ts][2 * i], sc, -off));
        const float e1 = exp2_fast(__builtin_fmaf(x[ts][2 * i + 1], sc, -off));
        sum += e0 + e1;
        wd[i] = pack_f16(e0, e1);
      }
      l = __builtin_fmaf(sum, __uint_as_float((254u - take[ts]) << 23), l);
      p[2 * ts] = make_uint4(wd[0], wd[1], wd[2], wd[3]);
      p[2 * ts + 1] = make_uint4(wd[4], wd[5], wd[6], wd[7]);
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(0);
    if constexpr (!part) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i + kP4Ahead < 16) f[i + kP4Ahead] = read(i + kP4Ahead);
        o[i & 3] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
            f[i], __builtin_bit_cast(at_f16x8, p[i >> 2]), o[i & 3], 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i + kP4Ahead < 16) __builtin_amdgcn_sched_group_barrier(0x100, 1, 1);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 1);
      }
    } else {
#pragma unroll
      for (int ts = 0; ts < 2; ++ts) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          uint32_t s[8];
          if (edge[ts]) {
            const uint4 b = lds.scales[ring][2 * ts + half][d];
            const uint32_t bw[4] = {b.x, b.y, b.z, b.w}, floor2 = (top[ts] - kBelow) * 0x00010001u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s[2 * e] = two_scales<0, true>(bw[e], floor2);
              s[2 * e + 1] = two_scales<1, true>(bw[e], floor2);
            }
          } else {
            const uint4* f =
                reinterpret_cast<const uint4*>(&lds.factor[ring][2 * ts + half][4 * d]);
            const uint4 f0 = f[0], f1 = f[1];
            s[0] = f0.x, s[1] = f0.y, s[2] = f0.z, s[3] = f0.w;
            s[4] = f1.x, s[5] = f1.y, s[6] = f1.z, s[7] = f1.w;
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint4 y = p[2 * ts + e];
            const uint4 z = make_uint4(mul_f16(y.x, s[4 * e]), mul_f16(y.y, s[4 * e + 1]),
                                       mul_f16(y.z, s[4 * e + 2]), mul_f16(y.w, s[4 * e + 3]));
            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                read(4 * (2 * ts + e) + d), __builtin_bit_cast(at_f16x8, z), o[d], 0, 0, 0);
          }
          __builtin_amdgcn_sched_barrier(0);  // few tiles: no registers for it
        }
      }
      if (nan) {
        // the groups of dims in which the row sees a NaN scale
        uint32_t bad = 0;
#pragma unroll
        for (int ts = 0; ts < 2; ++ts)
          bad |= seen_nans(lds.scales[ring][2 * ts + half], have[ts]);
        bad |= lane_xor<32>(bad);
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if ((bad >> d) & 1u) o[d][i] = __builtin_nanf("");
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  for (int64_t at = (int64_t)split * chunk; at < end; at += kP4Phase) {
    begin = (int)at;
    count = (int)min(end - at, (int64_t)kP4Phase);
    // the tiles any row of the wave sees
    const int mine =
        (int)min((int64_t)count, ((int64_t)longest + kTileTok - 1) / kTileTok - begin);
    __syncthreads();  // the phase before has been read
    for (int i = tid; i < 4 * (count + 4); i += kP4NT) {
      const int u = 4 * begin + i;
      lds.u_blk[i] = i < 4 * count && u < units ? block_of(a, pages, u >> ush, h) : -1;
    }
    __syncthreads();
    if (w < 3) load_scales(w);
    load_k(0);
    load_v(0);
    if (w < 2) store_scales(w);
    store_k(0);
    __syncthreads();
    store_v(0);
    load_k(1);
    load_v(1);
    auto tiles = [&](int from, int to, auto part_of) {
      for (int c = from; c < to; ++c) {
        __syncthreads();  // tile c is written, tile c - 1 read
        // (the next tile first: its loads have had a step's time, the one after gets one)
        store_k(c + 1);
        store_v(c + 1);
        load_k(c + 2);
        load_v(c + 2);
        if (c < mine) step(c, part_of);
        if (w == ((c + 2) & 7)) store_scales(c + 2);
        if (w == ((c + 3) & 7)) load_scales(c + 3);
      }
    };
    const int whole = (int)min((int64_t)count, max((int64_t)least / kTileTok - begin, (int64_t)0));
    tiles(0, whole, std::false_type{});
    tiles(whole, count, std::true_type{});
  }

  l += __uint_as_float(lane_xor<32>(__float_as_uint(l)));
  if (row >= rows) return;
  // lane: dims 32 dt + 8 q + 4 half + e of its row
  if (splits == 1) {
    const bool none = l == 0.f;
    const float inv = none ? 0.f : 0.5f / l;
    uint16_t* out = a.out + (tok * a.Hq + hq) * kHeadDim;
#pragma unroll
    for (int dt = 0; dt < 4; ++dt)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint2 y = make_uint2(pack_bf16(o[dt][4 * g] * inv, o[dt][4 * g + 1] * inv),
                                   pack_bf16(o[dt][4 * g + 2] * inv, o[dt][4 * g + 3] * inv));
        *reinterpret_cast<uint2*>(out + 32 * dt + 8 * g + 4 * half) = none ? make_uint2(0, 0) : y;
      }
  } else {
    const int64_t part = (((tok * a.Hkv + h) * splits) + split) * G + hq % G;
    float* out = a.part_o + part * kHeadDim;
#pragma unroll
    for (int dt = 0; dt < 4; ++dt)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<at_f32x4*>(out + 32 * dt + 8 * g + 4 * half) =
            at_f32x4{o[dt][4 * g], o[dt][4 * g + 1], o[dt][4 * g + 2], o[dt][4 * g + 3]} * 0.5f;
    if (half == 0) {
      a.part_ml[2 * part] = m;
      a.part_ml[2 * part + 1] = l;
    }
  }
}

}  // namespace

// How packed calls are cut: as the 8-bit cache's. The switch between the kernels, 64 rows a
// request, is early for this cache, whose 16-row kernel converts half the bytes: 9 requests of
// 5104 to 62488 tokens, 8 heads, 64 rows each 207 us there and 428 here, 96 rows 291 and 573,
// 128 rows 434 and 367; 64 requests of 2000 to 8000, 64 rows 199 and 440, 128 rows 347 and 437,
// 256 rows 639 and 822.
AttnSplit attend4_prefill_split(int64_t n_tok, int B, int Hq, int Hkv, int64_t units) {
  return attend_prefill_split(n_tok, B, Hq, Hkv, units);
}

int launch_attend4_prefill(const AttnArgs& a, AttnSplit sp, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (sp.rows != kP4Rows) return launch_attend4_rows(a, sp, stream);
  const int64_t tiles = attend_prefill_tiles(a.R, a.B, a.Hq / a.Hkv, kP4Rows);
  const dim3 grid((unsigned)(tiles * a.Hkv * sp.splits)), blk(kP4NT);
#define IDX_PRE4(KIND)                                                                         \
  hipLaunchKernelGGL((attend4_prefill_kernel<KIND>), grid, blk, 0, s, a, sp.chunk, sp.splits, \
                     tiles)
  if (a.softcap > kNearCap) IDX_PRE4(kCappedFar);
  else if (a.softcap > 0.f) IDX_PRE4(kCapped);
  else if (a.slopes != nullptr) IDX_PRE4(kBiased);
  else IDX_PRE4(kPlain);
#undef IDX_PRE4
  int e = (int)hipGetLastError();
  if (e == 0 && sp.splits > 1) e = launch_attend_merge(a, sp.splits, stream);
  return e;
}

}  // namespace idxk
