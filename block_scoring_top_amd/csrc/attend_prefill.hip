// Attention of packed prompt tokens over the paged 8-bit cache (include/idx_cache.h,
// idx_attend_prefill).
//
// A workgroup owns kPreRows rows (token, head of the KV head's group) of one request,
// 32 to a wave, and walks its tokens in tiles of 64.
//   - The tile's codes are converted once for the workgroup, on their way into LDS:
//     keys to bf16, values to fp16 (both exact), in the order in which the waves read
//     them as operands: 1 KB a product, 16 bytes a lane, free of bank conflicts. Two
//     buffers: a tile's loads are in flight while the one before it is computed.
//   - v_mfma_f32_32x32x16 with keys as A and queries as B: a lane holds one query row
//     and, of each 32 tokens, the 16 of one unit (row 8 q + 4 half + e of the product is
//     given token 4 q + e of unit `half`), so that the row's maximum takes one lane
//     swap, page scales are one number a lane, and the probabilities are the second
//     product's B operand as they stand.
//   - Scores stay unscaled: maxima are taken per unit and then scaled, and the page's
//     key scale, the row's maximum and the logarithm of the value scale enter with the
//     exponential's argument, one multiply-add a score. The sum of weights takes the
//     value scale back out, once a unit.
//   - The reference of a row is moved only when its maximum has grown by 2^kLazy or
//     more (sums are rescaled then); until that, probabilities reach up to 2^kLazy
//     times 2^kPBias, which fp16 holds.
// Two prompts of 8009 and 8192 tokens, 32 heads on 8: 1.15 ms, 0.93 PFLOP/s (a large
// library product reaches 1.21 on this card); 3.76 ms with 16 rows a product straight from
// the cache. Bound by the products and the exponentials beside them at the clock the card
// holds under them, about 2.05 GHz: running the two halves of the waves half a tile apart
// took 6 to 12 % fewer cycles (4464 against 5079 a tile) at a clock 10 % lower, the same
// time, and is not done; nor are four waves a workgroup (1.20 ms) or 128 rows straight
// from registers.
#include <hip/hip_runtime.h>

#include "attend.hpp"
#include "launch.h"

namespace idxk {

typedef float at_f32x16 __attribute__((ext_vector_type(16)));

namespace {

constexpr int kPreWaves = 8;
constexpr int kPreNT = kPreWaves * kWave;
constexpr int kPreRows = 32 * kPreWaves;
constexpr int kPackedMean = 64;               // rows a request, up to which they are few
constexpr int kCUs = 256;
constexpr int kPhase = 512;                   // tiles whose page data wait in LDS
constexpr int kPreUnits = 4 * (kPhase + 4);   // and for the tiles loaded ahead
static_assert(kPhase <= kPreNT, "a thread for each tile of a phase");
constexpr int kAhead = 4;                     // operands read from LDS before their use
constexpr int kFrag = kWave;                  // uint4s of one operand in LDS

struct PreLds {
  uint4 k[2][16][kFrag];  // [buffer][32-token half, 16-dim step]
  uint4 v[2][16][kFrag];  // [buffer][32-dim tile, 32-token half, 8 tokens of the units]
  int u_blk[kPreUnits];
  float u_ks[kPreUnits], u_lv[kPreUnits];
  float u_vmax[4 * kPhase];  // largest value scale of the phase's units up to each
  float red[kPreWaves];
  int longest[kPreWaves], shortest[kPreWaves];
  unsigned long long work[kPreWaves];
  // NaN value codes of a tile that some rows see only in part: which tile (plus one),
  // and for each dim and unit which of its 16 tokens
  int nan_tile[2];
  alignas(8) uint16_t nan_map[2][kHeadDim][4];
  int found;
};

__device__ __forceinline__ float halves_max(float v) {
  return fmaxf(v, __uint_as_float(lane_xor<32>(__float_as_uint(v))));
}

template <int KIND>
__global__ __launch_bounds__(kPreNT) void attend_prefill_kernel(AttnArgs a, int chunk,
                                                                int splits, int64_t n_tiles) {
  __shared__ PreLds lds;
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

  const RowTile rt = row_tile<kPreNT>(a, tile, G, kPreRows, &lds.found);
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
  // dims 16 s + 8 half .. + 7 of the row; a negative call scale turns the queries'
  // signs, so that scores keep their order under the (positive) scale of a unit
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

  int longest = len, shortest = row < rows ? len : 0x7FFFFFFF;  // of the wave's rows
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    longest = max(longest, __shfl_xor(longest, d));
    shortest = min(shortest, __shfl_xor(shortest, d));
  }
  // A cut call's stretches: the host knows only a bound of the lengths and cuts for that;
  // where the lengths give less than a stretch to each CU of that size, longer ones, equal
  // to a CU's share of the call, end together (and leave fewer partial sums). The work is
  // the requests' row tiles times the mean of their first and last row's tiles.
  unsigned long long work = 0;
  if (splits > 1) {
    for (int i = tid; i < a.B; i += kPreNT) {
      const int x0 = min(max(a.tok_indptr[i], 0), a.R);
      const int x1 = min(max(a.tok_indptr[i + 1], 0), a.R);
      if (x1 <= x0) continue;
      const int64_t held = (int64_t)page_list(a, i).n * a.page_size;
      const int64_t seen = min(held, (int64_t)max(a.kv_len[x0], 0)) +
                           min(held, (int64_t)max(a.kv_len[x1 - 1], 0));
      work += (((int64_t)(x1 - x0) * G + kPreRows - 1) / kPreRows) *
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
  for (int i = 0; i < kPreWaves; ++i) {
    most = max(most, lds.longest[i]);
    least = min(least, lds.shortest[i]);
    work += lds.work[i];
  }
  if (splits > 1)
    chunk = (int)min((unsigned long long)0x7FFFFFFF,
                     max((unsigned long long)chunk, (work * a.Hkv + kCUs - 1) / kCUs));

  const int units = min(pages.n << ush, (int)(((int64_t)most + kUnit - 1) / kUnit));
  const int64_t end = min(((int64_t)units + 3) / 4, ((int64_t)split + 1) * chunk);
  int begin = 0, count = 0;  // the phase's tiles

  // staging: thread -> (token, 16 dims) of the keys and (unit, dim) of the values
  const int64_t block = (int64_t)a.page_size * kHeadDim;
  const int sub = (1 << ush) - 1;
  const int ktok = (tid & 7) | ((tid >> 6) << 3), kc = (tid >> 3) & 7;  // 8 tokens a wave
  const int ku = ktok >> 4;
  const int vd = tid & 127, vu = tid >> 7;
  uint4 kreg, vreg;
  int vhave = 0;  // visible tokens of this thread's value unit
  bool kval = false;
  auto load_k = [&](int c) {  // c: tile of the phase
    const int kb = lds.u_blk[4 * c + ku];
    kval = kb >= 0;
    kreg = *reinterpret_cast<const uint4*>(
        a.k_cache + max(kb, 0) * block +
        ((((4 * (begin + c) + ku) & sub) * kUnit + (ktok & 15)) * kHeadDim + 16 * kc));
  };
  auto load_v = [&](int c) {
    const int vb = lds.u_blk[4 * c + vu], u = 4 * (begin + c) + vu;
    vhave = vb < 0 ? 0 : min(kUnit, most - u * kUnit);
    vreg = *reinterpret_cast<const uint4*>(a.v_cache + max(vb, 0) * block +
                                           (vd * a.page_size + (u & sub) * kUnit));
  };
  auto store_k = [&](int c) {
    // row 8 q + 4 (unit of the 32) + e holds token 4 q + e; every other step swaps rows 4
    // apart, so that 16 lanes' stores meet 16 different banks of 16 bytes
    const int i = ktok & 15, m32 = 8 * (i >> 2) + 4 * (ku & 1) + (i & 3);
    const uint4 x = kval ? kreg : make_uint4(0, 0, 0, 0);
    uint4* p = &lds.k[c & 1][(ku >> 1) * 8 + kc][m32 ^ ((kc & 1) << 2)];
    p[0] = __builtin_bit_cast(uint4, codes_bf16x8(x.x, x.y));
    p[32] = __builtin_bit_cast(uint4, codes_bf16x8(x.z, x.w));
  };
  auto store_v = [&](int c) {
    uint4 x = vhave == kUnit ? vreg : keep_tokens(vreg, vhave);
    if ((int64_t)(begin + c + 1) * kTileTok > least) {
      // A NaN value must reach the rows that see its token and no others, but all rows
      // share the product, where 0 x NaN is NaN: zero here, and noted.
      uint32_t word[4] = {x.x, x.y, x.z, x.w}, mask = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t bad = nan_codes(word[e]) >> 7;  // 1 in each NaN byte
        word[e] &= ~(bad * 0xFFu);
        // the four flags (bits 0, 8, 16, 24) side by side
        mask |= ((bad * 0x10204080u) >> 28) << (4 * e);
      }
      x = make_uint4(word[0], word[1], word[2], word[3]);
      lds.nan_map[c & 1][vd][vu] = (uint16_t)mask;
      if (mask != 0) lds.nan_tile[c & 1] = c + 1;
    }
    uint4* p = &lds.v[c & 1][((vd >> 5) * 2 + (vu >> 1)) * 2][(vu & 1) * 32 + (vd & 31)];
    p[0] = __builtin_bit_cast(uint4, codes_f16x8(x.x, x.y));
    p[kFrag] = __builtin_bit_cast(uint4, codes_f16x8(x.z, x.w));
  };

  // the wave's state
  at_f32x16 o[4];
#pragma unroll
  for (int dt = 0; dt < 4; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[dt][i] = 0.f;
  float m = -__builtin_inff(), l = 0.f;
  // the largest value scale of the units the row sees, up to the phase's end, and its
  // logarithm: o is in its units
  float vref = 0.f, lref = 0.f;
  float ksc[2], lv[2];  // scales of the tile

  // operands are read from LDS kAhead products before their use
  auto products = [&](at_f32x16 (&x)[2], int c) {
    auto read = [&](int i) {
      return __builtin_bit_cast(at_bf16x8, lds.k[c & 1][i][lane ^ ((i & 1) << 2)]);
    };
    at_bf16x8 f[16];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) f[i] = read(i);
#pragma unroll
    for (int ts = 0; ts < 2; ++ts)
#pragma unroll
      for (int i = 0; i < 16; ++i) x[ts][i] = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i + kAhead < 16) f[i + kAhead] = read(i + kAhead);
      x[i >> 3] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[i], q[i & 7], x[i >> 3], 0, 0, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i + kAhead < 16) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
  };
  // maxima, masks and the reference of tile c, whose products are in x
  auto reference = [&](at_f32x16 (&x)[2], int c) {
    int have[2];
    float top = -__builtin_inff();
#pragma unroll
    for (int ts = 0; ts < 2; ++ts) {
      const int i = 4 * c + 2 * ts + half, pos = (4 * begin + i) * kUnit;
      ksc[ts] = lds.u_ks[i];
      // (2^-60 below the reference fp16 holds nothing; nor does a unit without tokens)
      lv[ts] = fmaxf(lds.u_lv[i] - lref, -60.f);
      have[ts] = lds.u_blk[i] < 0 ? 0 : min(kUnit, len - pos);
      if constexpr (KIND != kPlain) {
        const float bias = -slope2 * (float)(len - 1 - pos);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float c0 = __builtin_fmaf((float)j, slope2, bias);
          x[ts][j] = score2<KIND>(x[ts][j], ksc[ts], cap, c0);
        }
        ksc[ts] = 1.f;
      }
      float mx = x[ts][0];
#pragma unroll
      for (int j = 1; j < 16; ++j) mx = fmaxf(mx, x[ts][j]);
      top = fmaxf(top, mx * ksc[ts]);
    }
    if (__any(have[0] < kUnit || have[1] < kUnit)) {
      top = -__builtin_inff();
#pragma unroll
      for (int ts = 0; ts < 2; ++ts) {
        // not 0, which would make NaN of the masked scores of a unit without tokens
        ksc[ts] = fmaxf(ksc[ts], 0x1p-126f);
        float mx = -__builtin_inff();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          x[ts][j] = j < have[ts] ? x[ts][j] : -__builtin_inff();
          mx = fmaxf(mx, x[ts][j]);
        }
        top = fmaxf(top, mx * ksc[ts]);
      }
    }
    top = halves_max(top);
    if (__any(top > m + kLazy)) {
      const float mn = top > m + kLazy ? top : m;
      const float f = exp2_fast(m - (mn == -__builtin_inff() ? 0.f : mn));
      m = mn;
      l *= f;
#pragma unroll
      for (int dt = 0; dt < 4; ++dt) o[dt] *= f;
    }
  };
  auto step = [&](int c) {
    at_f32x16 x[2];
    products(x, c);
    __builtin_amdgcn_sched_barrier(0);
    reference(x, c);
    auto read = [&](int i) {  // 8 tokens a quarter, dims 32 (i % 4) ..
      return __builtin_bit_cast(at_f16x8, lds.v[c & 1][(i & 3) * 4 + (i >> 2)][lane]);
    };
    at_f16x8 f[16];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) f[i] = read(i);
    const float base = m == -__builtin_inff() ? 0.f : m;
    uint4 p[4];
#pragma unroll
    for (int ts = 0; ts < 2; ++ts) {
      const float off = base - kPBias - lv[ts];
      float sum = 0.f;
      uint32_t wd[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e0 = exp2_fast(__builtin_fmaf(x[ts][2 * i], ksc[ts], -off));
        const float e1 = exp2_fast(__builtin_fmaf(x[ts][2 * i + 1], ksc[ts], -off));
        sum += e0 + e1;
        wd[i] = pack_f16(e0, e1);
      }
      l = __builtin_fmaf(sum, exp2_fast(-lv[ts]), l);
      p[2 * ts] = make_uint4(wd[0], wd[1], wd[2], wd[3]);
      p[2 * ts + 1] = make_uint4(wd[4], wd[5], wd[6], wd[7]);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i + kAhead < 16) f[i + kAhead] = read(i + kAhead);
      o[i & 3] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
          f[i], __builtin_bit_cast(at_f16x8, p[i >> 2]), o[i & 3], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i + kAhead < 16) __builtin_amdgcn_sched_group_barrier(0x100, 1, 1);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 1);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (lds.nan_tile[c & 1] == c + 1) {
      const int seen = min(max(len - (begin + c) * kTileTok, 0), kTileTok);
      const uint64_t sees = seen == kTileTok ? ~0ull : (1ull << seen) - 1;
#pragma unroll
      for (int dt = 0; dt < 4; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int d = 32 * dt + 8 * (i >> 2) + 4 * half + (i & 3);
          const uint64_t bad = *reinterpret_cast<const uint64_t*>(lds.nan_map[c & 1][d]);
          if ((bad & sees) != 0) o[dt][i] = __builtin_nanf("");
          __builtin_amdgcn_sched_barrier(0);  // a rare path: no registers for it
        }
    }
  };

  for (int64_t at = (int64_t)split * chunk; at < end; at += kPhase) {
    begin = (int)at;
    count = (int)min(end - at, (int64_t)kPhase);
    // the tiles any row of the wave sees
    const int mine =
        (int)min((int64_t)count, ((int64_t)longest + kTileTok - 1) / kTileTok - begin);
    __syncthreads();  // the phase before has been read
    if (tid < 2) lds.nan_tile[tid] = 0;
    for (int i = tid; i < 4 * (count + 4); i += kPreNT) {
      const int u = 4 * begin + i;
      const int blk = i < 4 * count && u < units ? block_of(a, pages, u >> ush, h) : -1;
      lds.u_blk[i] = blk;
      lds.u_ks[i] = blk < 0 ? 0.f : a.k_scale[blk] * call_scale;
      lds.u_lv[i] = blk < 0 ? 0.f : a.v_scale[blk];
    }
    __syncthreads();
    // The largest value scale up to each unit: a thread for each tile, whose four are
    // joined to those of the threads and waves before.
    float up[4], before = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      before = fmaxf(before, tid < count ? lds.u_lv[4 * tid + i] : 0.f);
      up[i] = before;
    }
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
      const float left = __shfl_up(before, d);
      if (lane >= d) before = fmaxf(before, left);
    }
    if (lane == kWave - 1) lds.red[w] = before;
    before = __shfl_up(before, 1);
    if (lane == 0) before = 0.f;
    __syncthreads();
    for (int i = 0; i < w; ++i) before = fmaxf(before, lds.red[i]);
    if (tid < count) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lds.u_vmax[4 * tid + i] = fmaxf(before, up[i]);
        lds.u_lv[4 * tid + i] = __log2f(lds.u_lv[4 * tid + i]);  // (no tokens: -infinity)
      }
    }
    __syncthreads();
    const int64_t seen = min(((int64_t)len + kUnit - 1) / kUnit - 4 * (int64_t)begin,
                             4 * (int64_t)count);
    const float vmax = seen > 0 ? lds.u_vmax[seen - 1] : 0.f;
    if (vmax > vref) {
      const float f = vref / vmax;
#pragma unroll
      for (int dt = 0; dt < 4; ++dt) o[dt] *= f;
      vref = vmax;
      lref = __log2f(vmax);
    }
    load_k(0);
    load_v(0);
    store_k(0);
    store_v(0);
    load_k(1);
    load_v(1);
    for (int c = 0; c < count; ++c) {
      __syncthreads();  // tile c is written, tile c - 1 read
      if (c < mine) step(c);
      store_k(c + 1);
      store_v(c + 1);
      load_k(c + 2);
      load_v(c + 2);
    }
  }

  l += __uint_as_float(lane_xor<32>(__float_as_uint(l)));
  if (row >= rows) return;
  // lane: dims 32 dt + 8 q + 4 half + e of its row
  if (splits == 1) {
    // (vref / l would lose its bits below fp32's normal range)
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t* out = a.out + (tok * a.Hq + hq) * kHeadDim;
#pragma unroll
    for (int dt = 0; dt < 4; ++dt)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = o[dt][4 * g + e] * inv * vref;
        *reinterpret_cast<uint2*>(out + 32 * dt + 8 * g + 4 * half) =
            make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
      }
  } else {
    const int64_t part = (((tok * a.Hkv + h) * splits) + split) * G + hq % G;
    float* out = a.part_o + part * kHeadDim;
#pragma unroll
    for (int dt = 0; dt < 4; ++dt)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<at_f32x4*>(out + 32 * dt + 8 * g + 4 * half) =
            at_f32x4{o[dt][4 * g], o[dt][4 * g + 1], o[dt][4 * g + 2], o[dt][4 * g + 3]} * vref;
    if (half == 0) {
      a.part_ml[2 * part] = m;
      a.part_ml[2 * part + 1] = l;
    }
  }
}

}  // namespace

int64_t attend_prefill_tiles(int64_t n_tok, int B, int G, int per) { return n_tok * G / per + B; }

// A call of fewer than two workgroups a CU is cut along its keys, into at most so many
// stretches as give about 512 workgroups of no less than 32 tiles; one of fewer workgroups
// than CUs down to four tiles (five tokens on 900 to 2777: 29 us at eight, 22 so). A
// workgroup's start and end cost four tiles' time, and its partial sums are written and
// read again (the two prompts of 8192, 2032 workgroups: 1.14 ms whole, 1.42 in two). The
// kernel lengthens the stretches to a CU's share of the call: chunks of 512 tokens on 4608
// and 30512, 32 heads on 8, 492 us before that and 418 so, 433 at 1024 wanted.
AttnSplit attend_prefill_split(int64_t n_tok, int B, int Hq, int Hkv, int64_t units) {
  const int G = Hq / Hkv;
  const int64_t tiles = (units + 3) / 4;
  // Few rows a request (drafted tokens): the kernel of single tokens, whose waves share out
  // the keys of 16 rows instead of the rows. 9 requests of 5104 to 62488 tokens, 8 heads:
  // 28 rows each 212 us against 417 here, 56 rows 295 against 464, 120 rows 525 against
  // 365; 64 requests of 2000 to 8000, 72 rows: 340 against 369.
  if (n_tok * G <= (int64_t)kPackedMean * B) {
    AttnSplit sp = attend_rows_split(attend_prefill_tiles(n_tok, B, G, 16), Hkv, units);
    sp.rows = 16;
    return sp;
  }
  const int64_t groups = attend_prefill_tiles(n_tok, B, G, kPreRows) * Hkv;
  auto most = [&](int64_t want, int64_t least) {
    const int64_t s = (want + groups - 1) / groups, t = tiles / least;
    return s < t ? s : t;
  };
  int64_t splits = 1;
  if (most(256, 4) > splits) splits = most(256, 4);
  if (most(512, 32) > splits) splits = most(512, 32);
  const int64_t chunk = (tiles + splits - 1) / splits;
  return {(int)chunk, (int)((tiles + chunk - 1) / chunk), kPreRows};
}

int launch_attend_prefill(const AttnArgs& a, AttnSplit sp, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (sp.rows != kPreRows) return launch_attend_rows(a, sp, stream);
  const int64_t tiles = attend_prefill_tiles(a.R, a.B, a.Hq / a.Hkv, kPreRows);
  const dim3 grid((unsigned)(tiles * a.Hkv * sp.splits)), blk(kPreNT);
#define IDX_PRE(KIND)                                                                         \
  hipLaunchKernelGGL((attend_prefill_kernel<KIND>), grid, blk, 0, s, a, sp.chunk, sp.splits, \
                     tiles)
  if (a.softcap > kNearCap) IDX_PRE(kCappedFar);
  else if (a.softcap > 0.f) IDX_PRE(kCapped);
  else if (a.slopes != nullptr) IDX_PRE(kBiased);
  else IDX_PRE(kPlain);
#undef IDX_PRE
  int e = (int)hipGetLastError();
  if (e == 0 && sp.splits > 1) e = launch_attend_merge(a, sp.splits, stream);
  return e;
}

}  // namespace idxk
