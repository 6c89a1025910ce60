// Attention of packed prompt tokens over the paged 8-bit cache (include/idx_cache.h,
// idx_attend_prefill).
//
// A workgroup owns kPreRows rows (token, head of the KV head's group) of one request,
// 32 to a wave, and walks its tokens in tiles of 64. Bound by the matrix products
// (512 operations a row and token pair of sums) and the softmax beside them.
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
//     times 2^kPreBias, which fp16 holds.
#include <hip/hip_runtime.h>

#include "attend.hpp"
#include "launch.h"

namespace idxk {

typedef float at_f32x16 __attribute__((ext_vector_type(16)));

namespace {

constexpr int kPreWaves = 8;
constexpr int kPreNT = kPreWaves * kWave;
constexpr int kPreRows = 32 * kPreWaves;
constexpr int kPhaseTiles = 64;               // tiles whose page data wait in LDS
constexpr int kPhaseUnits = 4 * kPhaseTiles;
constexpr float kPreBias = 9.f;
constexpr float kLazy = 6.f;
// what happens to a score beside its scale; capped ones may be biased too
constexpr int kPlain = 0, kBiased = 1, kCapped = 2;
constexpr int kFrag = kWave;                  // uint4s of one operand in LDS

struct PreLds {
  uint4 k[2][16][kFrag];  // [buffer][32-token half, 16-dim step]
  uint4 v[2][16][kFrag];  // [buffer][32-dim tile, 32-token half, 8 tokens of the units]
  int u_blk[kPhaseUnits];
  float u_ks[kPhaseUnits], u_lv[kPhaseUnits];
  float red[kPreWaves];
  int longest[kPreWaves], shortest[kPreWaves];
  // NaN value codes of a tile that some rows see only in part: which tile (plus one),
  // and for each dim and unit which of its 16 tokens
  int nan_tile[2];
  uint16_t nan_map[2][kHeadDim][4];
};

// First workgroup of request b: tiles never span requests, and
// floor(y / T) - floor(x / T) + 1 tiles hold any x..y rows.
__device__ __forceinline__ int64_t first_tile(const AttnArgs& a, int b, int G) {
  const int64_t p = min(max(a.tok_indptr[b], 0), a.R);
  return p * G / kPreRows + b;
}

__device__ __forceinline__ float halves_max(float v) {
  return fmaxf(v, __uint_as_float(lane_xor<32>(__float_as_uint(v))));
}

template <int KIND>
__global__ __launch_bounds__(kPreNT) void attend_prefill_kernel(AttnArgs a, int chunk,
                                                                int splits, int64_t n_tiles) {
  __shared__ PreLds lds;
  const int h = blockIdx.x % a.Hkv;
  const int rest = blockIdx.x / a.Hkv;
  const int split = rest % splits;
  const int64_t tile = n_tiles - 1 - rest / splits;  // a prompt's last tokens see most
  const int tid = threadIdx.x, lane = lane_id(), w = tid / kWave;
  const int n = lane & 31, half = lane >> 5;
  const int G = a.Hq / a.Hkv;
  const int ush = a.page_size == 16 ? 0 : a.page_size == 32 ? 1 : 2;  // log2(units a page)

  // the tile's request: the last b with first_tile(b) <= tile
  int b = 0;
  for (int lo = 0, hi = a.B; lo < hi;) {
    const int mid = (lo + hi) / 2;
    if (first_tile(a, mid, G) <= tile) {
      b = mid;
      lo = mid + 1;
    } else {
      hi = mid;
    }
  }
  const int t0 = min(max(a.tok_indptr[b], 0), a.R);
  const int t1 = min(max(a.tok_indptr[b + 1], 0), a.R);
  const int64_t row0 = (tile - first_tile(a, b, G)) * kPreRows;
  const int64_t rows = (int64_t)(t1 - t0) * G;
  if (row0 < 0 || row0 >= rows) return;

  const PageList pages = page_list(a, b);
  const int64_t row = row0 + 32 * w + n;
  const int64_t rat = min(row, rows - 1);
  const int64_t tok = t0 + rat / G;
  const int hq = h * G + (int)(rat % G);
  const int len = max(a.kv_len[tok], 0);
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

  int longest = len, shortest = len;  // of the wave's rows
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    longest = max(longest, __shfl_xor(longest, d));
    shortest = min(shortest, __shfl_xor(shortest, d));
  }
  if (lane == 0) {
    lds.longest[w] = longest;
    lds.shortest[w] = shortest;
  }
  if (tid < 2) lds.nan_tile[tid] = 0;
  __syncthreads();
  int most = 0, least = 0x7FFFFFFF;  // of the workgroup's rows
#pragma unroll
  for (int i = 0; i < kPreWaves; ++i) {
    most = max(most, lds.longest[i]);
    least = min(least, lds.shortest[i]);
  }

  at_f32x16 o[4];
#pragma unroll
  for (int dt = 0; dt < 4; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[dt][i] = 0.f;
  float m = -__builtin_inff(), l = 0.f, vref = 0.f;

  const int units = min(pages.n << ush, (int)(((int64_t)most + kUnit - 1) / kUnit));
  const int begin = split * chunk;
  const int end = min((units + 3) / 4, begin + chunk);

  // staging: thread -> (token, 16 dims) of the keys and (unit, dim) of the values
  const int64_t block = (int64_t)a.page_size * kHeadDim;
  const int sub = (1 << ush) - 1;
  const int ktok = (tid & 7) | ((tid >> 6) << 3), kc = (tid >> 3) & 7;  // 8 tokens a wave
  const int ku = ktok >> 4;
  const int vd = tid & 127, vu = tid >> 7;
  uint4 kreg, vreg;
  int vhave = 0;  // visible tokens of this thread's value unit
  bool kval = false;
  auto load = [&](int t, int phase) {
    const int i = (t - phase) * 4;
    const int kb = lds.u_blk[i + ku], vb = lds.u_blk[i + vu];
    kval = kb >= 0;
    vhave = vb < 0 ? 0 : min(kUnit, most - (4 * t + vu) * kUnit);
    kreg = *reinterpret_cast<const uint4*>(
        a.k_cache + max(kb, 0) * block +
        ((((4 * t + ku) & sub) * kUnit + (ktok & 15)) * kHeadDim + 16 * kc));
    vreg = *reinterpret_cast<const uint4*>(
        a.v_cache + max(vb, 0) * block + (vd * a.page_size + ((4 * t + vu) & sub) * kUnit));
  };
  auto store = [&](int buf, int t) {
    // keys: row 8 q + 4 (unit of the 32) + e holds token 4 q + e
    const int i = ktok & 15, m32 = 8 * (i >> 2) + 4 * (ku & 1) + (i & 3);
    const uint4 kx = kval ? kreg : make_uint4(0, 0, 0, 0);
    // every other step swaps rows 4 apart, so that 16 lanes' stores meet 16 banks of 16
    uint4* kp = &lds.k[buf][(ku >> 1) * 8 + kc][m32 ^ ((kc & 1) << 2)];
    kp[0] = __builtin_bit_cast(uint4, codes_bf16x8(kx.x, kx.y));
    kp[32] = __builtin_bit_cast(uint4, codes_bf16x8(kx.z, kx.w));
    uint4 vx = vhave == kUnit ? vreg : keep_tokens(vreg, vhave);
    if ((int64_t)(t + 1) * kTileTok > least) {
      // A NaN value must reach the rows that see its token and no others, but all rows
      // share the product, where 0 x NaN is NaN: zero here, and noted.
      uint32_t word[4] = {vx.x, vx.y, vx.z, vx.w}, mask = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t bad = nan_codes(word[e]) >> 7;  // 1 in each NaN byte
        word[e] &= ~(bad * 0xFFu);
        // the four flags (bits 0, 8, 16, 24) side by side
        mask |= ((bad * 0x10204080u) >> 28) << (4 * e);
      }
      vx = make_uint4(word[0], word[1], word[2], word[3]);
      lds.nan_map[buf][vd][vu] = (uint16_t)mask;
      if (mask != 0) lds.nan_tile[buf] = t + 1;
    }
    uint4* vp = &lds.v[buf][((vd >> 5) * 2 + (vu >> 1)) * 2][(vu & 1) * 32 + (vd & 31)];
    vp[0] = __builtin_bit_cast(uint4, codes_f16x8(vx.x, vx.y));
    vp[kFrag] = __builtin_bit_cast(uint4, codes_f16x8(vx.z, vx.w));
  };

  for (int phase = begin; phase < end; phase += kPhaseTiles) {
    // page data of the next tiles, and the largest value scale so far
    const int count = min(kPhaseTiles, end - phase);
    __syncthreads();  // the previous phase has been read
    float vmax = 0.f, vs = 0.f;
    if (tid < kPhaseUnits) {
      const int u = 4 * phase + tid;
      const int blk =
          tid < 4 * count && u < units ? block_of(a, pages, u >> ush, h) : -1;
      lds.u_blk[tid] = blk;
      lds.u_ks[tid] = blk < 0 ? 0.f : a.k_scale[blk] * call_scale;
      vs = blk < 0 ? 0.f : a.v_scale[blk];
      vmax = halves_max(vs);
#pragma unroll
      for (int d = 1; d < 32; d *= 2) vmax = fmaxf(vmax, __shfl_xor(vmax, d));
      if (lane == 0) lds.red[w] = vmax;
    }
    __syncthreads();
    float vtop = vref;
#pragma unroll
    for (int i = 0; i < kPhaseUnits / kWave; ++i) vtop = fmaxf(vtop, lds.red[i]);
    if (vtop > vref) {
      const float f = vref / vtop;
#pragma unroll
      for (int dt = 0; dt < 4; ++dt) o[dt] *= f;
      vref = vtop;
    }
    // value scales below 2^-60 of the largest: fp16 holds nothing of them
    if (tid < kPhaseUnits) lds.u_lv[tid] = vs == vtop ? 0.f : fmaxf(__log2f(vs / vtop), -60.f);
    load(phase, phase);
    store(0, phase);
    if (count > 1) load(phase + 1, phase);

    for (int c = 0; c < count; ++c) {
      const int buf = c & 1;
      __syncthreads();  // buffer `buf` is written, the other one read
      const int t = phase + c;
      if (t * kTileTok < longest) {  // (a tile starts below 2^31 - 64)
        at_f32x16 x[2];
#pragma unroll
        for (int ts = 0; ts < 2; ++ts) {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[ts][i] = 0.f;
#pragma unroll
          for (int s = 0; s < 8; ++s)
            x[ts] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                __builtin_bit_cast(at_bf16x8, lds.k[buf][ts * 8 + s][lane ^ ((s & 1) << 2)]), q[s],
                x[ts], 0, 0, 0);
        }
        float ksc[2], lv[2], bias[2];
        int have[2];
#pragma unroll
        for (int ts = 0; ts < 2; ++ts) {
          const int i = 4 * c + 2 * ts + half, pos = (4 * t + 2 * ts + half) * kUnit;
          ksc[ts] = lds.u_ks[i];
          lv[ts] = lds.u_lv[i];
          have[ts] = lds.u_blk[i] < 0 ? 0 : min(kUnit, len - pos);
          if constexpr (KIND != kPlain) bias[ts] = -slope2 * (float)(len - 1 - pos);
        }
        const bool whole = have[0] == kUnit && have[1] == kUnit;
        const bool any = !__all(whole);
        float top = -__builtin_inff();
#pragma unroll
        for (int ts = 0; ts < 2; ++ts) {
          if constexpr (KIND != kPlain) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float c0 = __builtin_fmaf((float)i, slope2, bias[ts]);
              x[ts][i] = KIND == kCapped ? capped(x[ts][i] * ksc[ts], a.softcap) + c0
                                         : __builtin_fmaf(x[ts][i], ksc[ts], c0);
            }
          }
          if (any) {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[ts][i] = i < have[ts] ? x[ts][i] : -__builtin_inff();
          }
          float mx = x[ts][0];
#pragma unroll
          for (int i = 1; i < 16; ++i) mx = fmaxf(mx, x[ts][i]);
          // a unit without tokens has scale 0: -inf there stays -inf
          top = fmaxf(top, KIND != kPlain || mx == -__builtin_inff() ? mx : mx * ksc[ts]);
        }
        top = halves_max(top);
        if (__any(top > m + kLazy)) {
          const float mn = fmaxf(m, top);
          const float f = exp2_fast(m - (mn == -__builtin_inff() ? 0.f : mn));
          m = mn;
          l *= f;
#pragma unroll
          for (int dt = 0; dt < 4; ++dt) o[dt] *= f;
        }
        const float base = m == -__builtin_inff() ? 0.f : m;
        uint4 p[2][2];
#pragma unroll
        for (int ts = 0; ts < 2; ++ts) {
          const float off = base - kPreBias - lv[ts];
          // not 0, which would make NaN of the masked scores of a unit without tokens
          const float sc = KIND != kPlain ? 1.f : fmaxf(ksc[ts], 1e-30f);
          float sum = 0.f;
          uint32_t wd[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float e0 = exp2_fast(__builtin_fmaf(x[ts][2 * i], sc, -off));
            const float e1 = exp2_fast(__builtin_fmaf(x[ts][2 * i + 1], sc, -off));
            sum += e0 + e1;
            wd[i] = pack_f16(e0, e1);
          }
          l = __builtin_fmaf(sum, exp2_fast(-lv[ts]), l);
          p[ts][0] = make_uint4(wd[0], wd[1], wd[2], wd[3]);
          p[ts][1] = make_uint4(wd[4], wd[5], wd[6], wd[7]);
        }
#pragma unroll
        for (int ts = 0; ts < 2; ++ts)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int dt = 0; dt < 4; ++dt)
              o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                  __builtin_bit_cast(at_f16x8, lds.v[buf][(dt * 2 + ts) * 2 + e][lane]),
                  __builtin_bit_cast(at_f16x8, p[ts][e]), o[dt], 0, 0, 0);
        if (lds.nan_tile[buf] == t + 1) {
          const int seen = min(max(len - t * kTileTok, 0), kTileTok);
          const uint64_t sees = seen == kTileTok ? ~0ull : (1ull << seen) - 1;
#pragma unroll
          for (int dt = 0; dt < 4; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int d = 32 * dt + 8 * (i >> 2) + 4 * half + (i & 3);
              const uint64_t bad = *reinterpret_cast<const uint64_t*>(lds.nan_map[buf][d]);
              if ((bad & sees) != 0) o[dt][i] = __builtin_nanf("");
            }
        }
      }
      if (c + 1 < count) store(buf ^ 1, t + 1);
      if (c + 2 < count) load(t + 2, phase);
    }
  }

  l += __uint_as_float(lane_xor<32>(__float_as_uint(l)));
  if (row >= rows) return;
  // lane: dims 32 dt + 8 q + 4 half + e of its row
  if (splits == 1) {
    const float inv = l == 0.f ? 0.f : vref / l;
    uint16_t* out = a.out + (tok * a.Hq + hq) * kHeadDim;
#pragma unroll
    for (int dt = 0; dt < 4; ++dt)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<uint2*>(out + 32 * dt + 8 * g + 4 * half) =
            make_uint2(pack_bf16(o[dt][4 * g] * inv, o[dt][4 * g + 1] * inv),
                       pack_bf16(o[dt][4 * g + 2] * inv, o[dt][4 * g + 3] * inv));
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

int64_t attend_prefill_tiles(int64_t n_tok, int B, int G) { return n_tok * G / kPreRows + B; }

AttnSplit attend_prefill_split(int64_t n_tok, int B, int Hq, int Hkv, int64_t units) {
  const int64_t tiles = (units + 3) / 4;
  const int64_t groups = attend_prefill_tiles(n_tok, B, Hq / Hkv) * Hkv;
  int64_t splits = (512 + groups - 1) / groups;
  splits = splits < tiles / 8 ? splits : tiles / 8;
  if (splits < 1) splits = 1;
  const int64_t chunk = (tiles + splits - 1) / splits;
  return {(int)chunk, (int)((tiles + chunk - 1) / chunk)};
}

int launch_attend_prefill(const AttnArgs& a, AttnSplit sp, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t tiles = attend_prefill_tiles(a.R, a.B, a.Hq / a.Hkv);
  const dim3 grid((unsigned)(tiles * a.Hkv * sp.splits)), blk(kPreNT);
#define IDX_PRE(KIND)                                                                         \
  hipLaunchKernelGGL((attend_prefill_kernel<KIND>), grid, blk, 0, s, a, sp.chunk, sp.splits, \
                     tiles)
  if (a.softcap > 0.f) IDX_PRE(kCapped);
  else if (a.slopes != nullptr) IDX_PRE(kBiased);
  else IDX_PRE(kPlain);
#undef IDX_PRE
  int e = (int)hipGetLastError();
  if (e == 0 && sp.splits > 1) e = launch_attend_merge(a, sp.splits, stream);
  return e;
}

}  // namespace idxk
