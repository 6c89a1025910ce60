// Attention of single tokens over a paged cache: the rows' kernel, over a policy of the
// cache's tiles (attend.hip: 8 bits, attend4.hip: 4 bits). A policy has
//   load_query, init   a row's operand, and what a state starts with
//   Tile               this lane's part of 64 tokens: load() asks for it, add() takes it
//                      into a state, by way of a wave's Scratch in LDS
//   dim_of, sums       the first dim of four, and the state's sums of them
//   kRowsInLds, rows   where add() finds the rows' operands: registers, or LDS, which all
//                      waves share
//   kWaves             waves a SIMD that an instance's registers are cut to
//
// One token's query heads of one KV head are the 16 or 32 rows of the products (above 32
// heads a group, two workgroups take 32 each); or, for prompt calls of few rows a request,
// 16 rows (token, head) of the request.
// Bound by reading the cache: each of a workgroup's four waves runs its own tiles, with its
// own softmax, joined in LDS at the end. Long rows are cut into chunks of tiles for several
// workgroups; their partial sums are joined by attend_merge_kernel (attend.hip).
#pragma once

#include "attend.hpp"
#include "launch.h"

namespace idxk {

constexpr int kAtNT = 256;
constexpr int kAtWaves = kAtNT / kWave;
constexpr int kPhase = 256;                   // tiles whose pages wait in LDS
constexpr int kPhaseUnits = 4 * kPhase;
constexpr int kRowPad = kHeadDim + 4;         // floats of a row of sums in LDS

template <class Cache, int NT, int KIND, bool PACKED>
__global__ __launch_bounds__(kAtNT, (Cache::template kWaves<NT, KIND, PACKED>)) void attend_rows_kernel(
    AttnArgs a, int chunk, int splits, int bands) {
  __shared__ int u_blk[kPhaseUnits], u_pos[kPhaseUnits];
  __shared__ float s_m[kAtWaves][16 * NT], s_l[kAtWaves][16 * NT];
  __shared__ __attribute__((aligned(16))) float s_o[16 * NT][kRowPad];
  __shared__ typename Cache::Scratch scratch[kAtWaves];
  __shared__ uint4 s_q[Cache::kRowsInLds ? 4 * NT : 1][kWave];

  const int band = blockIdx.x % bands;  // of 16 NT query heads of the group
  const int h = blockIdx.x / bands % a.Hkv;
  const int rest = blockIdx.x / bands / a.Hkv;
  const int split = rest % splits, r = rest / splits;  // packed: r is a row tile
  const int tid = threadIdx.x, lane = lane_id(), w = tid / kWave;
  const int n = lane & 15, g = lane >> 4;
  const int G = a.Hq / a.Hkv;
  const int upp = a.page_size / kUnit;

  // The request, and where row i of this workgroup's 16 NT lies: token row and head of the
  // group; rows past the last repeat it.
  RowTile rt{0, r, 16 * NT * band, G};
  bool known = true;
  if constexpr (PACKED) {
    __shared__ int found;
    rt = row_tile<kAtNT>(a, r, G, 16 * NT, &found);
    if (rt.row0 < 0 || rt.row0 >= rt.rows) return;
  } else {
    rt.b = a.row_req == nullptr ? r : a.row_req[r];
    known = rt.b >= 0 && rt.b < a.B;
  }
  const int rows = (int)min((int64_t)16 * NT, rt.rows - rt.row0);
  auto token_of = [&](int i) {
    return PACKED ? rt.t0 + (rt.row0 + min(i, rows - 1)) / G : (int64_t)r;
  };
  auto head_of = [&](int i) {
    const int64_t at = rt.row0 + min(i, rows - 1);
    return (int)(PACKED ? at % G : at);
  };
  const PageList pages = known ? page_list(a, rt.b) : PageList{0, 0};

  int len[NT];
  int seen = 0, shortest = 0x7FFFFFFF;  // longest and shortest visible length of the rows
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    len[j] = known ? max(a.kv_len[token_of(16 * j + n)], 0) : 0;
    seen = max(seen, len[j]);
    shortest = min(shortest, len[j]);
  }
  if constexpr (PACKED) {
#pragma unroll
    for (int d = 1; d < 16; d *= 2) {
      seen = max(seen, __shfl_xor(seen, d));
      shortest = min(shortest, __shfl_xor(shortest, d));
    }
  }
  const int64_t listed =
      a.ids != nullptr ? (int64_t)a.K * upp
                       : min((int64_t)pages.n * upp, ((int64_t)seen + kUnit - 1) / kUnit);
  const int64_t end = min(listed, ((int64_t)split + 1) * chunk * 4);
  auto part_of = [&](int row) {
    return ((token_of(row) * a.Hkv + h) * splits + split) * G + head_of(row);
  };
  // Chunks behind a row's last token leave no sums, a weight of zero alone (the join takes no
  // sums of those): calls are cut for a bound of the lengths, so there may be many (984 of 2048
  // workgroups in the rows of 4096 to 131072 tokens: 71.4 us with zeros stored for them, 69.7).
  if (splits > 1 && (int64_t)split * chunk * 4 >= end) {
    for (int row = tid; row < rows; row += kAtNT) {
      a.part_ml[2 * part_of(row)] = -__builtin_inff();
      a.part_ml[2 * part_of(row) + 1] = 0.f;
    }
    return;
  }

  const float call_scale = fabsf(a.score_scale);
  const Cap cap(a.softcap);
  at_bf16x8 q[NT][4];
  float slope2[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int hq = h * G + head_of(16 * j + n);
    Cache::load_query(a.q + token_of(16 * j + n) * a.q_stride + hq * kHeadDim, g,
                      a.score_scale < 0.f, q[j]);
    slope2[j] = KIND != kPlain ? slope_of(a, hq) : 0.f;
  }
  if (Cache::kRowsInLds && w == 0) {  // (the waves meet at the first phase)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) s_q[4 * j + i][lane] = __builtin_bit_cast(uint4, q[j][i]);
  }
  AttnState<NT> st;
  attn_init(st);
  Cache::init(st);

  // this workgroup's units, list slots or selected slots of 16 tokens each, a phase at a
  // time
  for (int64_t u0 = (int64_t)split * chunk * 4; u0 < end; u0 += kPhaseUnits) {
    const int units = (int)min(end - u0, (int64_t)kPhaseUnits);
    const int tiles = (units + 3) / 4;
    __syncthreads();  // the phase before has been read
    for (int i = tid; i < 4 * tiles; i += kAtNT) {
      int blk = -1, pos = 0;
      if (i < units) {
        const int64_t u = u0 + i;
        int slot = (int)(u / upp);
        const int sub = (int)(u % upp);
        if (a.ids != nullptr) slot = a.ids[(int64_t)r * a.K + slot];
        blk = block_of(a, pages, slot, h);
        if (blk >= 0) pos = slot * a.page_size + sub * kUnit;
        if (pos >= seen) blk = -1;
      }
      u_blk[i] = blk;
      u_pos[i] = blk < 0 ? 0 : pos;
    }
    __syncthreads();
    for (int t = w; t < tiles; t += kAtWaves) {
      const int ku = 4 * t + (n >> 2), vu = 4 * t + g;
      const int kblk = u_blk[ku], vblk = u_blk[vu], pos = u_pos[vu];
      const int have = vblk < 0 ? 0 : min(seen - pos, kUnit);
      if (__all(have == 0)) continue;
      typename Cache::Tile x;
      x.load(a, kblk, (u_pos[ku] & (a.page_size - 1)) / kUnit, vblk,
             (pos & (a.page_size - 1)) / kUnit, n, g);
      const bool any = !__all(have == kUnit && (!PACKED || pos + kUnit <= shortest));
      x.template add<NT, KIND, PACKED>(st, Cache::rows(q, s_q), vblk, call_scale, pos, have, len,
                                       slope2, cap, any, scratch[w]);
    }
  }

  // join the waves
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const float l = groups_sum(st.l[j]);
    if (g == 0) {
      s_m[w][16 * j + n] = st.m[j];
      s_l[w][16 * j + n] = l;
    }
  }
  __syncthreads();
  float f[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    float m = s_m[0][16 * j + n];
#pragma unroll
    for (int i = 1; i < kAtWaves; ++i) m = fmaxf(m, s_m[i][16 * j + n]);
    f[j] = st.m[j] == -__builtin_inff() ? 0.f : exp2_fast(st.m[j] - m) * st.vref;
  }
  for (int i = 0; i < kAtWaves; ++i) {
    if (w == i) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int dt = 0; dt < 8; ++dt) {
          at_f32x4* p = reinterpret_cast<at_f32x4*>(&s_o[16 * j + n][Cache::dim_of(dt, g)]);
          const at_f32x4 o = Cache::sums(st, j, dt) * f[j];
          *p = i == 0 ? o : *p + o;
        }
    }
    __syncthreads();
  }
  for (int item = tid; item < rows * 16; item += kAtNT) {
    const int row = item >> 4, d = (item & 15) * 8, g_row = head_of(row);
    const int64_t tok = token_of(row);
    const int64_t part = part_of(row);
    float m = s_m[0][row], l = 0.f;
#pragma unroll
    for (int i = 1; i < kAtWaves; ++i) m = fmaxf(m, s_m[i][row]);
    const float base = m == -__builtin_inff() ? 0.f : m;
#pragma unroll
    for (int i = 0; i < kAtWaves; ++i) l += scaled_down(s_l[i][row], s_m[i][row] - base);
    const float* o = &s_o[row][d];
    if (splits == 1) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint4 out;
      out.x = pack_bf16(o[0] * inv, o[1] * inv);
      out.y = pack_bf16(o[2] * inv, o[3] * inv);
      out.z = pack_bf16(o[4] * inv, o[5] * inv);
      out.w = pack_bf16(o[6] * inv, o[7] * inv);
      *reinterpret_cast<uint4*>(a.out + (tok * a.Hq + h * G + g_row) * kHeadDim + d) = out;
    } else {
      at_f32x4* p = reinterpret_cast<at_f32x4*>(a.part_o + part * kHeadDim + d);
      p[0] = *reinterpret_cast<const at_f32x4*>(o);
      p[1] = *reinterpret_cast<const at_f32x4*>(o + 4);
      if (d == 0) {
        a.part_ml[2 * part] = m;
        a.part_ml[2 * part + 1] = l;
      }
    }
  }
}

// Launches the rows' kernel of a cache, and the join of rows that were cut.
template <class Cache>
int launch_rows_of(const AttnArgs& a, AttnSplit sp, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int G = a.Hq / a.Hkv;
  const bool packed = a.tok_indptr != nullptr;
  const int bands = packed || G <= 32 ? 1 : 2;
  const int64_t rows = packed ? attend_prefill_tiles(a.R, a.B, G, sp.rows) : a.R;
  const dim3 grid((unsigned)(rows * a.Hkv * sp.splits * bands)), blk(kAtNT);
#define IDX_ROWS(NT, KIND, PACKED)                                                              \
  hipLaunchKernelGGL((attend_rows_kernel<Cache, NT, KIND, PACKED>), grid, blk, 0, s, a, sp.chunk, \
                     sp.splits, bands)
#define IDX_KINDS(NT, PACKED)                                  \
  if (a.softcap > kNearCap) IDX_ROWS(NT, kCappedFar, PACKED);  \
  else if (a.softcap > 0.f) IDX_ROWS(NT, kCapped, PACKED);     \
  else if (a.slopes != nullptr) IDX_ROWS(NT, kBiased, PACKED); \
  else IDX_ROWS(NT, kPlain, PACKED)
  if (packed) {
    IDX_KINDS(1, true);
  } else if (G <= 16) {
    IDX_KINDS(1, false);
  } else {
    IDX_KINDS(2, false);
  }
#undef IDX_KINDS
#undef IDX_ROWS
  int e = (int)hipGetLastError();
  if (e == 0 && sp.splits > 1) e = launch_attend_merge(a, sp.splits, stream);
  return e;
}

}  // namespace idxk
