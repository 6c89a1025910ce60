// Attention of single tokens over the paged 8-bit cache (include/idx_cache.h,
// idx_attend), and the join of partial results. The tile is in attend.hpp.
//
// One token's query heads of one KV head are the 16 or 32 rows of the products (above 32
// heads a group, two workgroups take 32 each); or, for prompt calls of few rows a request,
// 16 rows (token, head) of the request.
// Bound by reading the cache, 256 bytes a token and KV head: each of a workgroup's four
// waves runs its own tiles, with its own softmax, joined in LDS at the end. Long rows are
// cut into chunks of tiles for several workgroups; their partial sums are joined by
// attend_merge_kernel.
#include <hip/hip_runtime.h>

#include "attend.hpp"
#include "attend_args.h"
#include "launch.h"

namespace idxk {

namespace {

constexpr int kAtNT = 256;
constexpr int kAtWaves = kAtNT / kWave;
constexpr int kPhase = 256;                   // tiles whose pages wait in LDS
constexpr int kPhaseUnits = 4 * kPhase;
constexpr int kRowPad = kHeadDim + 4;         // floats of a row of sums in LDS

// Loads of one tile: this lane's key bytes (unit m / 4) and value bytes (unit g).
__device__ __forceinline__ void load_tile(const AttnArgs& a, int kblk, int ksub, int vblk,
                                          int vsub, int n, int g, uint4 (&k)[4][2],
                                          uint4 (&v)[8]) {
  const int64_t block = (int64_t)a.page_size * kHeadDim;
  const uint8_t* kp = a.k_cache + max(kblk, 0) * block + ksub * (kUnit * kHeadDim) +
                      (n & 3) * kHeadDim + 16 * g;
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int c = 0; c < 2; ++c)
      k[s][c] = *reinterpret_cast<const uint4*>(kp + s * (4 * kHeadDim) + 64 * c);
  const uint8_t* vp =
      a.v_cache + max(vblk, 0) * block + vsub * kUnit + (int64_t)n * a.page_size;
#pragma unroll
  for (int dt = 0; dt < 8; ++dt)
    v[dt] = *reinterpret_cast<const uint4*>(vp + (int64_t)dt * 16 * a.page_size);
}

template <int NT, int KIND, bool PACKED>
__global__ __launch_bounds__(kAtNT, 2) void attend_rows_kernel(AttnArgs a, int chunk, int splits,
                                                               int bands) {
  __shared__ int u_blk[kPhaseUnits], u_pos[kPhaseUnits];
  __shared__ float s_m[kAtWaves][16 * NT], s_l[kAtWaves][16 * NT];
  __shared__ __attribute__((aligned(16))) float s_o[16 * NT][kRowPad];

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

  const float call_scale = fabsf(a.score_scale);
  const Cap cap(a.softcap);
  at_bf16x8 q[NT][4];
  float slope2[NT];
  int len[NT];
  int seen = 0, shortest = 0x7FFFFFFF;  // longest and shortest visible length of the rows
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t tok = token_of(16 * j + n);
    const int hq = h * G + head_of(16 * j + n);
    load_query(a.q + tok * a.q_stride + hq * kHeadDim, g, a.score_scale < 0.f, q[j]);
    slope2[j] = KIND != kPlain ? slope_of(a, hq) : 0.f;
    len[j] = known ? max(a.kv_len[tok], 0) : 0;
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
  AttnState<NT> st;
  attn_init(st);

  // this workgroup's units, list slots or selected slots of 16 tokens each, a phase at a
  // time
  const int64_t listed =
      a.ids != nullptr ? (int64_t)a.K * upp
                       : min((int64_t)pages.n * upp, ((int64_t)seen + kUnit - 1) / kUnit);
  const int64_t end = min(listed, ((int64_t)split + 1) * chunk * 4);
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
      // (its scales are asked for with the codes, not while the units are listed: a
      // workgroup's start is a chain of loads already)
      uint4 k[4][2], v[8];
      const float ks = a.k_scale[max(vblk, 0)], vs = a.v_scale[max(vblk, 0)];
      load_tile(a, kblk, (u_pos[ku] & (a.page_size - 1)) / kUnit, vblk,
                (pos & (a.page_size - 1)) / kUnit, n, g, k, v);
      const bool any = !__all(have == kUnit && (!PACKED || pos + kUnit <= shortest));
      attn_tile<NT, KIND, PACKED>(st, q, k, v, vblk < 0 ? 0.f : ks * call_scale,
                                  vblk < 0 ? 0.f : vs, pos, have, len, slope2, cap, any);
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
          at_f32x4* p = reinterpret_cast<at_f32x4*>(&s_o[16 * j + n][16 * dt + 4 * g]);
          const at_f32x4 o = st.o[j][dt] * f[j];
          *p = i == 0 ? o : *p + o;
        }
    }
    __syncthreads();
  }
  for (int item = tid; item < rows * 16; item += kAtNT) {
    const int row = item >> 4, d = (item & 15) * 8, g_row = head_of(row);
    const int64_t tok = token_of(row);
    const int64_t part = (((tok * a.Hkv + h) * splits) + split) * G + g_row;
    float m = s_m[0][row], l = 0.f;
#pragma unroll
    for (int i = 1; i < kAtWaves; ++i) m = fmaxf(m, s_m[i][row]);
    const float base = m == -__builtin_inff() ? 0.f : m;
#pragma unroll
    for (int i = 0; i < kAtWaves; ++i) l += s_l[i][row] * exp2_fast(s_m[i][row] - base);
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

// The splits' sums of one (row, query head), each in units of its own maximum: TEAMS
// teams of 32 lanes, four dims a lane, take every TEAMS-th split, four at a time with
// their loads in flight, and are joined in LDS. Fixed orders: the same sums every time.
template <int TEAMS>
__global__ __launch_bounds__(kAtNT) void attend_merge_kernel(AttnArgs a, int64_t items,
                                                             int splits) {
  constexpr int kItems = kAtNT / 32 / TEAMS;  // of a workgroup
  __shared__ __attribute__((aligned(16))) float s_o[kAtNT / 32][kHeadDim];
  __shared__ float s_m[kAtNT / 32], s_l[kAtNT / 32];
  const int lane = threadIdx.x & 31, group = threadIdx.x / 32, team = group % TEAMS;
  const int64_t item = (int64_t)blockIdx.x * kItems + group / TEAMS;
  const int G = a.Hq / a.Hkv;
  const int64_t r = item / a.Hq;
  const int hq = (int)(item % a.Hq), h = hq / G;
  // prompt rows of no request keep their output
  const bool live = item < items && (a.tok_indptr == nullptr ||
                                     (r >= a.tok_indptr[0] && r < a.tok_indptr[a.B]));
  const int64_t first = ((r * a.Hkv + h) * splits) * G + hq % G;  // + s * G
  float m = -__builtin_inff(), l = 0.f;
  at_f32x4 o = {0.f, 0.f, 0.f, 0.f};
  if (live) {
    constexpr int kStep = 4;
    for (int s0 = team; s0 < splits; s0 += kStep * TEAMS) {
      at_f32x2 ml[kStep];
      at_f32x4 x[kStep];
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        const int s = s0 + i * TEAMS;
        const int64_t p = first + (int64_t)min(s, splits - 1) * G;
        ml[i] = *reinterpret_cast<const at_f32x2*>(a.part_ml + 2 * p);
        if (s >= splits) ml[i] = at_f32x2{-__builtin_inff(), 0.f};
      }
      // (a split without tokens has no weight: its sums, zeros, need not be read)
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        x[i] = at_f32x4{0.f, 0.f, 0.f, 0.f};
        if (ml[i][1] != 0.f) {
          const int64_t p = first + (int64_t)min(s0 + i * TEAMS, splits - 1) * G;
          x[i] = *reinterpret_cast<const at_f32x4*>(a.part_o + p * kHeadDim + 4 * lane);
        }
      }
      float top = m;
#pragma unroll
      for (int i = 0; i < kStep; ++i) top = fmaxf(top, ml[i][0]);
      const float base = top == -__builtin_inff() ? 0.f : top;
      const float f = exp2_fast(m - base);
      m = top;
      l *= f;
      o *= f;
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        const float w = exp2_fast(ml[i][0] - base);
        l += ml[i][1] * w;
        o += x[i] * w;
      }
    }
  }
  *reinterpret_cast<at_f32x4*>(&s_o[group][4 * lane]) = o;
  if (lane == 0) {
    s_m[group] = m;
    s_l[group] = l;
  }
  __syncthreads();
  if (!live || team != 0) return;
  float top = m;
#pragma unroll
  for (int i = 1; i < TEAMS; ++i) top = fmaxf(top, s_m[group + i]);
  const float base = top == -__builtin_inff() ? 0.f : top;
  const float f = exp2_fast(m - base);
  l *= f;
  o *= f;
#pragma unroll
  for (int i = 1; i < TEAMS; ++i) {
    const float w = exp2_fast(s_m[group + i] - base);
    l += s_l[group + i] * w;
    o += *reinterpret_cast<const at_f32x4*>(&s_o[group + i][4 * lane]) * w;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  reinterpret_cast<uint2*>(a.out + (r * a.Hq + hq) * kHeadDim)[lane] =
      make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
}

}  // namespace

// Rows are cut only when there are fewer than two workgroups a CU without it (the GQA
// batch of 128 rows on 4 heads, 256 pages each: 102 us whole, 108 in two). Then into
// chunks that would give eight a CU if all rows were of the longest length, so that
// ragged rows still balance (4 rows of 4096 to 131072 tokens on 8 heads: 148 us at two a
// CU, 136 at four, 123 at eight, 127 at sixteen; equal shares for all that the chip holds at
// once, worked out by the kernel, are slower, 130), down to a tile for each wave.
AttnSplit attend_rows_split(int64_t R, int Hkv, int64_t units) {
  const int64_t tiles = (units + 3) / 4;
  const int64_t pairs = R * Hkv;
  int64_t splits = pairs >= 512 ? 1 : (2048 + pairs - 1) / pairs;
  if (splits > tiles / kAtWaves) splits = tiles / kAtWaves;
  if (splits < 1) splits = 1;
  const int64_t chunk = (tiles + splits - 1) / splits;
  return {(int)chunk, (int)((tiles + chunk - 1) / chunk), 0};
}

int launch_attend_merge(const AttnArgs& a, int splits, void* stream) {
  const int64_t items = (int64_t)a.R * a.Hq;
  hipStream_t s = static_cast<hipStream_t>(stream);
  // few items of many splits: a workgroup for each (128 items of 32 splits: 18 us with a
  // wave for each and one split at a time, 4.8 so)
  const bool wide = splits > 8 && items <= 8192;
  const int per = wide ? 1 : 4;
  const dim3 grid((unsigned)((items + per - 1) / per)), blk(kAtNT);
  if (wide)
    hipLaunchKernelGGL((attend_merge_kernel<8>), grid, blk, 0, s, a, items, splits);
  else
    hipLaunchKernelGGL((attend_merge_kernel<2>), grid, blk, 0, s, a, items, splits);
  return (int)hipGetLastError();
}

int launch_attend_rows(const AttnArgs& a, AttnSplit sp, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int G = a.Hq / a.Hkv;
  const bool packed = a.tok_indptr != nullptr;
  const int bands = packed || G <= 32 ? 1 : 2;
  const int64_t rows = packed ? attend_prefill_tiles(a.R, a.B, G, sp.rows) : a.R;
  const dim3 grid((unsigned)(rows * a.Hkv * sp.splits * bands)), blk(kAtNT);
#define IDX_ROWS(NT, KIND, PACKED)                                                              \
  hipLaunchKernelGGL((attend_rows_kernel<NT, KIND, PACKED>), grid, blk, 0, s, a, sp.chunk, \
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
