// Attention of single tokens over the paged 8-bit cache (include/idx_cache.h,
// idx_attend), and the join of partial results. The kernel is in attend_rows.hpp, the tile
// in attend.hpp. Bound by reading the cache, 256 bytes a token and KV head.
#include <hip/hip_runtime.h>

#include "attend.hpp"
#include "attend_args.h"
#include "attend_rows.hpp"
#include "launch.h"

namespace idxk {

namespace {

// A lane's part of a tile: its key bytes (unit n / 4), value bytes (unit g) and that unit's
// scales.
struct Cache8 {
  static constexpr bool kRowsInLds = false;
  template <int NT, int KIND, bool PACKED>
  static constexpr int kWaves = 2;
  struct Scratch {};
  struct Tile {
    uint4 k[4][2], v[8];
    float ks, vs;
    __device__ __forceinline__ void load(const AttnArgs& a, int kblk, int ksub, int vblk, int vsub,
                                         int n, int g) {
      // (the scales are asked for with the codes, not while the units are listed: a
      // workgroup's start is a chain of loads already)
      ks = a.k_scale[max(vblk, 0)];
      vs = a.v_scale[max(vblk, 0)];
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
    template <int NT, int KIND, bool MIXED>
    __device__ __forceinline__ void add(AttnState<NT>& st, const at_bf16x8 (&q)[NT][4], int vblk,
                                        float call_scale, int pos, int have, const int (&len)[NT],
                                        const float (&slope2)[NT], const Cap& cap, bool any,
                                        Scratch&) {
      attn_tile<NT, KIND, MIXED>(st, q, k, v, vblk < 0 ? 0.f : ks * call_scale,
                                 vblk < 0 ? 0.f : vs, pos, have, len, slope2, cap, any);
    }
  };
  static __device__ __forceinline__ void load_query(const uint16_t* row, int g, bool negative,
                                                    at_bf16x8 (&q)[4]) {
    idxk::load_query(row, g, negative, q);
  }
  template <int NT>
  static __device__ __forceinline__ void init(AttnState<NT>&) {}
  template <int NT>
  static __device__ __forceinline__ const at_bf16x8 (&rows(const at_bf16x8 (&q)[NT][4],
                                                           const uint4 (&)[1][kWave]))[NT][4] {
    return q;
  }
  static __device__ __forceinline__ int dim_of(int dt, int g) { return 16 * dt + 4 * g; }
  template <int NT>
  static __device__ __forceinline__ at_f32x4 sums(const AttnState<NT>& st, int j, int dt) {
    return st.o[j][dt];
  }
};

// The splits' sums of one (row, query head), each in units of its own maximum: TEAMS
// teams of 32 lanes, four dims a lane, take every TEAMS-th split, four at a time, and are
// joined in LDS. Fixed orders: the same sums every time. Short: a launch and chains of loads
// (64 splits of 128 items: 4.9 us with eight splits' loads in flight, 5.7 with the sums behind
// the weights of four). A split's weights may reach 2^60 in its maximum's units (attend4.hpp), and
// count where its sums do not: scaled_down takes them where a factor of 2^-126 would leave
// more than 2^-29 of a row's weights, 2^-57 at the least (1024 items of 64 splits: 0.9 us if it
// always did).
constexpr float kHeavy = 0x1p40f;
template <int TEAMS, bool ALL>
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
    // A split without tokens has no weight: its sums are not taken, whatever they hold. Few
    // items (ALL) ask for two steps' weights and sums at once, many save those splits' bytes
    // (1024 items of 64 splits, 40 of them empty: 7.5 us, 8.5 with all sums read) and the
    // registers of the second step (51 against 82, eight waves a SIMD against five: 32 rows of
    // 8192 to 32768 tokens, 64 heads on 4, 152 us in all with it, 150 without).
    constexpr int kStep = 4, kLoads = ALL ? 2 : 1;
    for (int s0 = team; s0 < splits; s0 += kLoads * kStep * TEAMS) {
      at_f32x2 ml[kLoads * kStep];
      at_f32x4 x[kLoads * kStep];
#pragma unroll
      for (int i = 0; i < kLoads * kStep; ++i) {
        const int64_t p = first + (int64_t)min(s0 + i * TEAMS, splits - 1) * G;
        ml[i] = *reinterpret_cast<const at_f32x2*>(a.part_ml + 2 * p);
        if constexpr (ALL)
          x[i] = *reinterpret_cast<const at_f32x4*>(a.part_o + p * kHeadDim + 4 * lane);
        if (s0 + i * TEAMS >= splits) ml[i] = at_f32x2{-__builtin_inff(), 0.f};
      }
#pragma unroll
      for (int i = 0; i < kLoads * kStep; ++i) {
        if (ml[i][1] == 0.f) {
          x[i] = at_f32x4{0.f, 0.f, 0.f, 0.f};
        } else if (!ALL) {
          const int64_t p = first + (int64_t)min(s0 + i * TEAMS, splits - 1) * G;
          x[i] = *reinterpret_cast<const at_f32x4*>(a.part_o + p * kHeadDim + 4 * lane);
        }
      }
#pragma unroll
      for (int j = 0; j < kLoads * kStep; j += kStep) {
        float top = m;
#pragma unroll
        for (int i = j; i < j + kStep; ++i) top = fmaxf(top, ml[i][0]);
        const float base = top == -__builtin_inff() ? 0.f : top;
        const float f = exp2_fast(m - base);
        float most = l;
#pragma unroll
        for (int i = j; i < j + kStep; ++i) most = fmaxf(most, ml[i][1]);
        float w[kStep];
#pragma unroll
        for (int i = 0; i < kStep; ++i) w[i] = exp2_fast(ml[j + i][0] - base);
        if (__any(most > kHeavy)) {
          l = scaled_down(l, m - base);
#pragma unroll
          for (int i = 0; i < kStep; ++i)
            l += scaled_down(ml[j + i][1], ml[j + i][0] - base);
        } else {
          l *= f;
#pragma unroll
          for (int i = 0; i < kStep; ++i) l += ml[j + i][1] * w[i];
        }
        m = top;
        o *= f;
#pragma unroll
        for (int i = 0; i < kStep; ++i) o += x[j + i] * w[i];
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
  l = scaled_down(l, m - base);
  o *= f;
#pragma unroll
  for (int i = 1; i < TEAMS; ++i) {
    const float w = exp2_fast(s_m[group + i] - base);
    l += scaled_down(s_l[group + i], s_m[group + i] - base);
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
// CU, 136 at four, 123 at eight, 127 at sixteen; 114 at eight today; equal shares for all that
// the chip holds at once, worked out by the kernel, were slower, 130), down to a tile for each
// wave.
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
  if (wide && items * splits <= 8192)
    hipLaunchKernelGGL((attend_merge_kernel<8, true>), grid, blk, 0, s, a, items, splits);
  else if (wide)
    hipLaunchKernelGGL((attend_merge_kernel<8, false>), grid, blk, 0, s, a, items, splits);
  else
    hipLaunchKernelGGL((attend_merge_kernel<2, false>), grid, blk, 0, s, a, items, splits);
  return (int)hipGetLastError();
}

int launch_attend_rows(const AttnArgs& a, AttnSplit sp, void* stream) {
  return launch_rows_of<Cache8>(a, sp, stream);
}

}  // namespace idxk
