// Attention of single tokens over the paged 8-bit cache (include/idx_cache.h,
// idx_attend), and the join of partial results. The tile is in attend.hpp.
//
// One token's query heads of one KV head are the 16 (32, 64) rows of the products.
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
constexpr int kChunkTiles = 256;              // most tiles of one workgroup
constexpr int kChunkUnits = 4 * kChunkTiles;
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

template <int NT, bool EXTRA>
__global__ __launch_bounds__(kAtNT) void attend_rows_kernel(AttnArgs a, int chunk, int splits) {
  __shared__ int u_blk[kChunkUnits], u_pos[kChunkUnits];
  __shared__ float u_ks[kChunkUnits], u_vs[kChunkUnits];
  __shared__ float s_m[kAtWaves][16 * NT], s_l[kAtWaves][16 * NT];
  __shared__ __attribute__((aligned(16))) float s_o[16 * NT][kRowPad];

  const int h = blockIdx.x % a.Hkv;
  const int rest = blockIdx.x / a.Hkv;
  const int split = rest % splits, r = rest / splits;
  const int tid = threadIdx.x, lane = lane_id(), w = tid / kWave;
  const int n = lane & 15, g = lane >> 4;
  const int G = a.Hq / a.Hkv;
  const int upp = a.page_size / kUnit;

  int b = a.row_req == nullptr ? r : a.row_req[r];
  const bool known = b >= 0 && b < a.B;
  const PageList pages = known ? page_list(a, b) : PageList{0, 0};
  const int seen = known ? max(a.kv_len[r], 0) : 0;

  // this workgroup's units: list slots or selected slots, 16 tokens each
  const int64_t listed =
      a.ids != nullptr ? (int64_t)a.K * upp
                       : min((int64_t)pages.n * upp, ((int64_t)seen + kUnit - 1) / kUnit);
  const int64_t u0 = (int64_t)split * chunk * 4;
  const int units = (int)max((int64_t)0, min(listed - u0, (int64_t)chunk * 4));
  const int tiles = (units + 3) / 4;
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
    u_ks[i] = blk < 0 ? 0.f : a.k_scale[blk] * a.score_scale;
    u_vs[i] = blk < 0 ? 0.f : a.v_scale[blk];
  }

  at_bf16x8 q[NT][4];
  float slope2[NT];
  int len[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int hq = h * G + min(16 * j + n, G - 1);
    load_query(a.q + (int64_t)r * a.q_stride + hq * kHeadDim, g, q[j]);
    slope2[j] = EXTRA ? slope_of(a, hq) : 0.f;
    len[j] = seen;
  }
  AttnState<NT> st;
  attn_init(st);
  __syncthreads();

  for (int t = w; t < tiles; t += kAtWaves) {
    const int ku = 4 * t + (n >> 2), vu = 4 * t + g;
    const int kblk = u_blk[ku], vblk = u_blk[vu], pos = u_pos[vu];
    const int have = vblk < 0 ? 0 : min(seen - pos, kUnit);
    if (__all(have == 0)) continue;
    uint4 k[4][2], v[8];
    load_tile(a, kblk, (u_pos[ku] % a.page_size) / kUnit, vblk, (pos % a.page_size) / kUnit, n,
              g, k, v);
    const bool any = !__all(have == kUnit);
    if (any) {
#pragma unroll
      for (int dt = 0; dt < 8; ++dt) v[dt] = keep_tokens(v[dt], have);
    }
    attn_tile<NT, EXTRA>(st, q, k, v, u_ks[vu], u_vs[vu], pos, have, len, slope2, a.softcap,
                         any);
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
  const int64_t part = ((int64_t)r * a.Hkv + h) * splits + split;
  for (int item = tid; item < G * 16; item += kAtNT) {
    const int row = item >> 4, d = (item & 15) * 8;
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
      *reinterpret_cast<uint4*>(a.out + ((int64_t)r * a.Hq + h * G + row) * kHeadDim + d) = out;
    } else {
      at_f32x4* p = reinterpret_cast<at_f32x4*>(a.part_o + (part * G + row) * kHeadDim + d);
      p[0] = *reinterpret_cast<const at_f32x4*>(o);
      p[1] = *reinterpret_cast<const at_f32x4*>(o + 4);
      if (d == 0) {
        a.part_ml[2 * (part * G + row)] = m;
        a.part_ml[2 * (part * G + row) + 1] = l;
      }
    }
  }
}

// One wave per (row, query head): the splits' sums, each in units of its own maximum.
__global__ __launch_bounds__(kAtNT) void attend_merge_kernel(AttnArgs a, int64_t rows,
                                                             int splits) {
  const int64_t item = (int64_t)blockIdx.x * kAtWaves + threadIdx.x / kWave;
  if (item >= rows * a.Hq) return;
  const int lane = lane_id();
  const int G = a.Hq / a.Hkv;
  const int64_t r = item / a.Hq;
  // prompt rows of no request keep their output
  if (a.tok_indptr != nullptr && (r < a.tok_indptr[0] || r >= a.tok_indptr[a.B])) return;
  const int hq = (int)(item % a.Hq), h = hq / G, row = hq % G;
  const int64_t first = ((r * a.Hkv + h) * splits) * G + row;  // + s * G
  float m = -__builtin_inff();
  for (int s = lane; s < splits; s += kWave) m = fmaxf(m, a.part_ml[2 * (first + (int64_t)s * G)]);
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
  const float base = m == -__builtin_inff() ? 0.f : m;
  float l = 0.f;
  at_f32x2 o = {0.f, 0.f};
  for (int s = 0; s < splits; ++s) {
    const int64_t p = first + (int64_t)s * G;
    const float ls = a.part_ml[2 * p + 1];
    if (ls == 0.f) continue;
    const float f = exp2_fast(a.part_ml[2 * p] - base);
    l += ls * f;
    o += *reinterpret_cast<const at_f32x2*>(a.part_o + p * kHeadDim + 2 * lane) * f;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  reinterpret_cast<uint32_t*>(a.out + (r * a.Hq + hq) * kHeadDim)[lane] =
      pack_bf16(o[0] * inv, o[1] * inv);
}

}  // namespace

AttnSplit attend_rows_split(int64_t R, int Hkv, int64_t units) {
  const int64_t tiles = (units + 3) / 4;
  const int64_t pairs = R * Hkv;
  int64_t splits = (1024 + pairs - 1) / pairs;            // about four workgroups a CU
  splits = splits < tiles / 8 ? splits : tiles / 8;       // at least two tiles a wave
  if (splits < 1) splits = 1;
  int64_t chunk = (tiles + splits - 1) / splits;
  if (chunk > kChunkTiles) chunk = kChunkTiles;
  return {(int)chunk, (int)((tiles + chunk - 1) / chunk)};
}

int launch_attend_merge(const AttnArgs& a, int splits, void* stream) {
  const int64_t rows = a.R;
  const int64_t grid = (rows * a.Hq + kAtWaves - 1) / kAtWaves;
  hipLaunchKernelGGL(attend_merge_kernel, dim3((unsigned)grid), dim3(kAtNT), 0,
                     static_cast<hipStream_t>(stream), a, rows, splits);
  return (int)hipGetLastError();
}

int launch_attend_rows(const AttnArgs& a, AttnSplit sp, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int G = a.Hq / a.Hkv;
  const bool extra = a.softcap > 0.f || a.slopes != nullptr;
  const dim3 grid((unsigned)((int64_t)a.R * a.Hkv * sp.splits)), blk(kAtNT);
#define IDX_ROWS(NT, EX) \
  hipLaunchKernelGGL((attend_rows_kernel<NT, EX>), grid, blk, 0, s, a, sp.chunk, sp.splits)
  if (G <= 16) {
    if (extra) IDX_ROWS(1, true); else IDX_ROWS(1, false);
  } else if (G <= 32) {
    if (extra) IDX_ROWS(2, true); else IDX_ROWS(2, false);
  } else {
    if (extra) IDX_ROWS(4, true); else IDX_ROWS(4, false);
  }
#undef IDX_ROWS
  int e = (int)hipGetLastError();
  if (e == 0 && sp.splits > 1) e = launch_attend_merge(a, sp.splits, stream);
  return e;
}

}  // namespace idxk
