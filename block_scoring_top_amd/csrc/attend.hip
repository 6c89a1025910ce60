// Attention over the paged 8-bit cache (include/idx_cache.h: idx_attend,
// idx_attend_prefill). The tile that both kernels run is in attend.hpp.
//
// attend_rows_kernel: one token's query heads of one KV head are the 16 (32, 64)
// rows of the products. Bound by reading the cache, 256 bytes a token and KV head:
// each of a workgroup's four waves runs its own tiles, with its own softmax, joined
// in LDS at the end. Long rows are cut into chunks of tiles for several workgroups;
// their partial sums are joined by attend_merge_kernel.
//
// attend_prefill_kernel: 128 rows (token, head of the group) of one request share
// the tiles, 32 rows to a wave.
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

__device__ __forceinline__ float slope_of(const AttnArgs& a, int hq) {
  return a.slopes == nullptr ? 0.f : a.slopes[hq] * kLog2e;
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

constexpr int kPreRows = 128;  // rows of a workgroup, 32 to a wave

// First tile of request b in the grid: tiles never span requests, and
// floor(y / T) - floor(x / T) + 1 tiles hold any x..y rows.
__device__ __forceinline__ int64_t first_tile(const AttnArgs& a, int b, int G) {
  const int64_t p = min(max(a.tok_indptr[b], 0), a.R);
  return p * G / kPreRows + b;
}

template <bool EXTRA>
__global__ __launch_bounds__(kAtNT) void attend_prefill_kernel(AttnArgs a, int chunk,
                                                               int splits) {
  constexpr int NT = 2;
  const int h = blockIdx.x % a.Hkv;
  const int rest = blockIdx.x / a.Hkv;
  const int split = rest % splits;
  const int64_t tile = rest / splits;
  const int tid = threadIdx.x, lane = lane_id(), w = tid / kWave;
  const int n = lane & 15, g = lane >> 4;
  const int G = a.Hq / a.Hkv;
  const int upp = a.page_size / kUnit;

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
  at_bf16x8 q[NT][4];
  float slope2[NT];
  int len[NT];
  int64_t where[NT];  // output row, -1: none
  int longest = 0, shortest = 0x7FFFFFFF;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t row = row0 + 32 * w + 16 * j + n;
    const int64_t at = min(row, rows - 1);
    const int64_t tok = t0 + at / G;
    const int hq = h * G + (int)(at % G);
    load_query(a.q + tok * a.q_stride + hq * kHeadDim, g, q[j]);
    slope2[j] = EXTRA ? slope_of(a, hq) : 0.f;
    len[j] = max(a.kv_len[tok], 0);
    where[j] = row < rows ? tok * a.Hq + hq : -1;
    longest = max(longest, len[j]);
    shortest = min(shortest, len[j]);
  }
#pragma unroll
  for (int d = 1; d < 16; d *= 2) {
    longest = max(longest, __shfl_xor(longest, d));
    shortest = min(shortest, __shfl_xor(shortest, d));
  }
  AttnState<NT> st;
  attn_init(st);

  const int64_t units = min((int64_t)pages.n * upp, ((int64_t)longest + kUnit - 1) / kUnit);
  const int64_t tiles = (units + 3) / 4;
  const int64_t end = min(tiles, (int64_t)(split + 1) * chunk);
  for (int64_t t = (int64_t)split * chunk; t < end; ++t) {
    const int64_t ku = 4 * t + (n >> 2), vu = 4 * t + g;
    const int kblk = ku < units ? block_of(a, pages, (int)(ku / upp), h) : -1;
    const int vblk = vu < units ? block_of(a, pages, (int)(vu / upp), h) : -1;
    const int pos = vblk < 0 ? 0 : (int)vu * kUnit;
    const int have = vblk < 0 ? 0 : min(longest - pos, kUnit);
    const float ks = vblk < 0 ? 0.f : a.k_scale[vblk] * a.score_scale;
    const float vs = vblk < 0 ? 0.f : a.v_scale[vblk];
    uint4 k[4][2], v[8];
    load_tile(a, kblk, (int)(ku % upp), vblk, (int)(vu % upp), n, g, k, v);
    const bool any = !__all(have == kUnit && pos + kUnit <= shortest);
    if (any) {
#pragma unroll
      for (int dt = 0; dt < 8; ++dt) v[dt] = keep_tokens(v[dt], have);
      attn_nan_values<NT>(st, v, pos, have, len);
    }
    attn_tile<NT, EXTRA>(st, q, k, v, ks, vs, pos, have, len, slope2, a.softcap, any);
  }

#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const float l = groups_sum(st.l[j]);
    if (where[j] < 0) continue;
    if (splits == 1) {
      const float inv = l == 0.f ? 0.f : st.vref / l;
      uint16_t* o = a.out + where[j] * kHeadDim;
#pragma unroll
      for (int dt = 0; dt < 8; ++dt) {
        const at_f32x4 x = st.o[j][dt];
        *reinterpret_cast<uint2*>(o + 16 * dt + 4 * g) =
            make_uint2(pack_bf16(x[0] * inv, x[1] * inv), pack_bf16(x[2] * inv, x[3] * inv));
      }
    } else {
      const int64_t tok = where[j] / a.Hq;
      const int row = (int)(where[j] % a.Hq) % G;
      const int64_t part = (((tok * a.Hkv + h) * splits) + split) * G + row;
#pragma unroll
      for (int dt = 0; dt < 8; ++dt)
        *reinterpret_cast<at_f32x4*>(a.part_o + part * kHeadDim + 16 * dt + 4 * g) =
            st.o[j][dt] * st.vref;
      if (g == 0) {
        a.part_ml[2 * part] = st.m[j];
        a.part_ml[2 * part + 1] = l;
      }
    }
  }
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

AttnSplit attend_prefill_split(int64_t n_tok, int B, int Hq, int Hkv, int64_t units) {
  const int64_t tiles = (units + 3) / 4;
  const int64_t groups = attend_prefill_tiles(n_tok, B, Hq / Hkv) * Hkv;
  int64_t splits = (512 + groups - 1) / groups;
  splits = splits < tiles / 8 ? splits : tiles / 8;
  if (splits < 1) splits = 1;
  const int64_t chunk = (tiles + splits - 1) / splits;
  return {(int)chunk, (int)((tiles + chunk - 1) / chunk)};
}

int64_t attend_prefill_tiles(int64_t n_tok, int B, int G) { return n_tok * G / kPreRows + B; }

static int launch_merge(const AttnArgs& a, int64_t rows, int splits, hipStream_t s) {
  const int64_t grid = (rows * a.Hq + kAtWaves - 1) / kAtWaves;
  hipLaunchKernelGGL(attend_merge_kernel, dim3((unsigned)grid), dim3(kAtNT), 0, s, a, rows,
                     splits);
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
  if (e == 0 && sp.splits > 1) e = launch_merge(a, a.R, sp.splits, s);
  return e;
}

int launch_attend_prefill(const AttnArgs& a, AttnSplit sp, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool extra = a.softcap > 0.f || a.slopes != nullptr;
  const int64_t tiles = attend_prefill_tiles(a.R, a.B, a.Hq / a.Hkv);
  const dim3 grid((unsigned)(tiles * a.Hkv * sp.splits)), blk(kAtNT);
#define IDX_PRE(EX) \
  hipLaunchKernelGGL((attend_prefill_kernel<EX>), grid, blk, 0, s, a, sp.chunk, sp.splits)
  if (extra) IDX_PRE(true); else IDX_PRE(false);
#undef IDX_PRE
  int e = (int)hipGetLastError();
  if (e == 0 && sp.splits > 1) e = launch_merge(a, a.R, sp.splits, s);
  return e;
}

}  // namespace idxk
