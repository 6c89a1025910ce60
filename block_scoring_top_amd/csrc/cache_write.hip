// Quantising write of new keys and values into the paged 8-bit cache
// (include/idx_cache.h, idx_cache_write).
//
//   s = 2^k, the smallest with amax <= 448 s:  with amax = m 2^e, m in [0.5, 1),
//   and 448 = 0.875 * 2^9, k = e - 9 if m <= 0.875, else e - 8.
// Codes are e4m3(x / s), rounded to nearest even by the conversion instruction;
// |x / s| <= 448, so nothing saturates but an infinite x.
//
// A stream, bound by its bytes (prompts) or its chain of loads (single tokens). A wave
// quantises the keys or values of one page's tokens, a run of consecutive rows, for one KV
// head: lane = (four consecutive page offsets, 8 dims), so that a token's row is read and
// its key written in whole lines, the run's largest value takes one reduction over the
// wave, and the four tokens of a lane are one word of the transposed value page, in
// registers. Everything is read once: the run waits in registers for its scale.
// 56800 tokens of 8 heads (bf16, 349 MB in and out): 81 us, 4.3 TB/s (a large copy runs at
// 4.9); 4009 of them 10.3 us, a chain of loads, and 55 with a workgroup for each row and
// head that reads its elements twice; 128 single tokens of 4 heads 6.0 us.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "launch.h"

namespace idxk {

namespace {

constexpr int kWrNT = 256;
constexpr int kWrWaves = kWrNT / kWave;
constexpr float kE4M3Max = 448.f;

// the smallest power of two >= 2^IDX_CACHE_MIN_EXP with amax <= 448 s
__device__ __forceinline__ float scale_of(float amax) {
  int e;
  const float m = frexpf(amax, &e);
  int k = e - (m <= 0.875f ? 9 : 8);
  if (!(amax > 0.f) || k < -120) k = -120;
  return __uint_as_float((uint32_t)(k + 127) << 23);
}

__device__ __forceinline__ float clamp_e4m3(float x) {
  return x > kE4M3Max ? kE4M3Max : x < -kE4M3Max ? -kE4M3Max : x;  // NaN passes
}
// four values' codes in one word
__device__ __forceinline__ uint32_t codes_of(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(a), clamp_e4m3(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(c), clamp_e4m3(d), lo, true);
}
// four codes times f, as codes
__device__ __forceinline__ uint32_t rescaled(uint32_t w, float f) {
  return codes_of(__builtin_amdgcn_cvt_f32_fp8((int)w, 0) * f,
                  __builtin_amdgcn_cvt_f32_fp8((int)w, 1) * f,
                  __builtin_amdgcn_cvt_f32_fp8((int)w, 2) * f,
                  __builtin_amdgcn_cvt_f32_fp8((int)w, 3) * f);
}

// 8 values of a row, and the largest finite magnitude among them
template <bool BF16>
struct Eight {
  uint4 w[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const uint4* q = reinterpret_cast<const uint4*>(
        static_cast<const char*>(p) + i * (BF16 ? sizeof(uint16_t) : sizeof(float)));
    w[0] = q[0];
    if constexpr (!BF16) w[1] = q[1];
  }
  __device__ __forceinline__ float get(int e) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
    if constexpr (BF16) return (e & 1) ? bf16_hi(u[e >> 1]) : bf16_lo(u[e >> 1]);
    return __uint_as_float(u[e]);
  }
};

template <bool BF16, int PAGE>
__global__ __launch_bounds__(kWrNT) void cache_write_kernel(
    const void* __restrict__ k, const void* __restrict__ v, int64_t k_stride, int64_t v_stride,
    const int32_t* __restrict__ slots, uint8_t* __restrict__ k_cache,
    uint8_t* __restrict__ v_cache, float* __restrict__ k_scale, float* __restrict__ v_scale,
    int n_tok, int Hkv, int64_t n_slots, int span, int item_groups) {
  constexpr int PASSES = PAGE / 16;  // a wave holds 16 tokens a pass
  const int lane = lane_id();
  const int item = (blockIdx.x % item_groups) * kWrWaves +
                   __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int h = item >> 1;
  const bool keys = (item & 1) == 0;  // a wave for a head's keys, one for its values
  const int t0 = (blockIdx.x / item_groups) * span;
  if (h >= Hkv) return;
  const void* src = keys ? k : v;
  const int64_t stride = keys ? k_stride : v_stride;
  const int dim = 8 * (lane & 15), quad = lane >> 4;

  // Which rows from t0 on follow their predecessor in its page: one bit a row, for the
  // span and the longest run behind it.
  auto follows = [&](int i) {  // also whether row t0 + i has a slot
    const int t = t0 + i;
    const int s = t < n_tok ? slots[t] : -1, before = t < n_tok && t > 0 ? slots[t - 1] : -1;
    return make_int2(s >= 0 && s < n_slots, s % PAGE > 0 && before == s - 1);
  };
  const int2 mine = follows(lane);
  const uint64_t cont = ballot(mine.y != 0);
  uint64_t more = 0;  // rows 64.. of a span of several rows
  if (PAGE > 16 && span > 1) more = ballot(lane < PAGE && follows(kWave + lane).y != 0);
  for (uint64_t left = ballot(lane < span && mine.x != 0 && mine.y == 0); left != 0;
       left &= left - 1) {
    const int j = __builtin_ctzll(left), t = t0 + j;
    const int slot = __builtin_amdgcn_readfirstlane(slots[t]);
    const int first = slot % PAGE;
    const int page = slot / PAGE;
    // the bits behind j: a run ends where the page does, so 63 are enough
    const uint64_t bits = ((cont >> j) >> 1) | (j > 0 ? more << (63 - j) : 0);
    const int n = 1 + __builtin_ctzll(~bits | (1ull << 63));
    const int64_t blk = (int64_t)page * Hkv + h;
    const int64_t base = blk * (PAGE * kHeadDim);

    // offset o of the page is row t + o - first of the call
    uint8_t* cache = (keys ? k_cache : v_cache) + base;
    float* scale = (keys ? k_scale : v_scale) + blk;
    const float old = first > 0 ? *scale : 0.f;
    Eight<BF16> x[PASSES][4];
    float amax = 0.f;
#pragma unroll
    for (int p = 0; p < PASSES; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int o = 16 * p + 4 * quad + i;
        if (o >= first && o < first + n)
          x[p][i].load(src, (t + o - first) * stride + (int64_t)h * kHeadDim + dim);
      }
#pragma unroll
    for (int p = 0; p < PASSES; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int o = 16 * p + 4 * quad + i;
        if (o >= first && o < first + n)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float m = fabsf(x[p][i].get(e));
            if (m < __builtin_inff()) amax = fmaxf(amax, m);
          }
      }
    // (non-negative floats are in the order of their bits)
    float s = scale_of(__uint_as_float(wave_reduce_minmax<false>(__float_as_uint(amax))));
    if (first > 0) {
      s = fmaxf(s, old);
      if (s != old) {  // the page's earlier tokens move to the larger scale
        const float f = old / s;
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
          const int o = 16 * p + 4 * quad;
          if (keys) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (o + i < first) {
                uint2* w = reinterpret_cast<uint2*>(cache + (o + i) * kHeadDim + dim);
                *w = make_uint2(rescaled(w->x, f), rescaled(w->y, f));
              }
          } else if (o < first) {
            // bytes from `first` on keep their codes
            const uint32_t mine = first - o >= 4 ? ~0u : (1u << (8 * (first - o))) - 1;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              uint32_t* w = reinterpret_cast<uint32_t*>(cache + (dim + e) * PAGE + o);
              *w = (rescaled(*w, f) & mine) | (*w & ~mine);
            }
          }
        }
      }
    }
    auto write = [&](auto over) {
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int o = 16 * p + 4 * quad;
        if (keys) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (o + i >= first && o + i < first + n) {
              float y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = over(x[p][i].get(e));
              *reinterpret_cast<uint2*>(cache + (o + i) * kHeadDim + dim) =
                  make_uint2(codes_of(y[0], y[1], y[2], y[3]), codes_of(y[4], y[5], y[6], y[7]));
            }
        } else if (o + 4 > first && o < first + n) {
          const bool whole = o >= first && o + 4 <= first + n;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t w = codes_of(over(x[p][0].get(e)), over(x[p][1].get(e)),
                                        over(x[p][2].get(e)), over(x[p][3].get(e)));
            uint8_t* to = cache + (dim + e) * PAGE + o;
            if (whole) {
              *reinterpret_cast<uint32_t*>(to) = w;
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (o + i >= first && o + i < first + n) to[i] = (uint8_t)(w >> (8 * i));
            }
          }
        }
      }
    };
    // a power of two (all but calibrated scales that are kept): its inverse is exact, and a
    // division is a dozen instructions
    if ((__float_as_uint(s) & 0x007FFFFFu) == 0) {
      const float inv = 1.f / s;
      write([&](float y) { return y * inv; });
    } else {
      write([&](float y) { return y / s; });
    }
    if (lane == 0) *scale = s;
  }
}

}  // namespace

int launch_cache_write(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                       const int32_t* slots, uint8_t* k_cache, uint8_t* v_cache, float* k_scale,
                       float* v_scale, int n_tok, int Hkv, int n_pages, int page_size, bool bf16,
                       void* stream) {
  // prompts: a wave looks for runs among 16 rows (the 56800 tokens: 81 us, 97 with 8 rows,
  // 295 with one, 84 with 32); a few tokens: a wave for each row
  const int item_groups = (2 * Hkv + kWrWaves - 1) / kWrWaves;
  const int span = (int64_t)n_tok * item_groups > 8192 ? 16 : 1;
  const int64_t grid = (int64_t)((n_tok + span - 1) / span) * item_groups;
  if (grid > 0x7FFFFFFF) return (int)hipErrorInvalidConfiguration;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t n_slots = (int64_t)n_pages * page_size;
#define IDX_WRITE(BF, PAGE)                                                                    \
  hipLaunchKernelGGL((cache_write_kernel<BF, PAGE>), dim3((unsigned)grid), dim3(kWrNT), 0, s,  \
                     k, v, k_stride, v_stride, slots, k_cache, v_cache, k_scale, v_scale,      \
                     n_tok, Hkv, n_slots, span, item_groups)
  if (page_size == 16) {
    if (bf16) IDX_WRITE(true, 16); else IDX_WRITE(false, 16);
  } else if (page_size == 32) {
    if (bf16) IDX_WRITE(true, 32); else IDX_WRITE(false, 32);
  } else {
    if (bf16) IDX_WRITE(true, 64); else IDX_WRITE(false, 64);
  }
#undef IDX_WRITE
  return (int)hipGetLastError();
}

}  // namespace idxk
