// Quantising write of new keys and values into the paged 8-bit cache
// (include/idx_cache.h, idx_cache_write).
//
//   s = 2^k, the smallest with amax <= 448 s:  with amax = m 2^e, m in [0.5, 1),
//   and 448 = 0.875 * 2^9, k = e - 9 if m <= 0.875, else e - 8.
// Codes are e4m3(x / s), rounded to nearest even by the conversion instruction;
// |x / s| <= 448, so nothing saturates but an infinite x.
//
// One workgroup per token row and KV head; the rows that do not start a page's
// run of tokens leave at once, the others quantise the whole run: a thread owns
// one of the 128 dims of all its tokens.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "launch.h"

namespace idxk {

namespace {

constexpr int kWrNT = kHeadDim;
constexpr float kE4M3Max = 448.f;

template <bool BF16>
__device__ __forceinline__ float load_elem(const void* p, int64_t i) {
  if constexpr (BF16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  return static_cast<const float*>(p)[i];
}

// the smallest power of two >= 2^IDX_CACHE_MIN_EXP with amax <= 448 s
__device__ __forceinline__ float scale_of(float amax) {
  int e;
  const float m = frexpf(amax, &e);
  int k = e - (m <= 0.875f ? 9 : 8);
  if (!(amax > 0.f) || k < -120) k = -120;
  return __uint_as_float((uint32_t)(k + 127) << 23);
}

__device__ __forceinline__ uint8_t to_e4m3(float x) {
  x = x > kE4M3Max ? kE4M3Max : x < -kE4M3Max ? -kE4M3Max : x;  // NaN passes
  return (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(x, x, 0, false);
}

__device__ __forceinline__ float from_e4m3(uint8_t c) {
  return __builtin_amdgcn_cvt_f32_fp8((int)c, 0);
}

// largest value over the workgroup's 128 threads
__device__ __forceinline__ float block_max(float v, float* lds) {
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) v = fmaxf(v, __shfl_xor(v, d));
  __syncthreads();
  if ((threadIdx.x & (kWave - 1)) == 0) lds[threadIdx.x / kWave] = v;
  __syncthreads();
  return fmaxf(lds[0], lds[1]);
}

template <bool BF16>
__global__ __launch_bounds__(kWrNT) void cache_write_kernel(
    const void* __restrict__ k, const void* __restrict__ v, int64_t k_stride, int64_t v_stride,
    const int32_t* __restrict__ slots, uint8_t* __restrict__ k_cache,
    uint8_t* __restrict__ v_cache, float* __restrict__ k_scale, float* __restrict__ v_scale,
    int n_tok, int Hkv, int64_t n_slots, int page_size) {
  __shared__ float lds[2];
  const int t = blockIdx.x / Hkv, h = blockIdx.x - t * Hkv;
  const int d = threadIdx.x;
  const int slot = slots[t];
  if (slot < 0 || slot >= n_slots) return;
  const int first = slot % page_size;
  if (t > 0 && first > 0 && slots[t - 1] == slot - 1) return;  // inside a run
  const int page = slot / page_size;
  int n = 1;
  while (first + n < page_size && t + n < n_tok && slots[t + n] == slot + n) ++n;

  const int64_t blk = (int64_t)page * Hkv + h;
  const int64_t base = blk * page_size * kHeadDim;
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    const bool keys = pass == 0;
    const void* src = keys ? k : v;
    const int64_t stride = keys ? k_stride : v_stride;
    uint8_t* cache = (keys ? k_cache : v_cache) + base;
    float* scale = (keys ? k_scale : v_scale) + blk;
    // a token's code at this dim: keys are rows, values are columns
    const int64_t at0 = keys ? d : (int64_t)d * page_size;
    const int64_t step = keys ? kHeadDim : 1;
    float amax = 0.f;
    for (int i = 0; i < n; ++i) {
      const float a =
          fabsf(load_elem<BF16>(src, (t + i) * stride + (int64_t)h * kHeadDim + d));
      if (a < __builtin_inff()) amax = fmaxf(amax, a);
    }
    float s = scale_of(block_max(amax, lds));
    if (first > 0) {
      const float old = *scale;
      s = fmaxf(s, old);
      if (s != old) {
        const float f = old / s;
        for (int i = 0; i < first; ++i)
          cache[at0 + i * step] = to_e4m3(from_e4m3(cache[at0 + i * step]) * f);
      }
      __syncthreads();  // the old scale has been read
    }
    for (int i = 0; i < n; ++i) {
      const float x = load_elem<BF16>(src, (t + i) * stride + (int64_t)h * kHeadDim + d);
      cache[at0 + (first + i) * step] = to_e4m3(x / s);
    }
    if (d == 0) *scale = s;
  }
}

}  // namespace

int launch_cache_write(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                       const int32_t* slots, uint8_t* k_cache, uint8_t* v_cache, float* k_scale,
                       float* v_scale, int n_tok, int Hkv, int n_pages, int page_size, bool bf16,
                       void* stream) {
  const int64_t grid = (int64_t)n_tok * Hkv;
  if (grid > 0x7FFFFFFF) return (int)hipErrorInvalidConfiguration;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t n_slots = (int64_t)n_pages * page_size;
#define IDX_WRITE(BF)                                                                           \
  hipLaunchKernelGGL((cache_write_kernel<BF>), dim3((unsigned)grid), dim3(kWrNT), 0, s, k, v,   \
                     k_stride, v_stride, slots, k_cache, v_cache, k_scale, v_scale, n_tok, Hkv, \
                     n_slots, page_size)
  if (bf16) IDX_WRITE(true); else IDX_WRITE(false);
#undef IDX_WRITE
  return (int)hipGetLastError();
}

}  // namespace idxk
