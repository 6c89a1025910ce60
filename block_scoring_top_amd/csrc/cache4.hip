// The paged 4-bit cache's write and its reading back (include/idx_cache4.h,
// idx_cache4_write, idx_cache4_read).
//
//   s = 2^e, the smallest with amax <= 6 s: with amax = f 2^a, f in [1, 2), and
//   6 = 1.5 * 2^2, e = a - 2 if f <= 1.5, else a - 1.
// The magnitudes' bits order zero, finite values, infinity and NaN as integers, so one
// integer maximum over a block gives its scale byte and tells whether it holds a NaN.
// Codes are e2m1(x / s), rounded to nearest even and saturating, by the conversion
// instruction, whose scale operand is s itself.
//
// Streams, bound by their bytes (prompts) or a chain of loads (single tokens). A wave takes
// the keys or the values of one unit, up to 16 consecutive tokens of a page, for one KV head:
// lane = (four consecutive offsets, 8 dims), so that a token's row is read or written in
// whole lines and a block's maximum takes two lane moves. The values' columns come out of a
// transposition of 4 x 4 words between the wave's quarters, in registers: a lane then holds
// the 16 tokens of two dims, 16 bytes, and a unit's 1 KB is written (read) in one go where
// the page is the unit. 16396 tokens of 8 heads (bf16, 88 MB in and out): written in 13.5 us,
// read back in 12 (inputs partly in the last-level cache); 63280 read in 62, 5.3 TB/s (a
// large copy runs at 4.9); 128 single tokens of 4 heads 4.3 and 3.2 us.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "launch.h"

namespace idxk {

namespace {

constexpr int kC4NT = 256;
constexpr int kC4Waves = kC4NT / kWave;
constexpr int kC4Unit = 16;  // tokens
constexpr int kMinByte = 127 - 60, kMaxByte = 127 + 60;  // of the scales written

typedef __bf16 c4_bf16x2 __attribute__((ext_vector_type(2)));
typedef float c4_f32x2 __attribute__((ext_vector_type(2)));

// 8 consecutive values of a row
template <bool BF16>
struct Row8 {
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

// the scale byte of a block whose largest magnitude has the bits m
__device__ __forceinline__ uint32_t scale_byte(uint32_t m) {
  if (m > 0x7F800000u) return 255;
  const int b = (int)(m >> 23) - 2 + ((m & 0x007FFFFFu) > 0x00400000u ? 1 : 0);
  return (uint32_t)min(max(b, kMinByte), kMaxByte);
}
// eight codes in one word
template <bool BF16>
__device__ __forceinline__ uint32_t codes8(const Row8<BF16>& x, float s) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x.get(0), x.get(1), s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x.get(2), x.get(3), s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x.get(4), x.get(5), s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x.get(6), x.get(7), s, 3);
}

// w[j] of quarter q becomes w[q] of quarter j
__device__ __forceinline__ void transpose_quarters(uint32_t (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto r = __builtin_amdgcn_permlane32_swap(w[i], w[i + 2], false, false);
    w[i] = r[0];
    w[i + 2] = r[1];
  }
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const auto r = __builtin_amdgcn_permlane16_swap(w[i], w[i + 1], false, false);
    w[i] = r[0];
    w[i + 1] = r[1];
  }
}
// the low (high) halves of two words
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x05040100u);
}
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}
// 4 x 4 codes: v[i] holds token i's code of the dims 0..7, four bits each; out: for each
// pair of dims (2 p, 2 p + 1) the four tokens' codes of both, 16 bits each
__device__ __forceinline__ void codes_to_columns(const uint32_t (&v)[4], uint32_t (&w)[4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    uint32_t even = 0, odd = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      even |= ((v[i] >> (8 * p)) & 15u) << (4 * i);
      odd |= ((v[i] >> (8 * p + 4)) & 15u) << (4 * i);
    }
    w[p] = even | (odd << 16);
  }
}
__device__ __forceinline__ void columns_to_codes(const uint32_t (&w)[4], uint32_t (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t x = 0;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      x |= ((w[p] >> (4 * i)) & 15u) << (8 * p);
      x |= ((w[p] >> (16 + 4 * i)) & 15u) << (8 * p + 4);
    }
    v[i] = x;
  }
}
// the bits of the tokens first .. first + n of 16, four bits each
__device__ __forceinline__ uint64_t token_bits(int first, int n) {
  const uint64_t upto = first + n >= 16 ? ~0ull : (1ull << (4 * (first + n))) - 1;
  return upto & ~((1ull << (4 * first)) - 1);
}
// Those bits of a word. The others may be another wave's at the same time (tokens of a page
// in rows apart): each flips its own, which nobody else writes, from what they were. (2048
// tokens in as many pages, 8 heads: 25 us, 45 with an `and` and an `or`.)
__device__ __forceinline__ void put_bits(uint8_t* p, uint32_t w, uint32_t mine) {
  uint32_t* q = reinterpret_cast<uint32_t*>(p);
  if (mine == 0) return;
  if (mine == ~0u) {
    *q = w;
    return;
  }
  const uint32_t flip = (*q ^ w) & mine;
  if (flip != 0) __hip_atomic_fetch_xor(q, flip, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Which of the rows from t0 on follow their predecessor in its unit, and which of the
// first `span` lead a run: bits of the wave.
struct Runs {
  uint64_t follow, lead, absent;
};
__device__ __forceinline__ Runs runs_of(const int32_t* slots, int t0, int n_tok, int64_t n_slots,
                                        int span) {
  const int lane = lane_id(), t = t0 + lane;
  const int s = t < n_tok ? slots[t] : -1;
  const int before = t < n_tok && t > 0 ? slots[t - 1] : -1;
  const bool there = s >= 0 && s < n_slots;
  const bool follow = there && s % kC4Unit > 0 && before == s - 1;
  const bool mine = lane < span && t < n_tok;
  return {ballot(follow), ballot(mine && there && !follow), ballot(mine && !there)};
}

template <bool BF16>
__global__ __launch_bounds__(kC4NT) void cache4_write_kernel(
    const void* __restrict__ k, const void* __restrict__ v, int64_t k_stride, int64_t v_stride,
    const int32_t* __restrict__ slots, uint8_t* __restrict__ k_cache,
    uint8_t* __restrict__ v_cache, uint8_t* __restrict__ k_scale, uint8_t* __restrict__ v_scale,
    int n_tok, int Hkv, int64_t n_slots, int page_size, int span, int item_groups) {
  const int lane = lane_id();
  const int item = (blockIdx.x % item_groups) * kC4Waves +
                   __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int h = item >> 1;
  const bool keys = (item & 1) == 0;  // a wave for a head's keys, one for its values
  const int t0 = (blockIdx.x / item_groups) * span;
  if (h >= Hkv) return;
  const void* src = keys ? k : v;
  const int64_t stride = keys ? k_stride : v_stride;
  const int c = lane & 15, quad = lane >> 4;  // dims 8 c .., tokens 4 quad .. of the unit

  const Runs runs = runs_of(slots, t0, n_tok, n_slots, span);
  for (uint64_t left = runs.lead; left != 0; left &= left - 1) {
    const int j = __builtin_ctzll(left), t = t0 + j;
    const int slot = __builtin_amdgcn_readfirstlane(slots[t]);
    const int at = slot % page_size, first = slot % kC4Unit;
    const int64_t blk = (int64_t)(slot / page_size) * Hkv + h;
    // (a run is at most 16 rows, and leads are among the first 16 of 64)
    const int n = 1 + __builtin_ctzll(~((runs.follow >> j) >> 1));
    const int unit = at - first;  // the unit's first offset in its page

    Row8<BF16> x[4];
    uint32_t byte[4], code[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int o = 4 * quad + i;
#pragma unroll
      for (auto& w : x[i].w) w = make_uint4(0, 0, 0, 0);
      if (o >= first && o < first + n)
        x[i].load(src, (t + o - first) * stride + (int64_t)h * kHeadDim + 8 * c);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[i].get(e)) & 0x7FFFFFFFu);
      m = max(m, lane_xor<1>(m));
      m = max(m, lane_xor<2>(m));  // the block's four lanes
      byte[i] = scale_byte(m);
      code[i] = codes8(x[i], __uint_as_float(byte[i] << 23));
    }
    if (keys) {
      const int64_t row = blk * page_size + unit;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int o = 4 * quad + i;
        if (o < first || o >= first + n) continue;
        reinterpret_cast<uint32_t*>(k_cache + (row + o) * (kHeadDim / 2))[c] = code[i];
        if ((c & 3) == 0) k_scale[(row + o) * 4 + (c >> 2)] = (uint8_t)byte[i];
      }
      continue;
    }
    uint32_t w[4];
    codes_to_columns(code, w);
    transpose_quarters(w);
    // this lane's dims 8 c + 2 quad, and the next: 16 tokens of four bits each
    const int64_t half = page_size / 2;
    uint8_t* col = v_cache + blk * kHeadDim * half + (8 * c + 2 * quad) * half + unit / 2;
    const uint2 even = make_uint2(low_halves(w[0], w[1]), low_halves(w[2], w[3]));
    const uint2 odd = make_uint2(high_halves(w[0], w[1]), high_halves(w[2], w[3]));
    if (n == kC4Unit) {
      *reinterpret_cast<uint2*>(col) = even;
      *reinterpret_cast<uint2*>(col + half) = odd;
    } else {
      const uint64_t mine = token_bits(first, n);
      put_bits(col, even.x, (uint32_t)mine);
      put_bits(col + 4, even.y, (uint32_t)(mine >> 32));
      put_bits(col + half, odd.x, (uint32_t)mine);
      put_bits(col + half + 4, odd.y, (uint32_t)(mine >> 32));
    }
    if ((c & 3) == 0) {
      uint8_t* s = v_scale + (blk * 4 + (c >> 2)) * page_size + unit + 4 * quad;
      if (4 * quad >= first && 4 * quad + 4 <= first + n) {
        *reinterpret_cast<uint32_t*>(s) =
            byte[0] | (byte[1] << 8) | (byte[2] << 16) | (byte[3] << 24);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * quad + i >= first && 4 * quad + i < first + n) s[i] = (uint8_t)byte[i];
      }
    }
  }
}

// eight codes' values, times the scale, as a row's 8 values
template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t i, uint32_t code, uint32_t byte) {
  const float s = __uint_as_float(byte << 23);
  if constexpr (BF16) {
    auto two = [&](auto r) { return __builtin_bit_cast(uint32_t, r); };
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, s, 0)),
                   two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, s, 1)),
                   two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, s, 2)),
                   two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, s, 3)));
  } else {
    const c4_f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, s, 0);
    const c4_f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, s, 1);
    const c4_f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, s, 2);
    const c4_f32x2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, s, 3);
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(a[0], a[1], b[0], b[1]);
    q[1] = make_float4(d[0], d[1], e[0], e[1]);
  }
}

template <bool BF16>
__global__ __launch_bounds__(kC4NT) void cache4_read_kernel(
    const int32_t* __restrict__ slots, const uint8_t* __restrict__ k_cache,
    const uint8_t* __restrict__ v_cache, const uint8_t* __restrict__ k_scale,
    const uint8_t* __restrict__ v_scale, void* __restrict__ k, void* __restrict__ v,
    int64_t k_stride, int64_t v_stride, int n_tok, int Hkv, int64_t n_slots, int page_size,
    int span, int item_groups) {
  const int lane = lane_id();
  const int item = (blockIdx.x % item_groups) * kC4Waves +
                   __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int h = item >> 1;
  const bool keys = (item & 1) == 0;
  const int t0 = (blockIdx.x / item_groups) * span;
  void* dst = keys ? k : v;
  if (h >= Hkv || dst == nullptr) return;
  const int64_t stride = keys ? k_stride : v_stride;
  const int c = lane & 15, quad = lane >> 4;

  const Runs runs = runs_of(slots, t0, n_tok, n_slots, span);
  for (uint64_t left = runs.absent; left != 0; left &= left - 1)
    if (quad == 0)
      store8<BF16>(dst, (t0 + (int64_t)__builtin_ctzll(left)) * stride + (int64_t)h * kHeadDim +
                            8 * c, 0, 127);
  for (uint64_t left = runs.lead; left != 0; left &= left - 1) {
    const int j = __builtin_ctzll(left), t = t0 + j;
    const int slot = __builtin_amdgcn_readfirstlane(slots[t]);
    const int at = slot % page_size, first = slot % kC4Unit;
    const int64_t blk = (int64_t)(slot / page_size) * Hkv + h;
    const int n = 1 + __builtin_ctzll(~((runs.follow >> j) >> 1));
    const int unit = at - first;

    uint32_t byte[4], code[4];
    if (keys) {
      const int64_t row = blk * page_size + unit;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int o = 4 * quad + i;
        code[i] = reinterpret_cast<const uint32_t*>(k_cache + (row + o) * (kHeadDim / 2))[c];
        byte[i] = k_scale[(row + o) * 4 + (c >> 2)];
      }
    } else {
      const int64_t half = page_size / 2;
      const uint8_t* col = v_cache + blk * kHeadDim * half + (8 * c + 2 * quad) * half + unit / 2;
      const uint2 lo = *reinterpret_cast<const uint2*>(col);
      const uint2 hi = *reinterpret_cast<const uint2*>(col + half);
      const uint32_t s = *reinterpret_cast<const uint32_t*>(
          v_scale + (blk * 4 + (c >> 2)) * page_size + unit + 4 * quad);
      // (the pair of dims, for each quarter's four tokens)
      uint32_t w[4] = {low_halves(lo.x, hi.x), high_halves(lo.x, hi.x), low_halves(lo.y, hi.y),
                       high_halves(lo.y, hi.y)};
      transpose_quarters(w);
      columns_to_codes(w, code);
#pragma unroll
      for (int i = 0; i < 4; ++i) byte[i] = (s >> (8 * i)) & 255u;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int o = 4 * quad + i;
      if (o >= first && o < first + n)
        store8<BF16>(dst, (t + o - first) * stride + (int64_t)h * kHeadDim + 8 * c, code[i],
                     byte[i]);
    }
  }
}

}  // namespace

// Rows that a wave looks at for runs: 16 in long calls (16384 tokens in order, 8 heads: written
// in 16 us, 36 with four rows, 78 with one), one in those of a few tokens, each perhaps in a
// page of its own, which a wave takes in turn (128 of them: 5.3 us, 22 with 16 rows).
static int span_of(int n_tok, int item_groups) {
  return (int64_t)n_tok * item_groups > 8192 ? 16 : 1;
}

int launch_cache4_write(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                        const int32_t* slots, uint8_t* k_cache, uint8_t* v_cache,
                        uint8_t* k_scale, uint8_t* v_scale, int n_tok, int Hkv, int n_pages,
                        int page_size, bool bf16, void* stream) {
  const int item_groups = (2 * Hkv + kC4Waves - 1) / kC4Waves;
  const int span = span_of(n_tok, item_groups);
  const int64_t grid = ((int64_t)n_tok + span - 1) / span * item_groups;
  if (grid > 0x7FFFFFFF) return (int)hipErrorInvalidConfiguration;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t n_slots = (int64_t)n_pages * page_size;
#define IDX_WRITE4(BF)                                                                       \
  hipLaunchKernelGGL((cache4_write_kernel<BF>), dim3((unsigned)grid), dim3(kC4NT), 0, s, k, v, \
                     k_stride, v_stride, slots, k_cache, v_cache, k_scale, v_scale, n_tok, Hkv, \
                     n_slots, page_size, span, item_groups)
  if (bf16) IDX_WRITE4(true); else IDX_WRITE4(false);
#undef IDX_WRITE4
  return (int)hipGetLastError();
}

int launch_cache4_read(const int32_t* slots, const uint8_t* k_cache, const uint8_t* v_cache,
                       const uint8_t* k_scale, const uint8_t* v_scale, void* k, void* v,
                       int64_t k_stride, int64_t v_stride, int n_tok, int Hkv, int n_pages,
                       int page_size, bool bf16, void* stream) {
  const int item_groups = (2 * Hkv + kC4Waves - 1) / kC4Waves;
  const int span = span_of(n_tok, item_groups);
  const int64_t grid = ((int64_t)n_tok + span - 1) / span * item_groups;
  if (grid > 0x7FFFFFFF) return (int)hipErrorInvalidConfiguration;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t n_slots = (int64_t)n_pages * page_size;
#define IDX_READ4(BF)                                                                          \
  hipLaunchKernelGGL((cache4_read_kernel<BF>), dim3((unsigned)grid), dim3(kC4NT), 0, s, slots, \
                     k_cache, v_cache, k_scale, v_scale, k, v, k_stride, v_stride, n_tok, Hkv, \
                     n_slots, page_size, span, item_groups)
  if (bf16) IDX_READ4(true); else IDX_READ4(false);
#undef IDX_READ4
  return (int)hipGetLastError();
}

}  // namespace idxk
