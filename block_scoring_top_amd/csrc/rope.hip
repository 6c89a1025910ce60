// Rotary positions (include/idx_rope.h, idx_rope).
//
// A pair's angle in turns is p * T / 2^64, T the table's whole number: the low 64 bits of the
// product are its fraction, exact. The nearest quarter turn goes to the quadrant, what is
// left, at most an eighth of a turn, to the Taylor series of sine and cosine in fp32 (their
// next terms are 2^-29 and 2^-33 there).
//
// A stream: every element is read and written once. A workgroup has a token: a thread works
// the angle of one pair out, once for all heads, and leaves sine and cosine in LDS; then 8
// lanes take a head's row, 16 elements each: 8 pairs, or 16 elements that pass unchanged (four
// tokens a workgroup: 16384 tokens 69.8 us, 64.6 so). 16200 tokens of 32 + 8
// heads in bf16, 332 MB in and out: 61 us, 5.5 TB/s (a large copy runs at 4.9); 4100 tokens
// of 16 + 2 in fp32 17 us, 4.4 TB/s; 128 tokens of 16 + 4 3.2 us, a launch and two loads
// behind each other.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "launch.h"

namespace idxk {

namespace {

constexpr int kRopeNT = 256;
constexpr int kRopePairs = kHeadDim / 2;

typedef __bf16 rp_bf16x2 __attribute__((ext_vector_type(2)));
typedef float rp_f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  rp_f32x2 f = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, rp_bf16x2));
}

template <bool BF16>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&x)[8]) {
  if constexpr (BF16) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = bf16_lo(u[e]);
      x[2 * e + 1] = bf16_hi(u[e]);
    }
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = q[0], b = q[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
}
template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&x)[8]) {
  if constexpr (BF16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
  } else {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(x[0], x[1], x[2], x[3]);
    q[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// cosine and sine of p * turns / 2^64 turns
__device__ __forceinline__ float2 cos_sin(int p, uint64_t turns) {
  const uint64_t at = (uint64_t)(int64_t)p * turns;
  const uint32_t quadrant = (uint32_t)((at + (1ull << 61)) >> 62);
  const int64_t rest = (int64_t)(at - ((uint64_t)quadrant << 62));  // at most 2^61 in size
  // in radians: 2 pi / 2^64 a unit
  const float hi = (float)(int32_t)(rest >> 32), lo = (float)(uint32_t)rest;
  const float y = __builtin_fmaf(lo, 0x1p-32f, hi) * (6.283185307179586f * 0x1p-32f);
  const float z = y * y;
  float s = __builtin_fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
  s = __builtin_fmaf(z, s, 1.f / 120.f);
  s = __builtin_fmaf(z, s, -1.f / 6.f);
  s = __builtin_fmaf(z * y, s, y);
  float c = __builtin_fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
  c = __builtin_fmaf(z, c, -1.f / 720.f);
  c = __builtin_fmaf(z, c, 1.f / 24.f);
  c = __builtin_fmaf(z, c, -0.5f);
  c = __builtin_fmaf(z, c, 1.f);
  const float a = (quadrant & 1) ? s : c, b = (quadrant & 1) ? c : s;
  return make_float2((quadrant == 1 || quadrant == 2) ? -a : a, (quadrant & 2) ? -b : b);
}

template <bool BF16>
__global__ __launch_bounds__(kRopeNT) void rope_kernel(RopeArgs a, bool copy_q, bool copy_k) {
  __shared__ __attribute__((aligned(16))) float2 s_cs[kRopePairs];
  const int tid = threadIdx.x;
  const int64_t tok = blockIdx.x;
  const int pairs = a.rot / 2, len = a.tok_len[tok];
  if (len <= 0) return;
  if (tid < pairs) {
    float2 cs = cos_sin(len - 1, a.turns[tid]);
    cs.x *= a.factor;
    cs.y *= a.inverse ? -a.factor : a.factor;
    s_cs[tid] = cs;
  }
  __syncthreads();
  const int heads = a.Hq + a.Hkv;
  const int j = tid & 7;  // of the 8 lanes of a row
  for (int row = tid >> 3; row < heads; row += kRopeNT / 8) {
    const bool is_q = row < a.Hq;
    const int h = is_q ? row : row - a.Hq;
    const void* src = is_q ? a.q : a.k;
    void* dst = is_q ? a.q_out : a.k_out;
    const int64_t from = tok * (is_q ? a.q_stride : a.k_stride) + h * kHeadDim;
    const int64_t to = tok * (is_q ? a.q_out_stride : a.k_out_stride) + h * kHeadDim;
    float x[8], y[8];
    if (16 * j < a.rot) {
      float u[8], w[8];
      const float2* cs = &s_cs[8 * j];
      if (a.adjacent) {
        const int d = a.first + 16 * j;
        load8<BF16>(src, from + d, x);
        load8<BF16>(src, from + d + 8, y);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          u[2 * e] = x[2 * e] * cs[e].x - x[2 * e + 1] * cs[e].y;
          u[2 * e + 1] = x[2 * e + 1] * cs[e].x + x[2 * e] * cs[e].y;
          w[2 * e] = y[2 * e] * cs[e + 4].x - y[2 * e + 1] * cs[e + 4].y;
          w[2 * e + 1] = y[2 * e + 1] * cs[e + 4].x + y[2 * e] * cs[e + 4].y;
        }
        store8<BF16>(dst, to + d, u);
        store8<BF16>(dst, to + d + 8, w);
      } else {
        const int d = a.first + 8 * j;
        load8<BF16>(src, from + d, x);
        load8<BF16>(src, from + d + pairs, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          u[e] = x[e] * cs[e].x - y[e] * cs[e].y;
          w[e] = y[e] * cs[e].x + x[e] * cs[e].y;
        }
        store8<BF16>(dst, to + d, u);
        store8<BF16>(dst, to + d + pairs, w);
      }
    } else if (is_q ? copy_q : copy_k) {
      // the dims beside the rotated part, in two runs of 8, as they are
      int d = 16 * j - a.rot, e = d + 8;
      d += d < a.first ? 0 : a.rot;
      e += e < a.first ? 0 : a.rot;
      if constexpr (BF16) {  // (a conversion to float and back would quieten NaN)
        const uint16_t* p = static_cast<const uint16_t*>(src) + from;
        uint16_t* q = static_cast<uint16_t*>(dst) + to;
        const uint4 u = *reinterpret_cast<const uint4*>(p + d);
        const uint4 w = *reinterpret_cast<const uint4*>(p + e);
        *reinterpret_cast<uint4*>(q + d) = u;
        *reinterpret_cast<uint4*>(q + e) = w;
      } else {
        load8<BF16>(src, from + d, x);
        load8<BF16>(src, from + e, y);
        store8<BF16>(dst, to + d, x);
        store8<BF16>(dst, to + e, y);
      }
    }
  }
}

}  // namespace

int launch_rope(const RopeArgs& a, bool bf16, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool copy_q = a.q_out != a.q, copy_k = a.k_out != a.k;
  const dim3 grid((unsigned)a.n_tok), blk(kRopeNT);
  if (bf16)
    hipLaunchKernelGGL((rope_kernel<true>), grid, blk, 0, s, a, copy_q, copy_k);
  else
    hipLaunchKernelGGL((rope_kernel<false>), grid, blk, 0, s, a, copy_q, copy_k);
  return (int)hipGetLastError();
}

}  // namespace idxk
