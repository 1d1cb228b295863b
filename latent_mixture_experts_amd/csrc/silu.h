// silu.h -- SwiGLU's value and the loads of rows (shared by the kernels that
// quantise rows).
#pragma once

#include "device_common.h"

namespace moe {

// silu(g) * u, silu(g) = g / (1 + exp(-g)), through the exponential and
// reciprocal instructions (1 ulp each): the exponent's rounding error, up to
// |g| * 2^-24 of the result, is taken back by its low part. The exponent stops
// just below 128. The reciprocal instruction gives zero for what lies past 2^126
// (gates below -87.3), so it takes an eighth of the sum: its result times 1/8 is
// exact, or a denormal off by 2^-22 at most.
// PRECISE: the quotient's remainder is taken over the larger of the sum's two
// terms first (which leaves it nearly exact) and joins the product unrounded:
// 0.61 half steps of fp32 rms against 0.95 (0.88 by elementary fp32 operations).
// fp32 rows take it, where most of its time hides behind memory (16384 x 4096
// 119.8 us against 117.6); bf16 rows would pay more (32768 x 4096 146 us against
// 138), for codes whose errors come from elsewhere.
template <bool PRECISE>
__device__ __forceinline__ float silu_times(float g, float u) {
  constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f, kLn2 = 0.693147182f;
  constexpr float kOverflow = -0x1.62e43p+6f;  // from here down exp(-g) is infinite in fp32, the result zero
  const float b = __builtin_amdgcn_fmed3f(g, PRECISE ? -89.0f : -1e30f, 200.0f);
  const float t = fminf(-b * kLog2e, 0x1.fffffep+6f);
  const float low = fmaf(-b, kLog2eLow, fmaf(-b, kLog2e, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  if constexpr (PRECISE) {
    const float e8 = fmaf(e * (kLn2 * 0.125f), low, e * 0.125f);  // (finite: the bound on g)
    const float r = g > kOverflow ? __builtin_amdgcn_rcpf(e8 + 0.125f) : 0.0f;
    const float q = g * (r * 0.125f);
    const float rest = fmaf(-fminf(e8, 0.125f), q, fmaf(-fmaxf(e8, 0.125f), q, g * 0.125f));
    return fmaf(q, u, rest * r * u);
  } else {  // (what a gate asks beyond exponent 128 is in the low part, and makes the sum infinite)
    return g * (__builtin_amdgcn_rcpf(fmaf(fmaf(e * kLn2, low, e), 0.125f, 0.125f)) * 0.125f) * u;
  }
}

// Eight consecutive values. STREAM: values that nothing reads again soon pass the
// caches by (non-temporal).
template <bool STREAM>
__device__ __forceinline__ uint4 load16(const void* p) {
  if constexpr (STREAM)
    return __builtin_bit_cast(uint4, __builtin_nontemporal_load(static_cast<const u32x4*>(p)));
  else
    return *static_cast<const uint4*>(p);
}
template <bool F32, bool STREAM = false>
__device__ __forceinline__ void load8(const void* x, size_t at, float v[8]) {
  if constexpr (F32) {
    const float4 a = __builtin_bit_cast(float4, load16<STREAM>(static_cast<const float*>(x) + at));
    const float4 b = __builtin_bit_cast(float4, load16<STREAM>(static_cast<const float*>(x) + at + 4));
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = load16<STREAM>(static_cast<const uint16_t*>(x) + at);
    const uint32_t d[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(d[i] << 16);
      v[2 * i + 1] = __uint_as_float(d[i] & 0xFFFF0000u);
    }
  }
}

}  // namespace moe
