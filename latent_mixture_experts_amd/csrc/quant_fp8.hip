// quant_fp8.hip -- rows to E4M3 codes with one fp32 scale per 128 values,
// as they are or after SwiGLU (h = silu(gate) * up).
//
//   amax = max(2^-90, largest finite |v| of the group)
//   scale = amax / 448,   code = E4M3(v * (448 / amax)), to nearest, ties to even
//
// Both quotients are IEEE fp32 divisions, one each per group; 448 / amax is
// finite because amax >= 2^-90. A product can exceed 448 by its rounding only,
// which still rounds to 448. NaN and infinities (a format without infinities)
// become NaN codes and leave the group's scale to the finite values.
//
// Memory bound: each value is read once and held in registers between the
// maximum and the conversion. A group is one row of 16 lanes with 8 values
// each (16-byte loads of bf16, 8-byte stores), its maximum four DPP steps.
// 4096 x 8192 bf16: 18.3 us, 5.6 TB/s, fp32 31.3, 5.4; SwiGLU to 32768 x 4096 bf16
// 134 us, 5.0 TB/s (a large copy 5.1 TB/s); 32 x 4096: 2.2 us, a launch.
#include "device_common.h"
#include "fp8.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr float kE4m3Max = 448.0f;
constexpr uint32_t kTinyBits = 0x12800000u;  // 2^-90
constexpr uint32_t kInfBits = 0x7F800000u;

// Largest of the 16 lanes of a row, in every lane of it.
__device__ __forceinline__ uint32_t row16_max_u32(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xB1, 0xF, 0xF, false)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x4E, 0xF, 0xF, false)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x124, 0xF, 0xF, false)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x128, 0xF, 0xF, false)));
  return v;
}

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

// Eight consecutive values.
template <bool F32>
__device__ __forceinline__ void load8(const void* x, size_t at, float v[8]) {
  if constexpr (F32) {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + at + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at);
    const uint32_t d[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(d[i] << 16);
      v[2 * i + 1] = __uint_as_float(d[i] & 0xFFFF0000u);
    }
  }
}

// A workgroup's 16 groups: 2^log_g neighbouring groups of 16 >> log_g rows,
// and U such sets of rows, their loads issued together.
template <bool F32, bool SWIGLU, int U>
__global__ __launch_bounds__(256) void fp8_quant_kernel(Fp8Quant p, int log_g, int nkb) {
  const int l = threadIdx.x & 15, gi = threadIdx.x >> 4;
  const int b = (static_cast<int>(blockIdx.y) << log_g) + (gi & ((1 << log_g) - 1));
  const int rows_per_set = 16 >> log_g;
  const int row0 = static_cast<int>(blockIdx.x) * (rows_per_set * U) + (gi >> log_g);
  const int col = b * kFp8Block + l * 8;
  const bool live_col = col < p.cols;
  float v[U][8];
  float up[SWIGLU ? U : 1][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int row = row0 + u * rows_per_set;
    if (live_col && row < p.rows) {
      const size_t at = static_cast<size_t>(row) * p.ldx + col;
      load8<F32>(p.x, at, v[u]);
      if constexpr (SWIGLU) load8<F32>(p.x, at + p.cols, up[u]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[u][i] = 0.0f;
        if constexpr (SWIGLU) up[u][i] = 0.0f;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int row = row0 + u * rows_per_set;
    if constexpr (SWIGLU) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = silu_times<F32>(v[u][i], up[u][i]);
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[u][i]) & 0x7FFFFFFFu);
    m = row16_max_u32(m);
    const bool bad = m >= kInfBits;  // the same in all lanes of the group
    if (bad) {
      m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t a = __float_as_uint(v[u][i]) & 0x7FFFFFFFu;
        if (a < kInfBits) m = max(m, a);
      }
      m = row16_max_u32(m);
    }
    const float amax = __uint_as_float(max(m, kTinyBits));
    const float inv = kE4m3Max / amax;
    if (bad) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((__float_as_uint(v[u][i]) & 0x7FFFFFFFu) >= kInfBits) v[u][i] = __uint_as_float(0x7FC00000u);
    }
    uint32_t c[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float* q = &v[u][4 * h];
      int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0] * inv, q[1] * inv, 0, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2] * inv, q[3] * inv, w, true);
      c[h] = static_cast<uint32_t>(w);
    }
    if (live_col && row < p.rows) {
      *reinterpret_cast<uint2*>(p.codes + static_cast<size_t>(row) * p.cols + col) = uint2{c[0], c[1]};
      if (l == 0) p.scales[static_cast<size_t>(row) * nkb + b] = amax / kE4m3Max;
    }
  }
}

template <bool F32, bool SWIGLU>
hipError_t launch_quant(const Fp8Quant& q, hipStream_t st) {
  const int nkb = fp8_blocks(q.cols);
  int log_g = 0;
  while (log_g < 4 && (1 << log_g) < nkb) ++log_g;
  const int rows_per_set = 16 >> log_g;
  const unsigned gy = (nkb + (1 << log_g) - 1) >> log_g;
  constexpr int U = 4;
  // few rows: one set per workgroup, so that every CU gets some
  if (static_cast<int64_t>(gy) * ((q.rows + rows_per_set * U - 1) / (rows_per_set * U)) < 512) {
    const dim3 grid((q.rows + rows_per_set - 1) / rows_per_set, gy);
    MOE_LAUNCH((fp8_quant_kernel<F32, SWIGLU, 1>), grid, dim3(256), 0, st, q, log_g, nkb);
  } else {
    const dim3 grid((q.rows + rows_per_set * U - 1) / (rows_per_set * U), gy);
    MOE_LAUNCH((fp8_quant_kernel<F32, SWIGLU, U>), grid, dim3(256), 0, st, q, log_g, nkb);
  }
  return hipGetLastError();
}

}  // namespace

// A launch holds fewer than 2^32 threads, 16 per group: more than 2^24 rows take
// several.
hipError_t launch_fp8_quant(const Fp8Quant& all, hipStream_t st) {
  constexpr int kRows = 1 << 24;
  hipError_t e = hipSuccess;
  for (int64_t r = 0; r < all.rows && e == hipSuccess; r += kRows) {
    Fp8Quant q = all;
    q.x = static_cast<const uint8_t*>(all.x) + r * all.ldx * (all.f32 ? 4 : 2);
    q.codes += r * all.cols;
    q.scales += r * fp8_blocks(all.cols);
    q.rows = static_cast<int>(all.rows - r < kRows ? all.rows - r : kRows);
    if (q.swiglu)
      e = q.f32 ? launch_quant<true, true>(q, st) : launch_quant<false, true>(q, st);
    else
      e = q.f32 ? launch_quant<true, false>(q, st) : launch_quant<false, false>(q, st);
  }
  return e;
}

}  // namespace moe
