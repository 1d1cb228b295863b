// quant_fp4.hip -- rows to MXFP4 (E2M1 codes with one E8M0 scale per 32
// values), as they are or after SwiGLU (h = silu(gate) * up), and back.
//
//   m = largest |v| of the group, e = the exponent of m rounded to two
//   significant bits (what a code holds), X = 2^max(e - 2, -126)
//   scale = X as its biased exponent, code = E2M1(v / X), nearest, ties to even
//
// v / X is exact (or below the smallest code's half, when v is subnormal), so a
// code is v's nearest value in E2M1 times X; and because m rounds before its
// exponent is taken, |v / X| < 7 rounds to 6 at most: nothing saturates, each
// value is within half a step. E2M1 has neither NaN nor infinity: a group that
// holds one becomes NaN as a whole (scale 255, codes 0).
//
// Memory bound: each value is read once and held in registers between maximum
// and conversion. A lane holds 8 values (16-byte loads of bf16, 4-byte stores),
// a group is four lanes, its maximum two DPP steps, the conversion instruction
// takes the scale. Loads of values, and stores of them on the way back, pass the
// caches by (4096 x 8192 there and back 31.4 -> 30.4 us, SwiGLU 2% less; back and
// quantised again, 1024 rows 9.6 us, 9.5 with stores through the caches, 4096 rows 31.2
// and 30.7, 16384 rows 110 and 114). 4096 x 8192 bf16: 16 .. 18 us, 5 TB/s, and back
// 12 us (codes from the cache); SwiGLU to 32768 x 4096 bf16 101 us, 6.0 TB/s; 32 x
// 4096: 2.2 us, a launch.
#include "device_common.h"
#include "fp4.h"
#include "kernels.h"
#include "silu.h"

namespace moe {

namespace {

constexpr uint32_t kInfBits = 0x7F800000u;
constexpr int kBlock = 128;  // columns of a row of 16 lanes: four groups

// v of lane l ^ 1, l ^ 2: the largest of the four lanes of a group.
__device__ __forceinline__ uint32_t quad_max_u32(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xB1, 0xF, 0xF, false)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x4E, 0xF, 0xF, false)));
  return v;
}

// Bits set in any of the four lanes 4 apart of a row of 16, in every lane.
__device__ __forceinline__ uint32_t join_quads(uint32_t v) {
  v |= static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x124, 0xF, 0xF, false));
  v |= static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x128, 0xF, 0xF, false));
  return v;
}

// A workgroup's 16 rows of lanes: 2^log_g neighbouring blocks of 16 >> log_g
// rows, and U such sets of rows, their loads issued together.
template <bool F32, bool SWIGLU, int U>
__global__ __launch_bounds__(256) void fp4_quant_kernel(Fp4Quant p, int log_g, bool scale4) {
  const int l = threadIdx.x & 15, gi = threadIdx.x >> 4;
  const int b = (static_cast<int>(blockIdx.y) << log_g) + (gi & ((1 << log_g) - 1));
  const int rows_per_set = 16 >> log_g;
  const int row0 = static_cast<int>(blockIdx.x) * (rows_per_set * U) + (gi >> log_g);
  const int col = b * kBlock + l * 8;
  const bool live_col = col < p.cols;  // (whole groups: cols is a multiple of 32)
  float v[U][8];
  float up[SWIGLU ? U : 1][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int row = row0 + u * rows_per_set;
    if (live_col && row < p.rows) {
      const size_t at = static_cast<size_t>(row) * p.ldx + col;
      load8<F32, true>(p.x, at, v[u]);
      if constexpr (SWIGLU) load8<F32, true>(p.x, at + p.cols, up[u]);
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
    m = quad_max_u32(m);
    const bool bad = m >= kInfBits;  // the same in all lanes of the group
    // (adding a quarter to the significand carries into the exponent from 1.75 on)
    const uint32_t e = (m + 0x200000u) >> 23;
    const uint32_t byte = bad ? 255u : max(e, 3u) - 2u;
    const float scale = __uint_as_float(byte << 23);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[u][0], v[u][1], scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[u][2], v[u][3], scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[u][4], v[u][5], scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[u][6], v[u][7], scale, 3);
    if (bad) c = 0;
    const uint32_t four = join_quads(byte << (l / 4 * 8));
    if (live_col && row < p.rows) {
      *reinterpret_cast<uint32_t*>(p.codes + (static_cast<size_t>(row) * p.cols + col) / 2) = c;
      uint8_t* s = p.scales + (static_cast<size_t>(row) * p.cols + col) / kFp4Group;
      if (scale4) {  // (cols a multiple of 128, scales 4-byte aligned)
        if (l == 0) *reinterpret_cast<uint32_t*>(s) = four;
      } else if (l % 4 == 0) {
        *s = static_cast<uint8_t>(byte);
      }
    }
  }
}

template <bool F32, bool SWIGLU>
hipError_t launch_quant(const Fp4Quant& q, hipStream_t st) {
  const int nb = (q.cols + kBlock - 1) / kBlock;
  const bool scale4 = q.cols % kBlock == 0 && reinterpret_cast<uintptr_t>(q.scales) % 4 == 0;
  int log_g = 0;
  while (log_g < 4 && (1 << log_g) < nb) ++log_g;
  const int rows_per_set = 16 >> log_g;
  const unsigned gy = (nb + (1 << log_g) - 1) >> log_g;
  constexpr int U = 4;
  // few rows: one set per workgroup, so that every CU gets some
  if (static_cast<int64_t>(gy) * ((q.rows + rows_per_set * U - 1) / (rows_per_set * U)) < 512) {
    const dim3 grid((q.rows + rows_per_set - 1) / rows_per_set, gy);
    MOE_LAUNCH((fp4_quant_kernel<F32, SWIGLU, 1>), grid, dim3(256), 0, st, q, log_g, scale4);
  } else {
    const dim3 grid((q.rows + rows_per_set * U - 1) / (rows_per_set * U), gy);
    MOE_LAUNCH((fp4_quant_kernel<F32, SWIGLU, U>), grid, dim3(256), 0, st, q, log_g, scale4);
  }
  return hipGetLastError();
}

// Eight values a lane, the same arrangement.
template <bool F32, int U>
__global__ __launch_bounds__(256) void fp4_dequant_kernel(Fp4Dequant p, int log_g, bool wide) {
  const int l = threadIdx.x & 15, gi = threadIdx.x >> 4;
  const int b = (static_cast<int>(blockIdx.y) << log_g) + (gi & ((1 << log_g) - 1));
  const int rows_per_set = 16 >> log_g;
  const int row0 = static_cast<int>(blockIdx.x) * (rows_per_set * U) + (gi >> log_g);
  const int col = b * kBlock + l * 8;
  if (col >= p.cols) return;
  uint32_t c[U], s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int row = row0 + u * rows_per_set;
    c[u] = s[u] = 0;
    if (row < p.rows) {
      c[u] = *reinterpret_cast<const uint32_t*>(p.codes + (static_cast<size_t>(row) * p.cols + col) / 2);
      s[u] = p.scales[(static_cast<size_t>(row) * p.cols + col) / kFp4Group];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int row = row0 + u * rows_per_set;
    if (row >= p.rows) break;
    const float scale = __uint_as_float(s[u] << 23);  // (255: NaN, which the conversion gives)
    const size_t at = static_cast<size_t>(row) * p.ldo + col;
    if constexpr (F32) {
      float* o = static_cast<float*>(p.out) + at;
      const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], scale, 0);
      const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], scale, 1);
      const f32x2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], scale, 2);
      const f32x2 f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], scale, 3);
      const float q[8] = {a[0], a[1], d[0], d[1], e[0], e[1], f[0], f[1]};
      if (wide) {
        reinterpret_cast<float4*>(o)[0] = float4{q[0], q[1], q[2], q[3]};
        reinterpret_cast<float4*>(o)[1] = float4{q[4], q[5], q[6], q[7]};
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = q[i];
      }
    } else {
      uint16_t* o = static_cast<uint16_t*>(p.out) + at;
      const uint4 q = __builtin_bit_cast(uint4, mxfp4x8_to_bf16(c[u], scale));
      if (wide) {
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, q), reinterpret_cast<u32x4*>(o));
      } else {
        const uint32_t d[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = static_cast<uint16_t>(d[i / 2] >> (i % 2 * 16));
      }
    }
  }
}

template <bool F32>
hipError_t launch_dequant(const Fp4Dequant& q, hipStream_t st) {
  const int nb = (q.cols + kBlock - 1) / kBlock;
  const bool wide = q.ldo % (F32 ? 4 : 8) == 0 && reinterpret_cast<uintptr_t>(q.out) % 16 == 0;
  int log_g = 0;
  while (log_g < 4 && (1 << log_g) < nb) ++log_g;
  const int rows_per_set = 16 >> log_g;
  const unsigned gy = (nb + (1 << log_g) - 1) >> log_g;
  constexpr int U = 4;
  if (static_cast<int64_t>(gy) * ((q.rows + rows_per_set * U - 1) / (rows_per_set * U)) < 512) {
    const dim3 grid((q.rows + rows_per_set - 1) / rows_per_set, gy);
    MOE_LAUNCH((fp4_dequant_kernel<F32, 1>), grid, dim3(256), 0, st, q, log_g, wide);
  } else {
    const dim3 grid((q.rows + rows_per_set * U - 1) / (rows_per_set * U), gy);
    MOE_LAUNCH((fp4_dequant_kernel<F32, U>), grid, dim3(256), 0, st, q, log_g, wide);
  }
  return hipGetLastError();
}

constexpr int kRows = 1 << 24;  // a launch holds fewer than 2^32 threads, 16 per row and block

}  // namespace

hipError_t launch_fp4_quant(const Fp4Quant& all, hipStream_t st) {
  hipError_t e = hipSuccess;
  for (int64_t r = 0; r < all.rows && e == hipSuccess; r += kRows) {
    Fp4Quant q = all;
    q.x = static_cast<const uint8_t*>(all.x) + r * all.ldx * (all.f32 ? 4 : 2);
    q.codes += r * (all.cols / 2);
    q.scales += r * (all.cols / kFp4Group);
    q.rows = static_cast<int>(all.rows - r < kRows ? all.rows - r : kRows);
    if (q.swiglu)
      e = q.f32 ? launch_quant<true, true>(q, st) : launch_quant<false, true>(q, st);
    else
      e = q.f32 ? launch_quant<true, false>(q, st) : launch_quant<false, false>(q, st);
  }
  return e;
}

hipError_t launch_fp4_dequant(const Fp4Dequant& all, hipStream_t st) {
  hipError_t e = hipSuccess;
  for (int64_t r = 0; r < all.rows && e == hipSuccess; r += kRows) {
    Fp4Dequant q = all;
    q.codes += r * (all.cols / 2);
    q.scales += r * (all.cols / kFp4Group);
    q.out = static_cast<uint8_t*>(all.out) + r * all.ldo * (all.f32 ? 4 : 2);
    q.rows = static_cast<int>(all.rows - r < kRows ? all.rows - r : kRows);
    e = q.f32 ? launch_dequant<true>(q, st) : launch_dequant<false>(q, st);
  }
  return e;
}

}  // namespace moe
