// fp4_api.hip -- the C ABI of the 4-bit rows and their products
// (include/moe.h): argument checks and launches.
#include <stddef.h>
#include <stdint.h>

#include "api_checks.h"
#include "fp4.h"
#include "kernels.h"
#include "moe.h"

using namespace moe;

namespace {

// rows, columns and types of a call that has values on one side and codes on the other
int check_rows(int32_t rows, int32_t cols, int64_t ld, int64_t wide, int32_t type) {
  if (rows < 0 || cols <= 0) return MOE_EINVAL;
  MOE_TRY(type_ok(type));
  if (rows >= kMaxRows || cols % kFp4Group || cols > kMaxWidth) return MOE_EUNSUPPORTED;
  if (ld < wide) return MOE_EINVAL;
  return ld > kMaxPitch ? MOE_EUNSUPPORTED : MOE_OK;
}

int check_quant(int32_t rows, int32_t cols, int64_t wide, const void* x, int64_t ldx, int32_t type,
                const uint8_t* codes, const uint8_t* scales) {
  MOE_TRY(check_rows(rows, cols, ldx, wide, type));
  if (rows == 0) return MOE_OK;
  MOE_TRY(need(x, 16));
  MOE_TRY(need(codes, 16));
  MOE_TRY(need(scales, 1));
  return ldx % (type == MOE_TYPE_BF16 ? 8 : 4) ? MOE_EALIGN : MOE_OK;
}

int run_quant(int32_t rows, int32_t cols, const void* x, int64_t ldx, int32_t type, uint8_t* codes, uint8_t* scales,
              bool swiglu, void* stream) {
  if (rows == 0) return MOE_OK;
  Fp4Quant q{};
  q.x = x;
  q.ldx = ldx;
  q.codes = codes;
  q.scales = scales;
  q.rows = rows;
  q.cols = cols;
  q.f32 = type == MOE_TYPE_F32;
  q.swiglu = swiglu;
  return report_hip(launch_fp4_quant(q, static_cast<hipStream_t>(stream)));
}

int check_product(int32_t rows, int32_t N, int32_t K, const uint8_t* x, int64_t ldx, const uint8_t* xs,
                  const uint8_t* w, const uint8_t* ws, const void* out, int64_t ldo, int32_t type) {
  if (N <= 0 || K <= 0) return MOE_EINVAL;
  if (N > kMaxWidth) return MOE_EUNSUPPORTED;
  MOE_TRY(check_rows(rows, K, ldx, K / 2, type));
  if (ldo < N) return MOE_EINVAL;
  if (ldo > kMaxPitch) return MOE_EUNSUPPORTED;
  if (rows == 0) return MOE_OK;
  MOE_TRY(need(x, 16));
  MOE_TRY(need(xs, 1));
  MOE_TRY(need(w, 16));
  MOE_TRY(need(ws, 1));
  MOE_TRY(need(out, type_size(type)));
  return ldx % 16 ? MOE_EALIGN : MOE_OK;
}

Fp4Gemm product(int32_t rows, int32_t N, int32_t K, const uint8_t* x, int64_t ldx, const uint8_t* xs,
                const uint8_t* w, const uint8_t* ws, void* out, int64_t ldo, int32_t type) {
  Fp4Gemm g{};
  g.x = x;
  g.xs = xs;
  g.w = w;
  g.ws = ws;
  g.out = out;
  g.ldx = ldx;
  g.ldo = ldo;
  g.rows = g.x_rows = rows;
  g.experts = 1;
  g.N = N;
  g.K = K;
  g.index_div = 1;
  g.f32 = type == MOE_TYPE_F32;
  g.out_vec = ldo % 4 == 0 && aligned(out, g.f32 ? 16 : 8);
  g.out_vec8 = !g.f32 && ldo % 8 == 0 && aligned(out, 16);
  const auto start_at = [&](int n) { return K / kFp4Group % n == 0 && aligned(xs, n) && aligned(ws, n); };
  g.scales = start_at(16) ? kBy16 : start_at(4) ? kBy4 : kBy1;
  return g;
}

}  // namespace

extern "C" {

int moe_fp4_quantize_validate(int32_t rows, int32_t cols, const void* x, int64_t ldx, int32_t x_type,
                              const uint8_t* codes, const uint8_t* scales) {
  return check_quant(rows, cols, cols, x, ldx, x_type, codes, scales);
}

int moe_fp4_quantize(int32_t rows, int32_t cols, const void* x, int64_t ldx, int32_t x_type, uint8_t* codes,
                     uint8_t* scales, void* hip_stream) {
  MOE_TRY(moe_fp4_quantize_validate(rows, cols, x, ldx, x_type, codes, scales));
  return run_quant(rows, cols, x, ldx, x_type, codes, scales, false, hip_stream);
}

int moe_fp4_swiglu_validate(int32_t rows, int32_t inter, const void* gate_up, int64_t ld, int32_t type,
                            const uint8_t* codes, const uint8_t* scales) {
  return check_quant(rows, inter, 2 * static_cast<int64_t>(inter), gate_up, ld, type, codes, scales);
}

int moe_fp4_swiglu(int32_t rows, int32_t inter, const void* gate_up, int64_t ld, int32_t type, uint8_t* codes,
                   uint8_t* scales, void* hip_stream) {
  MOE_TRY(moe_fp4_swiglu_validate(rows, inter, gate_up, ld, type, codes, scales));
  return run_quant(rows, inter, gate_up, ld, type, codes, scales, true, hip_stream);
}

int moe_fp4_dequantize_validate(int32_t rows, int32_t cols, const uint8_t* codes, const uint8_t* scales,
                                const void* out, int64_t ldo, int32_t out_type) {
  MOE_TRY(check_rows(rows, cols, ldo, cols, out_type));
  if (rows == 0) return MOE_OK;
  MOE_TRY(need(codes, 16));
  MOE_TRY(need(scales, 1));
  return need(out, type_size(out_type));
}

int moe_fp4_dequantize(int32_t rows, int32_t cols, const uint8_t* codes, const uint8_t* scales, void* out,
                       int64_t ldo, int32_t out_type, void* hip_stream) {
  MOE_TRY(moe_fp4_dequantize_validate(rows, cols, codes, scales, out, ldo, out_type));
  if (rows == 0) return MOE_OK;
  Fp4Dequant q{};
  q.codes = codes;
  q.scales = scales;
  q.out = out;
  q.ldo = ldo;
  q.rows = rows;
  q.cols = cols;
  q.f32 = out_type == MOE_TYPE_F32;
  return report_hip(launch_fp4_dequant(q, static_cast<hipStream_t>(hip_stream)));
}

int moe_fp4_linear_validate(int32_t T, int32_t N, int32_t K, const uint8_t* x, int64_t ldx, const uint8_t* x_scales,
                            const uint8_t* w, const uint8_t* w_scales, const void* out, int64_t ldo,
                            int32_t out_type) {
  return check_product(T, N, K, x, ldx, x_scales, w, w_scales, out, ldo, out_type);
}

int moe_fp4_linear(int32_t T, int32_t N, int32_t K, const uint8_t* x, int64_t ldx, const uint8_t* x_scales,
                   const uint8_t* w, const uint8_t* w_scales, void* out, int64_t ldo, int32_t out_type,
                   void* hip_stream) {
  MOE_TRY(moe_fp4_linear_validate(T, N, K, x, ldx, x_scales, w, w_scales, out, ldo, out_type));
  if (T == 0) return MOE_OK;
  const Fp4Gemm g = product(T, N, K, x, ldx, x_scales, w, w_scales, out, ldo, out_type);
  return report_hip(launch_fp4_gemm(g, static_cast<hipStream_t>(hip_stream)));
}

int moe_fp4_grouped_validate(int32_t rows, int32_t n_experts, int32_t N, int32_t K, const int32_t* offsets,
                             const int32_t* row_index, int32_t index_div, int32_t x_rows, const uint8_t* x,
                             int64_t ldx, const uint8_t* x_scales, const uint8_t* w, const uint8_t* w_scales,
                             const void* out, int64_t ldo, int32_t out_type) {
  if (n_experts <= 0 || x_rows < 0 || index_div <= 0) return MOE_EINVAL;
  if (n_experts > kMaxExperts) return MOE_EUNSUPPORTED;
  MOE_TRY(check_product(rows, N, K, x, ldx, x_scales, w, w_scales, out, ldo, out_type));
  if (rows == 0) return MOE_OK;
  MOE_TRY(need(offsets, 4));
  if (row_index) {
    MOE_TRY(need(row_index, 4));
    if (x_rows == 0) return MOE_EINVAL;
    if (x_rows >= kMaxRows || x_rows * ldx >= kDescriptor) return MOE_EUNSUPPORTED;
  } else if (x_rows < rows || index_div != 1) {
    return MOE_EINVAL;
  }
  return MOE_OK;
}

int moe_fp4_grouped(int32_t rows, int32_t n_experts, int32_t N, int32_t K, const int32_t* offsets,
                    const int32_t* row_index, int32_t index_div, int32_t x_rows, const uint8_t* x, int64_t ldx,
                    const uint8_t* x_scales, const uint8_t* w, const uint8_t* w_scales, void* out, int64_t ldo,
                    int32_t out_type, void* hip_stream) {
  MOE_TRY(moe_fp4_grouped_validate(rows, n_experts, N, K, offsets, row_index, index_div, x_rows, x, ldx, x_scales, w,
                                   w_scales, out, ldo, out_type));
  if (rows == 0) return MOE_OK;
  Fp4Gemm g = product(rows, N, K, x, ldx, x_scales, w, w_scales, out, ldo, out_type);
  g.offsets = offsets;
  g.index = row_index;
  g.index_div = index_div;
  g.x_rows = x_rows;
  g.experts = n_experts;
  return report_hip(launch_fp4_gemm(g, static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
