// fp8_api.hip -- the C ABI of the 8-bit rows, their products and the balance
// loss (include/moe.h): argument checks and launches.
#include <stddef.h>
#include <stdint.h>

#include "api_checks.h"
#include "balance.h"
#include "fp8.h"
#include "kernels.h"
#include "moe.h"

using namespace moe;

namespace {

// The type of a product's out without MOE_SUM_F32.
int32_t out_type_of(int32_t type) { return type >= 0 ? type & ~MOE_SUM_F32 : type; }

int check_quant(int32_t rows, int32_t cols, int32_t wide, const void* x, int64_t ldx, int32_t type,
                const uint8_t* codes, const float* scales) {
  if (rows < 0 || cols <= 0) return MOE_EINVAL;
  MOE_TRY(type_ok(type));
  if (rows >= kMaxRows || cols % 16 || cols > kMaxWidth) return MOE_EUNSUPPORTED;
  if (ldx < wide) return MOE_EINVAL;
  if (ldx > kMaxPitch) return MOE_EUNSUPPORTED;
  if (rows == 0) return MOE_OK;
  MOE_TRY(need(x, 16));
  MOE_TRY(need(codes, 16));
  MOE_TRY(need(scales, 4));
  if (ldx % (type == MOE_TYPE_BF16 ? 8 : 4)) return MOE_EALIGN;
  return MOE_OK;
}

int run_quant(int32_t rows, int32_t cols, const void* x, int64_t ldx, int32_t type, uint8_t* codes, float* scales,
              bool swiglu, void* stream) {
  if (rows == 0) return MOE_OK;
  moe::Fp8Quant q{};
  q.x = x;
  q.ldx = ldx;
  q.codes = codes;
  q.scales = scales;
  q.rows = rows;
  q.cols = cols;
  q.f32 = type == MOE_TYPE_F32;
  q.swiglu = swiglu;
  return moe::report_hip(moe::launch_fp8_quant(q, static_cast<hipStream_t>(stream)));
}

int check_product(int32_t rows, int32_t N, int32_t K, const uint8_t* x, int64_t ldx, const float* xs,
                  const uint8_t* w, const float* ws, const void* out, int64_t ldo, int32_t type) {
  if (rows < 0 || N <= 0 || K <= 0) return MOE_EINVAL;
  MOE_TRY(type_ok(out_type_of(type)));
  if (rows >= kMaxRows || K % 16 || K > kMaxWidth || N > kMaxWidth) return MOE_EUNSUPPORTED;
  if (ldx < K || ldo < N) return MOE_EINVAL;
  if (ldx > kMaxPitch || ldo > kMaxPitch) return MOE_EUNSUPPORTED;
  if (rows == 0) return MOE_OK;
  MOE_TRY(need(x, 16));
  MOE_TRY(need(xs, 4));
  MOE_TRY(need(w, 16));
  MOE_TRY(need(ws, 4));
  MOE_TRY(need(out, out_type_of(type) == MOE_TYPE_F32 ? 4 : 2));
  if (ldx % 16) return MOE_EALIGN;
  return MOE_OK;
}

moe::Fp8Gemm product(int32_t rows, int32_t N, int32_t K, const uint8_t* x, int64_t ldx, const float* xs,
                     const uint8_t* w, const float* ws, void* out, int64_t ldo, int32_t type) {
  moe::Fp8Gemm g{};
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
  g.f32 = out_type_of(type) == MOE_TYPE_F32;
  g.exact = type != MOE_TYPE_BF16;
  g.out_vec = ldo % 4 == 0 && aligned(out, g.f32 ? 16 : 8);
  return g;
}

int check_balance(int32_t T, int32_t E, int32_t K) {
  if (T < 0 || E <= 0 || K <= 0) return MOE_EINVAL;
  if (T >= kMaxRows || E > moe::kFp8MaxExperts || K > 8 || K > E) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_fp8_quantize_validate(int32_t rows, int32_t cols, const void* x, int64_t ldx, int32_t x_type,
                              const uint8_t* codes, const float* scales) {
  return check_quant(rows, cols, cols, x, ldx, x_type, codes, scales);
}

int moe_fp8_quantize(int32_t rows, int32_t cols, const void* x, int64_t ldx, int32_t x_type, uint8_t* codes,
                     float* scales, void* hip_stream) {
  MOE_TRY(moe_fp8_quantize_validate(rows, cols, x, ldx, x_type, codes, scales));
  return run_quant(rows, cols, x, ldx, x_type, codes, scales, false, hip_stream);
}

int moe_fp8_swiglu_validate(int32_t rows, int32_t inter, const void* gate_up, int64_t ld, int32_t type,
                            const uint8_t* codes, const float* scales) {
  if (rows < 0 || inter <= 0) return MOE_EINVAL;
  if (inter > kMaxWidth) return MOE_EUNSUPPORTED;
  return check_quant(rows, inter, 2 * inter, gate_up, ld, type, codes, scales);
}

int moe_fp8_swiglu(int32_t rows, int32_t inter, const void* gate_up, int64_t ld, int32_t type, uint8_t* codes,
                   float* scales, void* hip_stream) {
  MOE_TRY(moe_fp8_swiglu_validate(rows, inter, gate_up, ld, type, codes, scales));
  return run_quant(rows, inter, gate_up, ld, type, codes, scales, true, hip_stream);
}

int moe_fp8_linear_validate(int32_t T, int32_t N, int32_t K, const uint8_t* x, int64_t ldx, const float* x_scales,
                            const uint8_t* w, const float* w_scales, const void* out, int64_t ldo,
                            int32_t out_type) {
  return check_product(T, N, K, x, ldx, x_scales, w, w_scales, out, ldo, out_type);
}

int moe_fp8_linear(int32_t T, int32_t N, int32_t K, const uint8_t* x, int64_t ldx, const float* x_scales,
                   const uint8_t* w, const float* w_scales, void* out, int64_t ldo, int32_t out_type,
                   void* hip_stream) {
  MOE_TRY(moe_fp8_linear_validate(T, N, K, x, ldx, x_scales, w, w_scales, out, ldo, out_type));
  if (T == 0) return MOE_OK;
  const moe::Fp8Gemm g = product(T, N, K, x, ldx, x_scales, w, w_scales, out, ldo, out_type);
  return moe::report_hip(moe::launch_fp8_gemm(g, static_cast<hipStream_t>(hip_stream)));
}

int moe_fp8_grouped_validate(int32_t rows, int32_t n_experts, int32_t N, int32_t K, const int32_t* offsets,
                             const int32_t* row_index, int32_t index_div, int32_t x_rows, const uint8_t* x,
                             int64_t ldx, const float* x_scales, const uint8_t* w, const float* w_scales,
                             const void* out, int64_t ldo, int32_t out_type) {
  if (n_experts <= 0 || x_rows < 0 || index_div <= 0) return MOE_EINVAL;
  if (n_experts > moe::kFp8MaxExperts) return MOE_EUNSUPPORTED;
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

int moe_fp8_grouped(int32_t rows, int32_t n_experts, int32_t N, int32_t K, const int32_t* offsets,
                    const int32_t* row_index, int32_t index_div, int32_t x_rows, const uint8_t* x, int64_t ldx,
                    const float* x_scales, const uint8_t* w, const float* w_scales, void* out, int64_t ldo,
                    int32_t out_type, void* hip_stream) {
  MOE_TRY(moe_fp8_grouped_validate(rows, n_experts, N, K, offsets, row_index, index_div, x_rows, x, ldx, x_scales, w,
                                   w_scales, out, ldo, out_type));
  if (rows == 0) return MOE_OK;
  moe::Fp8Gemm g = product(rows, N, K, x, ldx, x_scales, w, w_scales, out, ldo, out_type);
  g.offsets = offsets;
  g.index = row_index;
  g.index_div = index_div;
  g.x_rows = x_rows;
  g.experts = n_experts;
  return moe::report_hip(moe::launch_fp8_gemm(g, static_cast<hipStream_t>(hip_stream)));
}

size_t moe_balance_workspace_bytes(int32_t T, int32_t n_experts) {
  if (check_balance(T, n_experts, 1) != MOE_OK) return 0;
  return moe::balance_workspace(T, n_experts);
}

int moe_balance_loss_validate(int32_t T, int32_t n_experts, int32_t top_k, const float* logits,
                              const int32_t* topk_ids, const uint8_t* token_mask, const int32_t* counts,
                              const float* losses, const void* workspace, size_t workspace_bytes) {
  (void)token_mask;  // (any address)
  MOE_TRY(check_balance(T, n_experts, top_k));
  MOE_TRY(need(counts, 4));
  MOE_TRY(need(losses, 4));
  if (T > 0) {
    MOE_TRY(need(logits, 16));
    MOE_TRY(need(topk_ids, 4));
  }
  const size_t bytes = moe_balance_workspace_bytes(T, n_experts);
  if (bytes > 0) {
    MOE_TRY(need(workspace, 16));
    if (workspace_bytes < bytes) return MOE_EWORKSPACE;
  }
  return MOE_OK;
}

int moe_balance_loss(int32_t T, int32_t n_experts, int32_t top_k, const float* logits, const int32_t* topk_ids,
                     const uint8_t* token_mask, int32_t* counts, float* losses, void* workspace,
                     size_t workspace_bytes, void* hip_stream) {
  MOE_TRY(moe_balance_loss_validate(T, n_experts, top_k, logits, topk_ids, token_mask, counts, losses, workspace,
                                    workspace_bytes));
  moe::Balance b{};
  b.logits = logits;
  b.ids = topk_ids;
  b.mask = token_mask;
  b.T = T;
  b.E = n_experts;
  b.K = top_k;
  b.counts = counts;
  b.loss = losses;
  b.part = workspace;
  return moe::report_hip(moe::launch_balance_loss(b, static_cast<hipStream_t>(hip_stream)));
}

int moe_balance_loss_backward_validate(int32_t T, int32_t n_experts, int32_t top_k, const float* logits,
                                       const int32_t* topk_ids, const uint8_t* token_mask, const int32_t* counts,
                                       const float* grad_losses, const float* topk_w, const float* grad_topk_w,
                                       const float* grad_logits) {
  (void)token_mask;
  MOE_TRY(check_balance(T, n_experts, top_k));
  if (T == 0) return MOE_OK;
  MOE_TRY(need(logits, 16));
  MOE_TRY(need(counts, 4));
  MOE_TRY(need(grad_losses, 4));
  MOE_TRY(need(grad_logits, 16));
  if ((topk_w == nullptr) != (grad_topk_w == nullptr)) return MOE_EINVAL;
  if (topk_w) {
    MOE_TRY(need(topk_ids, 4));
    MOE_TRY(need(topk_w, 4));
    MOE_TRY(need(grad_topk_w, 4));
  }
  return MOE_OK;
}

int moe_balance_loss_backward(int32_t T, int32_t n_experts, int32_t top_k, const float* logits,
                              const int32_t* topk_ids, const uint8_t* token_mask, const int32_t* counts,
                              const float* grad_losses, const float* topk_w, const float* grad_topk_w,
                              float* grad_logits, void* hip_stream) {
  MOE_TRY(moe_balance_loss_backward_validate(T, n_experts, top_k, logits, topk_ids, token_mask, counts, grad_losses,
                                             topk_w, grad_topk_w, grad_logits));
  if (T == 0) return MOE_OK;
  moe::Balance b{};
  b.logits = logits;
  b.ids = topk_ids;
  b.mask = token_mask;
  b.T = T;
  b.E = n_experts;
  b.K = top_k;
  b.counts_in = counts;
  b.dloss = grad_losses;
  b.w = topk_w;
  b.dw = grad_topk_w;
  b.dlogits = grad_logits;
  return moe::report_hip(moe::launch_balance_backward(b, static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
