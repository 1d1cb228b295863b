// routes_api.hip -- the C ABI of the sort of routes and of the rows' way into
// expert order and back (include/moe.h): argument checks and launches.
#include <stddef.h>
#include <stdint.h>

#include "api_checks.h"
#include "kernels.h"
#include "moe.h"
#include "routes.h"

using namespace moe;

namespace {

constexpr int32_t kMaxTopK = 8;

int check_routes(int32_t T, int32_t top_k) {
  if (T < 0 || top_k <= 0) return MOE_EINVAL;
  return top_k > kMaxTopK || static_cast<int64_t>(T) * top_k >= kMaxRows ? MOE_EUNSUPPORTED : MOE_OK;
}

int check_rows(int32_t T, int32_t top_k, int32_t rows, int32_t cols) {
  MOE_TRY(check_routes(T, top_k));
  if (rows < 0 || cols <= 0) return MOE_EINVAL;
  return rows >= kMaxRows || cols > kMaxWidth ? MOE_EUNSUPPORTED : MOE_OK;
}

int check_matrix(int32_t n, int32_t cols, const void* p, int64_t ld, int32_t type) {
  MOE_TRY(type_ok(type));
  if (ld < cols) return MOE_EINVAL;
  if (ld > kMaxPitch) return MOE_EUNSUPPORTED;
  return n > 0 ? need(p, type_size(type)) : MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_sort_workspace_bytes(int32_t T, int32_t n_experts, int32_t top_k) {
  if (check_routes(T, top_k) != MOE_OK || n_experts <= 0 || n_experts > kMaxExperts) return 0;
  return sort_workspace(T * top_k);
}

int moe_sort_routes_validate(int32_t T, int32_t n_experts, int32_t top_k, const int32_t* topk_ids,
                             int32_t first_expert, const int32_t* expert_offsets, const int32_t* sorted_routes,
                             const int32_t* positions, const void* workspace, size_t workspace_bytes) {
  (void)first_expert;  // (any)
  MOE_TRY(check_routes(T, top_k));
  if (n_experts <= 0) return MOE_EINVAL;
  if (n_experts > kMaxExperts) return MOE_EUNSUPPORTED;
  MOE_TRY(need(expert_offsets, 4));
  if (T > 0) {
    MOE_TRY(need(topk_ids, 4));
    MOE_TRY(need(sorted_routes, 4));
    MOE_TRY(need(positions, 4));
  }
  const size_t bytes = moe_sort_workspace_bytes(T, n_experts, top_k);
  if (bytes > 0) {
    MOE_TRY(need(workspace, 16));
    if (workspace_bytes < bytes) return MOE_EWORKSPACE;
  }
  return MOE_OK;
}

int moe_sort_routes(int32_t T, int32_t n_experts, int32_t top_k, const int32_t* topk_ids, int32_t first_expert,
                    int32_t* expert_offsets, int32_t* sorted_routes, int32_t* positions, void* workspace,
                    size_t workspace_bytes, void* hip_stream) {
  MOE_TRY(moe_sort_routes_validate(T, n_experts, top_k, topk_ids, first_expert, expert_offsets, sorted_routes,
                                   positions, workspace, workspace_bytes));
  SortRoutes s{};
  s.ids = topk_ids;
  s.offsets = expert_offsets;
  s.sorted = sorted_routes;
  s.positions = positions;
  s.counts = static_cast<int32_t*>(workspace);
  s.R = T * top_k;
  s.E = n_experts;
  s.first = first_expert;
  return report_hip(launch_sort_routes(s, static_cast<hipStream_t>(hip_stream)));
}

int moe_gather_rows_validate(int32_t T, int32_t top_k, int32_t rows, int32_t cols, const void* x, int64_t ldx,
                             int32_t type, const int32_t* positions, const int32_t* n_taken, const void* out,
                             int64_t ldo) {
  MOE_TRY(check_rows(T, top_k, rows, cols));
  MOE_TRY(check_matrix(T, cols, x, ldx, type));
  MOE_TRY(check_matrix(rows, cols, out, ldo, type));
  if (T > 0) MOE_TRY(need(positions, 4));
  return n_taken ? need(n_taken, 4) : MOE_OK;
}

int moe_gather_rows(int32_t T, int32_t top_k, int32_t rows, int32_t cols, const void* x, int64_t ldx, int32_t type,
                    const int32_t* positions, const int32_t* n_taken, void* out, int64_t ldo, void* hip_stream) {
  MOE_TRY(moe_gather_rows_validate(T, top_k, rows, cols, x, ldx, type, positions, n_taken, out, ldo));
  if (rows == 0 || (T == 0 && !n_taken)) return MOE_OK;
  RouteRows p{};
  p.positions = positions;
  p.n_taken = n_taken;
  p.x = x;
  p.out = out;
  p.ldx = ldx;
  p.ldo = ldo;
  p.T = T;
  p.K = top_k;
  p.rows = rows;
  p.cols = cols;
  p.x_f32 = type == MOE_TYPE_F32;
  return report_hip(launch_gather_rows(p, static_cast<hipStream_t>(hip_stream)));
}

int moe_combine_rows_validate(int32_t T, int32_t top_k, int32_t rows, int32_t cols, const void* x, int64_t ldx,
                              int32_t type, const int32_t* positions, const float* topk_w, const void* out,
                              int64_t ldo, int32_t out_type) {
  MOE_TRY(check_rows(T, top_k, rows, cols));
  MOE_TRY(check_matrix(rows, cols, x, ldx, type));
  MOE_TRY(check_matrix(T, cols, out, ldo, out_type));
  if (T > 0) MOE_TRY(need(positions, 4));
  return T > 0 && topk_w ? need(topk_w, 4) : MOE_OK;
}

int moe_combine_rows(int32_t T, int32_t top_k, int32_t rows, int32_t cols, const void* x, int64_t ldx, int32_t type,
                     const int32_t* positions, const float* topk_w, void* out, int64_t ldo, int32_t out_type,
                     void* hip_stream) {
  MOE_TRY(moe_combine_rows_validate(T, top_k, rows, cols, x, ldx, type, positions, topk_w, out, ldo, out_type));
  if (T == 0) return MOE_OK;
  RouteRows p{};
  p.positions = positions;
  p.w = topk_w;
  p.x = x;
  p.out = out;
  p.ldx = ldx;
  p.ldo = ldo;
  p.T = T;
  p.K = top_k;
  p.rows = rows;
  p.cols = cols;
  p.x_f32 = type == MOE_TYPE_F32;
  p.out_f32 = out_type == MOE_TYPE_F32;
  return report_hip(launch_combine_rows(p, static_cast<hipStream_t>(hip_stream)));
}

int moe_combine_rows_backward_validate(int32_t T, int32_t top_k, int32_t rows, int32_t cols, const void* grad_out,
                                       int64_t ldg, int32_t grad_type, const void* x, int64_t ldx, int32_t type,
                                       const int32_t* positions, const float* topk_w, const int32_t* n_taken,
                                       const void* grad_rows, int64_t ldr, const float* grad_w) {
  MOE_TRY(check_rows(T, top_k, rows, cols));
  MOE_TRY(type_ok(type));
  MOE_TRY(check_matrix(T, cols, grad_out, ldg, grad_type));
  if (!grad_rows && !grad_w && rows > 0 && T > 0) return MOE_EINVAL;
  if (grad_rows) MOE_TRY(check_matrix(rows, cols, grad_rows, ldr, type));
  if (grad_w) {
    MOE_TRY(check_matrix(rows, cols, x, ldx, type));
    MOE_TRY(need(grad_w, 4));
  }
  if (T > 0) {
    MOE_TRY(need(positions, 4));
    if (topk_w) MOE_TRY(need(topk_w, 4));
  }
  return n_taken ? need(n_taken, 4) : MOE_OK;
}

int moe_combine_rows_backward(int32_t T, int32_t top_k, int32_t rows, int32_t cols, const void* grad_out,
                              int64_t ldg, int32_t grad_type, const void* x, int64_t ldx, int32_t type,
                              const int32_t* positions, const float* topk_w, const int32_t* n_taken,
                              void* grad_rows, int64_t ldr, float* grad_w, void* hip_stream) {
  MOE_TRY(moe_combine_rows_backward_validate(T, top_k, rows, cols, grad_out, ldg, grad_type, x, ldx, type, positions,
                                             topk_w, n_taken, grad_rows, ldr, grad_w));
  if (T == 0 && (!grad_rows || !n_taken || rows == 0)) return MOE_OK;
  RouteRows p{};
  p.positions = positions;
  p.w = topk_w;
  p.n_taken = n_taken;
  p.x = grad_w ? x : nullptr;
  p.out = rows > 0 ? grad_rows : nullptr;
  p.grad = grad_out;
  p.dw = grad_w;
  p.ldx = grad_w ? ldx : 0;
  p.ldo = grad_rows ? ldr : 0;
  p.ldg = ldg;
  p.T = T;
  p.K = top_k;
  p.rows = rows;
  p.cols = cols;
  p.x_f32 = type == MOE_TYPE_F32;
  p.out_f32 = grad_type == MOE_TYPE_F32;
  return report_hip(launch_combine_backward(p, static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
