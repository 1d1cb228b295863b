// routes.h -- launchers of the sort of routes by expert and of the rows' way
// into that order and back (internal to libmoe).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// Route r of the R = T * K routes goes to expert ids[r] - first if that lies in
// [0, E); offsets [E + 1], sorted [R] (-1 behind the last), positions [R] (-1:
// not to any of them).
struct SortRoutes {
  const int32_t* ids;
  int32_t* offsets;
  int32_t* sorted;
  int32_t* positions;
  int32_t* counts;  // workspace
  int R, E, first;
};
size_t sort_workspace(int R);
hipError_t launch_sort_routes(const SortRoutes& s, hipStream_t st);

// The rows of T tokens' K routes: row positions[t * K + k] of `rows` rows; a
// position outside [0, rows) is none.
struct RouteRows {
  const int32_t* positions;
  const float* w;          // [T][K], or null: 1
  const int32_t* n_taken;  // or null; rows from there on become zeros
  const void* x;           // gather: [T][cols]; combine and its gradient: [rows][cols]
  void* out;               // gather: [rows][cols]; combine: [T][cols]; gradient: [rows][cols] or null
  const void* grad;        // gradient: [T][cols]
  float* dw;               // gradient: [T][K] or null
  int64_t ldx, ldo, ldg;
  int T, K, rows, cols;
  bool x_f32, out_f32;     // types of rows and of tokens (gather: both x_f32)
};
hipError_t launch_gather_rows(const RouteRows& p, hipStream_t st);
hipError_t launch_combine_rows(const RouteRows& p, hipStream_t st);
hipError_t launch_combine_backward(const RouteRows& p, hipStream_t st);

}  // namespace moe
