// fp8.h -- launchers of the 8-bit float (E4M3) kernels and of the balance
// loss (internal to libmoe).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kFp8Block = 128;      // values per activation scale; weight blocks are 128 x 128
constexpr int kFp8MaxExperts = 256; // four experts per lane of the group search

inline int fp8_blocks(int n) { return (n + kFp8Block - 1) / kFp8Block; }

// rows x cols values (bf16, or fp32 when f32) to codes and scales; swiglu:
// x rows hold 2 * cols values, cols gate then cols up.
struct Fp8Quant {
  const void* x;
  int64_t ldx;
  uint8_t* codes;
  float* scales;
  int rows, cols;
  bool f32, swiglu;
};
hipError_t launch_fp8_quant(const Fp8Quant& q, hipStream_t st);

// out[r][n] = sum over blocks b of xs[x(r)][b] * ws[n / 128][b] * (codes of
// row x(r) . codes of weight row n over block b). offsets == nullptr: one
// group of all rows, x(r) = r. Else expert e takes rows offsets[e] ..
// offsets[e + 1] - 1 against its own weights, and x(r) = r, or
// index[r] / index_div when index is given.
struct Fp8Gemm {
  const uint8_t* x;
  const float* xs;
  const uint8_t* w;
  const float* ws;
  void* out;
  const int32_t* offsets;
  const int32_t* index;
  int64_t ldx, ldo;
  int rows, x_rows, experts, N, K, index_div;
  bool f32;       // out fp32, else bf16
  bool exact;     // blocks are summed in fp32 (always when f32)
  bool out_vec;   // out rows take four-value stores (base and pitch aligned)
};
hipError_t launch_fp8_gemm(const Fp8Gemm& g, hipStream_t st);

}  // namespace moe
