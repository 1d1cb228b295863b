// fp4.h -- launchers of the 4-bit float (MXFP4) rows and their products
// (internal to libmoe).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kFp4Group = 32;  // values per scale
enum { kBy16, kBy4, kBy1 };    // how many scales of a row one copy may take

// rows x cols values (bf16, or fp32 when f32) to codes [rows][cols/2] and
// scales [rows][cols/32]; swiglu: x rows hold 2 * cols values, cols gate then
// cols up.
struct Fp4Quant {
  const void* x;
  int64_t ldx;
  uint8_t* codes;
  uint8_t* scales;
  int rows, cols;
  bool f32, swiglu;
};
hipError_t launch_fp4_quant(const Fp4Quant& q, hipStream_t st);

// codes and scales back to values.
struct Fp4Dequant {
  const uint8_t* codes;
  const uint8_t* scales;
  void* out;
  int64_t ldo;
  int rows, cols;
  bool f32;
};
hipError_t launch_fp4_dequant(const Fp4Dequant& q, hipStream_t st);

// out[r][n] = sum over groups b of 32 of 2^(xs[x(r)][b] + ws[n][b] - 254) *
// (codes of row x(r) . codes of weight row n over group b). offsets ==
// nullptr: one group of all rows, x(r) = r. Else expert e takes rows
// offsets[e] .. offsets[e + 1] - 1 against its own weights, and x(r) = r, or
// index[r] / index_div when index is given.
struct Fp4Gemm {
  const uint8_t* x;
  const uint8_t* xs;
  const uint8_t* w;
  const uint8_t* ws;
  void* out;
  const int32_t* offsets;
  const int32_t* index;
  int64_t ldx, ldo;  // x: bytes between rows of codes; out: elements
  int rows, x_rows, experts, N, K, index_div;
  bool f32;       // out fp32, else bf16
  bool out_vec;   // out rows take four-value stores (base and pitch aligned)
  bool out_vec8;  // and eight-value ones (bf16)
  int scales;     // kBy16, kBy4: scale rows start at multiples of 16, 4 bytes, in x and w
};
hipError_t launch_fp4_gemm(const Fp4Gemm& g, hipStream_t st);

}  // namespace moe
