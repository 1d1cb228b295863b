// balance.h -- launchers of the balance loss (internal to libmoe).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

struct Balance {
  const float* logits;   // [T][E]
  const int32_t* ids;    // [T][K]
  const uint8_t* mask;   // [T] or null: tokens that count
  int T, E, K;
  // forward
  int32_t* counts;       // [E + 1]: routes per expert, tokens that count
  float* loss;           // [2]: balance, z
  void* part;            // workspace: partial sums of every workgroup
  // backward
  const int32_t* counts_in;
  const float* dloss;     // [2]
  const float* w;         // [T][K] gating weights, with
  const float* dw;        // [T][K] their gradients; both or neither
  float* dlogits;         // [T][E]
};
size_t balance_workspace(int T, int E);  // bytes; 0: none needed
hipError_t launch_balance_loss(const Balance& b, hipStream_t st);
hipError_t launch_balance_backward(const Balance& b, hipStream_t st);

}  // namespace moe
