// balance.hip -- the router's balance and z losses with the routes per
// expert, and the gradient of the router logits.
//
//   p = softmax(logits[t]),  lse = log sum exp(logits[t])
//   c_e = routes to expert e, N = tokens that count (mask; not all logits -inf)
//   f_e = E c_e / (K N),  P_e = sum_t p_te / N
//   balance = sum_e f_e P_e,  z = sum_t lse_t^2 / N
//   dlogits = g_b/N p (f - f . p) + 2 g_z/N lse p
//             + for each of the token's routes: w_k (dw_k - w . dw) at its expert
// (f carries no gradient: the counts are a step function of the logits.)
//
// Memory bound: a token's logits are read once into registers, one row of 16
// lanes per token (E <= 256: at most 16 per lane, four neighbouring ones per
// 16-byte load), so that a softmax costs four DPP steps per reduction. The
// probability sums stay in registers over all tokens of a lane row, then are
// joined over the workgroup in LDS in a fixed order and over the workgroups
// by a second launch in workgroup order; counts are integer atomics in LDS.
// Both are the same from run to run.
#include "balance.h"
#include "device_common.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kBW = 256;        // threads of a workgroup: 16 tokens at a time
constexpr int kBTokens = 16;    // tokens a workgroup takes at once
constexpr int kMaxE = 256;

template <int CTRL>
__device__ __forceinline__ float row_move(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float row16_max_f32(float v) {
  v = fmaxf(v, row_move<0xB1>(v));
  v = fmaxf(v, row_move<0x4E>(v));
  v = fmaxf(v, row_move<0x124>(v));
  return fmaxf(v, row_move<0x128>(v));
}

// Expert i (0..15) of lane l of a token's 16 lanes: four neighbouring ones
// per group of 64.
__device__ __forceinline__ int expert_of(int l, int i) { return (i >> 2) * 64 + l * 4 + (i & 3); }

template <bool VEC>  // rows of logits start at 16-byte boundaries
__device__ __forceinline__ void load_row(const float* row, int E, int l, float v[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = q * 64 + l * 4;
    if (VEC && e + 4 <= E) {
      const float4 a = *reinterpret_cast<const float4*>(row + e);
      v[4 * q] = a.x, v[4 * q + 1] = a.y, v[4 * q + 2] = a.z, v[4 * q + 3] = a.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * q + i] = e + i < E ? row[e + i] : -INFINITY;
    }
  }
}

// v -> exp(v - max); the sum and the maximum (0 where every logit is -inf:
// the sum is 0 then, and the token does not count).
__device__ __forceinline__ void row_softmax(float v[16], float& sum, float& top) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) m = fmaxf(m, v[i]);
  m = row16_max_f32(m);
  top = m == -INFINITY ? 0.0f : m;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] = expf(v[i] - top);
    s += v[i];
  }
  sum = row16_sum_f32(s);
}

// One workgroup's tokens: those of index blockIdx.x, blockIdx.x + gridDim.x,
// ... in units of kBTokens. ONE: the only workgroup, which writes the results.
template <bool VEC, bool ONE>
__global__ __launch_bounds__(kBW) void balance_kernel(Balance p) {
  __shared__ int32_t cnt[kMaxE + 1];
  __shared__ float red[kBTokens][kMaxE + 1];
  const int l = threadIdx.x & 15, row = threadIdx.x >> 4;
  for (int i = threadIdx.x; i <= kMaxE; i += kBW) cnt[i] = 0;
  __syncthreads();
  float acc[16], zz = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
  for (int t0 = static_cast<int>(blockIdx.x) * kBTokens; t0 < p.T; t0 += static_cast<int>(gridDim.x) * kBTokens) {
    const int t = t0 + row;
    const bool in = t < p.T && (!p.mask || p.mask[t]);
    float v[16];
    if (in) {
      load_row<VEC>(p.logits + static_cast<size_t>(t) * p.E, p.E, l, v);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = -INFINITY;
    }
    float sum, top;
    row_softmax(v, sum, top);
    if (sum == 0.0f) continue;  // masked, or every logit -inf (uniform over the token's lanes)
    const float inv = 1.0f / sum;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = fmaf(v[i], inv, acc[i]);
    if (l < p.K) {
      const int id = p.ids[static_cast<size_t>(t) * p.K + l];
      if (id >= 0 && id < p.E) atomicAdd(&cnt[id], 1);
    }
    if (l == 0) {
      const float lse = top + logf(sum);
      zz = fmaf(lse, lse, zz);
      atomicAdd(&cnt[kMaxE], 1);
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) red[row][expert_of(l, i)] = acc[i];
  if (l == 0) red[row][kMaxE] = zz;
  __syncthreads();
  // column sums, rows in order: expert threadIdx.x, and the z sum
  float ps = 0.0f, zs = 0.0f;
#pragma unroll
  for (int r = 0; r < kBTokens; ++r) {
    ps += red[r][threadIdx.x];
    zs += red[r][kMaxE];
  }
  if constexpr (ONE) {
    const int e = threadIdx.x;
    const float n = static_cast<float>(max(cnt[kMaxE], 1));
    const float f = static_cast<float>(cnt[e]) * static_cast<float>(p.E) / (static_cast<float>(p.K) * n);
    __syncthreads();
    float s = wave_sum_f32(e < p.E ? f * (ps / n) : 0.0f);
    if ((e & 63) == 0) red[0][e >> 6] = s;
    if (e < p.E) p.counts[e] = cnt[e];
    if (e == 0) p.counts[p.E] = cnt[kMaxE];
    __syncthreads();
    if (e == 0) {
      p.loss[0] = ((red[0][0] + red[0][1]) + red[0][2]) + red[0][3];
      p.loss[1] = zs / n;
    }
  } else {
    const size_t at = static_cast<size_t>(blockIdx.x) * (p.E + 1);
    const int e = threadIdx.x;
    if (e < p.E) {
      p.part[at + e] = ps;
      p.part_counts[at + e] = cnt[e];
    }
    if (e == 0) {
      p.part[at + p.E] = zs;
      p.part_counts[at + p.E] = cnt[kMaxE];
    }
  }
}

// The partial sums of G workgroups: thread (s, e) adds those of workgroups
// s, s + 4, ... for expert e, then the four in order.
constexpr int kJoin = 4;
__global__ __launch_bounds__(kJoin * kMaxE) void balance_join_kernel(Balance p, int G) {
  __shared__ float ps[kJoin][kMaxE], zsh[kJoin * kMaxE / 64], out[kMaxE / 64];
  __shared__ int32_t cs[kJoin][kMaxE], nsh[kJoin * kMaxE / 64];
  const int tid = threadIdx.x, e = tid & (kMaxE - 1), s = tid / kMaxE;
  const size_t pitch = p.E + 1;
  float a = 0.0f;
  int32_t c = 0;
  if (e < p.E) {
#pragma unroll 8
    for (int g = s; g < G; g += kJoin) {
      a += p.part[g * pitch + e];
      c += p.part_counts[g * pitch + e];
    }
  }
  ps[s][e] = a;
  cs[s][e] = c;
  float z = 0.0f;
  int32_t n = 0;
  for (int g = tid; g < G; g += kJoin * kMaxE) {
    z += p.part[g * pitch + p.E];
    n += p.part_counts[g * pitch + p.E];
  }
  z = wave_sum_f32(z);
#pragma unroll
  for (int d = 1; d < 64; d *= 2) n += wave_shfl_xor(n, d);
  if ((tid & 63) == 0) {
    zsh[tid / 64] = z;
    nsh[tid / 64] = n;
  }
  __syncthreads();
  int32_t total = 0;
  float zt = 0.0f;
#pragma unroll
  for (int i = 0; i < kJoin * kMaxE / 64; ++i) {
    total += nsh[i];
    zt += zsh[i];
  }
  const float nf = static_cast<float>(max(total, 1));
  if (s == 0) {
    int32_t ct = 0;
    float pt = 0.0f;
#pragma unroll
    for (int i = 0; i < kJoin; ++i) {
      ct += cs[i][e];
      pt += ps[i][e];
    }
    const float f = static_cast<float>(ct) * static_cast<float>(p.E) / (static_cast<float>(p.K) * nf);
    const float v = wave_sum_f32(e < p.E ? f * (pt / nf) : 0.0f);
    if ((e & 63) == 0) out[e >> 6] = v;
    if (e < p.E) p.counts[e] = ct;
  }
  __syncthreads();
  if (tid == 0) {
    p.loss[0] = ((out[0] + out[1]) + out[2]) + out[3];
    p.loss[1] = zt / nf;
    p.counts[p.E] = total;
  }
}

template <bool VEC>
__global__ __launch_bounds__(kBW) void balance_backward_kernel(Balance p) {
  const int l = threadIdx.x & 15, row = threadIdx.x >> 4;
  const float n = static_cast<float>(max(p.counts_in[p.E], 1));
  const float gb = p.dloss[0] / n, gz = 2.0f * p.dloss[1] / n;
  float f[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int e = expert_of(l, i);
    f[i] = e < p.E ? static_cast<float>(p.counts_in[e]) * static_cast<float>(p.E) / (static_cast<float>(p.K) * n) : 0.0f;
  }
  for (int t0 = static_cast<int>(blockIdx.x) * kBTokens; t0 < p.T; t0 += static_cast<int>(gridDim.x) * kBTokens) {
    const int t = t0 + row;
    if (t >= p.T) continue;  // (uniform over the token's lanes)
    const bool in = !p.mask || p.mask[t];
    float v[16];
    if (in) {
      load_row<VEC>(p.logits + static_cast<size_t>(t) * p.E, p.E, l, v);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = -INFINITY;
    }
    // the gating weights' part: lane k < K holds w_k (dw_k - w . dw)
    int id = -1;
    float gate = 0.0f;
    if (p.w && in) {
      float w = 0.0f, dw = 0.0f;
      if (l < p.K) {
        const size_t at = static_cast<size_t>(t) * p.K + l;
        id = p.ids[at];
        w = p.w[at];
        dw = p.dw[at];
      }
      gate = w * (dw - row16_sum_f32(w * dw));
    }
    float sum, top;
    row_softmax(v, sum, top);
    if (sum == 0.0f) {  // does not count: no gradient
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    } else {
      const float inv = 1.0f / sum, zl = gz * (top + logf(sum));
      float fp = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        v[i] *= inv;
        fp = fmaf(f[i], v[i], fp);
      }
      fp = row16_sum_f32(fp);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] *= fmaf(gb, f[i] - fp, zl);
      if (p.w) {
        for (int k = 0; k < p.K; ++k) {  // (a token's routes in order; one listed twice adds twice)
          const int e = __shfl(id, k, 16);
          const float a = __shfl(gate, k, 16);
          const int i0 = (e >> 6) * 4 + (e & 3);
          if (e >= 0 && e < p.E && ((e >> 2) & 15) == l) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (i == i0) v[i] += a;
          }
        }
      }
    }
    float* o = p.dlogits + static_cast<size_t>(t) * p.E;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int e = q * 64 + l * 4;
      if (VEC && e + 4 <= p.E) {
        *reinterpret_cast<float4*>(o + e) = float4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (e + i < p.E) o[e + i] = v[4 * q + i];
      }
    }
  }
}

}  // namespace

// One workgroup up to 64 tokens (one launch writes the results), else up to
// four per CU.
int balance_workgroups(int T) {
  if (T <= 4 * kBTokens) return 1;
  const int n = (T + kBTokens - 1) / kBTokens;
  return n < 512 ? n : 512;
}

hipError_t launch_balance_loss(const Balance& b, hipStream_t st) {
  const int G = balance_workgroups(b.T);
  const bool vec = b.E % 4 == 0;
  if (G == 1) {
    if (vec)
      MOE_LAUNCH((balance_kernel<true, true>), dim3(1), dim3(kBW), 0, st, b);
    else
      MOE_LAUNCH((balance_kernel<false, true>), dim3(1), dim3(kBW), 0, st, b);
    return hipGetLastError();
  }
  if (vec)
    MOE_LAUNCH((balance_kernel<true, false>), dim3(G), dim3(kBW), 0, st, b);
  else
    MOE_LAUNCH((balance_kernel<false, false>), dim3(G), dim3(kBW), 0, st, b);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  MOE_LAUNCH((balance_join_kernel), dim3(1), dim3(kJoin * kMaxE), 0, st, b, G);
  return hipGetLastError();
}

hipError_t launch_balance_backward(const Balance& b, hipStream_t st) {
  const int n = (b.T + kBTokens - 1) / kBTokens;
  const dim3 grid(n < 2048 ? n : 2048);
  if (b.E % 4 == 0)
    MOE_LAUNCH((balance_backward_kernel<true>), grid, dim3(kBW), 0, st, b);
  else
    MOE_LAUNCH((balance_backward_kernel<false>), grid, dim3(kBW), 0, st, b);
  return hipGetLastError();
}

}  // namespace moe
