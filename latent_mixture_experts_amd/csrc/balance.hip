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
// A token's logits are read once into registers, one row of 16 lanes per
// token (E <= 256: at most 16 per lane, four neighbouring ones per 16-byte
// load), so that a reduction costs four DPP steps. The probability sums stay
// in registers over all tokens of a lane row, then are joined over the
// workgroup in a fixed order, and over the workgroups by a second launch;
// counts are integer atomics in LDS. Both are the same from run to run.
// Bound by latency (by events over a captured graph; a trace of single launches
// says up to 1.7 us more each): 61 tokens of 16 experts 6.1 us forward (one
// workgroup), 4.7 backward; 4096 tokens of 256 experts 10.4 and 6.0; 32767 tokens
// 18.6 .. 19.2 (the join by one CU 7.6 of it) and 17.7, 3.8 TB/s.
#include "balance.h"
#include "device_common.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kMaxE = 256;
// Forward: 64 tokens at once, and at most one workgroup per CU, so that the one
// workgroup that joins their sums reads little.
constexpr int kFThreads = 1024, kFWaves = kFThreads / 64, kFTokens = kFThreads / 16, kFGroups = 256;
// Tokens of a lane row that are summed in fp32 before their sum is taken over
// into 64 bits: over thousands of like-signed additions an fp32 sum drifts (2^26
// tokens: 2.5e-5 and 4.6e-5 of the two losses). Calls with fewer take a kernel
// without the 64-bit sums, whose registers cost 0.4 .. 1 us (61 tokens 6.1 us
// against 6.5, 32767 tokens 18.6 against 19.7).
constexpr int kFRun = 32;
constexpr int kBThreads = 256, kBTokens = kBThreads / 16;  // backward

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

// exp(d) for d <= 0 through the exponential instruction (1 ulp); the error of
// the exponent's rounding, up to |d| * 2^-24 of the result, is taken back by
// its low part. Below -200 the result is 0 (the bound keeps -inf out of the low
// part); NaN stays NaN.
__device__ __forceinline__ float exp_neg(float d) {
  constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f, kLn2 = 0.693147182f;
  d = d < -200.0f ? -200.0f : d;
  const float t = d * kLog2e;
  const float low = fmaf(d, kLog2eLow, fmaf(d, kLog2e, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return fmaf(e * kLn2, low, e);
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
    v[i] = exp_neg(v[i] - top);
    s += v[i];
  }
  sum = row16_sum_f32(s);
}

struct Partial {  // of one workgroup and expert (the last: the z sum, the tokens that count)
  float p;
  int32_t n;
};
// Partials of one workgroup: even, so that pairs of them are 16-byte aligned.
__host__ __device__ inline size_t partial_pitch(int E) { return (static_cast<size_t>(E) + 2) & ~size_t{1}; }

// One workgroup's tokens: those of index blockIdx.x, blockIdx.x + gridDim.x,
// ... in units of kFTokens. ONE: the only workgroup, which writes the results.
// LONG: a lane row may take more than kFRun tokens.
template <bool VEC, bool ONE, bool LONG>
__global__ __launch_bounds__(kFThreads) void balance_kernel(Balance p) {
  __shared__ int32_t cnt[kMaxE + 1];
  __shared__ float red[kFWaves][kMaxE + 1];
  const int l = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = threadIdx.x; i <= kMaxE; i += kFThreads) cnt[i] = 0;
  __syncthreads();
  float acc[16], zz = 0.0f;
  [[maybe_unused]] double far[16], far_z = 0.0;
  [[maybe_unused]] int run = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    acc[i] = 0.0f;
    far[i] = 0.0;
  }
  for (int t0 = static_cast<int>(blockIdx.x) * kFTokens; t0 < p.T; t0 += static_cast<int>(gridDim.x) * kFTokens) {
    if (LONG && run++ == kFRun) {
      run = 1;
      far_z += zz;
      zz = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        far[i] += acc[i];
        acc[i] = 0.0f;
      }
    }
    const int t = t0 + row;
    const bool in = t < p.T && (!p.mask || p.mask[t]);
    float v[16];
    if (in) {
      load_row<VEC>(p.logits + static_cast<size_t>(t) * p.E, p.E, l, v);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = -INFINITY;
    }
    const int id = in && l < p.K ? p.ids[static_cast<size_t>(t) * p.K + l] : -1;
    float sum, top;
    row_softmax(v, sum, top);
    if (sum == 0.0f) continue;  // masked, or every logit -inf (uniform over the token's lanes)
    const float inv = 1.0f / sum;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = fmaf(v[i], inv, acc[i]);
    if (id >= 0 && id < p.E) atomicAdd(&cnt[id], 1);
    if (l == 0) {
      const float lse = top + logf(sum);
      zz = fmaf(lse, lse, zz);
      atomicAdd(&cnt[kMaxE], 1);
    }
  }
  if constexpr (LONG) {
    zz = static_cast<float>(far_z + zz);
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = static_cast<float>(far[i] + acc[i]);
  }
  // the wavefront's four tokens; lane row r keeps experts of i = 4r .. 4r+3
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    acc[i] += wave_shfl_xor(acc[i], 16);
    acc[i] += wave_shfl_xor(acc[i], 32);
    if ((i >> 2) == (lane >> 4)) red[wave][expert_of(l, i)] = acc[i];
  }
  zz += wave_shfl_xor(zz, 16);
  zz += wave_shfl_xor(zz, 32);
  if (lane == 0) red[wave][kMaxE] = zz;
  __syncthreads();
  // sums over the wavefronts, in order: expert threadIdx.x, and the z sum
  const int e = threadIdx.x;
  float ps = 0.0f, zs = 0.0f;
  if (e < kMaxE) {
#pragma unroll
    for (int r = 0; r < kFWaves; ++r) {
      ps += red[r][e];
      zs += red[r][kMaxE];
    }
  }
  if constexpr (ONE) {
    const float n = static_cast<float>(max(cnt[kMaxE], 1));
    float s = 0.0f;
    if (e < p.E) {
      s = static_cast<float>(cnt[e]) * static_cast<float>(p.E) / (static_cast<float>(p.K) * n) * (ps / n);
      p.counts[e] = cnt[e];
    }
    __syncthreads();
    s = wave_sum_f32(s);
    if (lane == 0) red[0][wave] = s;
    __syncthreads();
    if (e == 0) {
      p.loss[0] = ((red[0][0] + red[0][1]) + red[0][2]) + red[0][3];
      p.loss[1] = zs / n;
      p.counts[p.E] = cnt[kMaxE];
    }
  } else {
    Partial* out = static_cast<Partial*>(p.part) + blockIdx.x * partial_pitch(p.E);
    if (e < p.E) out[e] = Partial{ps, cnt[e]};
    if (e == 0) out[p.E] = Partial{zs, cnt[kMaxE]};
  }
}

// The partial sums of G workgroups: thread (s, c) adds those of workgroups s,
// s + S, ... for experts 2c and 2c + 1, S sets of 2^log_c threads (16-byte
// loads, up to 16 of them in flight per thread: one CU reads it all, at the rate
// of what it has outstanding), then the S sums in order.
constexpr int kJThreads = 1024;
__global__ __launch_bounds__(kJThreads) void balance_join_kernel(Balance p, int G, int log_c) {
  constexpr int kWaves = kJThreads / 64;
  __shared__ Partial ps[2 * kJThreads];
  __shared__ float zsh[kWaves], out[kMaxE / 64];
  __shared__ int32_t nsh[kWaves];
  static_assert(kFGroups <= kJThreads, "a thread per workgroup's z sum");
  const int tid = threadIdx.x, c = tid & ((1 << log_c) - 1), s = tid >> log_c, sets = kJThreads >> log_c;
  const Partial* in = static_cast<const Partial*>(p.part);
  const size_t pitch = partial_pitch(p.E);
  Partial a{0.0f, 0}, b{0.0f, 0};
  if (2 * c < p.E) {
#pragma unroll 16
    for (int g = s; g < G; g += sets) {
      const int4 v = *reinterpret_cast<const int4*>(in + g * pitch + 2 * c);
      a.p += __int_as_float(v.x);
      a.n += v.y;
      b.p += __int_as_float(v.z);
      b.n += v.w;
    }
  }
  ps[2 * tid] = a;
  ps[2 * tid + 1] = b;  // (past the last expert: the z sum or nothing, not used)
  Partial z{0.0f, 0};
  if (tid < G) z = in[tid * pitch + p.E];
  z.p = wave_sum_f32(z.p);
#pragma unroll
  for (int d = 1; d < 64; d *= 2) z.n += wave_shfl_xor(z.n, d);
  if ((tid & 63) == 0) {
    zsh[tid / 64] = z.p;
    nsh[tid / 64] = z.n;
  }
  __syncthreads();
  int32_t total = 0;
  float zt = 0.0f;
#pragma unroll
  for (int i = 0; i < (kFGroups + 63) / 64; ++i) {
    total += nsh[i];
    zt += zsh[i];
  }
  const float nf = static_cast<float>(max(total, 1));
  if (tid < kMaxE) {
    const int e = tid;
    Partial t{0.0f, 0};
    if (e < p.E)
      for (int i = 0; i < sets; ++i) {
        t.p += ps[(i << (log_c + 1)) + e].p;
        t.n += ps[(i << (log_c + 1)) + e].n;
      }
    const float f = static_cast<float>(t.n) * static_cast<float>(p.E) / (static_cast<float>(p.K) * nf);
    const float v = wave_sum_f32(e < p.E ? f * (t.p / nf) : 0.0f);
    if ((e & 63) == 0) out[e >> 6] = v;
    if (e < p.E) p.counts[e] = t.n;
  }
  __syncthreads();
  if (tid == 0) {
    p.loss[0] = ((out[0] + out[1]) + out[2]) + out[3];
    p.loss[1] = zt / nf;
    p.counts[p.E] = total;
  }
}

// Lane K of each row of 16 lanes, in every lane of the row.
template <int K>
__device__ __forceinline__ int row_lane(int v) {
  return __builtin_amdgcn_mov_dpp(v, 0x150 | K, 0xF, 0xF, false);
}

// Lane k's gate, plus those of the token's other routes to the same expert,
// in route order; -1 for the expert of all but the first of them, and of ids
// outside the experts.
template <int K = 0>
__device__ __forceinline__ void join_routes(int id, float gate, int l, float& sum, bool& first) {
  if constexpr (K < 8) {
    const bool same = row_lane<K>(id) == id;
    const float g = __builtin_bit_cast(float, row_lane<K>(__builtin_bit_cast(int, gate)));
    if (same) sum += g;
    if (same && K < l) first = false;
    join_routes<K + 1>(id, gate, l, sum, first);
  }
}

// LDS that other lanes of the wavefront wrote: the hardware keeps a wavefront's
// accesses in order, and this keeps the compiler to it.
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
}

// GATE: with the gating weights' part. Each token has a row of LDS for it,
// zero but for the experts its routes go to, which every lane reads beside
// its logits; the rows belong to one wavefront, so nothing is waited for.
template <bool VEC, bool GATE>
__global__ __launch_bounds__(kBThreads) void balance_backward_kernel(Balance p) {
  __shared__ __attribute__((aligned(16))) float gates[GATE ? kBTokens : 1][kMaxE];
  const int l = threadIdx.x & 15, row = threadIdx.x >> 4;
  if constexpr (GATE) {
#pragma unroll
    for (int q = 0; q < 4; ++q) *reinterpret_cast<float4*>(&gates[row][q * 64 + l * 4]) = float4{0.f, 0.f, 0.f, 0.f};
    wave_lds_order();
  }
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
    int id = -1;
    float w = 0.0f, dw = 0.0f;
    if (GATE && in && l < p.K) {
      const size_t at = static_cast<size_t>(t) * p.K + l;
      id = p.ids[at];
      if (id >= p.E) id = -1;
      w = p.w[at];
      dw = p.dw[at];
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
      if constexpr (GATE) {
        const float gate = w * (dw - row16_sum_f32(w * dw));  // (0 in lanes without a route)
        float joined = 0.0f;
        bool first = id >= 0;
        join_routes(id, gate, l, joined, first);
        if (first) gates[row][id] = joined;
        wave_lds_order();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 g = *reinterpret_cast<const float4*>(&gates[row][q * 64 + l * 4]);
          v[4 * q] += g.x, v[4 * q + 1] += g.y, v[4 * q + 2] += g.z, v[4 * q + 3] += g.w;
        }
        wave_lds_order();
        if (first) gates[row][id] = 0.0f;
        wave_lds_order();
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

// One workgroup up to 64 tokens (one launch writes the results).
int balance_workgroups(int T) {
  const int n = (T + kFTokens - 1) / kFTokens;
  return n < 1 ? 1 : n < kFGroups ? n : kFGroups;
}
size_t balance_workspace(int T, int E) {
  const int G = balance_workgroups(T);
  return G == 1 ? 0 : G * partial_pitch(E) * sizeof(Partial);
}

template <bool ONE, bool LONG>
hipError_t launch_sums(const Balance& b, int G, hipStream_t st) {
  if (b.E % 4 == 0)
    MOE_LAUNCH((balance_kernel<true, ONE, LONG>), dim3(G), dim3(kFThreads), 0, st, b);
  else
    MOE_LAUNCH((balance_kernel<false, ONE, LONG>), dim3(G), dim3(kFThreads), 0, st, b);
  return hipGetLastError();
}

hipError_t launch_balance_loss(const Balance& b, hipStream_t st) {
  const int G = balance_workgroups(b.T);
  if (G == 1) return launch_sums<true, false>(b, G, st);
  const bool many = b.T > kFRun * kFTokens * kFGroups;
  const hipError_t e = many ? launch_sums<false, true>(b, G, st) : launch_sums<false, false>(b, G, st);
  if (e != hipSuccess) return e;
  int log_c = 5;  // at least 32 pairs of experts, so at most 32 sets
  while ((2 << log_c) < b.E) ++log_c;
  MOE_LAUNCH((balance_join_kernel), dim3(1), dim3(kJThreads), 0, st, b, G, log_c);
  return hipGetLastError();
}

template <bool GATE>
hipError_t launch_backward(const Balance& b, hipStream_t st) {
  const int n = (b.T + kBTokens - 1) / kBTokens;
    // (32767 tokens of 256 experts: 22 us in workgroups of one pass, 17.6 in 1024)
  const dim3 grid(n < 1024 ? n : 1024);
  if (b.E % 4 == 0)
    MOE_LAUNCH((balance_backward_kernel<true, GATE>), grid, dim3(kBThreads), 0, st, b);
  else
    MOE_LAUNCH((balance_backward_kernel<false, GATE>), grid, dim3(kBThreads), 0, st, b);
  return hipGetLastError();
}
hipError_t launch_balance_backward(const Balance& b, hipStream_t st) {
  return b.w ? launch_backward<true>(b, st) : launch_backward<false>(b, st);
}

}  // namespace moe
