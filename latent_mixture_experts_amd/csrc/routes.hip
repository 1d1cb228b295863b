// routes.hip -- routes sorted by expert, the tokens' rows into that order, and
// back with their weights, with the gradients.
//
//   rows[positions[t][k]] = x[t]                               (gather)
//   out[t] = sum_k w[t][k] * rows[positions[t][k]]             (combine)
//   drows[positions[t][k]] = w[t][k] * dout[t]
//   dw[t][k] = <rows[positions[t][k]], dout[t]>                (its gradient)
// (gather's gradient is combine without weights.)
//
// All of them walk the tokens, so a token's own row is read (or written) once
// and its K routes' rows once each, which is the least there is; the rows of
// one token lie anywhere, each in whole lines. Sums are fp32, over a token's
// routes in rank order; nothing depends on the order in which workgroups run.
#include "device_common.h"
#include "kernels.h"
#include "route_small.h"
#include "routes.h"

namespace moe {

namespace {

// ---- sort ------------------------------------------------------------------
// A stable counting sort: within an expert routes ascend. Routes to no expert
// here are one more bucket behind the last, so that every entry of sorted is
// written. Lanes with the same bucket find each other with nine ballots, a
// lane's rank among them is a popcount.
constexpr int kSortWaves = 16;
constexpr int kBuckets = 257;

__device__ __forceinline__ int bucket_of(const SortRoutes& s, int r) {
  const int64_t e = static_cast<int64_t>(s.ids[r]) - s.first;
  return e >= 0 && e < s.E ? static_cast<int>(e) : s.E;
}

// The lanes in range with this lane's bucket.
__device__ __forceinline__ uint64_t same_bucket(int e, bool valid) {
  const uint64_t top = __ballot(valid && e == 256);
  const uint64_t low = same_id_mask(e & 255, valid && e != 256);
  return e == 256 ? top : low;
}

// Exclusive scan over the values of threads 0..256 (all 1024 call).
__device__ int scan_buckets(int v, int* sums) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int incl = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(incl, d, 64);
    if (lane >= d) incl += o;
  }
  if (lane == 63) sums[wave] = incl;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < wave && w < 5; ++w) base += sums[w];
  __syncthreads();
  return base + incl - v;
}

__global__ __launch_bounds__(1024) void sort_routes_kernel(SortRoutes s) {
  __shared__ int hist[kSortWaves][kBuckets];
  __shared__ int sums[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i < kSortWaves * kBuckets; i += 1024) (&hist[0][0])[i] = 0;
  __syncthreads();
  const int seg = ((s.R + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  const int64_t begin = static_cast<int64_t>(wave) * seg;
  const int64_t end = begin + seg < s.R ? begin + seg : s.R;
  for (int64_t b = begin; b < end; b += 64) {
    const int64_t r = b + lane;
    const bool valid = r < end;
    const int e = valid ? bucket_of(s, static_cast<int>(r)) : 0;
    const uint64_t same = same_bucket(e, valid);
    if (valid && (63 - __clzll(static_cast<long long>(same))) == lane) hist[wave][e] += __popcll(same);
  }
  __syncthreads();
  int total = 0;
  if (tid <= s.E)
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = hist[w][tid];
      hist[w][tid] = total;
      total += c;
    }
  const int off = scan_buckets(tid <= s.E ? total : 0, sums);
  if (tid <= s.E) {
    s.offsets[tid] = off;
    for (int w = 0; w < kSortWaves; ++w) hist[w][tid] += off;
  }
  __syncthreads();
  for (int64_t b = begin; b < end; b += 64) {
    const int64_t r = b + lane;
    const bool valid = r < end;
    const int e = valid ? bucket_of(s, static_cast<int>(r)) : 0;
    const uint64_t same = same_bucket(e, valid);
    if (valid) {
      const int at = hist[wave][e] + __popcll(same & ((1ull << lane) - 1ull));
      s.sorted[at] = e < s.E ? static_cast<int32_t>(r) : -1;
      s.positions[r] = e < s.E ? at : -1;
      if ((63 - __clzll(static_cast<long long>(same))) == lane) hist[wave][e] += __popcll(same);
    }
  }
}

// ---- rows ------------------------------------------------------------------
constexpr int kMaxK = 8;

template <bool F32, int V>
__device__ __forceinline__ void load_row(const void* x, int64_t at, float v[V]) {
  if constexpr (V == 1) {
    v[0] = F32 ? static_cast<const float*>(x)[at] : bf16_to_f32(static_cast<const uint16_t*>(x)[at]);
  } else if constexpr (F32) {
#pragma unroll
    for (int h = 0; h < V / 4; ++h) {
      const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + at + 4 * h);
      v[4 * h] = a.x, v[4 * h + 1] = a.y, v[4 * h + 2] = a.z, v[4 * h + 3] = a.w;
    }
  } else {
    static_assert(V == 8, "16 bytes");
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at);
    const uint32_t d[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(d[i] << 16);
      v[2 * i + 1] = __uint_as_float(d[i] & 0xFFFF0000u);
    }
  }
}
template <bool F32, int V>
__device__ __forceinline__ void store_row(void* x, int64_t at, const float v[V]) {
  if constexpr (V == 1) {
    if constexpr (F32)
      static_cast<float*>(x)[at] = v[0];
    else
      static_cast<__bf16*>(x)[at] = static_cast<__bf16>(v[0]);
  } else if constexpr (F32) {
#pragma unroll
    for (int h = 0; h < V / 4; ++h)
      *reinterpret_cast<float4*>(static_cast<float*>(x) + at + 4 * h) = float4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
  } else {
    bf16x8 b;
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = static_cast<__bf16>(v[i]);
    *reinterpret_cast<bf16x8*>(static_cast<uint16_t*>(x) + at) = b;
  }
}

// Rows from *n_taken on become zeros, by all workgroups.
template <bool F32, int V>
__device__ __forceinline__ void zero_rest(const RouteRows& p) {
  if (!p.n_taken) return;
  const float zero[V] = {};
  for (int64_t r = static_cast<int64_t>(max(*p.n_taken, 0)) + blockIdx.x; r < p.rows; r += gridDim.x)
    for (int c = threadIdx.x * V; c < p.cols; c += 256 * V) store_row<F32, V>(p.out, r * p.ldo + c, zero);
}

// A token's rows; -1: none.
__device__ __forceinline__ void positions_of(const RouteRows& p, int64_t t, int at[kMaxK]) {
#pragma unroll
  for (int k = 0; k < kMaxK; ++k) {
    const int v = k < p.K ? p.positions[t * p.K + k] : -1;
    at[k] = v >= 0 && v < p.rows ? v : -1;
  }
}

// One wavefront per token, over the columns.
template <bool F32, int V>
__global__ __launch_bounds__(256) void gather_rows_kernel(RouteRows p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + wave; t < p.T; t += static_cast<int64_t>(gridDim.x) * 4) {
    int at[kMaxK];
    positions_of(p, t, at);
    for (int c = lane * V; c < p.cols; c += 64 * V) {
      float v[V];
      load_row<F32, V>(p.x, t * p.ldx + c, v);
#pragma unroll
      for (int k = 0; k < kMaxK; ++k)
        if (at[k] >= 0) store_row<F32, V>(p.out, at[k] * p.ldo + c, v);
    }
  }
  zero_rest<F32, V>(p);
}

template <bool XF32, bool OF32, int V>
__global__ __launch_bounds__(256) void combine_rows_kernel(RouteRows p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + wave; t < p.T; t += static_cast<int64_t>(gridDim.x) * 4) {
    int at[kMaxK];
    positions_of(p, t, at);
    float w[kMaxK];
#pragma unroll
    for (int k = 0; k < kMaxK; ++k) w[k] = at[k] >= 0 && p.w ? p.w[t * p.K + k] : 1.0f;
    for (int c = lane * V; c < p.cols; c += 64 * V) {
      float v[kMaxK][V], sum[V] = {};
#pragma unroll
      for (int k = 0; k < kMaxK; ++k)
        if (at[k] >= 0) load_row<XF32, V>(p.x, at[k] * p.ldx + c, v[k]);
#pragma unroll
      for (int k = 0; k < kMaxK; ++k)
        if (at[k] >= 0) {
#pragma unroll
          for (int i = 0; i < V; ++i) sum[i] = fmaf(w[k], v[k][i], sum[i]);
        }
      store_row<OF32, V>(p.out, t * p.ldo + c, sum);
    }
  }
}

template <bool XF32, bool GF32, int V>
__global__ __launch_bounds__(256) void combine_backward_kernel(RouteRows p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + wave; t < p.T; t += static_cast<int64_t>(gridDim.x) * 4) {
    int at[kMaxK];
    positions_of(p, t, at);
    float w[kMaxK], dot[kMaxK] = {};
#pragma unroll
    for (int k = 0; k < kMaxK; ++k) w[k] = at[k] >= 0 && p.w ? p.w[t * p.K + k] : 1.0f;
    for (int c = lane * V; c < p.cols; c += 64 * V) {
      float g[V], v[kMaxK][V];
      load_row<GF32, V>(p.grad, t * p.ldg + c, g);
      if (p.dw) {
#pragma unroll
        for (int k = 0; k < kMaxK; ++k)
          if (at[k] >= 0) load_row<XF32, V>(p.x, at[k] * p.ldx + c, v[k]);
#pragma unroll
        for (int k = 0; k < kMaxK; ++k)
          if (at[k] >= 0) {
#pragma unroll
            for (int i = 0; i < V; ++i) dot[k] = fmaf(v[k][i], g[i], dot[k]);
          }
      }
      if (p.out) {
#pragma unroll
        for (int k = 0; k < kMaxK; ++k)
          if (at[k] >= 0) {
            float d[V];
#pragma unroll
            for (int i = 0; i < V; ++i) d[i] = w[k] * g[i];
            store_row<XF32, V>(p.out, at[k] * p.ldo + c, d);
          }
      }
    }
    if (p.dw) {
#pragma unroll
      for (int k = 0; k < kMaxK; ++k) {
        const float sum = wave_sum_f32(dot[k]);
        if (k < p.K && lane == 0) p.dw[t * p.K + k] = sum;
      }
    }
  }
  if (p.out) zero_rest<XF32, V>(p);
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Rows of eight values at a time: every row starts at a multiple of 16 bytes
// and holds whole eights.
bool eights(const RouteRows& p) {
  return p.cols % 8 == 0 && p.ldx % 8 == 0 && p.ldo % 8 == 0 && p.ldg % 8 == 0 && aligned16(p.x) && aligned16(p.out) &&
         aligned16(p.grad);
}

dim3 token_grid(int T) { return dim3(static_cast<unsigned>(T < 1 ? 1 : T < (1 << 22) ? (T + 3) / 4 : 1 << 20)); }

}  // namespace

size_t sort_workspace(int, int) { return 0; }

hipError_t launch_sort_routes(const SortRoutes& s, hipStream_t st) {
  MOE_LAUNCH((sort_routes_kernel), dim3(1), dim3(1024), 0, st, s);
  return hipGetLastError();
}

hipError_t launch_gather_rows(const RouteRows& p, hipStream_t st) {
  const dim3 grid = token_grid(p.T), block(256);
  if (p.x_f32)
    eights(p) ? MOE_LAUNCH((gather_rows_kernel<true, 8>), grid, block, 0, st, p)
              : MOE_LAUNCH((gather_rows_kernel<true, 1>), grid, block, 0, st, p);
  else
    eights(p) ? MOE_LAUNCH((gather_rows_kernel<false, 8>), grid, block, 0, st, p)
              : MOE_LAUNCH((gather_rows_kernel<false, 1>), grid, block, 0, st, p);
  return hipGetLastError();
}

template <bool XF32, bool OF32>
static void combine_as(const RouteRows& p, bool backward, hipStream_t st) {
  const dim3 grid = token_grid(p.T), block(256);
  if (backward)
    eights(p) ? MOE_LAUNCH((combine_backward_kernel<XF32, OF32, 8>), grid, block, 0, st, p)
              : MOE_LAUNCH((combine_backward_kernel<XF32, OF32, 1>), grid, block, 0, st, p);
  else
    eights(p) ? MOE_LAUNCH((combine_rows_kernel<XF32, OF32, 8>), grid, block, 0, st, p)
              : MOE_LAUNCH((combine_rows_kernel<XF32, OF32, 1>), grid, block, 0, st, p);
}
static hipError_t combine(const RouteRows& p, bool backward, hipStream_t st) {
  if (p.x_f32)
    p.out_f32 ? combine_as<true, true>(p, backward, st) : combine_as<true, false>(p, backward, st);
  else
    p.out_f32 ? combine_as<false, true>(p, backward, st) : combine_as<false, false>(p, backward, st);
  return hipGetLastError();
}
hipError_t launch_combine_rows(const RouteRows& p, hipStream_t st) { return combine(p, false, st); }
hipError_t launch_combine_backward(const RouteRows& p, hipStream_t st) { return combine(p, true, st); }

}  // namespace moe
