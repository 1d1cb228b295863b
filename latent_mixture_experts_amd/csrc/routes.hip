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
// A stable counting sort: within an expert routes ascend. Lanes with the same
// expert find each other with eight ballots, a lane's rank among them is a
// popcount. Routes to no expert here take no place; what lies behind the last
// place becomes -1.
//
// Up to kOneGroup routes: one workgroup, each wavefront a run of routes, walked
// twice (counts, places). More: chunks of kChunk routes, counted by a workgroup
// each; a second launch gives every chunk's places, its workgroups each adding
// up the chunks before their own (up to kFewChunks, where that is little), or
// after a launch that turns the counts into places first.
constexpr int kSortWaves = 16, kRun = 128, kChunk = kSortWaves * kRun;
constexpr int kOneGroup = 3 * kChunk, kFewChunks = 64, kExperts = 256;

__device__ __forceinline__ int expert_of(const SortRoutes& s, int64_t r, int64_t end) {
  if (r >= end) return -1;
  const int64_t e = static_cast<int64_t>(s.ids[r]) - s.first;
  return e >= 0 && e < s.E ? static_cast<int>(e) : -1;
}

// Adds the routes of [begin, end) to this wavefront's counts.
__device__ __forceinline__ void count_routes(const SortRoutes& s, int64_t begin, int64_t end, int* count) {
  const int lane = threadIdx.x & 63;
  for (int64_t b = begin; b < end; b += 64) {
    const int e = expert_of(s, b + lane, end);
    const uint64_t same = same_id_mask(e, e >= 0);
    if (e >= 0 && (63 - __clzll(static_cast<long long>(same))) == lane) count[e] += __popcll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // (another lane adds to it next time)
  }
}
// Gives them their places, from each expert's next one.
__device__ __forceinline__ void place_routes(const SortRoutes& s, int64_t begin, int64_t end, int* next) {
  const int lane = threadIdx.x & 63;
  for (int64_t b = begin; b < end; b += 64) {
    const int64_t r = b + lane;
    const int e = expert_of(s, r, end);
    const uint64_t same = same_id_mask(e, e >= 0);
    int at = -1;
    if (e >= 0) {
      at = next[e] + __popcll(same & ((1ull << lane) - 1ull));
      s.sorted[at] = static_cast<int32_t>(r);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // (every lane has read before one adds)
      if ((63 - __clzll(static_cast<long long>(same))) == lane) next[e] += __popcll(same);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (r < end) s.positions[r] = at;
  }
}

// Exclusive scan over the values of threads 0..255 (all 1024 call), and their sum.
__device__ int scan_experts(int v, int* sums, int* total) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int incl = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(incl, d, 64);
    if (lane >= d) incl += o;
  }
  if (lane == 63 && wave < 4) sums[wave] = incl;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < 4; ++w) base += w < wave ? sums[w] : 0;
  *total = sums[0] + sums[1] + sums[2] + sums[3];
  __syncthreads();
  return base + incl - v;
}

// hist[w][e], counts of wavefront w: each becomes its first place, base + those
// of the wavefronts before. Threads below E.
__device__ __forceinline__ void places_of_waves(int (*hist)[kExperts], int e, int base) {
  for (int w = 0; w < kSortWaves; ++w) {
    const int c = hist[w][e];
    hist[w][e] = base;
    base += c;
  }
}

__global__ __launch_bounds__(1024) void sort_one_kernel(SortRoutes s) {
  __shared__ int hist[kSortWaves][kExperts];
  __shared__ int sums[4];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int i = tid; i < kSortWaves * kExperts; i += 1024) (&hist[0][0])[i] = 0;
  __syncthreads();
  const int seg = ((s.R + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  const int begin = min(wave * seg, s.R), end = min(begin + seg, s.R);
  count_routes(s, begin, end, hist[wave]);
  __syncthreads();
  int total = 0, all;
  if (tid < s.E)
    for (int w = 0; w < kSortWaves; ++w) total += hist[w][tid];
  const int off = scan_experts(tid < s.E ? total : 0, sums, &all);
  if (tid < s.E) {
    s.offsets[tid] = off;
    places_of_waves(hist, tid, off);
  }
  if (tid == 0) s.offsets[s.E] = all;
  __syncthreads();
  place_routes(s, begin, end, hist[wave]);
  for (int i = all + tid; i < s.R; i += 1024) s.sorted[i] = -1;
}

// counts[c][e]: routes of chunk c to expert e
__global__ __launch_bounds__(1024) void sort_count_kernel(SortRoutes s) {
  __shared__ int hist[kSortWaves][kExperts];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int i = tid; i < kSortWaves * kExperts; i += 1024) (&hist[0][0])[i] = 0;
  __syncthreads();
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * kChunk + wave * kRun;
  count_routes(s, begin, begin + kRun < s.R ? begin + kRun : s.R, hist[wave]);
  __syncthreads();
  if (tid < s.E) {
    int total = 0;
    for (int w = 0; w < kSortWaves; ++w) total += hist[w][tid];
    s.counts[static_cast<size_t>(blockIdx.x) * kExperts + tid] = total;
  }
}

// Many chunks: counts[c][e] becomes the number of e's routes in the chunks
// before c; counts[G][e] their sum. A workgroup takes 16 experts, its threads 64
// runs of chunks of each.
__global__ __launch_bounds__(1024) void sort_scan_kernel(SortRoutes s, int G) {
  __shared__ int sums[64][16];
  const int e = static_cast<int>(blockIdx.x) * 16 + (threadIdx.x & 15), run = threadIdx.x >> 4;
  const int per = (G + 63) / 64, c0 = min(run * per, G), c1 = min(c0 + per, G);
  int total = 0;
  if (e < s.E)
    for (int c = c0; c < c1; ++c) total += s.counts[static_cast<size_t>(c) * kExperts + e];
  sums[run][threadIdx.x & 15] = total;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < run; ++i) before += sums[i][threadIdx.x & 15];
  if (e < s.E) {
    for (int c = c0; c < c1; ++c) {
      int* at = s.counts + static_cast<size_t>(c) * kExperts + e;
      const int n = *at;
      *at = before;
      before += n;
    }
    if (run == 63) s.counts[static_cast<size_t>(G) * kExperts + e] = before;
  }
}

// SCANNED: counts as sort_scan_kernel leaves them, else as counted.
template <bool SCANNED>
__global__ __launch_bounds__(1024) void sort_place_kernel(SortRoutes s, int G) {
  __shared__ int hist[kSortWaves][kExperts];
  __shared__ int sums[4];
  __shared__ int part[2][4][kExperts];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int chunk = static_cast<int>(blockIdx.x);
  for (int i = tid; i < kSortWaves * kExperts; i += 1024) (&hist[0][0])[i] = 0;
  if constexpr (!SCANNED) {  // four threads to an expert
    const int e = tid & 255, q = tid >> 8;
    int before = 0, total = 0;
    if (e < s.E) {
#pragma unroll 8
      for (int c = q; c < G; c += 4) {
        const int n = s.counts[static_cast<size_t>(c) * kExperts + e];
        total += n;
        before += c < chunk ? n : 0;
      }
    }
    part[0][q][e] = before;
    part[1][q][e] = total;
  }
  __syncthreads();
  const int64_t begin = static_cast<int64_t>(chunk) * kChunk + wave * kRun;
  const int64_t end = begin + kRun < s.R ? begin + kRun : s.R;
  count_routes(s, begin, end, hist[wave]);
  __syncthreads();
  int before = 0, total = 0, all;
  if (tid < s.E) {
    if constexpr (SCANNED) {
      before = s.counts[static_cast<size_t>(chunk) * kExperts + tid];
      total = s.counts[static_cast<size_t>(G) * kExperts + tid];
    } else {
      before = part[0][0][tid] + part[0][1][tid] + part[0][2][tid] + part[0][3][tid];
      total = part[1][0][tid] + part[1][1][tid] + part[1][2][tid] + part[1][3][tid];
    }
  }
  const int off = scan_experts(total, sums, &all);
  if (tid < s.E) {
    places_of_waves(hist, tid, off + before);
    if (chunk == 0) s.offsets[tid] = off;
  }
  if (chunk == 0 && tid == 0) s.offsets[s.E] = all;
  __syncthreads();
  place_routes(s, begin, end, hist[wave]);
  const int64_t stop = static_cast<int64_t>(chunk + 1) * kChunk < s.R ? static_cast<int64_t>(chunk + 1) * kChunk : s.R;
  for (int64_t i = static_cast<int64_t>(chunk) * kChunk + tid; i < stop; i += 1024)
    if (i >= all) s.sorted[i] = -1;
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

size_t sort_workspace(int R, int) {
  if (R <= kOneGroup) return 0;
  return static_cast<size_t>((R + kChunk - 1) / kChunk + 1) * kExperts * sizeof(int32_t);
}

hipError_t launch_sort_routes(const SortRoutes& s, hipStream_t st) {
  if (s.R <= kOneGroup) {
    MOE_LAUNCH((sort_one_kernel), dim3(1), dim3(1024), 0, st, s);
    return hipGetLastError();
  }
  const int G = (s.R + kChunk - 1) / kChunk;
  MOE_LAUNCH((sort_count_kernel), dim3(G), dim3(1024), 0, st, s);
  if (G <= kFewChunks) {
    MOE_LAUNCH((sort_place_kernel<false>), dim3(G), dim3(1024), 0, st, s, G);
  } else {
    MOE_LAUNCH((sort_scan_kernel), dim3((s.E + 15) / 16), dim3(1024), 0, st, s, G);
    MOE_LAUNCH((sort_place_kernel<true>), dim3(G), dim3(1024), 0, st, s, G);
  }
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
