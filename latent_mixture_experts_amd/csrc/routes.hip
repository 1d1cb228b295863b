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
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "kernels.h"
#include "route_small.h"
#include "routes.h"
#include "silu.h"

namespace moe {

namespace {

// ---- sort ------------------------------------------------------------------
// A stable counting sort: within an expert routes ascend. Lanes with the same
// expert find each other with eight ballots, a lane's rank among them is a
// popcount. Routes to no expert here take no place; what lies behind the last
// place becomes -1.
//
// Up to kOneGroup routes: one workgroup, each wavefront a run of routes, walked
// twice (counts, places; 2048 routes 5.9 us against 7.2 in two launches, 2560 7.4
// against 7.3, 4096 8.8 against 7.3). More: chunks of a run for each of a workgroup's
// wavefronts, counted by a workgroup each; a second launch gives every chunk's
// places, its workgroups each adding up the chunks before their own (up to
// kFewRoutes, where that is little, in runs of one step), or after a launch that
// turns the counts into places first (longer runs: fewer counts to write and
// read). All latency: 64 routes 3.9 us, 4096 7.9, 32768 8.6 (runs of two steps 11.3),
// 262136 13.3; 8 million 103 us (runs of two steps 125, of one 167).
constexpr int kSortWaves = 16, kOneGroup = 2560, kFewRoutes = 1 << 18, kExperts = 256;
constexpr int kShortRun = 64, kLongRun = 256;
__host__ __device__ constexpr int chunk_of(int R) { return kSortWaves * (R <= kFewRoutes ? kShortRun : kLongRun); }

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
  const int run = chunk_of(s.R) / kSortWaves;
  const int64_t begin = (static_cast<int64_t>(blockIdx.x) * kSortWaves + wave) * run;
  count_routes(s, begin, begin + run < s.R ? begin + run : s.R, hist[wave]);
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
  const int run = chunk_of(s.R) / kSortWaves;
  const int64_t begin = (static_cast<int64_t>(chunk) * kSortWaves + wave) * run;
  const int64_t end = begin + run < s.R ? begin + run : s.R;
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
  const int64_t first = static_cast<int64_t>(chunk) * kSortWaves * run, after = first + kSortWaves * run;
  for (int64_t i = first + tid; i < (after < s.R ? after : s.R); i += 1024)
    if (i >= all) s.sorted[i] = -1;
}

// ---- rows ------------------------------------------------------------------
// A wavefront takes spans of kSpan columns of a token, eight values a lane: eight
// neighbours where rows allow it (VEC), else 64 apart. Tokens start at different
// spans: their rows lie a power of two apart as a rule, and wavefronts that walk
// them in step meet on the same memory channels. Stores of whole pieces pass the
// caches by, which leaves those to the rows that are read (4096 tokens of 8 rows of
// 4096 bf16, in one stream: sort, gather and its gradient 149 -> 124 us, combine and
// its gradient 183 -> 160; loads that do so instead: 130 and 180; 8352 tokens of 7 rows
// of 376 fp32, combine and its gradient: 62 -> 56, loads 69). What reads the stored
// rows next pays for it or not: gather, then moe_fp4_quantize of its rows, 4096 tokens
// 111 us (107 with stores through the caches, which make the gather alone 61 instead
// of 53), 1024 tokens 33 (29), 128 tokens 9.2 (10.1); combine, then its quantisation,
// 68 (70), 21 (20) and 7.9 (7.7).
constexpr int kMaxK = 8, kSpan = 512;

__device__ __forceinline__ void store16(void* p, uint4 v) {
  __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), static_cast<u32x4*>(p));
}

template <bool F32, bool VEC>
__device__ __forceinline__ void load_span(const void* x, int64_t row, int c, int cols, float v[8]) {
  if constexpr (VEC) {
    load8<F32>(x, row + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t at = row + c + 64 * i;
      v[i] = 0.0f;
      if (c + 64 * i < cols) v[i] = F32 ? static_cast<const float*>(x)[at] : bf16_to_f32(static_cast<const uint16_t*>(x)[at]);
    }
  }
}
template <bool F32, bool VEC>
__device__ __forceinline__ void store_span(void* x, int64_t row, int c, int cols, const float v[8]) {
  if constexpr (VEC) {
    if constexpr (F32) {
      float* o = static_cast<float*>(x) + row + c;
      store16(o, __builtin_bit_cast(uint4, f32x4{v[0], v[1], v[2], v[3]}));
      store16(o + 4, __builtin_bit_cast(uint4, f32x4{v[4], v[5], v[6], v[7]}));
    } else {
      bf16x8 b;
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = static_cast<__bf16>(v[i]);
      store16(static_cast<uint16_t*>(x) + row + c, __builtin_bit_cast(uint4, b));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t at = row + c + 64 * i;
      if (c + 64 * i < cols) {
        if constexpr (F32)
          static_cast<float*>(x)[at] = v[i];
        else
          static_cast<__bf16*>(x)[at] = static_cast<__bf16>(v[i]);
      }
    }
  }
}
// A lane's first column in a span.
template <bool VEC>
__device__ __forceinline__ int span_column(int span, int lane) {
  return span * kSpan + (VEC ? lane * 8 : lane);
}

// Rows from *n_taken on become zeros, by all workgroups.
template <bool F32, bool VEC>
__device__ __forceinline__ void zero_rest(const RouteRows& p) {
  if (!p.n_taken) return;
  const float zero[8] = {};
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, spans = (p.cols + kSpan - 1) / kSpan;
  for (int64_t r = static_cast<int64_t>(max(*p.n_taken, 0)) + blockIdx.x; r < p.rows; r += gridDim.x)
    for (int s = wave; s < spans; s += 4) {
      const int c = span_column<VEC>(s, lane);
      if (c < p.cols) store_span<F32, VEC>(p.out, r * p.ldo, c, p.cols, zero);
    }
}

// A token's rows (-1: none) and, asked for, its weights: lane k loads those of
// route k, and all of them go to scalar registers (one load's latency, not K).
struct TokenRoutes {
  int at[kMaxK];
  float w[kMaxK];
};
template <bool WEIGHTS>
__device__ __forceinline__ TokenRoutes routes_of(const RouteRows& p, int t, int lane) {
  const int v = lane < p.K ? p.positions[t * p.K + lane] : -1, mine = v >= 0 && v < p.rows ? v : -1;
  const float w = WEIGHTS && p.w && lane < p.K ? p.w[t * p.K + lane] : 1.0f;
  TokenRoutes r;
#pragma unroll
  for (int k = 0; k < kMaxK; ++k) {
    r.at[k] = __builtin_amdgcn_readlane(mine, k);
    r.w[k] = WEIGHTS ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), k)) : 1.0f;
  }
  return r;
}

// A workgroup's four wavefronts take 2^log spans of 4 >> log tokens, and
// neighbouring workgroups the same tokens' next spans (nq workgroups to a set of
// tokens), so that a row is read as a whole at about one time.
struct Walk {
  int token, step;  // first token of this wavefront (T: none), and to its next
  int span, spans;  // its span before the token's turn, of so many
};
__device__ __forceinline__ Walk walk_of(const RouteRows& p, int wave, int log, int nq) {
  Walk w;
  w.spans = (p.cols + kSpan - 1) / kSpan;
  const int set = static_cast<int>(blockIdx.x) / nq, q = static_cast<int>(blockIdx.x) - set * nq;
  w.token = set * (4 >> log) + (wave >> log);
  w.step = static_cast<int>(gridDim.x) / nq * (4 >> log);
  w.span = (q << log) + (wave & ((1 << log) - 1));
  if (w.span >= w.spans) w.token = p.T;
  return w;
}

// (bits as they are: no conversion on the way)
template <bool F32, bool VEC>
__global__ __launch_bounds__(256) void gather_rows_kernel(RouteRows p, int log, int nq) {
  using Bits = std::conditional_t<F32, uint32_t, uint16_t>;
  constexpr int kWords = F32 ? 2 : 1;  // 16-byte pieces of eight values
  const Bits* x = static_cast<const Bits*>(p.x);
  Bits* out = static_cast<Bits*>(p.out);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Walk walk = walk_of(p, wave, log, nq);
  for (int t = walk.token; t < p.T; t += walk.step) {
    const TokenRoutes r = routes_of<false>(p, t, lane);
    const int c = span_column<VEC>((walk.span + t) % walk.spans, lane);
    if (c >= p.cols) continue;
    uint4 piece[kWords];
    Bits v[8];
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) piece[i] = load16<false>(x + t * p.ldx + c + i * (16 / sizeof(Bits)));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = c + 64 * i < p.cols ? x[t * p.ldx + c + 64 * i] : 0;
    }
#pragma unroll
    for (int k = 0; k < kMaxK; ++k)
      if (r.at[k] >= 0) {
        Bits* o = out + r.at[k] * p.ldo + c;
        if constexpr (VEC) {
#pragma unroll
          for (int i = 0; i < kWords; ++i) store16(o + i * (16 / sizeof(Bits)), piece[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + 64 * i < p.cols) o[64 * i] = v[i];
        }
      }
  }
  zero_rest<F32, VEC>(p);
}

template <bool XF32, bool OF32, bool VEC>
__global__ __launch_bounds__(256) void combine_rows_kernel(RouteRows p, int log, int nq) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Walk walk = walk_of(p, wave, log, nq);
  for (int t = walk.token; t < p.T; t += walk.step) {
    const TokenRoutes r = routes_of<true>(p, t, lane);
    const int c = span_column<VEC>((walk.span + t) % walk.spans, lane);
    if (c >= p.cols) continue;
    float v[kMaxK][8], sum[8] = {};
#pragma unroll
    for (int k = 0; k < kMaxK; ++k)
      if (r.at[k] >= 0) load_span<XF32, VEC>(p.x, r.at[k] * p.ldx, c, p.cols, v[k]);
#pragma unroll
    for (int k = 0; k < kMaxK; ++k)
      if (r.at[k] >= 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = fmaf(r.w[k], v[k][i], sum[i]);
      }
    store_span<OF32, VEC>(p.out, t * p.ldo, c, p.cols, sum);
  }
}

// WPT wavefronts to a token: 4, or 1 where a token has one span. A token's dot
// products are joined over the lanes, then over the wavefronts in order.
template <bool XF32, bool GF32, bool VEC, int WPT>
__global__ __launch_bounds__(256) void combine_backward_kernel(RouteRows p) {
  __shared__ float part[WPT][kMaxK];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int kTokens = 4 / WPT;
  const int spans = (p.cols + kSpan - 1) / kSpan;
  for (int t = static_cast<int>(blockIdx.x) * kTokens + wave / WPT; t < p.T; t += static_cast<int>(gridDim.x) * kTokens) {
    const TokenRoutes r = routes_of<true>(p, t, lane);
    float dot[kMaxK] = {};
    for (int s = wave % WPT; s < spans; s += WPT) {
      const int c = span_column<VEC>((s + t) % spans, lane);
      if (c >= p.cols) continue;
      float g[8], v[kMaxK][8];
      load_span<GF32, VEC>(p.grad, t * p.ldg, c, p.cols, g);
      if (p.dw) {
#pragma unroll
        for (int k = 0; k < kMaxK; ++k)
          if (r.at[k] >= 0) load_span<XF32, VEC>(p.x, r.at[k] * p.ldx, c, p.cols, v[k]);
#pragma unroll
        for (int k = 0; k < kMaxK; ++k)
          if (r.at[k] >= 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[k] = fmaf(v[k][i], g[i], dot[k]);
          }
      }
      if (p.out) {
#pragma unroll
        for (int k = 0; k < kMaxK; ++k)
          if (r.at[k] >= 0) {
            float d[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = r.w[k] * g[i];
            store_span<XF32, VEC>(p.out, r.at[k] * p.ldo, c, p.cols, d);
          }
      }
    }
    if (p.dw) {
      float sum = 0.0f;  // lane k: route k's
#pragma unroll
      for (int k = 0; k < kMaxK; ++k) {
        const float all = wave_sum_f32(dot[k]);
        sum = lane == k ? all : sum;
      }
      if constexpr (WPT > 1) {
        if (lane < kMaxK) part[wave][lane] = sum;
        __syncthreads();
        if (wave == 0 && lane < kMaxK) sum = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
        __syncthreads();  // (the next token's are written then)
      }
      if (wave % WPT == 0 && lane < p.K) p.dw[t * p.K + lane] = sum;
    }
  }
  if (p.out) zero_rest<XF32, VEC>(p);
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Rows of eight values at a time: every row starts at a multiple of 16 bytes
// and holds whole eights.
bool eights(const RouteRows& p) {
  return p.cols % 8 == 0 && p.ldx % 8 == 0 && p.ldo % 8 == 0 && p.ldg % 8 == 0 && aligned16(p.x) && aligned16(p.out) &&
         aligned16(p.grad);
}

constexpr int kMostBlocks = 1 << 22;  // (a launch holds fewer than 2^32 threads)

// Workgroups of `tokens` tokens each, nq to one set of them; more tokens than that
// take turns.
int token_grid(int T, int tokens, int nq) { return nq * std::max(1, std::min((T + tokens - 1) / tokens, kMostBlocks / nq)); }

struct Spans {
  int log, nq;
  explicit Spans(int cols) {
    const int spans = (cols + kSpan - 1) / kSpan;
    log = spans >= 3 ? 2 : spans - 1;
    nq = (spans + (1 << log) - 1) >> log;
  }
};

}  // namespace

size_t sort_workspace(int R) {
  if (R <= kOneGroup) return 0;
  return static_cast<size_t>((R + chunk_of(R) - 1) / chunk_of(R) + 1) * kExperts * sizeof(int32_t);
}

hipError_t launch_sort_routes(const SortRoutes& s, hipStream_t st) {
  if (s.R <= kOneGroup) {
    MOE_LAUNCH((sort_one_kernel), dim3(1), dim3(1024), 0, st, s);
    return hipGetLastError();
  }
  const int G = (s.R + chunk_of(s.R) - 1) / chunk_of(s.R);
  MOE_LAUNCH((sort_count_kernel), dim3(G), dim3(1024), 0, st, s);
  if (s.R <= kFewRoutes) {
    MOE_LAUNCH((sort_place_kernel<false>), dim3(G), dim3(1024), 0, st, s, G);
  } else {
    MOE_LAUNCH((sort_scan_kernel), dim3((s.E + 15) / 16), dim3(1024), 0, st, s, G);
    MOE_LAUNCH((sort_place_kernel<true>), dim3(G), dim3(1024), 0, st, s, G);
  }
  return hipGetLastError();
}

hipError_t launch_gather_rows(const RouteRows& p, hipStream_t st) {
  const Spans sp(p.cols);
  const dim3 grid(token_grid(p.T, 4 >> sp.log, sp.nq)), block(256);
  if (p.x_f32)
    eights(p) ? MOE_LAUNCH((gather_rows_kernel<true, true>), grid, block, 0, st, p, sp.log, sp.nq)
              : MOE_LAUNCH((gather_rows_kernel<true, false>), grid, block, 0, st, p, sp.log, sp.nq);
  else
    eights(p) ? MOE_LAUNCH((gather_rows_kernel<false, true>), grid, block, 0, st, p, sp.log, sp.nq)
              : MOE_LAUNCH((gather_rows_kernel<false, false>), grid, block, 0, st, p, sp.log, sp.nq);
  return hipGetLastError();
}

template <bool XF32, bool OF32, bool VEC>
static void combine_as(const RouteRows& p, bool backward, hipStream_t st) {
  const Spans sp(p.cols);
  const dim3 block(256);
  if (!backward)
    MOE_LAUNCH((combine_rows_kernel<XF32, OF32, VEC>), dim3(token_grid(p.T, 4 >> sp.log, sp.nq)), block, 0, st, p, sp.log, sp.nq);
  else if (p.cols > kSpan)
    MOE_LAUNCH((combine_backward_kernel<XF32, OF32, VEC, 4>), dim3(token_grid(p.T, 1, 1)), block, 0, st, p);
  else
    MOE_LAUNCH((combine_backward_kernel<XF32, OF32, VEC, 1>), dim3(token_grid(p.T, 4, 1)), block, 0, st, p);
}
template <bool XF32, bool OF32>
static void combine_types(const RouteRows& p, bool backward, hipStream_t st) {
  eights(p) ? combine_as<XF32, OF32, true>(p, backward, st) : combine_as<XF32, OF32, false>(p, backward, st);
}
static hipError_t combine(const RouteRows& p, bool backward, hipStream_t st) {
  if (p.x_f32)
    p.out_f32 ? combine_types<true, true>(p, backward, st) : combine_types<true, false>(p, backward, st);
  else
    p.out_f32 ? combine_types<false, true>(p, backward, st) : combine_types<false, false>(p, backward, st);
  return hipGetLastError();
}
hipError_t launch_combine_rows(const RouteRows& p, hipStream_t st) { return combine(p, false, st); }
hipError_t launch_combine_backward(const RouteRows& p, hipStream_t st) { return combine(p, true, st); }

}  // namespace moe
