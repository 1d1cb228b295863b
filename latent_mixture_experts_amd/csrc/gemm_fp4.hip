// gemm_fp4.hip -- products of MXFP4 rows with MXFP4 weights (E2M1 codes, one
// E8M0 scale per 32 values of either), dense and per expert.
//
//   out[r][n] = sum_b 2^(xs[r][b] + ws[n][b] - 254) * sum_{k in group b} x[r][k] w[n][k]
//
// The matrix instruction 16x16x128 takes both operands' codes and scales as
// they are stored and adds to an fp32 sum. Products of codes are multiples of
// 1/4 up to 36, so a group's sum is exact whatever its order; scaled groups are
// added in fp32 (measured: 128 products with scales of 2^-27 .. 2^23 are within
// 6.5e-8 of their sizes, denormal and vanishing results as IEEE rounding gives
// them, a scale of 255 gives NaN).
#include <algorithm>
#include <cmath>

#include "device_common.h"
#include "fp4.h"
#include "grouped.h"
#include "kernels.h"

namespace moe {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// An operand fragment: 16 bytes (one group of 32 codes) of row l % 16 per lane.
__device__ __forceinline__ i32x8 codes16(uint4 v) {
  return i32x8{static_cast<int>(v.x), static_cast<int>(v.y), static_cast<int>(v.z), static_cast<int>(v.w), 0, 0, 0, 0};
}
// D(16x16, fp32) += A(16x128) * B(128x16)^T with a scale per lane's group (byte
// BYTE of its word): lane l holds group l/16 of row l%16 of both, and receives
// rows 4*(l/16) .. +3 of A against row l%16 of B.
template <int BYTE = 0>
__device__ __forceinline__ f32x4 mfma_fp4(uint4 a, uint32_t sa, uint4 b, uint32_t sb, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(codes16(a), codes16(b), c, 4, 4, BYTE, static_cast<int>(sa), BYTE,
                                                          static_cast<int>(sb));
}

// ---- few rows: the weights stream once from HBM ----------------------------
// A wavefront takes 16 weight rows x up to 16 rows over a run of K's chunks of
// 512 values; KS wavefronts of a workgroup split K and are joined through LDS
// in order, and the workgroup's 8 / KS such teams take neighbouring weight
// rows. A group of more rows takes them in passes. Grid: (weight row tiles,
// groups).
constexpr int kFW = 8;      // wavefronts
constexpr int kChunk = 512; // values of a chunk: 256 bytes of codes, 16 scales

template <int KS, int D, bool F32, bool SVEC>
__global__ __launch_bounds__(64 * kFW, 4) void fp4_stream_kernel(Fp4Gemm p) {
  constexpr int kTeams = kFW / KS;
  __shared__ f32x4 part[KS > 1 ? kFW : 1][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nl = lane & 15, g = lane >> 4;
  const Group grp = p.offsets ? find_group(p, static_cast<int>(blockIdx.y), 1 << 30) : Group{0, 0, p.rows};
  if (grp.expert < 0) return;
  const int ks = wave % KS;
  const int n0 = (static_cast<int>(blockIdx.x) * kTeams + wave / KS) * 16;
  const int kbytes = p.K / 2, kscales = p.K / kFp4Group;  // of a row
  const int nch = (p.K + kChunk - 1) / kChunk;
  const int per = (nch + KS - 1) / KS;
  const int c0 = min(ks * per, nch), n_c = min(per, nch - c0);
  // (a team past the last weight row reads and writes nothing)
  const int wrows = min(max(p.N - n0, 0), 16);
  const size_t wrow = static_cast<size_t>(grp.expert) * p.N + n0;
  const rsrc_t w_r = make_rsrc(p.w + wrow * kbytes, static_cast<uint32_t>(wrows * kbytes));
  const rsrc_t ws_r = make_rsrc(p.ws + wrow * kscales, static_cast<uint32_t>(wrows * kscales));
  const uint32_t w_off = static_cast<uint32_t>(nl * kbytes) + g * 16, ws_off = static_cast<uint32_t>(nl * kscales);

  for (int r0 = grp.begin; r0 < grp.end; r0 += 16) {
    const int base = p.index ? 0 : r0;  // the descriptors start at this row of x
    const int xrows = p.index ? p.x_rows : min(grp.end - r0, 16);
    const rsrc_t x_r = make_rsrc(p.x + static_cast<size_t>(base) * p.ldx,
                                 static_cast<uint32_t>(static_cast<size_t>(xrows - 1) * p.ldx + kbytes));
    const rsrc_t xs_r = make_rsrc(p.xs + static_cast<size_t>(base) * kscales, static_cast<uint32_t>(xrows) * kscales);
    // (lanes without a row read nothing)
    const int row = r0 + nl;
    const int src = row < grp.end ? source_row(p, row) - base : 0;
    const uint32_t x_off = row < grp.end ? static_cast<uint32_t>(src * p.ldx) + g * 16 : kOutOfRange;
    const uint32_t xs_off = row < grp.end ? static_cast<uint32_t>(src) * kscales : kOutOfRange;
    f32x4 acc{0.f, 0.f, 0.f, 0.f};

    uint4 wv[D][4], xv[D][4];
    uint32_t wsv[D][4], xsv[D][4];
    auto load = [&](int u, int i) __attribute__((always_inline)) {
      const int c = c0 + i;
#pragma unroll
      for (int s = 0; s < 4; ++s) {  // (pieces past the last value: zeros in both operands)
        const int at = c * (kChunk / 2) + s * 64;
        const bool in = at + g * 16 < kbytes;
        wv[u][s] = buf_load16<kAuxStream>(w_r, in ? w_off + at : kOutOfRange);
        xv[u][s] = buf_load16<kAuxDefault>(x_r, in ? x_off + at : kOutOfRange);
        if constexpr (!SVEC) {
          const uint32_t sat = c * 16 + s * 4 + g;
          wsv[u][s] = buf_load8<kAuxDefault>(ws_r, in ? ws_off + sat : kOutOfRange);
          xsv[u][s] = buf_load8<kAuxDefault>(xs_r, in ? xs_off + sat : kOutOfRange);
        }
      }
      if constexpr (SVEC) {
        const uint4 a = buf_load16<kAuxDefault>(ws_r, ws_off + c * 16), b = buf_load16<kAuxDefault>(xs_r, xs_off + c * 16);
        wsv[u][0] = a.x, wsv[u][1] = a.y, wsv[u][2] = a.z, wsv[u][3] = a.w;
        xsv[u][0] = b.x, xsv[u][1] = b.y, xsv[u][2] = b.z, xsv[u][3] = b.w;
      }
    };
    auto consume = [&](int u) __attribute__((always_inline)) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint32_t a = SVEC ? wsv[u][s] >> (8 * g) : wsv[u][s], b = SVEC ? xsv[u][s] >> (8 * g) : xsv[u][s];
        acc = mfma_fp4(wv[u][s], a, xv[u][s], b, acc);
      }
    };
#pragma unroll
    for (int u = 0; u < D; ++u)
      if (u < n_c) load(u, u);
    int i = 0;
    for (; i + 2 * D <= n_c; i += D) {  // (no branches inside: the waits stay D chunks deep)
#pragma unroll
      for (int u = 0; u < D; ++u) {
        consume(u);
        load(u, i + D + u);
      }
    }
#pragma unroll
    for (int u = 0; u < D; ++u)
      if (i + u < n_c) {
        consume(u);
        if (i + D + u < n_c) load(u, i + D + u);
      }
    i += D;
#pragma unroll
    for (int u = 0; u < D; ++u)
      if (i + u < n_c) consume(u);

    if constexpr (KS == 1) {
      if (row < grp.end && n0 + 4 * g < p.N) store4<F32>(p, row, n0 + 4 * g, acc);
    } else {
      part[wave][lane] = acc;
      __syncthreads();
      if (ks == 0) {
#pragma unroll
        for (int v = 1; v < KS; ++v) acc += part[wave + v][lane];
        if (row < grp.end && n0 + 4 * g < p.N) store4<F32>(p, row, n0 + 4 * g, acc);
      }
      __syncthreads();  // (the next pass writes part again)
    }
  }
}

template <int KS, int D, bool F32>
void launch_stream_as(const Fp4Gemm& g, dim3 grid, hipStream_t st) {
  if (g.scale_vec)
    MOE_LAUNCH((fp4_stream_kernel<KS, D, F32, true>), grid, dim3(64 * kFW), 0, st, g);
  else
    MOE_LAUNCH((fp4_stream_kernel<KS, D, F32, false>), grid, dim3(64 * kFW), 0, st, g);
}
template <int KS, int D>
hipError_t launch_stream_ks(const Fp4Gemm& g, int tiles, int groups, hipStream_t st) {
  const dim3 grid((tiles * KS + kFW - 1) / kFW, groups);
  if (g.f32)
    launch_stream_as<KS, D, true>(g, grid, st);
  else
    launch_stream_as<KS, D, false>(g, grid, st);
  return hipGetLastError();
}

// K is split over wavefronts until about 16 of them per CU have work.
hipError_t launch_stream(const Fp4Gemm& g, int groups, hipStream_t st) {
  const int tiles = (g.N + 15) / 16;
  const int64_t waves = static_cast<int64_t>(tiles) * groups;
  if (waves >= 4096) return launch_stream_ks<1, 1>(g, tiles, groups, st);
  if (waves >= 2048) return launch_stream_ks<2, 1>(g, tiles, groups, st);
  if (waves >= 1024) return launch_stream_ks<4, 1>(g, tiles, groups, st);
  return launch_stream_ks<8, 1>(g, tiles, groups, st);
}

}  // namespace

hipError_t launch_fp4_gemm(const Fp4Gemm& g, hipStream_t st) {
  return launch_stream(g, std::min(g.rows, g.experts), st);
}

}  // namespace moe
