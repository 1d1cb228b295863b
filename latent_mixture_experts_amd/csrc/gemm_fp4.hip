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
//
// What bounds it: one to 16 rows, the weights' way from HBM and a launch's start
// (4096 x 8192: 6.7 us); few rows per expert, HBM (32 tokens' down projection, 163
// experts of 4096 x 4096, 1.45 GB: 219 us, 6.6 TB/s); thousands of rows, the latency
// of the copies from L2 into LDS with two stages held (4096 x 4096 x 8192: 67 us,
// 4.1 PFLOP/s, of which the matrix unit is busy 27 us at 2.4 GHz and LDS three
// tenths of the time; 570 MB pass into LDS at 8.5 TB/s, in 6.3e6 requests to L2, a
// third of them for 16 bytes of scales each).
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
// rows. Dense products of at most 16 rows only: it reads neither offsets nor an
// index, which one expert, too, may come with. Grid: weight row tiles.
constexpr int kFW = 8;      // wavefronts
constexpr int kChunk = 512; // values of a chunk: 256 bytes of codes, 16 scales

template <int KS, int D, bool F32, bool SVEC>
__global__ __launch_bounds__(64 * kFW, 2) void fp4_stream_kernel(Fp4Gemm p) {
  constexpr int kTeams = kFW / KS;
  __shared__ f32x4 part[kFW][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nl = lane & 15, g = lane >> 4;
  const int ks = wave % KS;
  const int n0 = (static_cast<int>(blockIdx.x) * kTeams + wave / KS) * 16;
  const int kbytes = p.K / 2, kscales = p.K / kFp4Group;  // of a row
  const int nch = (p.K + kChunk - 1) / kChunk;
  const int per = (nch + KS - 1) / KS;
  const int c0 = min(ks * per, nch), n_c = min(per, nch - c0);
  // (a team past the last weight row reads and writes nothing)
  const int wrows = min(max(p.N - n0, 0), 16);
  const rsrc_t w_r = make_rsrc(p.w + static_cast<size_t>(n0) * kbytes, static_cast<uint32_t>(wrows * kbytes));
  const rsrc_t ws_r = make_rsrc(p.ws + static_cast<size_t>(n0) * kscales, static_cast<uint32_t>(wrows * kscales));
  const uint32_t w_off = static_cast<uint32_t>(nl * kbytes) + g * 16, ws_off = static_cast<uint32_t>(nl * kscales);

  const rsrc_t x_r = make_rsrc(p.x, static_cast<uint32_t>(static_cast<size_t>(p.rows - 1) * p.ldx + kbytes));
  const rsrc_t xs_r = make_rsrc(p.xs, static_cast<uint32_t>(p.rows * kscales));
  // (lanes without a row read nothing)
  const bool live = nl < p.rows;
  const uint32_t x_off = live ? static_cast<uint32_t>(nl * p.ldx) + g * 16 : kOutOfRange;
  const uint32_t xs_off = live ? static_cast<uint32_t>(nl * kscales) : kOutOfRange;
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

  part[wave][lane] = acc;
  __syncthreads();
  if (ks == 0) {
#pragma unroll
    for (int v = 1; v < KS; ++v) acc += part[wave + v][lane];
    if (live && n0 + 4 * g < p.N) store4<F32>(p, nl, n0 + 4 * g, acc);
  }
}

// ---- many rows: LDS-staged tiles -------------------------------------------
// Workgroup tile: WT x WW wavefronts, each FT x FW fragments of 16 rows x 16
// weight rows; a tile's row fragments are dealt to the wavefront rows in turn,
// so a partly filled tile loads them evenly. A stage holds KG blocks of 256
// values, each the work of a wavefront group of its own (WT x WW), joined
// through LDS at the end. Both operands' 128 bytes of a row and block are copied
// straight from global memory into LDS in a ring of R stages (the copies run
// R - 1 ahead). A lane takes 16-byte pieces 2g and 2g+1 of its row, one matrix
// instruction each, so that their two scales are one 16-bit read; piece 2g + i of
// row r lies at place (g + 4i) ^ ((r/2) % 8) of the row's eight, so that the rows
// one read touches start in distinct banks (in the order of the pieces half the
// banks met twice: 4096 x 4096 x 8192 81 -> 79 us).
// Scales: in sets of 16 bytes, the scales of 512 values of a row: of two stages (KG
// = 1, two such sets in turn), or of (half of) one; 16 bytes per copy where rows'
// scales start at multiples of 16 bytes (kBy16), else of 4 (kBy4). Else (kBy1) byte
// by byte, each into a word of its own, with the codes they belong to.
constexpr int kBlockValues = 256, kRowBytes = 128, kPieces = 8;  // of a row and block

__device__ __forceinline__ int piece_at(int r, int c) { return (r * 8 + ((c >> 1 | (c & 1) << 2) ^ ((r >> 1) & 7))) * 16; }
// The piece at place i of row r.
__device__ __forceinline__ int piece_of(int r, int i) {
  const int v = i ^ ((r >> 1) & 7);
  return (v & 3) << 1 | v >> 2;
}

// a and b of the lane rows g = 0 .. 3 of 16: (a0, a2, b0, b2) and (a1, a3, b1, b3).
__device__ __forceinline__ uint2 swap_rows(uint32_t a, uint32_t b) {
  const auto h = __builtin_amdgcn_permlane32_swap(a, b, false, false);  // (a0, a1, b0, b1), (a2, a3, b2, b3)
  const auto q = __builtin_amdgcn_permlane16_swap(h[0], h[1], false, false);
  return uint2{q[0], q[1]};
}

// Waits until every LDS read has returned.
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xC07F); }

// As lds_copy16, past the caches (non-temporal).
__device__ __forceinline__ void lds_copy16_once(rsrc_t r, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dwordx4 %0, %1, 0 offen nt lds" ::"v"(voff), "s"(r), "s"(lds) : "memory");
}
// As lds_copy16: one byte per lane, to a word of its own (upper bytes zero).
__device__ __forceinline__ void lds_copy1(rsrc_t r, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_ubyte %0, %1, 0 offen lds" ::"v"(voff), "s"(r), "s"(lds) : "memory");
}

template <int WT, int WW, int FT, int FW, int R, int KG, int SCALES, bool EARLY, bool ONCE>
__global__ __launch_bounds__(64 * WT * WW * KG) void fp4_tile_kernel(Fp4Gemm p, int n_row_tiles, int n_col_tiles, int chunk) {
  constexpr int kGroup = WT * WW, NW = kGroup * KG, BM = WT * FT * 16, BN = WW * FW * 16;
  constexpr bool WIDE = SCALES != kBy1;
  // 1-KiB copies per wavefront and stage (its group's block); of the rows' some
  // wavefronts may have one fewer
  constexpr int kXOps = (BM / 8 + kGroup - 1) / kGroup, kXLeast = BM / 8 / kGroup, kWOps = BN / 8 / kGroup;
  constexpr int kOps = kXOps + kWOps, kLeast = (kXLeast + kWOps) * (WIDE ? 1 : 2);
  static_assert(!EARLY || (R == 2 && KG == 1), "two stages held");
  static_assert(kWOps * 8 * kGroup == BN && kXLeast > 0, "whole copies");
  static_assert(R >= 2 && R <= 4 && (R - 2) * kLeast < 64, "vmcnt field; scale sets land in time");
  constexpr int kXSlot = KG * BM * kRowBytes, kWSlot = KG * BN * kRowBytes;  // bytes of a stage
  // scale sets: stages of one, sets held, 16-byte halves of a row, blocks of 64 rows, copies of one
  constexpr bool kPairs = WIDE && KG == 1;
  constexpr int kSets = kPairs ? 2 : R, kHalves = WIDE && KG == 4 ? 2 : 1, kParts = SCALES == kBy4 ? 4 : 1;
  constexpr int kXC = (BM + 63) / 64, kWC = (BN + 63) / 64;
  constexpr int kSxSlot = WIDE ? kHalves * kXC * 1024 : KG * BM * kPieces * 4;
  constexpr int kSwSlot = WIDE ? kHalves * kWC * 1024 : KG * BN * kPieces * 4;
  constexpr int kSOps = (kParts * kHalves * (kXC + kWC) + NW - 1) / NW;  // WIDE: copies per wavefront and set
  __shared__ __attribute__((aligned(1024))) uint8_t Xs[R][kXSlot];
  __shared__ __attribute__((aligned(1024))) uint8_t Ws[R][kWSlot];
  __shared__ __attribute__((aligned(1024))) uint8_t Sx[kSets][kSxSlot];
  __shared__ __attribute__((aligned(1024))) uint8_t Sw[kSets][kSwSlot];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nl = lane & 15, g = lane >> 4;
  const int kg = wave / kGroup, wt = wave % kGroup % WT, ww = wave % kGroup / WT;

  int mt, nt;
  if (p.offsets) {
    const int logical = xcd_tile(chunk);
    mt = logical / n_col_tiles;
    nt = logical % n_col_tiles;
  } else {
    const TileRC t = dense_tile_of(static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x), n_row_tiles,
                                   n_col_tiles, 4);
    mt = t.mt;
    nt = t.nt;
    if (mt < 0) return;
  }
  const Group grp = find_group(p, mt, BM);
  if (grp.expert < 0) return;
  const int nrows = grp.end - grp.begin, n0 = nt * BN, ncols = min(BN, p.N - n0);
  const int kbytes = p.K / 2, kscales = p.K / kFp4Group;  // of a row
  const int nst = (p.K + KG * kBlockValues - 1) / (KG * kBlockValues);
  const size_t wrow = static_cast<size_t>(grp.expert) * p.N + n0;
  const uint8_t* w_base = p.w + wrow * kbytes;
  const uint32_t w_bytes = static_cast<uint32_t>(ncols * kbytes);
  const rsrc_t ws_r = make_rsrc(p.ws + wrow * kscales, static_cast<uint32_t>(ncols * kscales));
  const int base = p.index ? 0 : grp.begin;
  const int xrows = p.index ? p.x_rows : nrows;
  const uint8_t* x_base = p.x + static_cast<size_t>(base) * p.ldx;
  const uint32_t x_bytes = static_cast<uint32_t>(static_cast<size_t>(xrows - 1) * p.ldx + kbytes);
  const rsrc_t xs_r = make_rsrc(p.xs + static_cast<size_t>(base) * kscales, static_cast<uint32_t>(xrows) * kscales);
  auto row_of = [&](int r) -> int { return r < nrows ? source_row(p, grp.begin + r) - base : -1; };

  // Copy o of a scale set: of half `half` of block `block` of 64 rows (the rows', then
  // the weights'), all of them, or 16 with a word per lane.
  struct SetCopy {
    int block, half, part;
    __device__ __forceinline__ explicit SetCopy(int o) : block(o / kParts / kHalves), half(o / kParts % kHalves), part(o % kParts) {}
  };
  // Source offsets of this wavefront's copies in the first stage; the
  // descriptors of the codes step along K, so a copy costs no vector arithmetic.
  uint32_t xoff[kXOps], woff[kWOps];
  uint32_t sxoff[WIDE ? 1 : kXOps], swoff[WIDE ? 1 : kWOps], soff[WIDE ? kSOps : 1];
#pragma unroll
  for (int i = 0; i < kXOps; ++i) {
    const int r = (i * kGroup + wave % kGroup) * 8 + (lane >> 3), src = row_of(r);
    xoff[i] = src < 0 ? kOutOfRange : static_cast<uint32_t>(src * p.ldx) + kg * kRowBytes + piece_of(r, lane & 7) * 16;
    if constexpr (!WIDE) sxoff[i] = src < 0 ? kOutOfRange : static_cast<uint32_t>(src * kscales + kg * kPieces + (lane & 7));
  }
#pragma unroll
  for (int i = 0; i < kWOps; ++i) {
    const int r = (i * kGroup + wave % kGroup) * 8 + (lane >> 3);
    woff[i] = static_cast<uint32_t>(r * kbytes) + kg * kRowBytes + piece_of(r, lane & 7) * 16;
    if constexpr (!WIDE) swoff[i] = static_cast<uint32_t>(r * kscales + kg * kPieces + (lane & 7));
  }
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < kSOps; ++i) {
      const SetCopy o(i * NW + wave);
      const int r = (o.block < kXC ? o.block : o.block - kXC) * 64 + (SCALES == kBy4 ? o.part * 16 + lane / 4 : lane);
      const int src = o.block < kXC ? row_of(r) : r < ncols ? r : -1;
      soff[i] = src < 0 ? kOutOfRange : static_cast<uint32_t>(src * kscales + o.half * 16 + (SCALES == kBy4 ? lane % 4 * 4 : 0));
    }
  }
  const uint32_t lds_x = lds_address(&Xs[0][0]), lds_w = lds_address(&Ws[0][0]);
  const uint32_t lds_sx = lds_address(&Sx[0][0]), lds_sw = lds_address(&Sw[0][0]);
  // Copies of one stage: descriptors, and the LDS slot they fill. Stages past
  // the last have empty descriptors, so their copies read nothing (zeros into a
  // slot that no product reads) and every stage counts the same.
  struct Stage {
    rsrc_t x, w, sx, sw;
    int slot;
  };
  const bool partial = p.K % (KG * kBlockValues) != 0;
  auto stage_of = [&](int st, int slot) __attribute__((always_inline)) {
    const uint32_t k0 = static_cast<uint32_t>(st) * (KG * kRowBytes), s0 = static_cast<uint32_t>(st) * (KG * kPieces);
    if (partial && st == nst - 1) {  // the last one that reads: its pieces past K read nothing, zeros in both operands
      const int left = (kbytes - static_cast<int>(k0) - kg * kRowBytes) / 16;  // pieces
      auto in = [&](int q) { return piece_of(q * 8 + (lane >> 3), lane & 7) < left; };
#pragma unroll
      for (int i = 0; i < kXOps; ++i) {
        if (!in(i * kGroup + wave % kGroup)) xoff[i] = kOutOfRange;
        if constexpr (!WIDE)
          if ((lane & 7) >= left) sxoff[i] = kOutOfRange;
      }
#pragma unroll
      for (int i = 0; i < kWOps; ++i) {
        if (!in(i * kGroup + wave % kGroup)) woff[i] = kOutOfRange;
        if constexpr (!WIDE)
          if ((lane & 7) >= left) swoff[i] = kOutOfRange;
      }
    }
    const bool none = st >= nst;
    Stage s{make_rsrc(none ? x_base : x_base + k0, none ? 0 : x_bytes - k0),
            make_rsrc(none ? w_base : w_base + k0, none ? 0 : w_bytes - k0), xs_r, ws_r, slot};
    if constexpr (!WIDE) {
      const uint8_t* xs = p.xs + static_cast<size_t>(base) * kscales;
      const uint8_t* ws = p.ws + wrow * kscales;
      s.sx = make_rsrc(none ? xs : xs + s0, none ? 0 : static_cast<uint32_t>(xrows) * kscales - s0);
      s.sw = make_rsrc(none ? ws : ws + s0, none ? 0 : static_cast<uint32_t>(ncols * kscales) - s0);
    }
    return s;
  };
  // this wavefront's copy c (0 .. kOps-1) of a stage
  auto copy = [&](const Stage& s, int c) __attribute__((always_inline)) {
    const int i = c < kXOps ? c : c - kXOps, q = i * kGroup + wave % kGroup;  // 8-row block of the tile
    if (c < kXOps) {
      if (kXOps == kXLeast || q < BM / 8) {
        if constexpr (!WIDE)
          lds_copy1(s.sx, sxoff[c < kXOps ? c : 0],
                    __builtin_amdgcn_readfirstlane(lds_sx + s.slot * kSxSlot + kg * (BM * kPieces * 4) + q * 256));
        lds_copy16(s.x, xoff[c < kXOps ? c : 0],
                   __builtin_amdgcn_readfirstlane(lds_x + s.slot * kXSlot + kg * (BM * kRowBytes) + q * 1024));
      }
    } else {
      if constexpr (!WIDE)
        lds_copy1(s.sw, swoff[c < kXOps ? 0 : c - kXOps],
                  __builtin_amdgcn_readfirstlane(lds_sw + s.slot * kSwSlot + kg * (BN * kPieces * 4) + q * 256));
      const uint32_t off = woff[c < kXOps ? 0 : c - kXOps];
      const uint32_t to = __builtin_amdgcn_readfirstlane(lds_w + s.slot * kWSlot + kg * (BN * kRowBytes) + q * 1024);
      if constexpr (ONCE)
        lds_copy16_once(s.w, off, to);
      else
        lds_copy16(s.w, off, to);
    }
  };
  // WIDE: set `set` of the scales into place `at` (scales past K: none)
  auto issue_set = [&](int set, int at) __attribute__((always_inline)) {
    if constexpr (WIDE) {
#pragma unroll
      for (int i = 0; i < kSOps; ++i) {
        const SetCopy o(i * NW + wave);
        const int s0 = (set * kHalves + o.half) * 16 + (SCALES == kBy4 ? lane % 4 * 4 : 0);  // first scale
        const uint32_t off = s0 < kscales ? soff[i] + set * (kHalves * 16) : kOutOfRange;
        const bool of_x = o.block < kXC;
        if (of_x || o.block < kXC + kWC) {
          const uint32_t to = __builtin_amdgcn_readfirstlane(
              (of_x ? lds_sx + at * kSxSlot + o.half * (kXC * 1024) + o.block * 1024
                    : lds_sw + at * kSwSlot + o.half * (kWC * 1024) + (o.block - kXC) * 1024) + o.part * 256);
          if constexpr (SCALES == kBy4)
            of_x ? lds_copy4(xs_r, off, to) : lds_copy4(ws_r, off, to);
          else
            of_x ? lds_copy16(xs_r, off, to) : lds_copy16(ws_r, off, to);
        }
      }
    }
  };

  f32x4 acc[FT][FW];
#pragma unroll
  for (int t = 0; t < FT; ++t)
#pragma unroll
    for (int f = 0; f < FW; ++f) acc[t][f] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Stage st lives in slot st % R. The stages overlap: before the last row
  // fragment's products of a stage every wavefront has read its slot to
  // registers; there they meet, the first fragments of stage st + 1 (landed by
  // then) are read under those last products, and the slot takes the copies of
  // stage st + R, spread over the following products. Within a stage the next row
  // fragment's reads run under the products of this one.
  auto kloop = [&](auto live_tag) __attribute__((always_inline)) {
    constexpr int LIVE = decltype(live_tag)::value;
    constexpr int kProducts = LIVE * FW;  // of a wavefront and stage (pairs of matrix instructions)
    // copy c goes out with product at(c), counted from the meeting
    auto at = [](int c) constexpr { return kProducts >= 2 * kOps ? 2 * c : c * kProducts / kOps; };
    auto copies_at = [&](const Stage& s, int q) __attribute__((always_inline)) {
#pragma unroll
      for (int c = 0; c < kOps; ++c)
        if (at(c) == q) copy(s, c);
    };
    if constexpr (kPairs) issue_set(0, 0);
#pragma unroll
    for (int s = 0; s < (EARLY ? R : R - 1); ++s) {
      if constexpr (!kPairs) issue_set(s, s);
      const Stage g = stage_of(s, s);
#pragma unroll
      for (int c = 0; c < kOps; ++c) copy(g, c);
    }
    if constexpr (!kPairs && !EARLY) issue_set(R - 1, R - 1);
    if constexpr (kPairs) issue_set(1, 1);
    Stage ahead = stage_of(EARLY ? R : R - 1, EARLY ? 0 : R - 1);
    if constexpr (!EARLY) {
#pragma unroll
      for (int q = 0; q < (LIVE > 0 ? FW : 1); ++q) copies_at(ahead, q);
    }
    wait_vm_lds<EARLY ? kLeast : (R - 2) * kLeast>();  // (stage 0 and its scales; the others are younger)
    __syncthreads();
    // the copies of stage st + 1 have landed, in every wavefront
    auto meet = [&](int st, int slot) __attribute__((always_inline)) {
      wait_vm_lds<EARLY ? kWOps * (WIDE ? 1 : 2) : (R - 2) * kLeast>();
      __syncthreads();
      if constexpr (!kPairs) issue_set(st + R, slot);
      // (of pairs: set j is read until stage 2j + 1's meeting and takes set j + 2
      // there, two stages of copies before the meeting that lets it be read)
      if constexpr (kPairs)
        if (st & 1) issue_set(st / 2 + 2, st / 2 & 1);
      if constexpr (!EARLY) ahead = stage_of(st + R, slot);
    };
    // EARLY: every wavefront has read its weights of stage st, whose place takes
    // those of stage st + 2 at once, the rows' place theirs after the meeting
    auto turn = [&](int st, int slot) __attribute__((always_inline)) {
      wait_lds();
      __syncthreads();
      ahead = stage_of(st + R, slot);
    };
    auto copy_weights = [&](int q, int per) __attribute__((always_inline)) {
#pragma unroll
      for (int c = 0; c < kWOps; ++c)
        if (c / per == q) copy(ahead, kXOps + c);
    };
    auto copy_rows = [&](int q, int per) __attribute__((always_inline)) {
#pragma unroll
      for (int c = 0; c < kXOps; ++c)
        if (c / per == q) copy(ahead, c);
    };
    if constexpr (LIVE == 0) {
      for (int st = 0, slot = 0; st < nst; ++st, slot = slot == R - 1 ? 0 : slot + 1) {
        if constexpr (EARLY) {
          turn(st, slot);
          copy_weights(0, kWOps);
        }
        meet(st, slot);
        if constexpr (EARLY)
          copy_rows(0, kXOps);
        else
          copies_at(ahead, 0);
      }
    } else {
      // (rows 16 apart keep their swizzle: constant offsets from one address)
      const int xp0 = piece_at(wt * 16 + nl, 2 * g), xp1 = piece_at(wt * 16 + nl, 2 * g + 1);
      const int wp0 = piece_at(ww * FW * 16 + nl, 2 * g), wp1 = piece_at(ww * FW * 16 + nl, 2 * g + 1);
      struct Operand {
        uint4 v[2];
        uint32_t s[WIDE ? 1 : 2];  // WIDE: both scales in one word
      };
      auto read_scales = [&](Operand& o, const uint8_t* b, int slot_bytes, int copies, int rows, int st, int slot, int row, int step)
                             __attribute__((always_inline)) {
        if constexpr (WIDE) {
          const int set = kPairs ? (st >> 1) & 1 : slot, half = KG == 4 ? kg >> 1 : 0, eight = kPairs ? st & 1 : kg & 1;
          o.s[0] = *reinterpret_cast<const uint16_t*>(b + set * slot_bytes + half * (copies * 1024) + eight * 8 + row * 16 + 2 * g + step * 256);
        } else {
          const uint2 s = *reinterpret_cast<const uint2*>(b + slot * slot_bytes + kg * (rows * kPieces * 4) + row * 32 + 8 * g + step * 512);
          o.s[0] = s.x;
          o.s[1] = s.y;
        }
      };
      auto read_x = [&](Operand& o, int st, int slot, int t) __attribute__((always_inline)) {
        const uint8_t* b = &Xs[0][0] + slot * kXSlot + kg * (BM * kRowBytes);
        o.v[0] = *reinterpret_cast<const uint4*>(b + xp0 + t * WT * 2048);
        o.v[1] = *reinterpret_cast<const uint4*>(b + xp1 + t * WT * 2048);
        read_scales(o, &Sx[0][0], kSxSlot, kXC, BM, st, slot, wt * 16 + nl, t * WT);
      };
      auto read_w = [&](Operand& o, int st, int slot, int f) __attribute__((always_inline)) {
        const uint8_t* b = &Ws[0][0] + slot * kWSlot + kg * (BN * kRowBytes);
        o.v[0] = *reinterpret_cast<const uint4*>(b + wp0 + f * 2048);
        o.v[1] = *reinterpret_cast<const uint4*>(b + wp1 + f * 2048);
        read_scales(o, &Sw[0][0], kSwSlot, kWC, BN, st, slot, ww * FW * 16 + nl, f);
      };
      auto product = [&](const Operand& a, const Operand& b, int s, f32x4 c) __attribute__((always_inline)) {
        if constexpr (WIDE)
          return s == 0 ? mfma_fp4<0>(a.v[0], a.s[0], b.v[0], b.s[0], c) : mfma_fp4<1>(a.v[1], a.s[0], b.v[1], b.s[0], c);
        else
          return mfma_fp4<0>(a.v[s], a.s[s], b.v[s], b.s[s], c);
      };
      Operand wv[FW], xv, next;
#pragma unroll
      for (int f = 0; f < FW; ++f) read_w(wv[f], 0, 0, f);
      read_x(next, 0, 0, 0);
      for (int st = 0, slot = 0; st < nst; ++st) {
        const int after = slot == R - 1 ? 0 : slot + 1;
#pragma unroll
        for (int t = 0; t < LIVE; ++t) {
          xv = next;
          if constexpr (EARLY) {
            if (t == (LIVE > 1 ? 1 : 0)) turn(st, slot);
            if (LIVE <= 2 && t + 1 == LIVE) copy_weights(0, kWOps);
          }
          if (t + 1 < LIVE) {
            read_x(next, st, slot, t + 1);
          } else {
            meet(st, slot);
            read_x(next, st + 1, after, 0);  // (after the last stage: what the slot held, not used)
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int f = 0; f < FW; ++f) {
            acc[t][f] = product(wv[f], xv, 0, acc[t][f]);
            acc[t][f] = product(wv[f], xv, 1, acc[t][f]);
            __builtin_amdgcn_sched_barrier(0);
            if (t + 1 == LIVE) read_w(wv[f], st + 1, after, f);
            if constexpr (EARLY) {
              if (LIVE > 2 && t == 1) copy_weights(f, (kWOps + FW - 1) / FW);
              if (t + 1 == LIVE) copy_rows(f, (kXOps + FW - 1) / FW);
            } else {
              copies_at(ahead, t + 1 == LIVE ? f : t * FW + f + FW);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        slot = after;
      }
    }
    wait_vm_lds<0>();  // (a last scale set and empty copies may still be on their way into this workgroup's LDS)
  };
  // fragments of this wavefront that hold rows
  const int live = ((nrows + 15) / 16 + WT - 1 - wt) / WT;
  if (live > FT * 3 / 4)
    kloop(std::integral_constant<int, FT>{});
  else if (live > FT / 2)
    kloop(std::integral_constant<int, (FT > 2 ? FT * 3 / 4 : FT)>{});
  else if (live > FT / 4)
    kloop(std::integral_constant<int, (FT > 1 ? FT / 2 : 1)>{});
  else if (live > 0)
    kloop(std::integral_constant<int, (FT > 4 ? FT / 4 : 1)>{});
  else
    kloop(std::integral_constant<int, 0>{});

  if constexpr (KG > 1) {  // the groups' sums in order, through the LDS that held the stages
    static_assert((KG - 1) * kGroup * FT * FW * 1024 <= R * kWSlot, "sums fit");
    f32x4* part = reinterpret_cast<f32x4*>(&Ws[0][0]);
    __syncthreads();  // (every wavefront's copies have landed and its reads are done)
    if (kg > 0) {
#pragma unroll
      for (int t = 0; t < FT; ++t)
#pragma unroll
        for (int f = 0; f < FW; ++f) part[((wave - kGroup) * FT * FW + t * FW + f) * 64 + lane] = acc[t][f];
    }
    __syncthreads();
    if (kg > 0) return;
#pragma unroll
    for (int v = 1; v < KG; ++v)
#pragma unroll
      for (int t = 0; t < FT; ++t)
#pragma unroll
        for (int f = 0; f < FW; ++f) acc[t][f] += part[((wave + (v - 1) * kGroup) * FT * FW + t * FW + f) * 64 + lane];
  }
  auto store = [&](auto f32_tag) __attribute__((always_inline)) {
    constexpr bool F32 = decltype(f32_tag)::value;
    const int n1 = n0 + ww * (FW * 16) + 4 * g;
    const bool whole = p.out_vec && n0 + BN <= p.N;  // (no part of the tile lies past the last weight row)
#pragma unroll
    for (int t = 0; t < FT; ++t) {
      const int r = (t * WT + wt) * 16 + nl;
      const bool live_row = r < nrows;
      auto* o = static_cast<typename Out4<F32>::type*>(p.out) + static_cast<size_t>(grp.begin + r) * p.ldo;
      if constexpr (!F32 && FW % 2 == 0) {
        if (p.out_vec8 && n0 + BN <= p.N) {
          // two fragments' values dealt out anew over the four lanes of a row: eight neighbours each
#pragma unroll
          for (int f = 0; f < FW; f += 2) {
            const Out4<false> x(acc[t][f]), y(acc[t][f + 1]);
            const uint2 a = __builtin_bit_cast(uint2, x.v), b = __builtin_bit_cast(uint2, y.v);
            const auto lo = swap_rows(a.x, b.x), hi = swap_rows(a.y, b.y);
            if (live_row)
              *reinterpret_cast<uint4*>(o + n0 + ww * (FW * 16) + f * 16 + 8 * g) = uint4{lo.x, hi.x, lo.y, hi.y};
          }
          continue;
        }
      }
      if (live_row) {
#pragma unroll
        for (int f = 0; f < FW; ++f) {
          if (whole) {
            const Out4<F32> x(acc[t][f]);
            *reinterpret_cast<decltype(x.v)*>(o + n1 + f * 16) = x.v;
          } else if (n1 + f * 16 < p.N) {
            store4<F32>(p, grp.begin + r, n1 + f * 16, acc[t][f]);
          }
        }
      }
    }
  };
  if (p.f32)
    store(std::true_type{});
  else
    store(std::false_type{});
}

template <int KS, int D, bool F32>
void launch_stream_as(const Fp4Gemm& g, dim3 grid, hipStream_t st) {
  if (g.scales == kBy16)
    MOE_LAUNCH((fp4_stream_kernel<KS, D, F32, true>), grid, dim3(64 * kFW), 0, st, g);
  else
    MOE_LAUNCH((fp4_stream_kernel<KS, D, F32, false>), grid, dim3(64 * kFW), 0, st, g);
}
template <int KS, int D>
hipError_t launch_stream_ks(const Fp4Gemm& g, int tiles, hipStream_t st) {
  const dim3 grid((tiles * KS + kFW - 1) / kFW);
  if (g.f32)
    launch_stream_as<KS, D, true>(g, grid, st);
  else
    launch_stream_as<KS, D, false>(g, grid, st);
  return hipGetLastError();
}

// K is split over wavefronts until about 16 of them per CU have work.
hipError_t launch_stream(const Fp4Gemm& g, hipStream_t st) {
  const int tiles = (g.N + 15) / 16;
  if (tiles >= 2048) return launch_stream_ks<2, 2>(g, tiles, st);
  if (tiles >= 1024) return launch_stream_ks<4, 2>(g, tiles, st);
  return launch_stream_ks<8, 2>(g, tiles, st);
}

template <int WT, int WW, int FT, int FW, int R, int KG, int SCALES, bool EARLY = false>
hipError_t launch_tile_as(const Fp4Gemm& g, hipStream_t st) {
  constexpr int BM = WT * FT * 16, BN = WW * FW * 16;
  const int nct = (g.N + BN - 1) / BN;
  int nrt = (g.rows + BM - 1) / BM, grid, chunk = 1;
  if (g.offsets) {
    nrt = g.rows / BM + std::min(g.rows, g.experts);  // every expert may end in a partial tile
    // Tiles dealt to the XCDs: with an expert in one or two row tiles, both with
    // all their column tiles to one XCD, so that its weights enter one L2.
    if (nrt > 32 && g.rows < static_cast<int64_t>(2 * BM) * g.experts) chunk = 2 * nct;
    grid = xcd_grid(nrt * nct, chunk);
  } else {
    grid = (nrt * nct + 7) / 8 * 8;
  }
  // Weights that about one row tile reads pass the caches by (down projection with
  // its quantisation, 32 tokens 246 -> 225 us, 4096 tokens 677 -> 643); weights that
  // many tiles read do not (4096 dense rows 93 -> 99). Experts get their rows unevenly:
  // where more than about four in ten start a second row tile the weights of those
  // cost more than that gains (128 rows on average in tiles of 128: 622 -> 715 us).
  // Only the mean is known here, and skewed routing takes what it asks for: with half
  // of the routes on 16 of 256 experts of 4096 x 4096, 512 tokens take 433 us (routed
  // evenly 430), 4096 tokens 677 (591); 512 tokens on 8192 x 4096 943 (891).
  const dim3 block(64 * WT * WW * KG);
  const double mean = static_cast<double>(g.rows) / g.experts;
  if (SCALES != kBy1 && (g.experts > 1 ? mean + 0.3 * std::sqrt(mean) : mean) <= BM)
    MOE_LAUNCH((fp4_tile_kernel<WT, WW, FT, FW, R, KG, SCALES, EARLY, SCALES != kBy1>), dim3(grid), block, 0, st, g, nrt, nct, chunk);
  else
    MOE_LAUNCH((fp4_tile_kernel<WT, WW, FT, FW, R, KG, SCALES, EARLY, false>), dim3(grid), block, 0, st, g, nrt, nct, chunk);
  return hipGetLastError();
}
// RB: stages held with scales by bytes, which take more LDS (two of them: EARLY, 64
// experts of 128 rows x 4096 x 2880 188 -> 174 us).
template <int WT, int WW, int FT, int FW, int R, int KG, int RB = R, bool EARLY = false>
hipError_t launch_tile(const Fp4Gemm& g, hipStream_t st) {
  if (g.scales == kBy16) return launch_tile_as<WT, WW, FT, FW, R, KG, kBy16, EARLY>(g, st);
  if (g.scales == kBy4) return launch_tile_as<WT, WW, FT, FW, R, KG, kBy4, EARLY>(g, st);
  return launch_tile_as<WT, WW, FT, FW, RB, KG, kBy1, RB == 2>(g, st);
}

// The tiles: rows, weight rows, and what one takes in ns: start and end, and per
// block of 256 of K with up to one workgroup per CU (`one`) or as many as share it
// (`full`; per_cu of them). The second set: with scales copied by bytes. Single
// kernels, N = 4096, K = 8192, us:
//   rows   32x32  32x64  64x64  64x128  128x128  128x128, 2 per CU  128x256  256x256
//     64     10     14     16      24       24          25             35       40
//    128     17     14     16      23       28          28             40       43
//    256     31     20     16      23       27          28             39       57
//    512     60     36     28      23       27          30             38       57
//   1024    117     65     56      36       28          31             36       57
//   2048    207    114    107      67       53          45             41       57
//   4096    386    209    186     124      106          88             82       67
// Small tiles win while they fit one round, their stages being mostly latency;
// for thousands of rows what counts is how often an operand enters LDS (12 .. 16
// TB/s over the chip with tiles of up to 128 x 128, 10 with 128 x 256, 8.5 with 256 x
// 256, whose stages wait for their copies' latency). N = 8192, K = 4096, 4096 rows:
// 128x256 96, 256x256 76. Experts of 128 rows (4096 tokens' down projection): 654, 622 and 576 with the last
// three. Over 13 widths, dense and per expert, 1 .. 4096 rows, the choice costs at
// most 1.15 times the best of them.
struct TileCost {
  int per_cu;
  double ends, one, full;
};
struct TileShape {
  int rows, cols;
  TileCost wide, bytes;
};
enum { T32x32, T32x64, T64x64, T64x128, T128x128, T128x128Two, T128x256, T256x256, kNTiles };
constexpr TileShape kTiles[kNTiles] = {{32, 32, {1, 4800, 160, 160}, {1, 4800, 180, 180}},
                                       {32, 64, {2, 3500, 320, 510}, {1, 3500, 430, 430}},
                                       {64, 64, {1, 4800, 340, 340}, {1, 4800, 550, 550}},
                                       {64, 128, {2, 5800, 525, 940}, {1, 5800, 610, 610}},
                                       {128, 128, {1, 5700, 680, 680}, {1, 5700, 1090, 1090}},
                                       {128, 128, {2, 5000, 850, 1300}, {2, 3800, 1540, 2100}},
                                       {128, 256, {1, 6600, 1140, 1140}, {1, 6600, 2270, 2270}},
                                       {256, 256, {1, 8100, 1850, 1850}, {1, 8100, 1850, 1850}}};

int best_tile(const Fp4Gemm& g) {
  // rows of one group: experts get theirs unevenly, by about the root of the mean
  const double mean = static_cast<double>(g.rows) / g.experts;
  const double rows = g.experts > 1 ? mean + std::sqrt(mean) : mean;
  const int groups = std::min(g.rows, g.experts);
  const double blocks = (g.K + kBlockValues - 1) / kBlockValues;
  int best = 0;
  double least = 1e300;
  for (int i = 0; i < kNTiles; ++i) {
    const TileShape& t = kTiles[i];
    const double per_group = std::ceil(std::max(rows, 1.0) / t.rows);
    const double tiles = groups * per_group * std::ceil(static_cast<double>(g.N) / t.cols);
    if (i == T256x256 && g.scales != kBy16) continue;  // (no registers to spare)
    const TileCost& c = g.scales == kBy1 ? t.bytes : t.wide;
    const double round = 256.0 * c.per_cu, whole = std::floor(tiles / round), rest = tiles - whole * round;
    const double full = c.ends + blocks * c.full, one = c.ends + blocks * c.one;
    const double ns = whole * full + (rest == 0 ? 0 : rest <= 256 ? one : full);
    // (a tile without rows in its lower part still streams its weights)
    const double fill = std::max(rows, 1.0) / (per_group * t.rows);
    const double cost = ns * (0.55 + 0.45 * fill);
    if (cost < least) {
      least = cost;
      best = i;
    }
  }
  return best;
}

// Up to 16 dense rows: the streaming kernel, while it has little to stream (a
// wavefront reads the rows beside its 16 weight rows, which costs the more the
// more rows * K they are and the more wavefronts share a CU). us, streaming kernel
// / best tiles:
//   rows   4096x4128   4096x8192   8192x4096   16384x1024   28672x8192   512x14336
//      1   5.2 / 7.5    6.8 / 8.9   6.1 / 7.1    4.5 / 5.3    31.6 / 30.6   7.4 / 8.7
//      8        -       7.5 / 9.1       -        4.8 / 5.4    37.9 / 31.3       -
//     16   6.6 / 8.6    8.4 / 9.4   8.0 / 7.2    5.2 / 5.6    45.2 / 31.6  10.0 / 8.9
// The step at N = 4096 is where a second workgroup joins a CU. Over N = 4096 .. 12288,
// K = 1024, 4096 and 8192, 1 .. 16 rows, the limits cost at most 1.11 times the better
// kernel (4112 x 4096, 8 rows: 5.9 / 6.5, and tiles taken).
// Per expert the tiles are level with it (8 routes of one token, N = 4096, K =
// 4096: 18.9 / 16.4) or better (32 tokens' 163 experts 296 / 252).
bool streams(const Fp4Gemm& g) {
  return !g.offsets && g.rows <= 16 && static_cast<int64_t>(g.rows) * g.K <= (g.N <= 4096 ? 128 << 10 : 16 << 10);
}

}  // namespace

hipError_t launch_fp4_gemm(const Fp4Gemm& g, hipStream_t st) {
  if (streams(g)) return launch_stream(g, st);
  switch (best_tile(g)) {
    case T32x32: return launch_tile<1, 2, 2, 1, 3, 4>(g, st);
    case T32x64: return launch_tile<1, 4, 2, 1, 3, 2>(g, st);
    case T64x64: return launch_tile<2, 2, 2, 2, 3, 2>(g, st);
    case T64x128: return launch_tile<2, 4, 2, 2, 3, 1>(g, st);
    case T128x128: return launch_tile<2, 4, 4, 2, 3, 1>(g, st);
    case T128x128Two: return launch_tile<2, 2, 4, 4, 2, 1, 2, true>(g, st);
    case T128x256: return launch_tile<2, 4, 4, 4, 3, 1, 2>(g, st);
    default: return launch_tile_as<4, 2, 4, 8, 2, 1, kBy16, true>(g, st);  // (by 16 only: no registers to spare)
  }
}

}  // namespace moe
