// gemm_fp8.hip -- products of E4M3 rows with E4M3 weights, one fp32 scale per
// 128 values of a row and one per 128 x 128 block of the weights, dense and
// per expert.
//
//   out[r][n] = sum_b xs[r][b] * ws[n/128][b] * sum_{k in block b} x[r][k] w[n][k]
//
// A block's sum leaves the matrix unit before it meets its scales (a scale that
// is no power of two cannot enter it) and is added in fp32 on the vector unit.
// The weights are the A operand and the rows the B operand, so a lane holds
// four neighbouring outputs of ONE row: its scale product is one value per row
// fragment and block, not one per output.
//
// Two ways to sum a block. The E4M3 MFMA 16x16x128 takes it in one
// instruction at twice the bf16 rate, but adds each eight neighbouring products
// on a grid 2^-14 of the largest of them and drops what lies below (measured; the
// eights are then added in fp32): each eight may come out 7 * 2^-14 of its
// largest product off, a block up to 2^-7.2 of its largest. For normal operands a
// sum is 1.5e-5 of the sums' norm off, which a bf16 rounding (half a step: up to
// 2^-8 of the value) hides; where the terms cancel it may be all that is left. The
// tiles with bf16 out take it, whatever bounds them, unless the caller asks for
// fp32 sums (MOE_SUM_F32) or there are at most 16 dense rows. Those, fp32 outs and
// the streaming kernel turn the codes into bf16 (exact) and sum the block to fp32 by four bf16 MFMAs 16x16x32
// (measured: 1e-8 of the norm).
#include <algorithm>
#include <cmath>

#include "device_common.h"
#include "fp8.h"
#include "grouped.h"
#include "kernels.h"

namespace moe {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8 pair16(uint4 lo, uint4 hi) {
  return i32x8{static_cast<int>(lo.x), static_cast<int>(lo.y), static_cast<int>(lo.z), static_cast<int>(lo.w),
               static_cast<int>(hi.x), static_cast<int>(hi.y), static_cast<int>(hi.z), static_cast<int>(hi.w)};
}

// Eight E4M3 codes as bf16, exactly.
__device__ __forceinline__ bf16x8 e4m3x8_to_bf16(int lo, int hi) {
  const uint32_t l = static_cast<uint32_t>(lo), h = static_cast<uint32_t>(hi);
  const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(l, 1.0f, false);
  const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(l, 1.0f, true);
  const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(h, 1.0f, false);
  const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(h, 1.0f, true);
  return bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// An operand fragment, 16 rows x one block, as the matrix instructions take it:
// the codes, or (EXACT) their bf16 values, decoded once for all the products it
// enters, for sums in fp32. Lane l holds 32 bytes of row l%16; which 32 of the block's 128 lane
// group l/16 holds is free as long as both operands agree, since the block is
// summed whole.
template <bool EXACT>
struct Operand {
  i32x8 codes;
  __device__ __forceinline__ void set(i32x8 c) { codes = c; }
};
template <>
struct Operand<true> {
  bf16x8 v[4];
  __device__ __forceinline__ void set(i32x8 c) {
#pragma unroll
    for (int s = 0; s < 4; ++s) v[s] = e4m3x8_to_bf16(c[2 * s], c[2 * s + 1]);
  }
};
// D(16x16, fp32) = A(16x128) * B(128x16)^T: lane l receives rows 4*(l/16) .. +3
// of A against row l%16 of B.
__device__ __forceinline__ f32x4 mfma_block(const Operand<false>& a, const Operand<false>& b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.codes, b.codes, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_block(const Operand<true>& a, const Operand<true>& b) {
  f32x4 d{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < 4; ++s) d = mfma16x16x32(a.v[s], b.v[s], d);
  return d;
}

// ---- few rows: the weights stream once from HBM ----------------------------
// A wavefront takes 16 weight rows x up to 16 rows over a run of K's blocks;
// KS wavefronts of a workgroup split K and are joined through LDS in order, and
// the workgroup's 8 / KS such teams take neighbouring weight rows. Everything a
// block needs (codes of both operands, scales) is loaded to registers D blocks
// ahead, so each wavefront keeps D * 2 KiB of weights in flight and waits for
// nothing else. A group of more rows takes them in passes. Grid: (weight row
// tiles, groups).
constexpr int kFW = 8;  // wavefronts

template <int KS, int D, bool F32>
__global__ __launch_bounds__(64 * kFW, 4) void fp8_stream_kernel(Fp8Gemm p) {
  constexpr int kTeams = kFW / KS;
  __shared__ f32x4 part[KS > 1 ? kFW : 1][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nl = lane & 15, g = lane >> 4;
  const Group grp = p.offsets ? find_group(p, static_cast<int>(blockIdx.y), 1 << 30) : Group{0, 0, p.rows};
  if (grp.expert < 0) return;
  const int ks = wave % KS;
  const int n0 = (static_cast<int>(blockIdx.x) * kTeams + wave / KS) * 16;
  const int nkb = (p.K + kFp8Block - 1) / kFp8Block;
  const int per = (nkb + KS - 1) / KS;
  const int kb0 = min(ks * per, nkb), n_kb = min(per, nkb - kb0);
  const size_t K = static_cast<size_t>(p.K);
  // (a team past the last weight row reads and writes nothing)
  const int wrows = min(max(p.N - n0, 0), 16);
  const rsrc_t w_r = make_rsrc(p.w + (static_cast<size_t>(grp.expert) * p.N + n0) * K, static_cast<uint32_t>(wrows * K));
  const rsrc_t ws_r = make_rsrc(
      p.ws + (static_cast<size_t>(grp.expert) * ((p.N + kFp8Block - 1) / kFp8Block) + n0 / kFp8Block) * nkb,
      wrows > 0 ? nkb * 4u : 0u);
  const uint32_t w_off = static_cast<uint32_t>(nl) * p.K + g * 16;
  // Wavefronts that take all of K start at different blocks: weight rows lie a
  // power of two apart as a rule, and wavefronts that walk them in step meet on
  // the same memory channels (8 tokens' down projection 213 -> 193 us).
  const int turn =
      KS == 1 ? __builtin_amdgcn_readfirstlane((5 * (static_cast<int>(blockIdx.x) + wave) + static_cast<int>(blockIdx.y)) % nkb) : 0;

  for (int r0 = grp.begin; r0 < grp.end; r0 += 16) {
    const int base = p.index ? 0 : r0;  // the descriptors start at this row of x
    const int xrows = p.index ? p.x_rows : min(grp.end - r0, 16);
    const rsrc_t x_r = make_rsrc(p.x + static_cast<size_t>(base) * p.ldx,
                                 static_cast<uint32_t>(static_cast<size_t>(xrows - 1) * p.ldx + K));
    const rsrc_t xs_r = make_rsrc(p.xs + static_cast<size_t>(base) * nkb, static_cast<uint32_t>(xrows) * nkb * 4u);
    // (lanes without a row read nothing)
    const int row = r0 + nl;
    const int src = row < grp.end ? source_row(p, row) - base : 0;
    const uint32_t x_off = row < grp.end ? static_cast<uint32_t>(src * p.ldx) + g * 16 : kOutOfRange;
    const uint32_t xs_off = row < grp.end ? static_cast<uint32_t>(src) * nkb * 4u : kOutOfRange;
    f32x4 acc{0.f, 0.f, 0.f, 0.f};

    uint4 wv[D][2], xv[D][2];
    float xsv[D], wsv[D];
    auto load = [&](int u, int i) __attribute__((always_inline)) {
      const int turned = i + turn;
      const int kb = kb0 + (turned >= n_kb ? turned - n_kb : turned);
      const uint32_t at = static_cast<uint32_t>(kb) * kFp8Block;
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // (pieces past the last value: zeros in both operands)
        const bool in = static_cast<int>(at) + h * 64 + g * 16 < p.K;
        wv[u][h] = buf_load16<kAuxStream>(w_r, in ? w_off + at + h * 64 : kOutOfRange);
        xv[u][h] = buf_load16<kAuxDefault>(x_r, in ? x_off + at + h * 64 : kOutOfRange);
      }
      xsv[u] = __uint_as_float(buf_load4<kAuxDefault>(xs_r, xs_off + kb * 4));
      wsv[u] = __uint_as_float(buf_load4<kAuxDefault>(ws_r, kb * 4));
    };
    auto consume = [&](int u) __attribute__((always_inline)) {
      Operand<true> wf, xf;
      wf.set(pair16(wv[u][0], wv[u][1]));
      xf.set(pair16(xv[u][0], xv[u][1]));
      const f32x4 d = mfma_block(wf, xf);
      const float s = xsv[u] * wsv[u];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(d[i], s, acc[i]);
    };
#pragma unroll
    for (int u = 0; u < D; ++u)
      if (u < n_kb) load(u, u);
    int i = 0;
    for (; i + 2 * D <= n_kb; i += D) {  // (no branches inside: the waits stay D blocks deep)
#pragma unroll
      for (int u = 0; u < D; ++u) {
        consume(u);
        load(u, i + D + u);
      }
    }
#pragma unroll
    for (int u = 0; u < D; ++u)
      if (i + u < n_kb) {
        consume(u);
        if (i + D + u < n_kb) load(u, i + D + u);
      }
    i += D;
#pragma unroll
    for (int u = 0; u < D; ++u)
      if (i + u < n_kb) consume(u);

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

// ---- many rows: LDS-staged tiles -------------------------------------------
// Workgroup tile: WT x WW wavefronts, each FT x FW fragments of 16 rows x 16
// weight rows; a tile's row fragments are dealt to the wavefront rows in
// turn, so a partly filled tile loads them evenly. KG blocks of K per stage,
// each the work of a wavefront group of its own (WT x WW), joined through LDS at
// the end: with few tiles a stage's length is the time its parts wait for each
// other, and a stage of four blocks takes little longer than one of one. Both
// operands' 128-byte rows are copied straight from global memory into LDS in a
// ring of R stages (the copies run R - 1 ahead), 16-byte piece c of row r at
// position r*8 + (c ^ ((r/2) % 8)), so that the 16 rows one read touches start
// in distinct banks. The scales follow the same way: with one block per stage
// in sets of four stages, [row][stage], two sets in turn; else with their stage,
// [row][block].

__device__ __forceinline__ int fpos(int r, int c) { return (r * 8 + (c ^ ((r >> 1) & 7))) * 16; }

template <int WT, int WW, int FT, int FW, int R, int KG, bool F32, bool EXACT>
__global__ __launch_bounds__(64 * WT * WW * KG) void fp8_tile_kernel(Fp8Gemm p, int n_row_tiles, int n_col_tiles, int chunk) {
  constexpr int kGroup = WT * WW, NW = kGroup * KG, BM = WT * FT * 16, BN = WW * FW * 16;
  // 1-KiB copies per wavefront and stage (its group's block); of the rows' some
  // wavefronts may have one fewer
  constexpr int kXOps = (BM / 8 + kGroup - 1) / kGroup, kXLeast = BM / 8 / kGroup, kWOps = BN / 8 / kGroup;
  constexpr int kFSet = KG == 1 ? 4 : KG;                          // blocks of a scale set
  constexpr int kSetRows = 64 / kFSet, kSets = KG == 1 ? 2 : R;    // rows of one 64-scale copy; sets held
  constexpr int kSOps = (BM / kSetRows + NW - 1) / NW;             // such copies per wavefront and set
  static_assert((BN % kFp8Block == 0 || kFp8Block % BN == 0) && BN * kFSet <= 64 * kFp8Block, "tiles within weight blocks");
  static_assert(kWOps * 8 * kGroup == BN && BM % kSetRows == 0 && kXLeast > 0, "whole copies");
  constexpr int kOps = kXOps + kWOps, kLeast = kXLeast + kWOps;
  static_assert((R - 2) * kLeast < 64, "vmcnt field");
  // (KG = 1: a set is asked for four stages before its first use, and the wait
  // of the third of them leaves at most the copies of R - 2 stages outstanding,
  // all younger)
  static_assert(R >= 2 && R <= 4, "scale sets land in time");
  constexpr int kXSlot = KG * BM * kFp8Block, kWSlot = KG * BN * kFp8Block;  // bytes of a stage
  __shared__ __attribute__((aligned(1024))) uint8_t Xs[R][kXSlot];
  __shared__ __attribute__((aligned(1024))) uint8_t Ws[R][kWSlot];
  __shared__ __attribute__((aligned(256))) float Sx[kSets][BM * kFSet];
  __shared__ __attribute__((aligned(256))) float Sw[kSets][64];
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
  const int nkb = (p.K + kFp8Block - 1) / kFp8Block, nst = (nkb + KG - 1) / KG;
  const size_t K = static_cast<size_t>(p.K);
  const int nnb = (n0 % kFp8Block + ncols + kFp8Block - 1) / kFp8Block;  // weight blocks of the tile that exist
  const uint8_t* w_base = p.w + (static_cast<size_t>(grp.expert) * p.N + n0) * K;
  const uint32_t w_bytes = static_cast<uint32_t>(ncols * K);
  const rsrc_t ws_r = make_rsrc(
      p.ws + (static_cast<size_t>(grp.expert) * ((p.N + kFp8Block - 1) / kFp8Block) + n0 / kFp8Block) * nkb,
      static_cast<uint32_t>(nnb * nkb) * 4u);
  const int base = p.index ? 0 : grp.begin;
  const int xrows = p.index ? p.x_rows : nrows;
  const uint8_t* x_base = p.x + static_cast<size_t>(base) * p.ldx;
  const uint32_t x_bytes = static_cast<uint32_t>(static_cast<size_t>(xrows - 1) * p.ldx + K);
  const rsrc_t xs_r = make_rsrc(p.xs + static_cast<size_t>(base) * nkb, static_cast<uint32_t>(xrows) * nkb * 4u);
  auto row_of = [&](int r) -> int { return r < nrows ? source_row(p, grp.begin + r) - base : -1; };

  // Source offsets of this wavefront's copies in the first stage; the
  // descriptors step along K, so a copy costs no vector arithmetic.
  uint32_t xoff[kXOps], woff[kWOps], soff[kSOps];
#pragma unroll
  for (int i = 0; i < kXOps; ++i) {
    const int r = (i * kGroup + wave % kGroup) * 8 + (lane >> 3), src = row_of(r);
    xoff[i] = src < 0 ? kOutOfRange : static_cast<uint32_t>(src * p.ldx) + kg * kFp8Block + ((lane & 7) ^ ((r >> 1) & 7)) * 16;
  }
#pragma unroll
  for (int i = 0; i < kWOps; ++i) {
    const int r = (i * kGroup + wave % kGroup) * 8 + (lane >> 3);
    woff[i] = static_cast<uint32_t>(r) * p.K + kg * kFp8Block + ((lane & 7) ^ ((r >> 1) & 7)) * 16;
  }
#pragma unroll
  for (int i = 0; i < kSOps; ++i) {
    const int src = row_of((kSOps * wave + i) * kSetRows + lane / kFSet);
    soff[i] = src < 0 ? kOutOfRange : static_cast<uint32_t>(src) * nkb * 4u + (lane % kFSet) * 4;
  }
  const uint32_t lds_x = lds_address(&Xs[0][0]), lds_w = lds_address(&Ws[0][0]);
  const uint32_t lds_sx = lds_address(&Sx[0][0]), lds_sw = lds_address(&Sw[0][0]);
  // Copies of one stage: descriptors, and the LDS slot they fill. Stages past
  // the last have empty descriptors, so their copies read nothing (zeros into a
  // slot that no product reads) and every stage counts the same.
  struct Stage {
    rsrc_t x, w;
    int slot;
  };
  const bool partial = p.K % (KG * kFp8Block) != 0;
  auto stage_of = [&](int st, int slot) __attribute__((always_inline)) {
    const uint32_t k0 = static_cast<uint32_t>(st) * (KG * kFp8Block);
    if (partial && st == nst - 1) {  // the last one that reads: its pieces past K read nothing, zeros in both operands
      const int left = p.K - static_cast<int>(k0) - kg * kFp8Block;
      auto in = [&](int q) { return ((lane & 7) ^ (((q * 8 + (lane >> 3)) >> 1) & 7)) * 16 < left; };
#pragma unroll
      for (int i = 0; i < kXOps; ++i)
        if (!in(i * kGroup + wave % kGroup)) xoff[i] = kOutOfRange;
#pragma unroll
      for (int i = 0; i < kWOps; ++i)
        if (!in(i * kGroup + wave % kGroup)) woff[i] = kOutOfRange;
    }
    const bool none = st >= nst;
    return Stage{make_rsrc(none ? x_base : x_base + k0, none ? 0 : x_bytes - k0),
                 make_rsrc(none ? w_base : w_base + k0, none ? 0 : w_bytes - k0), slot};
  };
  // this wavefront's copy c (0 .. kOps-1) of a stage
  auto copy = [&](const Stage& s, int c) __attribute__((always_inline)) {
    const int i = c < kXOps ? c : c - kXOps, q = i * kGroup + wave % kGroup;  // 8-row block of the tile
    if (c < kXOps) {
      if (kXOps == kXLeast || q < BM / 8)
        lds_copy16(s.x, xoff[c < kXOps ? c : 0],
                   __builtin_amdgcn_readfirstlane(lds_x + s.slot * kXSlot + kg * (BM * kFp8Block) + q * 1024));
    } else {
      lds_copy16(s.w, woff[c < kXOps ? 0 : c - kXOps],
                 __builtin_amdgcn_readfirstlane(lds_w + s.slot * kWSlot + kg * (BN * kFp8Block) + q * 1024));
    }
  };
  auto issue_set = [&](int set, int at) __attribute__((always_inline)) {
    const bool in = set * kFSet + lane % kFSet < nkb;
#pragma unroll
    for (int i = 0; i < kSOps; ++i)
      if (kSOps * wave + i < BM / kSetRows)
        lds_copy4(xs_r, in ? soff[i] + set * (kFSet * 4) : kOutOfRange,
                  __builtin_amdgcn_readfirstlane(lds_sx + at * (BM * kFSet * 4) + (kSOps * wave + i) * 256));
    if (wave == 0)
      lds_copy4(ws_r, in && lane / kFSet < nnb ? (lane / kFSet * nkb + set * kFSet + lane % kFSet) * 4u : kOutOfRange,
                __builtin_amdgcn_readfirstlane(lds_sw + at * 256));
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
  // stage st + R, spread over the following products (together they would fill
  // the memory pipe's queue and hold the wavefront up). Within a stage a
  // product's four scaled additions run under the matrix instructions of the two
  // products after it, and the next row fragment's reads under those of this
  // one; the scheduling barriers keep that order (left alone, the compiler puts
  // all additions behind all products).
  auto kloop = [&](auto live_tag) __attribute__((always_inline)) {
    constexpr int LIVE = decltype(live_tag)::value;
    constexpr int kProducts = LIVE * FW;  // of a wavefront and stage
    // copy c goes out with product at(c), counted from the meeting
    auto at = [](int c) constexpr { return kProducts >= 2 * kOps ? 2 * c : c * kProducts / kOps; };
    auto copies_at = [&](const Stage& s, int q) __attribute__((always_inline)) {
#pragma unroll
      for (int c = 0; c < kOps; ++c)
        if (at(c) == q) copy(s, c);
    };
    if constexpr (KG == 1) issue_set(0, 0);
#pragma unroll
    for (int s = 0; s < R - 1; ++s) {
      if constexpr (KG > 1) issue_set(s, s);
      const Stage g = stage_of(s, s);
#pragma unroll
      for (int c = 0; c < kOps; ++c) copy(g, c);
    }
    if constexpr (KG > 1) issue_set(R - 1, R - 1);
    Stage ahead = stage_of(R - 1, R - 1);
#pragma unroll
    for (int q = 0; q < (LIVE > 0 ? FW : 1); ++q) copies_at(ahead, q);
    wait_vm_lds<0>();
    __syncthreads();
    // the copies of stage st + 1 have landed, in every wavefront
    auto meet = [&](int st, int slot) __attribute__((always_inline)) {
      wait_vm_lds<(R - 2) * kLeast>();
      __syncthreads();
      if constexpr (KG > 1) issue_set(st + R, slot);
      ahead = stage_of(st + R, slot);
    };
    // KG = 1: the set after stage st's, when st is the first of its set (every
    // wavefront has read the last scales of the set this one replaces)
    auto next_set = [&](int st) __attribute__((always_inline)) {
      if (KG == 1 && st % kFSet == 0) issue_set(st / kFSet + 1, (st / kFSet + 1) & 1);
    };
    if constexpr (LIVE == 0) {
      for (int st = 0, slot = 0; st < nst; ++st, slot = slot == R - 1 ? 0 : slot + 1) {
        next_set(st);
        meet(st, slot);
        copies_at(ahead, 0);
      }
    } else {
      // (rows 16 apart keep their swizzle: constant offsets from one address)
      const int xp0 = fpos(wt * 16 + nl, g), xp1 = fpos(wt * 16 + nl, 4 + g);
      const int wp0 = fpos(ww * FW * 16 + nl, g), wp1 = fpos(ww * FW * 16 + nl, 4 + g);
      auto read_x = [&](int slot, int t) __attribute__((always_inline)) {
        const uint8_t* b = &Xs[0][0] + slot * kXSlot + kg * (BM * kFp8Block);
        return pair16(*reinterpret_cast<const uint4*>(b + xp0 + t * WT * 2048), *reinterpret_cast<const uint4*>(b + xp1 + t * WT * 2048));
      };
      auto read_w = [&](int slot, int f) __attribute__((always_inline)) {
        const uint8_t* b = &Ws[0][0] + slot * kWSlot + kg * (BN * kFp8Block);
        return pair16(*reinterpret_cast<const uint4*>(b + wp0 + f * 2048), *reinterpret_cast<const uint4*>(b + wp1 + f * 2048));
      };
      auto scale_x = [&](int st, int slot, int t) __attribute__((always_inline)) {
        const int set = KG == 1 ? (st / kFSet) & 1 : slot, blk = KG == 1 ? st % kFSet : kg;
        return (&Sx[set][(wt * 16 + nl) * kFSet + blk])[t * WT * 16 * kFSet];
      };
      auto scale_w = [&](int st, int slot) __attribute__((always_inline)) {
        const int set = KG == 1 ? (st / kFSet) & 1 : slot, blk = KG == 1 ? st % kFSet : kg;
        return Sw[set][(n0 % kFp8Block + ww * (FW * 16)) / kFp8Block * kFSet + blk];
      };
      Operand<EXACT> wv[FW], xv;
#pragma unroll
      for (int f = 0; f < FW; ++f) wv[f].set(read_w(0, f));
      i32x8 next = read_x(0, 0);
      float next_s = scale_x(0, 0, 0), next_w = scale_w(0, 0);
      constexpr int kLag = FW < 2 ? FW : 2;  // (two row fragments' scales are held)
      for (int st = 0, slot = 0; st < nst; ++st) {
        const int after = slot == R - 1 ? 0 : slot + 1;
        const float wsc = next_w;
        next_set(st);
        f32x4 d[kLag + 1];
        float s[2];
        auto add = [&](int j) __attribute__((always_inline)) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[j / FW][j % FW][i] = fmaf(d[j % (kLag + 1)][i], s[(j / FW) & 1], acc[j / FW][j % FW][i]);
            asm volatile("" : "+v"(acc[j / FW][j % FW][i]));  // (not moved behind the branches below)
          }
        };
#pragma unroll
        for (int t = 0; t < LIVE; ++t) {
          xv.set(next);
          s[t & 1] = next_s * wsc;
          if (t + 1 < LIVE) {
            next = read_x(slot, t + 1);
            next_s = scale_x(st, slot, t + 1);
          } else {
            meet(st, slot);
            next = read_x(after, 0);  // (after the last stage: what the slot held, not used)
            next_s = scale_x(st + 1, after, 0);
            next_w = scale_w(st + 1, after);
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int f = 0; f < FW; ++f) {
            const int j = t * FW + f;
            d[j % (kLag + 1)] = mfma_block(wv[f], xv);
            __builtin_amdgcn_sched_barrier(0);
            if (t + 1 == LIVE) wv[f].set(read_w(after, f));
            if (j >= kLag) add(j - kLag);
            copies_at(ahead, t + 1 == LIVE ? f : j + FW);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
#pragma unroll
        for (int j = kProducts > kLag ? kProducts - kLag : 0; j < kProducts; ++j) add(j);
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
  const int n1 = n0 + ww * (FW * 16) + 4 * g;
  if (p.out_vec && n0 + BN <= p.N) {  // (no part of the tile lies past the last weight row)
#pragma unroll
    for (int t = 0; t < FT; ++t) {
      const int r = (t * WT + wt) * 16 + nl;
      auto* o = static_cast<typename Out4<F32>::type*>(p.out) + static_cast<size_t>(grp.begin + r) * p.ldo + n1;
      if (r < nrows) {
#pragma unroll
        for (int f = 0; f < FW; ++f) {
          const Out4<F32> x(acc[t][f]);
          *reinterpret_cast<decltype(x.v)*>(o + f * 16) = x.v;
        }
      }
    }
  } else {
#pragma unroll
    for (int t = 0; t < FT; ++t) {
      const int r = (t * WT + wt) * 16 + nl;
      if (r < nrows) {
#pragma unroll
        for (int f = 0; f < FW; ++f)
          if (n1 + f * 16 < p.N) store4<F32>(p, grp.begin + r, n1 + f * 16, acc[t][f]);
      }
    }
  }
}

template <int KS, int D>
hipError_t launch_stream_ks(const Fp8Gemm& g, int tiles, int groups, hipStream_t st) {
  const dim3 grid((tiles * KS + kFW - 1) / kFW, groups), block(64 * kFW);
  if (g.f32)
    MOE_LAUNCH((fp8_stream_kernel<KS, D, true>), grid, block, 0, st, g);
  else
    MOE_LAUNCH((fp8_stream_kernel<KS, D, false>), grid, block, 0, st, g);
  return hipGetLastError();
}

// K is split over wavefronts until about 16 of them per CU have work (one
// token's gate/up, 8 experts x 512 tiles: no split 57 us, split by two 59);
// a wavefront with all of K keeps four blocks in flight, one with a part two
// (one pooler token 9.3 -> 8.8 us, fewer registers).
hipError_t launch_stream(const Fp8Gemm& g, int groups, hipStream_t st) {
  const int tiles = (g.N + 15) / 16;
  const int64_t waves = static_cast<int64_t>(tiles) * groups;
  if (waves >= 4096) return launch_stream_ks<1, 4>(g, tiles, groups, st);
  if (waves >= 2048) return launch_stream_ks<2, 2>(g, tiles, groups, st);
  if (waves >= 1024) return launch_stream_ks<4, 2>(g, tiles, groups, st);
  return launch_stream_ks<8, 2>(g, tiles, groups, st);
}

template <int WT, int WW, int FT, int FW, int R, int KG, bool F32, bool EXACT>
hipError_t launch_tile_as(const Fp8Gemm& g, hipStream_t st) {
  constexpr int BM = WT * FT * 16, BN = WW * FW * 16;
  const int nct = (g.N + BN - 1) / BN;
  int nrt = (g.rows + BM - 1) / BM, grid, chunk = 1;
  if (g.offsets) {
    nrt = g.rows / BM + std::min(g.rows, g.experts);  // every expert may end in a partial tile
    // Tiles dealt to the XCDs: with an expert in one or two row tiles, both with
    // all their column tiles to one XCD, so that its weights enter one L2. With
    // more, or too few to go round, single tiles: a column tile then meets the
    // same XCD for every row tile as a rule (2000 tokens on 16 experts 206 ->
    // 196 us, one token's 8 routes 38 -> 26).
    if (nrt > 32 && g.rows < static_cast<int64_t>(2 * BM) * g.experts) chunk = 2 * nct;
    grid = xcd_grid(nrt * nct, chunk);
  } else {
    grid = (nrt * nct + 7) / 8 * 8;
  }
  MOE_LAUNCH((fp8_tile_kernel<WT, WW, FT, FW, R, KG, F32, EXACT>), dim3(grid), dim3(64 * WT * WW * KG), 0, st, g, nrt, nct, chunk);
  return hipGetLastError();
}
template <int WT, int WW, int FT, int FW, int R, int KG>
hipError_t launch_tile_exact(const Fp8Gemm& g, hipStream_t st) {
  return g.f32 ? launch_tile_as<WT, WW, FT, FW, R, KG, true, true>(g, st)
               : launch_tile_as<WT, WW, FT, FW, R, KG, false, true>(g, st);
}
template <int WT, int WW, int FT, int FW, int R, int KG>
hipError_t launch_tile(const Fp8Gemm& g, hipStream_t st) {
  return g.exact ? launch_tile_exact<WT, WW, FT, FW, R, KG>(g, st)
                 : launch_tile_as<WT, WW, FT, FW, R, KG, false, false>(g, st);
}

// The tiles: rows, weight rows, and what one block of K takes in ns: in the
// first round of workgroups, and in each further one (the 32 x 64 ones share a CU
// with others, so their further rounds overlap). `one`: for a single round
// only, with stages of several blocks. Measured at N = 4096, K = 8192 in bf16 out
// and taken to go the same way at other widths; fp32 sums take 1.2 times as long
// for 64 rows, 1.5 for 256, 1.7 for 2048, 2.1 for 4096. Small tiles win while they
// fit one round: each has a CU to itself. What bounds them is not the matrix unit:
// their operands enter LDS at 11 .. 15 TB/s over the chip whichever tile is taken,
// with stages that wait on memory and on each other. N = 4096, K = 8192, us:
//   rows   32x32 one  32x64 one  64x64 one  64x128 one  32x64  64x128  128x128  128x256  256x256
//     64       11        15         18          23        22      28       29       38       71
//    128        -        15         18          23        22      28       35       53       71
//    256        -        29         20          24        30      29       36       53       88
//    512        -        53         36          27        50      31       37       54       88
//   2048        -         -          -           -       204     119       82       71       99
//   4096        -         -          -           -         -       -        -      155      117
// (48 x 32: 33 rows of N = 8192, K = 4096 10.2 us against 11.0 with 32 x 64.)
// 144 x 256 stands for experts of about 128 rows, half of which would take a
// second, nearly empty tile of 128 (4096 tokens' down projection 6% less time than
// with 128 x 256, experts of 109 rows the same).
struct TileShape {
  int rows, cols, first_ns, more_ns;
  bool one;
};
enum { T32x32, T48x32, T32x64, T64x64, T64x128, T32x64Rounds, T64x128Rounds, T128x128, T128x256, T144x256, T256x256, kNTiles };
constexpr TileShape kTiles[kNTiles] = {
    {32, 32, 175, 0, true},        {48, 32, 195, 0, true},        {32, 64, 230, 0, true},
    {64, 64, 300, 0, true},        {64, 128, 420, 0, true},       {32, 64, 340, 210, false},
    {64, 128, 450, 450, false},    {128, 128, 620, 620, false},   {128, 256, 1100, 1100, false},
    {144, 256, 1200, 1200, false}, {256, 256, 1800, 1800, false}};

int best_tile(const Fp8Gemm& g) {
  // rows of one group: experts get theirs unevenly, by about the root of the mean
  const double mean = static_cast<double>(g.rows) / g.experts;
  const double rows = g.experts > 1 ? mean + std::sqrt(mean) : mean;
  const int groups = std::min(g.rows, g.experts);
  int best = T32x64Rounds;
  double least = 1e30;
  for (int i = 0; i < kNTiles; ++i) {
    const TileShape& t = kTiles[i];
    // 256 x 256: its sums fill the registers, no room for bf16 operands; and
    // partly filled ones waste most (experts of 128 rows: 10% more time)
    if (t.rows == 256 && (g.exact || (g.experts > 1 && mean < 512))) continue;
    const double tiles = groups * std::ceil(rows / t.rows) * std::ceil(static_cast<double>(g.N) / t.cols);
    if (t.one && tiles > 256.0) continue;
    const double rounds = t.more_ns == t.first_ns ? std::ceil(tiles / 256.0) : std::max(1.0, tiles / 256.0);
    const double ns = t.first_ns + (rounds - 1.0) * t.more_ns;
    if (ns < least) {
      least = ns;
      best = i;
    }
  }
  return best;
}

// Few rows and little to stream: the streaming kernel or the tiles. Per expert
// (8 tokens on 4 experts 12.8 us against 12.0 .. 13.0) the streaming kernel,
// until the weights fill the chip: there the tiles read faster, whole 128-byte
// lines at a time (32 tokens' down projection 480 us against 510).
//
// Dense: a streaming wavefront reads the rows beside its 16 weight rows, so what
// it costs grows with rows * K. Up to 4096 weight rows each of its workgroups has
// a CU to itself and that is little; beyond, they share CUs, two on some and one
// on others, and the tiles win but for the shortest products. In between: weight
// rows a multiple of 4096 bytes apart meet on the same memory channels, which
// costs the tiles a tenth (N = 28672: 4.1 TB/s at K = 8192, 5.0 at 7168), while the
// CUs' last round of streaming workgroups is nearly full. The limits are where
// the two cross over 18 widths N of 512 .. 28672 and 9 of K of 512 .. 14336 at
// 1 .. 16 rows, weights from HBM (mean loss over the better of the two 0.5%, at
// most 1.17 times). us, streaming kernel / tiles, fp32 sums:
//   rows   4096x4096   4096x8192   5120x7168   8192x1024   8192x4096   16384x8192
//      1   7.0 / 8.8    9.9 / 13.2  13.7 / 12.6   4.6 / 5.7    9.7 / 11.0  28.4 / 33.5
//      4   7.2 / 8.9   10.7 / 13.4  14.7 / 12.7   4.6 / 5.7   10.6 / 10.9  31.9 / 33.7
//     16   8.1 / 9.3   13.6 / 14.1  20.4 / 13.4   5.6 / 5.9   13.4 / 11.1  44.1 / 34.3
bool streams(const Fp8Gemm& g) {
  if (g.experts > 1) return true;
  const int64_t values = static_cast<int64_t>(g.rows) * g.K;
  if (g.N <= 4096) return values <= 128 << 10;
  const int tiles = (g.N + 15) / 16, rounds = (tiles + 255) / 256;
  if (g.K % 4096 == 0 && tiles * 8 >= rounds * 256 * 7) return values <= 16 << 10;
  return values <= 8 << 10;
}

}  // namespace

hipError_t launch_fp8_gemm(const Fp8Gemm& call, hipStream_t st) {
  Fp8Gemm g = call;
  // Up to 16 dense rows are summed in fp32 by either kernel, so that few tokens'
  // results do not go by the widths (tiles: 8192 x 4096 11.1 -> 11.5 us).
  if (g.experts == 1 && g.rows <= 16) g.exact = true;
  const int groups = std::min(g.rows, g.experts);
  const int mean = (g.rows - 1) / g.experts + 1;
  if (g.rows <= 64 && mean <= 16 && static_cast<int64_t>(groups) * ((g.N + 63) / 64) < 2048 && streams(g))
    return launch_stream(g, groups, st);
  switch (best_tile(g)) {
    case T32x32: return launch_tile<1, 2, 2, 1, 3, 4>(g, st);
    case T48x32: return launch_tile<1, 2, 3, 1, 3, 4>(g, st);
    // (four blocks per stage where their decoding is the longer part: 33 rows in
    // fp32, N = 8192, K = 4096, 12.4 us against 13.6; bf16 11.0 against 10.5)
    case T32x64: return g.exact ? launch_tile_exact<1, 4, 2, 1, 3, 4>(g, st) : launch_tile_as<1, 4, 2, 1, 4, 2, false, false>(g, st);
    case T64x64: return launch_tile<2, 2, 2, 2, 3, 2>(g, st);
    case T64x128: return launch_tile<2, 4, 2, 2, 3, 2>(g, st);
    case T32x64Rounds: return launch_tile<1, 4, 2, 1, 4, 1>(g, st);
    case T64x128Rounds: return launch_tile<2, 4, 2, 2, 4, 1>(g, st);
    case T128x128: return launch_tile<2, 4, 4, 2, 4, 1>(g, st);
    case T128x256: return launch_tile<2, 4, 4, 4, 3, 1>(g, st);
    case T144x256: return launch_tile<1, 8, 9, 2, 3, 1>(g, st);
    // (wavefronts of 64 rows x 128 weight rows: 117 us for 4096 rows against 124
    // with 128 x 64, half the row scales to read and multiply)
    default: return launch_tile_as<4, 2, 4, 8, 2, 1, false, false>(g, st);
  }
}

}  // namespace moe
