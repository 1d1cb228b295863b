// grouped.h -- what the products of 8-bit and of 4-bit rows share: the group of
// rows that a workgroup takes, the row that an output row reads, stores of four
// neighbouring outputs, waits and copies into LDS. P: a product's arguments
// (Fp8Gemm, Fp4Gemm).
#pragma once

#include "device_common.h"

namespace moe {

// Waits until at most the N most recent vector-memory instructions are
// outstanding (N < 64: vmcnt's high two bits are bits 14 and 15) and every LDS
// read has returned.
template <int N>
__device__ __forceinline__ void wait_vm_lds() {
  static_assert(N >= 0 && N < 64, "vmcnt field");
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));
}

// The rows a workgroup takes: tile `tile` of the list that gives every
// expert ceil(rows / tile_rows) tiles, experts ascending. Every wavefront
// finds it by itself: four experts per lane, a scan of the tile counts over
// the lanes, a ballot. Offsets are clamped into [0, rows], so a bad list
// cannot lead outside the buffers. expert < 0: no such tile.
struct Group {
  int expert, begin, end;
};
template <typename P>
__device__ __forceinline__ Group find_group(const P& p, int tile, int tile_rows) {
  if (!p.offsets) {
    const int b = tile * tile_rows;
    return b < p.rows ? Group{0, b, min(p.rows - b, tile_rows) + b} : Group{-1, 0, 0};
  }
  const int lane = threadIdx.x & 63;
  int off[5], cnt[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 5; ++i) off[i] = min(max(p.offsets[min(4 * lane + i, p.experts)], 0), p.rows);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = off[i + 1] - off[i];
    cnt[i] = n > 0 ? (n - 1) / tile_rows + 1 : 0;  // (lanes past the last expert: no rows)
    sum += cnt[i];
  }
  int upto = sum;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int v = __shfl_up(upto, d, 64);
    if (lane >= d) upto += v;
  }
  int left = tile - (upto - sum);
  const uint64_t mine = __ballot(left >= 0 && left < sum);
  if (mine == 0) return Group{-1, 0, 0};
  int e = 4 * lane, b = off[0], n = off[1];
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (e == 4 * lane + i && left >= cnt[i]) {
      left -= cnt[i];
      e = 4 * lane + i + 1;
      b = off[i + 1];
      n = off[i + 2];
    }
  b += left * tile_rows;
  const int src = __builtin_ctzll(mine);
  Group g;
  g.expert = __builtin_amdgcn_readlane(e, src);
  g.begin = __builtin_amdgcn_readlane(b, src);
  g.end = min(__builtin_amdgcn_readlane(n, src), g.begin + min(tile_rows, p.rows));
  return g;
}

// The row of x that output row r reads (an index outside x is clamped into it).
template <typename P>
__device__ __forceinline__ int source_row(const P& p, int r) {
  if (!p.index) return r;
  const int v = p.index[r] / p.index_div;
  return min(max(v, 0), p.x_rows - 1);
}

// Four neighbouring outputs as they are stored (bf16: to nearest even, by the
// conversion instruction).
template <bool F32>
struct Out4 {
  typedef float type;
  f32x4 v;
  __device__ __forceinline__ explicit Out4(f32x4 a) : v(a) {}
};
template <>
struct Out4<false> {
  typedef __bf16 type;
  __attribute__((__vector_size__(4 * sizeof(__bf16)))) __bf16 v;
  __device__ __forceinline__ explicit Out4(f32x4 a)
      : v{static_cast<__bf16>(a[0]), static_cast<__bf16>(a[1]), static_cast<__bf16>(a[2]), static_cast<__bf16>(a[3])} {}
};

// Outputs n .. n+3 of one row, those that exist.
template <bool F32, typename P>
__device__ __forceinline__ void store4(const P& p, int row, int n, f32x4 a) {
  const Out4<F32> x(a);
  auto* o = static_cast<typename Out4<F32>::type*>(p.out) + static_cast<size_t>(row) * p.ldo + n;
  if (p.out_vec && n + 4 <= p.N) {
    *reinterpret_cast<decltype(x.v)*>(o) = x.v;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < p.N) o[i] = x.v[i];
  }
}

// As lds_copy16, 4 bytes per lane.
__device__ __forceinline__ void lds_copy4(rsrc_t r, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dword %0, %1, 0 offen lds" ::"v"(voff), "s"(r), "s"(lds) : "memory");
}
template <typename T>
__device__ __forceinline__ uint32_t lds_address(const T* p) {
  return static_cast<uint32_t>(reinterpret_cast<size_t>((__attribute__((address_space(3))) T*)(p)));
}

}  // namespace moe
