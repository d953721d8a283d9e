// Tiles of the kernels that write transposed codes (quantize.hip,
// act_grad.hip): 128 rows x 64 columns, 256 threads; thread t holds rows
// 4 (t / 8) .. + 3 of columns 8 (t % 8) .. + 7.  LDS (transposed codes): 64
// columns x 32 words; word w of column c holds rows 4w .. 4w + 3 and sits at
// c * 32 + (w ^ (8 * ((c / 8) & 3))).
#pragma once
#include "fp8mi_device.h"

namespace fp8mi {

constexpr int kTileR = 128, kTileC = 64, kTileThreads = 256;

// Bias-gradient partials in LDS: row group g (32 of them, 4 rows each) and
// column c at g * 64 + (c ^ (g & 7)).  A write instruction (fixed column
// offset e, lanes over 8 row groups x 8 column groups) then spreads over 32
// distinct 8-byte bank pairs, and a read (one row group, 64 consecutive
// columns) stays a permutation of one 512-byte row.
__device__ __forceinline__ int bg_index(int g, int c) { return g * 64 + (c ^ (g & 7)); }

__device__ __forceinline__ int lds_t_index(int c, int w) { return c * 32 + (w ^ (8 * ((c >> 3) & 3))); }

// Tile origin (row, column) of a tile index: 32-bit division whenever the
// tile count fits (every tensor a GPU can hold), 64-bit otherwise; the
// branch is uniform across the workgroup.
__device__ __forceinline__ void tile_origin(int64_t tile, int64_t tiles_c, int64_t ntiles, int64_t& r0,
                                            int64_t& c0) {
  if (ntiles <= 0xFFFFFFFFll) {
    const uint32_t t = (uint32_t)tile, tc = (uint32_t)tiles_c;
    const uint32_t q = t / tc;
    r0 = (int64_t)q * kTileR;
    c0 = (int64_t)(t - q * tc) * kTileC;
  } else {
    r0 = (tile / tiles_c) * kTileR;
    c0 = (tile % tiles_c) * kTileC;
  }
}

// One-shot dual grids: workgroups are dealt to the 8 XCDs round-robin, and a
// tile's row codes fill one half of each 128-byte line, the column
// neighbour's tile the other.  Workgroups b and b + 8 (the same XCD, launched
// one after the other) take tiles 2k and 2k + 1 of each group of 16, so the two
// halves of a line meet in one L2 and leave it together; the XCDs still take
// neighbouring pairs in turn.  (Measured at bf16 8192 x 1536, alternating
// libraries on one box: dual 14.5 -> 14.25 us with a ring, 12.4 -> 12.1 us with
// a scale; giving each XCD one contiguous range of tiles instead gained about
// as much for the dual and slowed the transposed layout by 6-9%.)
__device__ __forceinline__ uint32_t dual_pair_block(uint32_t b, uint32_t nb) {
  const uint32_t full = nb / 16u * 16u;
  if (b >= full) return b;
  const uint32_t r = b % 16u;
  return b - r + 2u * (r % 8u) + r / 8u;
}

// 4 x 4 byte transpose: words a, b, c, d hold 4 consecutive codes of rows 0..3;
// col[k] receives byte k of each, row 0 in its low byte.  Two stages of
// v_perm_b32 (byte k of the result picks byte sel_k of {hi, lo}, 0-3 from lo,
// 4-7 from hi): interleave row pairs, then take the matching halves.
__device__ __forceinline__ void transpose4x4_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t (&col)[4]) {
  const uint32_t ab_lo = __builtin_amdgcn_perm(b, a, 0x05010400u);  // a0 b0 a1 b1
  const uint32_t ab_hi = __builtin_amdgcn_perm(b, a, 0x07030602u);  // a2 b2 a3 b3
  const uint32_t cd_lo = __builtin_amdgcn_perm(d, c, 0x05010400u);  // c0 d0 c1 d1
  const uint32_t cd_hi = __builtin_amdgcn_perm(d, c, 0x07030602u);  // c2 d2 c3 d3
  col[0] = __builtin_amdgcn_perm(cd_lo, ab_lo, 0x05040100u);         // a0 b0 c0 d0
  col[1] = __builtin_amdgcn_perm(cd_lo, ab_lo, 0x07060302u);         // a1 b1 c1 d1
  col[2] = __builtin_amdgcn_perm(cd_hi, ab_hi, 0x05040100u);         // a2 b2 c2 d2
  col[3] = __builtin_amdgcn_perm(cd_hi, ab_hi, 0x07060302u);         // a3 b3 c3 d3
}

}  // namespace fp8mi
