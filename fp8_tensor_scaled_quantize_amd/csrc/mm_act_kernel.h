// The fused epilogue of fp8_mm_act: bias, pre-activation output, activation
// (optionally gated), residual, then one bf16 rounding or the output
// quantization, on the accumulators of mm_tile (mm_fp8_kernel.h).
//
//   t_ij = acc_ij fl32(sa_i sb_j) + bias_j                 (z_out = bf16(t))
//   y_ij = act(t_ij) + res_ij, or gated y_ij = act(t_i,2j) t_i,2j+1 + res_ij
// in fp32 throughout.  A gated pair is always in one lane.
#pragma once
#include "activation.h"
#include "mm_fp8_kernel.h"
#include "vec_io.h"

namespace fp8mi {

// The accumulators of one 16-row strip, regrouped so that a lane holds
// consecutive columns of its row.  Lane l = 16 g + r of an MFMA tile holds
// columns 4g .. 4g + 3 of row r; tiles are taken in pairs (32 columns), and one
// v_permlane16_swap per value pair exchanges the odd 16-lane rows of the
// first tile's register with the even ones of the second's: lane group g ends
// with columns 8 (g / 2) .. + 7 of tile g & 1.  No LDS and no barrier: each wave
// reads and writes its own rows, 64 contiguous bytes (of bf16) of a row per
// four lanes and instruction.  (Staged through LDS with 8-column stores of
// whole rows, the epilogue held 128 + 128 values live and spilled: 8192 x 6912
// x 1536 without activation 171 us, regrouped 92 us, the plain GEMM 87 us.)
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap16(float& a, float& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
// Columns per lane and pair, pairs per strip (a strip of one tile is taken as
// it is, 4 columns per lane).
constexpr int pair_cols(int tj) { return tj == 1 ? 4 : 8; }
constexpr int strip_pairs(int tj) { return (tj + 1) / 2; }
template <int TJ> __device__ __forceinline__ void lane_columns(const v4f (&acc)[TJ], int c, float (&t)[pair_cols(TJ)]) {
  static_assert(TJ == 1 || TJ % 2 == 0, "whole pairs");
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if constexpr (TJ == 1) {
      t[r] = acc[0][r];
    } else {
      t[r] = acc[2 * c][r];
      t[4 + r] = acc[2 * c + 1][r];
      swap16(t[r], t[4 + r]);
    }
  }
}
template <int TJ> __device__ __forceinline__ int lane_column(int g, int c) {
  return TJ == 1 ? 4 * g : 32 * c + 16 * (g & 1) + 8 * (g >> 1);
}

// W words to element-aligned memory (EB bytes per element), n of the W * 4 / EB
// elements; W = 1, 2, 4 or 8.  STREAM: non-temporal.
template <int W, int EB, bool STREAM = false> __device__ __forceinline__ void store_words(uint8_t* g, const uint32_t (&w)[W], int n) {
  if (n >= W * 4 / EB) {
    if constexpr (W >= 4) {
#pragma unroll
      for (int c = 0; c < W / 4; ++c) {
        const u32x4_byte v = {w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]};
        if constexpr (STREAM) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_byte*>(g) + c);
        else reinterpret_cast<u32x4_byte*>(g)[c] = v;
      }
    } else if constexpr (W == 2) {
      if constexpr (STREAM) __builtin_nontemporal_store(u32x2_byte{w[0], w[1]}, reinterpret_cast<u32x2_byte*>(g));
      else *reinterpret_cast<u32x2_byte*>(g) = u32x2_byte{w[0], w[1]};
    } else {
      typedef uint32_t u32_byte __attribute__((aligned(1)));
      *reinterpret_cast<u32_byte*>(g) = w[0];
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < W * 4 / EB - 1; ++e) {
    if (e < n) {
      if constexpr (EB == 2) reinterpret_cast<uint16_t*>(g)[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
      else g[e] = (uint8_t)(w[e / 4] >> (8 * (e & 3)));
    }
  }
}

// C consecutive 16-bit residual values as stored, n of them inside the matrix.
template <int C> struct Res16 {
  uint32_t w[C / 2];
};
template <int C> __device__ __forceinline__ void load_res16(Res16<C>& o, const MmActArgs& p, int64_t row, int64_t col, int n) {
  const uint16_t* q = static_cast<const uint16_t*>(p.res) + row * p.ld_res + col;
  if (n >= C) {
    if constexpr (C == 8) {
      const u32x4_any v = *reinterpret_cast<const u32x4_any*>(q);
#pragma unroll
      for (int e = 0; e < 4; ++e) o.w[e] = v[e];
    } else if constexpr (C == 4) {
      const u32x2_any v = *reinterpret_cast<const u32x2_any*>(q);
      o.w[0] = v[0];
      o.w[1] = v[1];
    } else {
      typedef uint32_t u32_any __attribute__((aligned(2)));
      o.w[0] = *reinterpret_cast<const u32_any*>(q);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < C / 2; ++e) o.w[e] = 0u;
#pragma unroll
  for (int e = 0; e < C - 1; ++e)
    if (e < n) o.w[e / 2] |= (uint32_t)q[e] << (16 * (e & 1));
}
template <int C> __device__ __forceinline__ void add_res16(float (&y)[C], const Res16<C>& r, bool bf16) {
#pragma unroll
  for (int e = 0; e < C; e += 2) {
    float a, b;
    if (bf16) widen2<kBF16>(r.w[e / 2], a, b);
    else widen2<kF16>(r.w[e / 2], a, b);
    y[e] += a;
    y[e + 1] += b;
  }
}
template <int C> __device__ __forceinline__ void add_res32(float (&y)[C], const MmActArgs& p, int64_t row, int64_t col, int n) {
  const float* q = static_cast<const float*>(p.res) + row * p.ld_res + col;
  typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
  if (C % 4 == 0 && n >= C) {
#pragma unroll
    for (int c = 0; c < C / 4; ++c) {
      const f32x4_any v = reinterpret_cast<const f32x4_any*>(q)[c];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[4 * c + e] += v[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < C; ++e)
      if (e < n) y[e] += q[e];
  }
}

template <int C> __device__ __forceinline__ void pack_bf16(uint32_t (&w)[C / 2], const float (&f)[C]) {
#pragma unroll
  for (int e = 0; e < C; e += 2) {
    const f32x2 v = {f[e], f[e + 1]};
    w[e / 2] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
  }
}

// Everything of one wave's strips for one activation.  Returns the largest |y|
// inside the matrix, NaN left out (0 for a bf16 output).
template <int ACT, int OUT, bool GATED, int TI, int TJ>
__device__ __forceinline__ float act_strips(const MmActArgs& p, const v4f (&acc)[TI][TJ], const float* bias_s,
                                            const float* col_s, int64_t row0, int64_t col0, int rows_in, int cols_in,
                                            float s_c) {
  constexpr int G = GATED ? 2 : 1;  // t columns per output column
  constexpr int C = pair_cols(TJ), CO = C / G, NP = strip_pairs(TJ);
  // packed words of a lane's outputs per pair; two pairs' narrow outputs are
  // joined by v_permlane32_swap, so that a lane stores 16 consecutive t columns
  constexpr int WO = OUT < 0 ? CO / 2 : (CO + 3) / 4, EB = OUT < 0 ? 2 : 1;
  constexpr bool JOIN = NP == 2 && WO < 4;
  // The big tiles' 16-byte stores of pre-activations and bf16 outputs bypass
  // the L2's keeping (their sizes pass it by far, the operand panels stay):
  // 8192 x 6912 x 1536 gelu to fp8 with pre-activations 140 -> 121 us over three
  // sets of buffers in turn, bf16 output without them 107 -> 100.  Narrower
  // stores fill a line in several steps and lose by it (98 -> 105).
  constexpr bool STREAM = TI * TJ >= 24;
  const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
  const auto clip = [](int v, int most) { return v < 0 ? 0 : (v < most ? v : most); };
  const float sa = p.a_scale_inv && !p.a_rows ? *p.a_scale_inv : 1.0f;
  // Three pairs (the 128 x 192 tile): bias and scales are read from LDS strip
  // by strip, the registers would not suffice.
  constexpr bool LEAN = NP > 2;
  int n[NP];  // the lane's columns inside the matrix
  int64_t col[NP];
  float bias[NP][C], cs[NP][C];
  auto load_cols = [&]() {
#pragma unroll
    for (int c = 0; c < NP; ++c) {
      const int at = lane_column<TJ>(g, c);
#pragma unroll
      for (int e = 0; e < C; e += 4) {
        const float4 b4 = *reinterpret_cast<const float4*>(bias_s + at + e);
        const float4 c4 = *reinterpret_cast<const float4*>(col_s + at + e);
        bias[c][e] = b4.x; bias[c][e + 1] = b4.y; bias[c][e + 2] = b4.z; bias[c][e + 3] = b4.w;
        // fl32(sa sb); row scales of A are multiplied in strip by strip
        cs[c][e] = sa * c4.x; cs[c][e + 1] = sa * c4.y; cs[c][e + 2] = sa * c4.z; cs[c][e + 3] = sa * c4.w;
      }
    }
  };
#pragma unroll
  for (int c = 0; c < NP; ++c) {
    const int at = lane_column<TJ>(g, c);
    n[c] = clip(cols_in - at, C);
    col[c] = col0 + at;
  }
  if constexpr (!LEAN) load_cols();
  const bool sreg = OUT >= 0 && scale_regular(s_c);
  float amax = 0.0f;
  // A 16-bit residual's next strips are in flight while one is finished: as many
  // as the registers that the epilogue leaves free hold.  Over three sets of
  // buffers in turn, without a residual -> with it (us): 8192 x 6912 x 1536
  // 91 -> 130, 4096 x 3584 x 4096 48 -> 52, 8192 x 1536 x 6912 78 -> 92 (one
  // strip ahead 97), 8192^3 383 -> 421; brought into the L2 during the last K
  // steps by waves that load nothing else 136, 55, 91 and 432.
  constexpr int AHEAD = (LEAN ? 2 : 4) - (OUT < 0 ? 0 : 1);
  const bool res16 = p.res && p.res_dt != kF32;
  Res16<CO> raw[AHEAD][NP];
  auto fetch = [&](Res16<CO> (&to)[NP], int i) {
#pragma unroll
    for (int c = 0; c < NP; ++c)
      load_res16<CO>(to[c], p, row0 + 16 * i + r16, col[c] / G, 16 * i + r16 < rows_in ? n[c] / G : 0);
  };
  if (res16) {
#pragma unroll
    for (int i = 0; i < (AHEAD < TI ? AHEAD : TI); ++i) fetch(raw[i], i);
  }
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int lr = 16 * i + r16;
    const bool in = lr < rows_in;
    const int64_t row = row0 + lr;
    const float ra = p.a_rows ? p.a_scale_inv[in ? row : row0] : 1.0f;
    // step by step over the whole strip: few, long basic blocks, so that the
    // chains of exp2 and reciprocal of different values overlap
    float t[NP][C], y[NP][CO];
    if constexpr (LEAN) load_cols();
#pragma unroll
    for (int c = 0; c < NP; ++c) lane_columns<TJ>(acc[i], c, t[c]);
    if (p.a_rows) {
#pragma unroll
      for (int c = 0; c < NP; ++c)
#pragma unroll
        for (int e = 0; e < C; ++e) t[c][e] = fmaf(t[c][e], ra * cs[c][e], bias[c][e]);
    } else {
#pragma unroll
      for (int c = 0; c < NP; ++c)
#pragma unroll
        for (int e = 0; e < C; ++e) t[c][e] = fmaf(t[c][e], cs[c][e], bias[c][e]);
    }
    if (p.z && in) {
#pragma unroll
      for (int c = 0; c < NP; ++c) {
        uint32_t w[C / 2];
        pack_bf16<C>(w, t[c]);
        store_words<C / 2, 2, STREAM>(reinterpret_cast<uint8_t*>(p.z + row * p.ld_z + col[c]), w, n[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < NP; ++c)
#pragma unroll
      for (int e = 0; e < CO; ++e)
        y[c][e] = GATED ? act_value<ACT>(t[c][G * e]) * t[c][G * e + G - 1] : act_value<ACT>(t[c][e]);
    if (res16) {
#pragma unroll
      for (int c = 0; c < NP; ++c) add_res16<CO>(y[c], raw[i % AHEAD][c], p.res_dt == kBF16);
      if (i + AHEAD < TI) fetch(raw[i % AHEAD], i + AHEAD);
    } else if (p.res) {
#pragma unroll
      for (int c = 0; c < NP; ++c) add_res32<CO>(y[c], p, row, col[c] / G, in ? n[c] / G : 0);
    }
    uint32_t w[NP][WO];
    if constexpr (OUT < 0) {
#pragma unroll
      for (int c = 0; c < NP; ++c) pack_bf16<CO>(w[c], y[c]);
    } else {
      // columns past the edge hold y = 0 (zero weights, no bias, no residual);
      // rows past it hold the bias's values: left out lane by lane
      float m = 0.0f;  // a NaN kept: it picks the exact encoder
#pragma unroll
      for (int c = 0; c < NP; ++c)
#pragma unroll
        for (int e = 0; e < CO; ++e) m = __builtin_elementwise_maximum(m, fabsf(y[c][e]));
      const bool nan = m != m;
      if (nan) {
        m = 0.0f;
#pragma unroll
        for (int c = 0; c < NP; ++c)
#pragma unroll
          for (int e = 0; e < CO; ++e)
            if (e < n[c] / G) m = fmaxf(m, fabsf(y[c][e]));
      }
      if (!in) m = 0.0f;
      amax = fmaxf(amax, m);
      auto encode = [&](auto enc) {
#pragma unroll
        for (int c = 0; c < NP; ++c)
#pragma unroll
          for (int e = 0; e < CO; e += 4) {
            const float y2 = CO > 2 ? y[c][(e + 2) % CO] : 0.0f, y3 = CO > 2 ? y[c][(e + 3) % CO] : 0.0f;
            w[c][e / 4] = enc(y[c][e] * s_c, y[c][e + 1] * s_c, y2 * s_c, y3 * s_c);
          }
      };
      if (!__any(nan) && sreg) {
        // no clamp where fl32(max |y| |s|), the largest of them, is in range
        if (!__any(m * fabsf(s_c) > FmtTraits<OUT>::kMax))
          encode([](float a, float b, float c, float d) { return cvt4_inrange<OUT>(a, b, c, d); });
        else
          encode([](float a, float b, float c, float d) { return cvt4<OUT>(a, b, c, d); });
      } else {
        encode([](float a, float b, float c, float d) { return enc4_exact<OUT>(a, b, c, d); });
      }
    }
    const int64_t at = row * p.ldc;
    if constexpr (JOIN) {
      uint32_t o[2 * WO];
#pragma unroll
      for (int k = 0; k < WO; ++k) {
        swap32(w[0][k], w[1][k]);
        o[k] = w[0][k];
        o[WO + k] = w[1][k];
      }
      if (in)
        store_words<2 * WO, EB>(static_cast<uint8_t*>(p.c) + (at + (col0 + 16 * g) / G) * EB, o,
                                clip(cols_in - 16 * g, 16) / G);
    } else if (in) {
#pragma unroll
      for (int c = 0; c < NP; ++c)  // two codes alone (gated, one tile a wave) fill half their word
        store_words<WO, EB, STREAM && OUT < 0 && WO == 4>(static_cast<uint8_t*>(p.c) + (at + col[c] / G) * EB, w[c], n[c] / G);
    }
    __builtin_amdgcn_sched_barrier(0);  // one strip's registers at a time
  }
  return amax;
}

// One wave's strips, the activation chosen once.
template <int OUT, bool GATED, int TI, int TJ>
__device__ __forceinline__ float act_strips_any(const MmActArgs& p, const v4f (&acc)[TI][TJ], const float* bias_s,
                                                const float* col_s, int64_t row0, int64_t col0, int rows_in,
                                                int cols_in, float s_c) {
  switch (p.act) {
    case kActRelu: return act_strips<kActRelu, OUT, GATED>(p, acc, bias_s, col_s, row0, col0, rows_in, cols_in, s_c);
    case kActGelu: return act_strips<kActGelu, OUT, GATED>(p, acc, bias_s, col_s, row0, col0, rows_in, cols_in, s_c);
    case kActSilu: return act_strips<kActSilu, OUT, GATED>(p, acc, bias_s, col_s, row0, col0, rows_in, cols_in, s_c);
    default: return act_strips<kActNone, OUT, GATED>(p, acc, bias_s, col_s, row0, col0, rows_in, cols_in, s_c);
  }
}

// The output scale; read before this workgroup's amax can be folded.
template <int OUT> __device__ __forceinline__ float act_out_scale(const MmActArgs& p) {
  return OUT < 0 ? 1.0f : (p.c_ring ? __uint_as_float(p.c_ring[p.c_H]) : *p.c_scale);
}

// A workgroup's share of the output's amax and scale bookkeeping; every thread
// calls it.  red: NT / 64 + 1 words of LDS.
template <int OUT, int NT>
__device__ __forceinline__ void act_finish(const MmActArgs& p, float amax, float s_c, float* red) {
  if constexpr (OUT >= 0) {
    if (p.c_ring || p.c_amax_out) {
      const float bmax = block_max<NT>(amax, red);
      if (p.c_ring) {
        ring_block_done<OUT>(p.c_ring, p.c_H, bmax, s_c, p.c_scale_inv_out, p.c_amax_out,
                             reinterpret_cast<uint32_t*>(red + NT / 64));
        return;
      }
      if (threadIdx.x == 0) publish_max(reinterpret_cast<uint32_t*>(p.c_amax_out), bmax);
    }
    if (threadIdx.x == 0 && p.c_scale_inv_out && blockIdx.x + blockIdx.y == 0) *p.c_scale_inv_out = 1.0f / s_c;
  }
}

template <int BM, int BN, int WAVES_M, int WAVES_N, int DEEP, int OUT, int TI, int TJ, class P>
__device__ __forceinline__ void act_epilogue(const P& p, v4f (&acc)[TI][TJ], uint8_t* pool, const int64_t m0,
                                             const int64_t n0) {
  constexpr bool GATED = P::kGated;
  constexpr int NWAVES = WAVES_M * WAVES_N, NT = 64 * NWAVES;
  constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
  using Lds = TileLds<BM, BN, NWAVES, DEEP>;
  const int tid = threadIdx.x;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wid / WAVES_N, wn = wid % WAVES_N;
  const float* const bias_s = reinterpret_cast<const float*>(pool + Lds::kActBias) + wn * WN;
  const float* const col_s = reinterpret_cast<const float*>(pool + Lds::kActCol) + wn * WN;
  const int64_t row0 = m0 + wm * WM, col0 = n0 + wn * WN;
  const int64_t rl = p.M - row0, cl = p.N - col0;
  const int rows_in = rl < WM ? (int)rl : WM, cols_in = cl < WN ? (int)cl : WN;  // negative: none
  const float s_c = act_out_scale<OUT>(p);
  float amax = 0.0f;
  if (rows_in > 0)
    amax = act_strips_any<OUT, GATED>(p, acc, bias_s, col_s, row0, col0, rows_in, cols_in, s_c);
  act_finish<OUT, NT>(p, amax, s_c, reinterpret_cast<float*>(pool + Lds::kActRed));
}

// Gating fixed at compile time (it decides the output tile's shape).
template <bool GATED> struct MmActTyped : MmActArgs {
  static constexpr bool kGated = GATED;
};

template <int BM, int BN, int WM_, int WN_, int MINB, int OUT, class P, bool PREC = false, int DEEP = 0>
static hipError_t launch_act_tile(const P& p0, hipStream_t st) {
  const int64_t tiles_m = (p0.M + BM - 1) / BM, tiles_n = (p0.N + BN - 1) / BN;
  P p = p0;
  p.early_loads = tiles_m * tiles_n > (int64_t)device_cu_count();  // more than one round
  hipLaunchKernelGGL((mm_fp8_dma<kE4M3, kE4M3, BM, BN, WM_, WN_, MINB, OUT, 0, PREC, DEEP, P>),
                     dim3((unsigned)(tiles_m * tiles_n)), dim3(64 * WM_ * WN_), 0, st, p, tiles_m, tiles_n, BM == 128 ? 8 : 4);
  return hipGetLastError();
}

// ===========================================================================
// Few rows (serving): bound by reading the weights once.  A workgroup takes 16
// weight rows and 16 TI rows of A, its NW waves every NW-th K step
// of 128; fragments come straight from global memory into registers, U steps in
// flight per wave, no LDS and no barrier before the end.  Lane group g of a
// fragment takes k = 16 g .. + 15 and 64 + 16 g .. + 15 of the step instead of
// 32 g .. + 31, A and B alike: the sums are over the same products, and each
// load instruction reads 64 contiguous bytes of a row.  The waves'
// sums meet in LDS, added in wave order, and the epilogue is that of one
// 16-column strip per 16 rows.  (32 x 1536 x 6912 with residual, graph replay:
// 16.7 us in 64 x 32 tiles, whose rows are half empty and whose 48 workgroups
// leave most CUs idle.)
// ===========================================================================
template <int OUT, bool GATED, int TI, int NW>
__global__ void __launch_bounds__(64 * NW) mm_act_rows(MmActArgs p) {
  constexpr int NT = 64 * NW, U = 4;
  static_assert(NW >= TI, "one wave per 16 rows finishes them");
  __shared__ float4 part[NW][TI][64];
  __shared__ float bias_s[16], col_s[16];
  __shared__ float red[NW + 1];
  const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * 16 * TI;
  // raw buffers: rows past an edge and chunks past K read as zero
  const int ext_a = (int)p.a_extent_from(0), ext_b = (int)p.b_extent_from(n0);
  const auto rsa = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p.a), 0, ext_a, 0x00020000);
  const auto rsb = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p.b + n0 * p.ldb), 0, ext_b, 0x00020000);
  const int K = (int)p.K, steps = (K + kBK - 1) / kBK;
  const uint32_t ob = (uint32_t)r16 * (uint32_t)p.ldb + 16 * g;
  uint32_t oa[TI];  // a row past M - 1 starts at or beyond the extent
#pragma unroll
  for (int i = 0; i < TI; ++i) oa[i] = m0 + 16 * i + r16 < p.M ? (uint32_t)(m0 + 16 * i + r16) * (uint32_t)p.lda + 16 * g : (uint32_t)ext_a;
  const bool b_in = n0 + r16 < p.N;
  auto frag = [&](__amdgpu_buffer_rsrc_t rs, uint32_t off, int ext, int kt) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const int k = kt * kBK + 16 * g;
    const u32x4 lo = __builtin_amdgcn_raw_buffer_load_b128(rs, k < K ? off + kt * kBK : ext, 0, 0);
    const u32x4 hi = __builtin_amdgcn_raw_buffer_load_b128(rs, k + 64 < K ? off + kt * kBK + 64 : ext, 0, 0);
    v8i r;
    r[0] = (int)lo[0]; r[1] = (int)lo[1]; r[2] = (int)lo[2]; r[3] = (int)lo[3];
    r[4] = (int)hi[0]; r[5] = (int)hi[1]; r[6] = (int)hi[2]; r[7] = (int)hi[3];
    return r;
  };
  v4f acc[TI];
#pragma unroll
  for (int i = 0; i < TI; ++i) acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  v8i bf[U], af[U][TI];
  auto load = [&](int kt) {  // a step past the end reads nothing (k >= K)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      bf[u] = frag(rsb, b_in ? ob : (uint32_t)ext_b, ext_b, kt + u * NW);
#pragma unroll
      for (int i = 0; i < TI; ++i) af[u][i] = frag(rsa, oa[i], ext_a, kt + u * NW);
    }
    __builtin_amdgcn_sched_barrier(0);  // all in flight before anything waits
  };
  // the residual's lines are on their way to the L2 before the weights' loads:
  // otherwise the epilogue waits for HBM once more
  uint32_t warm = 0u;
  if (p.res && wid < TI && g == 0 && m0 + 16 * wid + r16 < p.M)
    warm = static_cast<const uint8_t*>(p.res)[((m0 + 16 * wid + r16) * p.ld_res + n0 / (GATED ? 2 : 1)) *
                                              (p.res_dt == kF32 ? 4 : 2)];
  load(wid);
  // bias and column scales: read behind the first steps' loads, parked after the K loop
  const int64_t pc = n0 + (lane & 15);
  const bool col_in = tid < 16 && pc < p.N;
  const uint32_t bias_bits = p.bias && col_in ? load_bias_bits(p, pc) : 0u;
  float col_scale = 1.0f;
  if (p.b_scale_inv) col_scale = p.b_scale_inv[p.b_rows ? (pc < p.N ? pc : n0) : 0];
  for (int kt = wid; kt < steps;) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < TI; ++i) acc[i] = mfma_nt<kE4M3, kE4M3>(bf[u], af[u][i], acc[i]);
    kt += U * NW;
    if (kt < steps) load(kt);
  }
#pragma unroll
  for (int i = 0; i < TI; ++i) part[wid][i][lane] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
  if (tid < 16) {
    bias_s[tid] = col_in && p.bias ? decode_bias(p, bias_bits, 1.0f) : 0.0f;
    col_s[tid] = col_scale;
  }
  const float s_c = act_out_scale<OUT>(p);
  asm volatile("" ::"v"(warm));
  __syncthreads();
  float amax = 0.0f;
  const int64_t row0 = m0 + 16 * wid;
  if (wid < TI && row0 < p.M) {
    v4f sum[1][1];
    const float4 f = part[0][wid][lane];
    sum[0][0] = v4f{f.x, f.y, f.z, f.w};
#pragma unroll
    for (int w = 1; w < NW; ++w) {
      const float4 q = part[w][wid][lane];
      sum[0][0][0] += q.x; sum[0][0][1] += q.y; sum[0][0][2] += q.z; sum[0][0][3] += q.w;
    }
    const int rows_in = p.M - row0 < 16 ? (int)(p.M - row0) : 16;
    const int cols_in = p.N - n0 < 16 ? (int)(p.N - n0) : 16;
    amax = act_strips_any<OUT, GATED>(p, sum, bias_s, col_s, row0, n0, rows_in, cols_in, s_c);
  }
  act_finish<OUT, NT>(p, amax, s_c, red);
}

// Blocks of 16 rows by 16 columns, a workgroup each, while every one has a CU of
// its own: each then reads 16 rows of either operand.  Graph replay over twelve
// sets of buffers, 32-row blocks or tiles -> this (us): 24 x 1536 x 6912 11.8 ->
// 9.8, 32 x 1536 x 6912 12.9 -> 9.8, 48 x 1024 x 6912 16.3 -> 9.8, 64 x 1024 x
// 4096 11.7 -> 8.0, 64 x 512 x 512 5.6 -> 3.7, 40 x 512 x 8192 18.4 -> 10.4,
// 256 x 256 x 4096 11.7 -> 7.9, 4096 x 16 x 512 5.4 -> 3.7.
// With two workgroups per CU the others win: 32 x 3584 x 2048 7.0 against 8.1,
// 48 x 1536 x 6912 16.4 against 16.7.
static inline bool act_row_blocks(const MmActArgs& p) {
  return (p.N + 15) / 16 * ((p.M + 15) / 16) <= device_cu_count();
}
template <int OUT, bool GATED, int TI> static hipError_t launch_act_rows_ti(const MmActArgs& p, hipStream_t st) {
  const dim3 grid((unsigned)((p.N + 15) / 16), (unsigned)((p.M + 16 * TI - 1) / (16 * TI)));
  const int64_t wgs = (int64_t)grid.x * grid.y;
  // waves per workgroup: enough of them over the chip, no more than K steps
  const int64_t steps = (p.K + kBK - 1) / kBK;
  if (wgs >= 768 || steps <= 8) hipLaunchKernelGGL((mm_act_rows<OUT, GATED, TI, 4>), grid, dim3(256), 0, st, p);
  else if (wgs >= 384 || steps <= 16) hipLaunchKernelGGL((mm_act_rows<OUT, GATED, TI, 8>), grid, dim3(512), 0, st, p);
  else hipLaunchKernelGGL((mm_act_rows<OUT, GATED, TI, 16>), grid, dim3(1024), 0, st, p);
  return hipGetLastError();
}
template <int OUT, bool GATED> static hipError_t launch_act_rows(const MmActArgs& p, hipStream_t st) {
  return p.M <= 16 || act_row_blocks(p) ? launch_act_rows_ti<OUT, GATED, 1>(p, st) : launch_act_rows_ti<OUT, GATED, 2>(p, st);
}
// Every column of workgroups reads all of A, which the tiles share through LDS: taken for
// at most 8 rows, for 16 while the weights are small, for 32 while there is
// at most one workgroup per CU, beyond that in blocks (act_row_blocks).  Graph replay, tiles -> this (us): 1 x 13824 x
// 1536 9.6 -> 7.5, 8 x 4096 x 4096 11.4 -> 7.7, 16 x 1536 x 6912 16.0 -> 9.6,
// 32 x 4096 x 4096 11.4 -> 10.8; and where the
// tiles stay: 16 x 28672 x 8192 50 against 59, 32 x 8192 x 2048 8.3 against
// 10.6, 64 x 1536 x 6912 16.2 against 19.6.
static inline bool act_few_rows(const MmActArgs& p) {
  if (p.M <= 8) return true;
  if (p.M <= 16) return p.N * p.K <= (int64_t)32 << 20;
  return (p.M <= 32 && p.N <= 16 * (int64_t)device_cu_count()) || act_row_blocks(p);
}

// The plain GEMM's tile (pick_tile) for small problems; for large ones 256 x
// 256 (0), its mixed grid (7), or 128 x 192 tiles of four waves (4), two
// workgroups per CU, so that one's epilogue passes under the other's K loop.
// Costs are in 1/256 of a round of 256 x 256 tiles: a round of two 128 x 192
// tiles per CU takes 202 (a last round at most half full 0.6 of it, its
// workgroups having a CU each), 27% more where K is long and the smaller
// tile's L2 traffic counts.  The mixed grid's band costs 150 in place of a
// last round, but not with plain fp8 outputs, where it measured slower than
// its count.  Both sides measured, over three sets of buffers in turn (us,
// others -> 128 x 192): 8192 x 6912 x 1536 gelu to fp8 115 -> 102, with
// pre-activations 120 -> 111; 6144 x 6144 x 1536 gelu 72 -> 68, to fp8 83 -> 67;
// 4096 x 2560 x 2048 gelu to fp8 34 -> 29; 8192 x 1536 x 1536 residual 31 -> 28;
// and where the rule keeps the others: 8192 x 6912 x 1536 with residual 137
// against 157, 4096 x 3584 x 4096 gelu 52 against 70, 8192 x 13824 x 1536 with
// pre-activations 237 against 268, 8192^3 400 against 494.
static inline int pick_act_tile(const MmActArgs& p, bool plain_q8, int ncu) {
  static const int forced = env_int_in("FP8MI_MM_TILE", 0, 8, -1);
  if (forced >= 0) return forced;
  int base = pick_tile(p, ncu);
  if (base != 0 && base != 3 && base != 7) return base;
  base = mixed_band_cols(p, ncu) > 0 ? 7 : 0;
  const int64_t r256 = (((p.M + 255) / 256) * ((p.N + 255) / 256) + ncu - 1) / ncu;
  const int64_t cost = base == 7 && !plain_q8 ? (r256 - 1) * 256 + 150 : r256 * 256;
  const int64_t t = ((p.M + 127) / 128) * ((p.N + 191) / 192), full = t / (2 * ncu), rest = t % (2 * ncu);
  int64_t own = full * 202 + (rest == 0 ? 0 : (rest <= ncu ? 121 : 202));
  if (p.K > 2048) own += own * 27 / 100;
  return own < cost ? 4 : base;
}

template <int OUT, bool GATED> static hipError_t launch_act_family(const MmActArgs& args, hipStream_t st) {
  using P = MmActTyped<GATED>;
  if (!mm_precise(args) && act_few_rows(args)) return launch_act_rows<OUT, GATED>(args, st);
  P p;
  static_cast<MmActArgs&>(p) = args;
  const int tile = mm_precise(p) ? pick_tile(p, device_cu_count())
                                 : pick_act_tile(p, OUT >= 0 && !GATED, device_cu_count());
  if (mm_precise(p)) {
    switch (tile) {
      case 5: return launch_act_tile<64, 64, 1, 4, 2, OUT, P, true>(p, st);
      case 2: return launch_act_tile<64, 128, 1, 4, 2, OUT, P, true>(p, st);
      default: return launch_act_tile<128, 128, 2, 2, 2, OUT, P, true>(p, st);
    }
  }
  switch (tile) {
    case 0:
    case 3: return launch_act_tile<256, 256, 2, 4, 1, OUT, P>(p, st);
    case 1: return launch_act_tile<128, 128, 2, 2, 2, OUT, P>(p, st);
    case 4: return launch_act_tile<128, 192, 2, 2, 2, OUT, P>(p, st);
    case 5: return launch_act_tile<64, 64, 1, 4, 2, OUT, P>(p, st);
    case 6: return launch_act_tile<64, 64, 1, 4, 1, OUT, P, false, 8>(p, st);
    case 8: return launch_act_tile<64, 32, 4, 1, 1, OUT, P, false, 8>(p, st);
    case 7: {
      const int64_t cb = mixed_band_cols(p, device_cu_count());
      if (cb == 0) return launch_act_tile<256, 256, 2, 4, 1, OUT, P>(p, st);
      p.early_loads = 1;  // at least two rounds
      const int64_t tiles_m = (p.M + 255) / 256, tiles_n = (p.N + 255) / 256 - cb, band_m = (p.M + 127) / 128;
      hipLaunchKernelGGL((mm_fp8_mixed<kE4M3, kE4M3, OUT, 0, P>), dim3((unsigned)(tiles_m * tiles_n + band_m * cb)),
                         dim3(512), 0, st, p, tiles_m, tiles_n, band_m, cb, tiles_n * 256, 4);
      return hipGetLastError();
    }
    default: return launch_act_tile<64, 128, 1, 4, 2, OUT, P>(p, st);
  }
}

}  // namespace fp8mi
