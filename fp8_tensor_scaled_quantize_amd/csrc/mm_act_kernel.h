// The fused epilogue of fp8_mm_act: bias, pre-activation output, activation
// (optionally gated), residual, then one bf16 rounding or the output
// quantization, on the accumulators of mm_tile (mm_fp8_kernel.h).
//
//   t_ij = acc_ij fl32(sa_i sb_j) + bias_j                 (z_out = bf16(t))
//   y_ij = act(t_ij) + res_ij, or gated y_ij = act(t_i,2j) t_i,2j+1 + res_ij
// in fp32 throughout.  A lane holds 4 consecutive columns of a row, so a gated
// pair is always in one lane.
#pragma once
#include "activation.h"
#include "mm_fp8_kernel.h"
#include "vec_io.h"

namespace fp8mi {

// Rows of a tile staged in LDS (PITCH bytes apart, ROWB bytes each) to global
// memory at dst, ld bytes apart: 16 bytes per lane and step, whole rows by
// consecutive lanes; rows_in x cols_in_b bytes of the tile lie inside the
// matrix, EB bytes per element.
template <int ROWB, int PITCH, int EB, int NT>
__device__ __forceinline__ void store_rows(const uint8_t* S, uint8_t* dst, int64_t ld, int rows_in, int cols_in_b,
                                           int tid) {
  constexpr int PPR = ROWB / 16;
  static_assert(ROWB % 16 == 0 && PITCH % 16 == 0, "16-byte pieces");
  for (int q = tid; q < rows_in * PPR; q += NT) {
    const int r = q / PPR, c = 16 * (q % PPR);
    if (c >= cols_in_b) continue;
    const uint4 v = *reinterpret_cast<const uint4*>(S + r * PITCH + c);
    uint8_t* g = dst + r * ld + c;
    if (c + 16 <= cols_in_b) {
      if constexpr (EB == 2) *reinterpret_cast<u32x4_any*>(g) = u32x4_any{v.x, v.y, v.z, v.w};
      else *reinterpret_cast<u32x4_byte*>(g) = u32x4_byte{v.x, v.y, v.z, v.w};
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 16 / EB - 1; ++e) {
        if (c + (e + 1) * EB > cols_in_b) break;
        if constexpr (EB == 2) reinterpret_cast<uint16_t*>(g)[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
        else g[e] = (uint8_t)(w[e / 4] >> (8 * (e & 3)));
      }
    }
  }
}

// W consecutive residual values of one row starting at column c, n of them
// inside the matrix.
template <int W> __device__ __forceinline__ void load_res(float (&f)[W], const MmActArgs& p, int64_t row, int64_t c, int n) {
#pragma unroll
  for (int e = 0; e < W; ++e) f[e] = 0.0f;
  const int64_t at = row * p.ld_res + c;
  if (p.res_dt == kF32) {
    const float* q = static_cast<const float*>(p.res) + at;
#pragma unroll
    for (int e = 0; e < W; ++e)
      if (e < n) f[e] = q[e];
    return;
  }
  uint32_t w[W / 2];
  const uint16_t* q = static_cast<const uint16_t*>(p.res) + at;
  if (n >= W) {
    if constexpr (W == 4) {
      const u32x2_any v = *reinterpret_cast<const u32x2_any*>(q);
      w[0] = v[0];
      w[1] = v[1];
    } else {
      typedef uint32_t u32_any __attribute__((aligned(2)));
      w[0] = *reinterpret_cast<const u32_any*>(q);
    }
  } else {
#pragma unroll
    for (int e = 0; e < W / 2; ++e) w[e] = 0u;
#pragma unroll
    for (int e = 0; e < W; ++e)
      if (e < n) w[e / 2] |= (uint32_t)q[e] << (16 * (e & 1));
  }
#pragma unroll
  for (int e = 0; e < W / 2; ++e) {
    if (p.res_dt == kBF16) widen2<kBF16>(w[e], f[2 * e], f[2 * e + 1]);
    else widen2<kF16>(w[e], f[2 * e], f[2 * e + 1]);
  }
}

// y in place of t: acc[..][0 .. W - 1] hold the lane's W output columns.
template <int ACT, bool GATED, int TI, int TJ> __device__ __forceinline__ void apply_act(v4f (&acc)[TI][TJ]) {
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      if constexpr (GATED) {
        acc[i][j][0] = act_value<ACT>(acc[i][j][0]) * acc[i][j][1];
        acc[i][j][1] = act_value<ACT>(acc[i][j][2]) * acc[i][j][3];
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = act_value<ACT>(acc[i][j][r]);
      }
    }
}

template <int BM, int BN, int WAVES_M, int WAVES_N, int DEEP, int OUT, int TI, int TJ, class P>
__device__ __forceinline__ void act_epilogue(const P& p, v4f (&acc)[TI][TJ], uint8_t* pool, const int64_t m0,
                                             const int64_t n0) {
  constexpr bool GATED = P::kGated;
  constexpr int NWAVES = WAVES_M * WAVES_N, NT = 64 * NWAVES;
  constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
  constexpr int G = GATED ? 2 : 1;     // t columns per output column
  constexpr int W = 4 / G, BNO = BN / G;  // output columns per lane and MFMA tile / per tile
  using Lds = TileLds<BM, BN, NWAVES, DEEP>;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wid / WAVES_N, wn = wid % WAVES_N;
  const int r16 = lane & 15, ng = lane >> 4;
  const int64_t No = p.N / G, o0 = n0 / G;
  const int rows_in = p.M - m0 < BM ? (int)(p.M - m0) : BM;  // the tile's part inside the matrices
  const int cols_in = p.N - n0 < BN ? (int)(p.N - n0) : BN;
  const int outs_in = cols_in / G;
  const float* const bias_s = reinterpret_cast<const float*>(pool + Lds::kBias);
  const float* const col_s = reinterpret_cast<const float*>(pool + Lds::kCol);

  // t, in place
  const float sa = p.a_scale_inv && !p.a_rows ? *p.a_scale_inv : 1.0f;
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int lm = wm * WM + 16 * i + r16;
    float ra = sa;
    if (p.a_rows) ra = p.a_scale_inv[m0 + (lm < rows_in ? lm : 0)];
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const float4 b4 = *reinterpret_cast<const float4*>(&bias_s[wn * WN + 16 * j + 4 * ng]);
      const float4 c4 = *reinterpret_cast<const float4*>(&col_s[wn * WN + 16 * j + 4 * ng]);
      acc[i][j][0] = fmaf(acc[i][j][0], ra * c4.x, b4.x);
      acc[i][j][1] = fmaf(acc[i][j][1], ra * c4.y, b4.y);
      acc[i][j][2] = fmaf(acc[i][j][2], ra * c4.z, b4.z);
      acc[i][j][3] = fmaf(acc[i][j][3], ra * c4.w, b4.w);
    }
  }
  if (p.z) {
    constexpr int PITCH = 2 * (BN + 8);
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        *reinterpret_cast<uint2*>(pool + (wm * WM + 16 * i + r16) * PITCH + 2 * (wn * WN + 16 * j + 4 * ng)) =
            bf16x4_rne(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
    __syncthreads();
    store_rows<2 * BN, PITCH, 2, NT>(pool, reinterpret_cast<uint8_t*>(p.z + m0 * p.ld_z + n0), 2 * p.ld_z, rows_in,
                                     2 * cols_in, tid);
    __syncthreads();
  }
  switch (p.act) {
    case kActRelu: apply_act<kActRelu, GATED>(acc); break;
    case kActGelu: apply_act<kActGelu, GATED>(acc); break;
    case kActSilu: apply_act<kActSilu, GATED>(acc); break;
    default:
      if constexpr (GATED) apply_act<kActNone, true>(acc);
      break;
  }
  if (p.res) {
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int lm = wm * WM + 16 * i + r16;
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const int lo = (wn * WN + 16 * j + 4 * ng) / G;
        float f[W];
        load_res<W>(f, p, m0 + lm, o0 + lo, lm < rows_in ? outs_in - lo : 0);
#pragma unroll
        for (int r = 0; r < W; ++r) acc[i][j][r] += f[r];
      }
    }
  }
  if constexpr (OUT < 0) {
    constexpr int PITCH = 2 * (BNO + 8);
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        uint8_t* q = pool + (wm * WM + 16 * i + r16) * PITCH + 2 * ((wn * WN + 16 * j + 4 * ng) / G);
        const uint2 v = bf16x4_rne(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
        if constexpr (GATED) *reinterpret_cast<uint32_t*>(q) = v.x;
        else *reinterpret_cast<uint2*>(q) = v;
      }
    __syncthreads();
    uint16_t* C = static_cast<uint16_t*>(p.c) + m0 * p.ldc + o0;
    store_rows<2 * BNO, PITCH, 2, NT>(pool, reinterpret_cast<uint8_t*>(C), 2 * p.ldc, rows_in, 2 * outs_in, tid);
    return;
  } else {
    // quantized like an fp32 tensor; the workgroup's amax is published before
    // any code is stored (see mm_tile's quantizing epilogue)
    constexpr int PITCH = BNO + 16;
    float* const red = reinterpret_cast<float*>(pool + Lds::kRed);
    const float s_c = p.c_ring ? __uint_as_float(p.c_ring[p.c_H]) : *p.c_scale;
    auto tile_max = [&](auto maxop) {
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        const bool row_in = wm * WM + 16 * i + r16 < rows_in;
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
          const int lo = (wn * WN + 16 * j + 4 * ng) / G;
#pragma unroll
          for (int r = 0; r < W; ++r)
            if (row_in && lo + r < outs_in) m = maxop(m, fabsf(acc[i][j][r]));
        }
      }
      return m;
    };
    float amax = tile_max([](float a, float b) { return __builtin_elementwise_maximum(a, b); });
    const bool fast = !__any(amax != amax) && scale_regular(s_c);
    if (!fast) amax = tile_max([](float a, float b) { return fmaxf(a, b); });
    uint32_t pub = __builtin_nondeterministic_value(0u);  // read by thread 0 only
    if (p.c_ring) {
      const float bmax = block_max<NT>(amax, red);
      if (tid == 0) pub = ring_publish(p.c_ring, p.c_H, bmax);
    }
    auto encode = [&](auto enc) {
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
          const v4f y = acc[i][j];
          uint8_t* q = pool + (wm * WM + 16 * i + r16) * PITCH + (wn * WN + 16 * j + 4 * ng) / G;
          if constexpr (GATED) *reinterpret_cast<uint16_t*>(q) = (uint16_t)enc(y[0] * s_c, y[1] * s_c, 0.0f, 0.0f);
          else *reinterpret_cast<uint32_t*>(q) = enc(y[0] * s_c, y[1] * s_c, y[2] * s_c, y[3] * s_c);
        }
    };
    if (fast) encode([](float a, float b, float c, float d) { return cvt4<OUT>(a, b, c, d); });
    else encode([](float a, float b, float c, float d) { return enc4_exact<OUT>(a, b, c, d); });
    __syncthreads();
    store_rows<BNO, PITCH, 1, NT>(pool, static_cast<uint8_t*>(p.c) + m0 * p.ldc + o0, p.ldc, rows_in, outs_in, tid);
    if (p.c_ring) {
      ring_block_finish<OUT>(p.c_ring, p.c_H, pub, s_c, p.c_scale_inv_out, p.c_amax_out,
                             reinterpret_cast<uint32_t*>(red + NWAVES));
    } else {
      if (p.c_amax_out) {
        const float bmax = block_max<NT>(amax, red);
        if (tid == 0) publish_max(reinterpret_cast<uint32_t*>(p.c_amax_out), bmax);
      }
      if (tid == 0 && p.c_scale_inv_out && blockIdx.x == 0) *p.c_scale_inv_out = 1.0f / s_c;
    }
  }
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
                     dim3((unsigned)(tiles_m * tiles_n)), dim3(64 * WM_ * WN_), 0, st, p, tiles_m, tiles_n, 4);
  return hipGetLastError();
}

// The tile rule of the plain GEMM (pick_tile): the K loop dominates both.
template <int OUT, bool GATED> static hipError_t launch_act_family(const MmActArgs& args, hipStream_t st) {
  using P = MmActTyped<GATED>;
  P p;
  static_cast<MmActArgs&>(p) = args;
  const int tile = pick_tile(p, device_cu_count());
  if (mm_precise(p)) {
    switch (tile) {
      case 5: return launch_act_tile<64, 64, 1, 4, 2, OUT, P, true>(p, st);
      case 2: return launch_act_tile<64, 128, 1, 4, 2, OUT, P, true>(p, st);
      default: return launch_act_tile<128, 128, 2, 2, 2, OUT, P, true>(p, st);
    }
  }
  switch (tile) {
    case 0: return launch_act_tile<256, 256, 2, 4, 1, OUT, P>(p, st);
    case 3: return launch_act_tile<256, 192, 2, 4, 1, OUT, P>(p, st);
    case 1: return launch_act_tile<128, 128, 2, 2, 2, OUT, P>(p, st);
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
