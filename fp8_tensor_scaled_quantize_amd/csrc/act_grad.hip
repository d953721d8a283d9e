// Gradient through the activation of a fused epilogue, quantized for the two
// products of the backward pass:
//   dz_ij = dy_ij act'(z_ij), or gated (gate and value interleaved in z)
//   dz_i,2j = dy_ij act'(z_i,2j) z_i,2j+1,  dz_i,2j+1 = dy_ij act(z_i,2j),
//   codes = enc(fl32(dz s)) in row and transposed layout, amax = max |dz|
// (folded into the gradient's ring, or to the caller's word) and the bias
// gradient's column sums of dz, all from one read of dy and z.
//
// Bound by HBM: 4 bytes read (2 + 1 per dz element gated) and 2 written per
// element.  The tile (tile.h) is the dual quantize's; each thread computes its
// 4 x 8 values in registers, publishes the workgroup's amax before it encodes
// them, stores the row codes directly and the transposed ones through LDS.
// Stores are non-temporal (8192 x 6912 with the bias gradient 88.0 -> 81.8 us
// over three sets of buffers in turn), the gated form's row codes excepted: they
// gain nothing by it (68.9 against 68.7 us) and the products that follow lose (a
// gated block's step at 8192 x 1536 x 6912 1062 -> 1080 us).
#include "activation.h"
#include "fp8mi_internal.h"
#include "tile.h"
#include "vec_io.h"

namespace fp8mi {

// Six workgroups a CU: 80 registers.  The form with the bias gradient needs 84 and
// spills 12 to 16; with five a CU (no spill) it takes 80.9 us in place of 81.7 at
// 8192 x 6912 and 128.0 in place of 130.2 at 8192 x 13824 gated, the form without
// it the same at either (80.0, 130.4).
template <int DT, int FMT, int ACT, bool GATED, bool BG>
__global__ void __launch_bounds__(kTileThreads, 6) act_grad_kernel(ActGradArgs p, int64_t tiles_c, int64_t ntiles) {
  __shared__ float red[kTileThreads / 64];
  __shared__ __align__(16) uint32_t lds_t[kTileC * 32];
  __shared__ float bg_part[BG ? kTileR / 4 * kTileC : 1];  // [row group][column], swizzled
  const int t = threadIdx.x, cg = t & 7, rg = t >> 3;
  const float s = p.ring ? __uint_as_float(p.ring[p.H]) : *p.scale;
  int64_t r0 = 0, c0 = 0;
  const int64_t tile = dual_pair_block(blockIdx.x, gridDim.x);
  if (ntiles > 0) tile_origin(tile, tiles_c, ntiles, r0, c0);
  const int64_t cc = c0 + 8 * cg;  // this thread's first column
  const int n = cc >= p.cols ? 0 : (p.cols - cc >= 8 ? 8 : (int)(p.cols - cc));

  // all loads first
  constexpr int NDY = GATED ? 4 : 8;
  Raw8<DT> rd[4];
  Raw8<kBF16> rz[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + 4 * rg + i;
    const int ni = r < p.rows ? n : 0;
    if (ni == 8) {
      load8(rz[i], p.z, r * p.ld_z + cc);
      if constexpr (GATED) {
        zero8(rd[i]);
        const u32x2_any v = *reinterpret_cast<const u32x2_any*>(static_cast<const uint16_t*>(p.dy) + r * p.ld_dy +
                                                                cc / 2);
        rd[i].w[0] = v[0];
        rd[i].w[1] = v[1];
      } else {
        load8(rd[i], p.dy, r * p.ld_dy + cc);
      }
    } else {
      load8_tail(rz[i], p.z, r * p.ld_z + cc, ni);
      load8_tail(rd[i], p.dy, r * p.ld_dy + (GATED ? cc / 2 : cc), GATED ? ni / 2 : ni);
    }
  }
  float d[4][8];
  float m = 0.0f;  // max |dz| with a NaN kept
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float g[8], z[8];
    widen8(rd[i], g);
    widen8(rz[i], z);
#pragma unroll
    for (int e = 0; e < NDY; ++e) {
      float v, sl;
      if constexpr (GATED) {
        act_value_slope<ACT>(z[2 * e], v, sl);
        d[i][2 * e] = g[e] * z[2 * e + 1] * sl;
        d[i][2 * e + 1] = g[e] * v;
      } else {
        act_value_slope<ACT>(z[e], v, sl);
        d[i][e] = g[e] * sl;
      }
    }
    // rows and columns outside the tensor hold dy = z = 0, so dz = 0
#pragma unroll
    for (int e = 0; e < 8; ++e) m = __builtin_elementwise_maximum(m, fabsf(d[i][e]));
  }
  const bool nan = m != m;
  if (nan) {
    m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(d[i][e]));
  }
  // the amax is published before the codes are stored: the slot atomic's round
  // trip passes under them
  uint32_t pub = __builtin_nondeterministic_value(0u);  // read by thread 0 only
  const bool want_amax = p.ring || p.amax_out;
  float bmax = 0.0f;
  if (want_amax) bmax = block_max<kTileThreads>(m, red);
  if (p.ring && t == 0) pub = ring_publish(p.ring, p.H, bmax);

  uint32_t rw[4][2];
  if (!nan && scale_regular(s) && m * fabsf(s) <= FmtTraits<FMT>::kMax) {
    // no clamp needed: fl32(|dz| |s|) <= fl32(m |s|)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        rw[i][h] = cvt4_inrange<FMT>(d[i][4 * h] * s, d[i][4 * h + 1] * s, d[i][4 * h + 2] * s, d[i][4 * h + 3] * s);
  } else if (!nan && scale_regular(s)) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        rw[i][h] = cvt4<FMT>(d[i][4 * h] * s, d[i][4 * h + 1] * s, d[i][4 * h + 2] * s, d[i][4 * h + 3] * s);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        rw[i][h] = enc4_exact<FMT>(d[i][4 * h] * s, d[i][4 * h + 1] * s, d[i][4 * h + 2] * s, d[i][4 * h + 3] * s);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + 4 * rg + i;
    if (r < p.rows && n > 0) store_codes8<!GATED>(p.out_row + r * p.ld_row + cc, rw[i][0], rw[i][1], n);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t col[4];
    transpose4x4_bytes(rw[0][h], rw[1][h], rw[2][h], rw[3][h], col);
#pragma unroll
    for (int k = 0; k < 4; ++k) lds_t[lds_t_index(8 * cg + 4 * h + k, rg)] = col[k];
  }
  if constexpr (BG) {
    // bias gradient: this thread's 4 rows in fp32, then the 32 row groups (and
    // the tiles) in fp64, in a fixed order
#pragma unroll
    for (int e = 0; e < 8; ++e)
      bg_part[bg_index(rg, 8 * cg + e)] = (d[0][e] + d[1][e]) + (d[2][e] + d[3][e]);
  }
  __syncthreads();
  if constexpr (BG) {
    if (t < kTileC && c0 + t < p.cols && ntiles > 0) {
      double v = 0.0;
#pragma unroll 8
      for (int g = 0; g < kTileR / 4; ++g) v += (double)bg_part[bg_index(g, t)];
      p.bias_ws[(r0 / kTileR) * p.cols + c0 + t] = v;
    }
  }
  // 64 transposed rows (one per column) x 128 bytes; lane: row cl, 16 bytes at 16q
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    const int cl = (t >> 3) + 32 * pass, q = t & 7;
    const int64_t c = c0 + cl, rr = r0 + 16 * q;
    if (c < p.cols && rr < p.rows) {
      const uint4 v = *reinterpret_cast<const uint4*>(&lds_t[lds_t_index(cl, 4 * q)]);
      uint8_t* dst = p.out_t + c * p.ld_t + rr;
      if (rr + 16 <= p.rows) {
        const u32x4_byte w = {v.x, v.y, v.z, v.w};
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4_byte*>(dst));
      } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 15; ++e)
          if (rr + e < p.rows) dst[e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
      }
    }
  }
  if (p.ring) {
    ring_block_finish<FMT>(p.ring, p.H, pub, s, p.scale_inv_out, p.amax_out, reinterpret_cast<uint32_t*>(red));
  } else if (t == 0) {
    if (p.amax_out) publish_max(reinterpret_cast<uint32_t*>(p.amax_out), bmax);
    if (p.scale_inv_out && blockIdx.x == 0) *p.scale_inv_out = 1.0f / s;
  }
}

template <int DT, int FMT, int ACT, bool GATED> static hipError_t launch_one(const ActGradArgs& p, hipStream_t st) {
  const int64_t tiles_c = (p.cols + kTileC - 1) / kTileC;
  const int64_t ntiles = ((p.rows + kTileR - 1) / kTileR) * tiles_c;
  const dim3 grid((unsigned)(ntiles > 0 ? ntiles : 1));  // nothing to do: the scale's bookkeeping alone
  if (p.bias_ws)
    hipLaunchKernelGGL((act_grad_kernel<DT, FMT, ACT, GATED, true>), grid, dim3(kTileThreads), 0, st, p, tiles_c,
                       ntiles);
  else
    hipLaunchKernelGGL((act_grad_kernel<DT, FMT, ACT, GATED, false>), grid, dim3(kTileThreads), 0, st, p, tiles_c,
                       ntiles);
  return hipGetLastError();
}

template <int DT, int FMT> static hipError_t launch_fmt(const ActGradArgs& p, int act, bool gated, hipStream_t st) {
  if (gated) {
    switch (act) {
      case kActRelu: return launch_one<DT, FMT, kActRelu, true>(p, st);
      case kActGelu: return launch_one<DT, FMT, kActGelu, true>(p, st);
      case kActSilu: return launch_one<DT, FMT, kActSilu, true>(p, st);
      default: return launch_one<DT, FMT, kActNone, true>(p, st);
    }
  }
  switch (act) {
    case kActRelu: return launch_one<DT, FMT, kActRelu, false>(p, st);
    case kActGelu: return launch_one<DT, FMT, kActGelu, false>(p, st);
    default: return launch_one<DT, FMT, kActSilu, false>(p, st);
  }
}

hipError_t launch_act_grad(const ActGradArgs& p, int dt, int fmt, int act, bool gated, hipStream_t st) {
  if (!p.ring && p.amax_out) {
    const hipError_t e = launch_zero_word(p.amax_out, st);
    if (e != hipSuccess) return e;
  }
  if (dt == kF16) return fmt == kE4M3 ? launch_fmt<kF16, kE4M3>(p, act, gated, st) : launch_fmt<kF16, kE5M2>(p, act, gated, st);
  return fmt == kE4M3 ? launch_fmt<kBF16, kE4M3>(p, act, gated, st) : launch_fmt<kBF16, kE5M2>(p, act, gated, st);
}

}  // namespace fp8mi
