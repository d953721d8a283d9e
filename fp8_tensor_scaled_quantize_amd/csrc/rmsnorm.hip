// Root-mean-square norm with the residual's addition and an fp8 output, and
// its gradient.
//
//   h_ij = x_ij + r_ij,  rstd_i = 1 / sqrt(mean_j h_ij^2 + eps),
//   y_ij = (h_ij rstd_i) w_j,  code_ij = enc(fl32(y_ij s)).
// s is one scale per tensor (the caller's, or the ring's with this call's
// amax folded by the last workgroup) or one per row, s_i = fmt_max / max_j
// |y_ij|, measured while the row is still in registers.
//
// Gradient, with g_ij = dy_ij w_j and n columns:
//   dx_ij = rstd_i g_ij - rstd_i^3 (sum_j g_ij h_ij / n) h_ij + dsum_ij,
//   dw_j  = sum_i dy_ij (h_ij rstd_i).
//
// Both are bound by HBM: every element is read once and written once.  A row
// is held in the registers of WPR waves (NV vectors of 8 elements per lane),
// so the sums that need the whole row (and the row's maximum) cost no second
// read.  With WPR = 1 a row's sums stay inside one wave: no barrier, no LDS.
// All sums are fp32.
#include "fp8mi_internal.h"
#include "vec_io.h"

namespace fp8mi {

// Sum (maximum) over the WPR waves of a row, in wave order; red has WPR words
// that no other value uses before the next barrier but one.
template <int WPR> __device__ __forceinline__ float row_sum(float v, float* red, int wr, int lane) {
  v = wave_sum(v);
  if constexpr (WPR > 1) {
    if (lane == 0) red[wr] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < WPR; ++i) v += red[i];
  }
  return v;
}
template <int WPR> __device__ __forceinline__ float row_max(float v, float* red, int wr, int lane) {
  v = wave_max(v);
  if constexpr (WPR > 1) {
    if (lane == 0) red[wr] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < WPR; ++i) v = fmaxf(v, red[i]);
  }
  return v;
}

// Eight codes of y * s.  exact: some y is NaN or the scale is not regular.
template <int FMT> __device__ __forceinline__ uint2 encode8(const float (&y)[8], float s, bool exact) {
  if (!exact)
    return make_uint2(cvt4<FMT>(y[0] * s, y[1] * s, y[2] * s, y[3] * s),
                      cvt4<FMT>(y[4] * s, y[5] * s, y[6] * s, y[7] * s));
  return make_uint2(enc4_exact<FMT>(y[0] * s, y[1] * s, y[2] * s, y[3] * s),
                    enc4_exact<FMT>(y[4] * s, y[5] * s, y[6] * s, y[7] * s));
}

// A workgroup of NT threads holds NT / 64 / WPR rows.
template <int DT, int FMT, int WPR, int NV, int NT>
__global__ void __launch_bounds__(NT) rmsnorm_kernel(NormArgs p) {
  constexpr int RPB = NT / 64 / WPR;
  static_assert(RPB >= 1 && (WPR == 1 || RPB == 1), "a row of several waves takes the whole workgroup");
  __shared__ float red[2][2][WPR];
  __shared__ float blk[NT / 64 + 1];
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int wr = WPR == 1 ? 0 : wid;
  const int li = wr * 64 + lane;
  const float s_t = p.row_scaled ? 1.0f : (p.ring ? __uint_as_float(p.ring[p.H]) : *p.scale);
  float amax = 0.0f;
  int parity = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < p.rows; row0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = row0 + (WPR == 1 ? wid : 0);
    if (row >= p.rows) break;  // one row per wave: no barrier inside the loop
    Raw8<DT> rx[NV], rr[NV];
    int n[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t c = 8 * (int64_t)(v * 64 * WPR + li);
      n[v] = c >= p.cols ? 0 : (p.cols - c >= 8 ? 8 : (int)(p.cols - c));
      if (n[v] == 8) load8(rx[v], p.x, row * p.ld_x + c);
      else load8_tail(rx[v], p.x, row * p.ld_x + c, n[v]);
      if (p.res) {
        if (n[v] == 8) load8(rr[v], p.res, row * p.ld_res + c);
        else load8_tail(rr[v], p.res, row * p.ld_res + c, n[v]);
      }
    }
    float f[NV][8];
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      widen8(rx[v], f[v]);
      if (p.res) {
        float r[8];
        widen8(rr[v], r);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[v][e] += r[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(f[v][e], f[v][e], ss);
    }
    ss = row_sum<WPR>(ss, red[parity][0], wr, lane);
    const float rstd = 1.0f / sqrtf(ss / p.n_cols + p.eps);
    float m = 0.0f;  // max |y| with a NaN kept
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t c = 8 * (int64_t)(v * 64 * WPR + li);
      if (p.sum_out && n[v] > 0) {  // h, before it is scaled in place
        Raw8<DT> o;
        narrow8(o, f[v]);
        store8(p.sum_out, row * p.ld_sum + c, o, n[v]);
      }
      float w[8];
      if (p.weight) {
        load8_rt(w, p.weight, p.weight_dt, n[v] > 0 ? c : 0, n[v]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[v][e] = (f[v][e] * rstd) * w[e];
        // lanes past the row's end hold zeros, which rstd = inf would make NaN
        m = __builtin_elementwise_maximum(m, e < n[v] ? fabsf(f[v][e]) : 0.0f);
      }
    }
    const bool nan = m != m;
    if (nan) {
      m = 0.0f;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < n[v]) m = fmaxf(m, fabsf(f[v][e]));
    }
    float s = s_t;
    if (p.row_scaled) {
      const float rm = row_max<WPR>(m, red[parity][1], wr, lane);
      s = scale_from_max<FMT>(rm);
      if (li == 0) {
        p.scale_inv_out[row] = 1.0f / s;
        if (p.amax_out) p.amax_out[row] = rm;
      }
    } else {
      amax = fmaxf(amax, m);
    }
    if (p.rstd_out && li == 0) p.rstd_out[row] = rstd;
    const bool exact = nan || !scale_regular(s);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (n[v] > 0) {
        const uint2 q = encode8<FMT>(f[v], s, exact);
        store_codes8(p.out + row * p.ld_out + 8 * (int64_t)(v * 64 * WPR + li), q.x, q.y, n[v]);
      }
    }
    parity ^= 1;
  }
  if (p.row_scaled) return;
  const float bmax = block_max<NT>(amax, blk);
  if (p.ring) {
    ring_block_done<FMT>(p.ring, p.H, bmax, s_t, p.scale_inv_out, p.amax_out, reinterpret_cast<uint32_t*>(blk));
  } else if (threadIdx.x == 0) {
    if (p.amax_out) publish_max(reinterpret_cast<uint32_t*>(p.amax_out), bmax);
    if (p.scale_inv_out && blockIdx.x == 0) *p.scale_inv_out = 1.0f / s_t;
  }
}

// Gradient.  A wave (WPR = 1) or the workgroup walks over rows and keeps the
// weight gradient's sums of its columns in registers; each workgroup then
// writes one fp32 partial row, and rmsnorm_dw adds those in a fixed order.
template <int DT, int WPR, int NV, int NT>
__global__ void __launch_bounds__(NT) rmsnorm_grad_kernel(NormGradArgs p) {
  constexpr int RPB = NT / 64 / WPR;
  static_assert(RPB >= 1 && (WPR == 1 || RPB == 1), "a row of several waves takes the whole workgroup");
  __shared__ float red[2][WPR];
  __shared__ float part[WPR == 1 ? NV * 512 : 1];
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int wr = WPR == 1 ? 0 : wid;
  const int li = wr * 64 + lane;
  float dw[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[v][e] = 0.0f;
  int parity = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < p.rows; row0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = row0 + (WPR == 1 ? wid : 0);
    if (row >= p.rows) break;  // one row per wave: no barrier inside the loop
    Raw8<DT> rd[NV], rh[NV], rs[NV];
    int n[NV];
    const float rstd = p.rstd[row];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t c = 8 * (int64_t)(v * 64 * WPR + li);
      n[v] = c >= p.cols ? 0 : (p.cols - c >= 8 ? 8 : (int)(p.cols - c));
      if (n[v] == 8) {
        load8(rd[v], p.dy, row * p.ld_dy + c);
        load8(rh[v], p.h, row * p.ld_h + c);
        if (p.dsum) load8(rs[v], p.dsum, row * p.ld_dsum + c);
      } else {
        load8_tail(rd[v], p.dy, row * p.ld_dy + c, n[v]);
        load8_tail(rh[v], p.h, row * p.ld_h + c, n[v]);
        if (p.dsum) load8_tail(rs[v], p.dsum, row * p.ld_dsum + c, n[v]);
      }
    }
    float g[NV][8];
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t c = 8 * (int64_t)(v * 64 * WPR + li);
      float h[8], w[8];
      widen8(rd[v], g[v]);
      widen8(rh[v], h);
      if (p.weight) {
        load8_rt(w, p.weight, p.weight_dt, n[v] > 0 ? c : 0, n[v]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e < n[v]) dw[v][e] = fmaf(g[v][e], h[e] * rstd, dw[v][e]);
        g[v][e] *= w[e];
        dot = fmaf(g[v][e], h[e], dot);
      }
    }
    dot = row_sum<WPR>(dot, red[parity], wr, lane);
    const float k = -(rstd * rstd) * rstd * (dot / p.n_cols);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (n[v] == 0) continue;
      float h[8], o[8];
      widen8(rh[v], h);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = fmaf(k, h[e], rstd * g[v][e]);
      if (p.dsum) {
        float t[8];
        widen8(rs[v], t);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += t[e];
      }
      Raw8<DT> q;
      narrow8(q, o);
      store8(p.dx, row * p.ld_dx + 8 * (int64_t)(v * 64 * WPR + li), q, n[v]);
    }
    parity ^= 1;
  }
  if (!p.parts) return;
  float* dst = p.parts + (int64_t)blockIdx.x * p.cols;
  if constexpr (WPR == 1) {
    // the waves add their sums one after the other, in wave order
    for (int w = 0; w < NT / 64; ++w) {
      if (wid == w) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float* q = part + (v * 8 + e) * 64 + lane;
            *q = w == 0 ? dw[v][e] : *q + dw[v][e];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < p.cols; c += NT) dst[c] = part[((c >> 9) * 8 + (c & 7)) * 64 + ((c >> 3) & 63)];
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t c = 8 * (int64_t)(v * 64 * WPR + li);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < p.cols) dst[c + e] = dw[v][e];
    }
  }
}

// Adds the workgroups' partial rows, in order, in fp64: 32 columns per
// workgroup, 8 sub-lanes per column over contiguous ranges of partials.
constexpr int kDwCols = 32, kDwSplit = 8;
__global__ void __launch_bounds__(kDwCols * kDwSplit) rmsnorm_dw(const float* parts, int64_t nparts, int64_t cols,
                                                                 float* out) {
  __shared__ double red[kDwSplit][kDwCols];
  const int c = threadIdx.x % kDwCols, q = threadIdx.x / kDwCols;
  const int64_t col = (int64_t)blockIdx.x * kDwCols + c;
  const int64_t per = (nparts + kDwSplit - 1) / kDwSplit;
  const int64_t k0 = q * per, k1 = k0 + per < nparts ? k0 + per : nparts;
  double t = 0.0;
  if (col < cols) {
#pragma unroll 8
    for (int64_t k = k0; k < k1; ++k) t += (double)parts[k * cols + col];
  }
  red[q][c] = t;
  __syncthreads();
  if (q == 0 && col < cols) {
    double v = red[0][c];
#pragma unroll
    for (int j = 1; j < kDwSplit; ++j) v += red[j][c];
    out[col] = (float)v;
  }
}

// ---------------------------------------------------------------------------
// Host launchers.
// ---------------------------------------------------------------------------
static int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int DT, int FMT, int WPR, int NV, int NT>
static void launch_norm_one(const NormArgs& p, int64_t most_blocks, hipStream_t st) {
  constexpr int RPB = NT / 64 / WPR;
  int64_t blocks = cdiv(p.rows, RPB);
  if (blocks > most_blocks) blocks = most_blocks;
  if (blocks < 1) blocks = 1;
  hipLaunchKernelGGL((rmsnorm_kernel<DT, FMT, WPR, NV, NT>), dim3((unsigned)blocks), dim3(NT), 0, st, p);
}

// Waves per row: one while the rows alone give the chip its waves and a row
// fits 6 vectors per lane; else four (rows of at most 8192 columns) or
// sixteen (at most kNormMaxCols).
template <int DT, int FMT> static hipError_t launch_norm(const NormArgs& p, hipStream_t st) {
  const int64_t ncu = device_cu_count();
  const int64_t most = 8 * ncu;
  const int64_t v1 = cdiv(p.cols, 512), v4 = cdiv(p.cols, 2048), v16 = cdiv(p.cols, 8192);
  if (v1 <= 1 || (v1 <= 6 && p.rows >= 4 * ncu)) {
    switch (v1) {
      case 0:
      case 1: launch_norm_one<DT, FMT, 1, 1, 256>(p, most, st); break;
      case 2: launch_norm_one<DT, FMT, 1, 2, 256>(p, most, st); break;
      case 3: launch_norm_one<DT, FMT, 1, 3, 256>(p, most, st); break;
      case 4: launch_norm_one<DT, FMT, 1, 4, 256>(p, most, st); break;
      default: launch_norm_one<DT, FMT, 1, 6, 256>(p, most, st); break;
    }
  } else if (v4 <= 4) {
    switch (v4) {
      case 1: launch_norm_one<DT, FMT, 4, 1, 256>(p, most, st); break;
      case 2: launch_norm_one<DT, FMT, 4, 2, 256>(p, most, st); break;
      default: launch_norm_one<DT, FMT, 4, 4, 256>(p, most, st); break;
    }
  } else {
    if (v16 <= 2) launch_norm_one<DT, FMT, 16, 2, 1024>(p, most, st);
    else launch_norm_one<DT, FMT, 16, 4, 1024>(p, most, st);
  }
  return hipGetLastError();
}

template <int DT> static hipError_t launch_norm_dt(const NormArgs& p, int fmt, hipStream_t st) {
  return fmt == kE4M3 ? launch_norm<DT, kE4M3>(p, st) : launch_norm<DT, kE5M2>(p, st);
}

hipError_t launch_rmsnorm(const NormArgs& p, int dt, int fmt, hipStream_t st) {
  if (p.row_scaled && p.rows == 0) return hipSuccess;
  if (!p.row_scaled && !p.ring && p.amax_out) {
    const hipError_t e = launch_zero_word(p.amax_out, st);
    if (e != hipSuccess) return e;
  }
  switch (dt) {
    case kF32: return launch_norm_dt<kF32>(p, fmt, st);
    case kF16: return launch_norm_dt<kF16>(p, fmt, st);
    default: return launch_norm_dt<kBF16>(p, fmt, st);
  }
}

// Workgroups of the gradient's main pass (one partial row of the weight's
// gradient each): one per row (or per 8 rows of one wave each) up to
// kGradBlocks.
constexpr int64_t kGradBlocks = 512;
static bool grad_one_wave(int64_t rows, int64_t cols) { return cols <= 512 || (cols <= 2048 && rows >= 2048); }
static int64_t grad_blocks(int64_t rows, int64_t cols) {
  const int64_t b = grad_one_wave(rows, cols) ? cdiv(rows, 8) : rows;
  return b > kGradBlocks ? kGradBlocks : b;
}

int64_t rmsnorm_grad_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  return grad_blocks(rows, cols) * cols * (int64_t)sizeof(float);
}

template <int DT> static void launch_norm_grad(const NormGradArgs& p, unsigned nb, hipStream_t st) {
  const int64_t v1 = cdiv(p.cols, 512), v4 = cdiv(p.cols, 2048), v16 = cdiv(p.cols, 8192);
  const dim3 g(nb);
  if (grad_one_wave(p.rows, p.cols)) {
    switch (v1) {
      case 1: hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, 1, 1, 512>), g, dim3(512), 0, st, p); break;
      case 2: hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, 1, 2, 512>), g, dim3(512), 0, st, p); break;
      case 3: hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, 1, 3, 512>), g, dim3(512), 0, st, p); break;
      default: hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, 1, 4, 512>), g, dim3(512), 0, st, p); break;
    }
  } else if (v4 <= 4) {
    switch (v4) {
      case 1: hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, 4, 1, 256>), g, dim3(256), 0, st, p); break;
      case 2: hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, 4, 2, 256>), g, dim3(256), 0, st, p); break;
      default: hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, 4, 4, 256>), g, dim3(256), 0, st, p); break;
    }
  } else {
    if (v16 <= 2) hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, 16, 2, 1024>), g, dim3(1024), 0, st, p);
    else hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, 16, 4, 1024>), g, dim3(1024), 0, st, p);
  }
}

hipError_t launch_rmsnorm_grad(const NormGradArgs& p0, int dt, float* dweight, void* workspace, hipStream_t st) {
  if (p0.cols == 0) return hipSuccess;
  const int64_t nb = p0.rows > 0 ? grad_blocks(p0.rows, p0.cols) : 0;
  NormGradArgs p = p0;
  // one workgroup: its sums are the gradient
  p.parts = !dweight ? nullptr : (nb == 1 ? dweight : static_cast<float*>(workspace));
  if (nb > 0) {
    switch (dt) {
      case kF32: launch_norm_grad<kF32>(p, (unsigned)nb, st); break;
      case kF16: launch_norm_grad<kF16>(p, (unsigned)nb, st); break;
      default: launch_norm_grad<kBF16>(p, (unsigned)nb, st); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (dweight && nb != 1)
    hipLaunchKernelGGL(rmsnorm_dw, dim3((unsigned)cdiv(p.cols, kDwCols)), dim3(kDwCols * kDwSplit), 0, st,
                       static_cast<const float*>(workspace), nb, p.cols, dweight);
  return hipGetLastError();
}

}  // namespace fp8mi
