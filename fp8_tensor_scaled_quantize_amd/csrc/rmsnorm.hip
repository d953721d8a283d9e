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
//
// Four vectors a lane at sixteen waves a row (above 16384 columns) pass the 128
// registers a lane has there: fp32 rows spill in the norm (512 x 32768 63 us for
// 218 MB), every type in the gradient (1024 x 20480 bf16 154 us for 168 MB, where
// two vectors a lane take 66 us for the 268 MB of 2048 x 16384).  The one-wave
// fp32 gradient of 1537 to 2048 columns spills too (8192 x 2048 86 us for 268 MB).
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

// A lane's NV vectors of one row: elements 8 (v 64 WPR + li) .. + 7, n[v] of
// them inside the row; the others read as zero.
template <int DT, int NV> struct RowRaw {
  Raw8<DT> v[NV];
};
template <int DT, int WPR, int NV>
__device__ __forceinline__ void load_row(RowRaw<DT, NV>& r, const void* base, int64_t at, int li, const int (&n)[NV]) {
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (n[v] == 8) load8(r.v[v], base, at + 8 * (v * 64 * WPR + li));
    else load8_tail(r.v[v], base, at + 8 * (v * 64 * WPR + li), n[v]);
  }
}
// Weights of the lane's columns: as stored (W32: fp32, else two bytes each).
template <bool W32, int WPR, int NV>
__device__ __forceinline__ void load_weight(RowRaw<W32 ? kF32 : kBF16, NV>& r, const void* w, int li, const int (&n)[NV]) {
  if (w) {
    load_row<W32 ? kF32 : kBF16, WPR, NV>(r, w, 0, li, n);
  } else {  // ones (fp32: the launch picks W32)
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < Raw8<W32 ? kF32 : kBF16>::kWords; ++e) r.v[v].w[e] = 0x3F800000u;
  }
}
template <bool W32> __device__ __forceinline__ void widen_weight(const Raw8<W32 ? kF32 : kBF16>& r, int dt, float (&f)[8]) {
  if constexpr (W32) {
    widen8(r, f);
  } else if (dt == kBF16) {
    widen8(r, f);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) widen2<kF16>(r.w[e], f[2 * e], f[2 * e + 1]);
  }
}

// A workgroup of NT threads holds NT / 64 / WPR rows at a time.
template <int DT, bool W32, int WPR, int NV, int NT>
__global__ void __launch_bounds__(NT) rmsnorm_kernel(NormArgs p) {
  constexpr int RPB = NT / 64 / WPR;
  static_assert(RPB >= 1 && (WPR == 1 || RPB == 1), "a row of several waves takes the whole workgroup");
  __shared__ float red[2][2][WPR];
  __shared__ float blk[NT / 64 + 1];
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int wr = WPR == 1 ? 0 : wid;
  const int li = wr * 64 + lane;
  int n[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int64_t c = 8 * (int64_t)(v * 64 * WPR + li);
    n[v] = c >= p.cols ? 0 : (p.cols - c >= 8 ? 8 : (int)(p.cols - c));
  }
  const float s_t = p.row_scaled ? 1.0f : (p.ring ? __uint_as_float(p.ring[p.H]) : *p.scale);
  // one pass over the rows: the workgroup's amax is published as soon as it is
  // known, its atomic's round trip passing under the encoding and the stores
  const bool early = p.ring && !p.row_scaled && p.rows <= (int64_t)gridDim.x * RPB;
  uint32_t pub = __builtin_nondeterministic_value(0u);  // read by thread 0 only
  RowRaw<W32 ? kF32 : kBF16, NV> rw;
  float amax = 0.0f;
  int parity = 0;
  int64_t row = (int64_t)blockIdx.x * RPB + (WPR == 1 ? wid : 0);
  // with early every wave takes the loop's first turn, rows or not (a barrier)
  for (bool first = true; row < p.rows || (early && first); row += (int64_t)gridDim.x * RPB) {
    const bool have = row < p.rows;
    RowRaw<DT, NV> rx, rr;
    float f[NV][8];
    float ss = 0.0f;
    if (have) {
      load_row<DT, WPR, NV>(rx, p.x, row * p.ld_x, li, n);
      if (p.res) load_row<DT, WPR, NV>(rr, p.res, row * p.ld_res, li, n);
      if (first) load_weight<W32, WPR, NV>(rw, p.weight, li, n);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        widen8(rx.v[v], f[v]);
        if (p.res) {
          float r[8];
          widen8(rr.v[v], r);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[v][e] += r[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(f[v][e], f[v][e], ss);
      }
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) f[v][e] = 0.0f;
    }
    first = false;
    ss = row_sum<WPR>(ss, red[parity][0], wr, lane);
    const float rstd = 1.0f / sqrtf(ss / p.n_cols + p.eps);
    float m = 0.0f;  // max |y| with a NaN kept
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (p.sum_out && n[v] > 0 && have) {  // h, before it is scaled in place
        Raw8<DT> o;
        narrow8(o, f[v]);
        store8(p.sum_out, row * p.ld_sum + 8 * (v * 64 * WPR + li), o, n[v]);
      }
      if (have) {
        float w[8];
        widen_weight<W32>(rw.v[v], p.weight_dt, w);
        // elements past the row's end are zeros, NaN only where rstd is inf
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f[v][e] = (f[v][e] * rstd) * w[e];
          m = __builtin_elementwise_maximum(m, fabsf(f[v][e]));
        }
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
      s = p.fmt == kE4M3 ? scale_from_max<kE4M3>(rm) : scale_from_max<kE5M2>(rm);
      if (li == 0) {
        p.scale_inv_out[row] = 1.0f / s;
        if (p.amax_out) p.amax_out[row] = rm;
      }
    } else {
      amax = fmaxf(amax, m);
    }
    if (early) {  // uniform over the workgroup
      const float bmax = block_max<NT>(amax, blk);
      if (threadIdx.x == 0) pub = ring_publish(p.ring, p.H, bmax);
    }
    if (p.rstd_out && li == 0 && have) p.rstd_out[row] = rstd;
    const bool exact = nan || !scale_regular(s);
    if (have) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (n[v] > 0) {
          // not streamed: the product that follows reads them (19.3 us streamed,
          // 19.8 so, and 256 rows' product 0.25 us slower)
          const uint2 q = p.fmt == kE4M3 ? encode8<kE4M3>(f[v], s, exact) : encode8<kE5M2>(f[v], s, exact);
          store_codes8(p.out + row * p.ld_out + 8 * (v * 64 * WPR + li), q.x, q.y, n[v]);
        }
      }
    }
    parity ^= 1;
  }
  if (p.row_scaled) return;
  uint32_t* const flag = reinterpret_cast<uint32_t*>(blk);
  if (p.ring) {
    if (!early) {
      const float bmax = block_max<NT>(amax, blk);
      if (threadIdx.x == 0) pub = ring_publish(p.ring, p.H, bmax);
    }
    if (p.fmt == kE4M3) ring_block_finish<kE4M3>(p.ring, p.H, pub, s_t, p.scale_inv_out, p.amax_out, flag);
    else ring_block_finish<kE5M2>(p.ring, p.H, pub, s_t, p.scale_inv_out, p.amax_out, flag);
    return;
  }
  if (p.amax_out) {
    const float bmax = block_max<NT>(amax, blk);
    if (threadIdx.x == 0) publish_max(reinterpret_cast<uint32_t*>(p.amax_out), bmax);
  }
  if (threadIdx.x == 0 && p.scale_inv_out && blockIdx.x == 0) *p.scale_inv_out = 1.0f / s_t;
}

// The weight gradient of few rows, straight from dy and h: workgroups past the
// rows' own take 16 columns each, NT / 16 row lanes per column, so a second
// launch is saved for a second read (from the L2).
constexpr int kDirectCols = 16;
template <int DT, int NT> __device__ __forceinline__ void dw_direct(const NormGradArgs& p, int64_t c0, float* red) {
  constexpr int RL = NT / kDirectCols, U = 4;
  const int c = threadIdx.x % kDirectCols, rl = threadIdx.x / kDirectCols;
  const int64_t col = c0 + c;
  float s = 0.0f;
  if (col < p.cols) {
    for (int64_t r = rl; r < p.rows; r += U * RL) {
      float d[U], h[U], k[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t q = r + u * RL < p.rows ? r + u * RL : r;
        d[u] = load1<DT>(p.dy, q * p.ld_dy + col);
        h[u] = load1<DT>(p.h, q * p.ld_h + col);
        k[u] = p.rstd[q];
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (r + u * RL < p.rows) s = fmaf(d[u], h[u] * k[u], s);
    }
  }
  red[threadIdx.x] = s;
  __syncthreads();
  if (rl == 0 && col < p.cols) {
    double v = (double)red[c];
    for (int i = 1; i < RL; ++i) v += (double)red[i * kDirectCols + c];
    p.dw_direct[col] = (float)v;
  }
}

// Gradient.  A wave (WPR = 1) or the workgroup walks over rows, the next row's
// loads in flight while one is finished, and keeps the weights and the weight
// gradient's sums of its columns in registers; each workgroup then writes one
// fp32 partial row, and rmsnorm_dw adds those in a fixed order.
template <int DT, bool W32, int WPR, int NV, int NT>
__global__ void __launch_bounds__(NT) rmsnorm_grad_kernel(NormGradArgs p) {
  constexpr int RPB = NT / 64 / WPR;
  static_assert(RPB >= 1 && (WPR == 1 || RPB == 1), "a row of several waves takes the whole workgroup");
  __shared__ float red[2][WPR];
  __shared__ float part[WPR == 1 && NV * 512 > NT ? NV * 512 : NT];
  if ((int64_t)blockIdx.x >= p.row_blocks) {
    dw_direct<DT, NT>(p, ((int64_t)blockIdx.x - p.row_blocks) * kDirectCols, part);
    return;
  }
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int wr = WPR == 1 ? 0 : wid;
  const int li = wr * 64 + lane;
  int n[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int64_t c = 8 * (int64_t)(v * 64 * WPR + li);
    n[v] = c >= p.cols ? 0 : (p.cols - c >= 8 ? 8 : (int)(p.cols - c));
  }
  RowRaw<W32 ? kF32 : kBF16, NV> rw;
  load_weight<W32, WPR, NV>(rw, p.weight, li, n);
  float dw[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[v][e] = 0.0f;
  const int64_t step = p.row_blocks * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + (WPR == 1 ? wid : 0);
  RowRaw<DT, NV> rd, rh, rs;
  float rstd = 0.0f;
  auto load = [&](int64_t r) {
    rstd = p.rstd[r];
    load_row<DT, WPR, NV>(rd, p.dy, r * p.ld_dy, li, n);
    load_row<DT, WPR, NV>(rh, p.h, r * p.ld_h, li, n);
    if (p.dsum) load_row<DT, WPR, NV>(rs, p.dsum, r * p.ld_dsum, li, n);
  };
  // (a row of sixteen waves leaves no registers for the next one)
  constexpr bool AHEAD = WPR < 16;
  if (AHEAD && row < p.rows) load(row);
  int parity = 0;
  for (; row < p.rows; row += step) {
    if (!AHEAD) load(row);
    float g[NV][8], o[NV][8];
    float dot = 0.0f;
    const float rk = rstd;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float w[8], h[8];
      widen8(rd.v[v], g[v]);
      widen8(rh.v[v], h);
      widen_weight<W32>(rw.v[v], p.weight_dt, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dw[v][e] = fmaf(g[v][e], h[e] * rk, dw[v][e]);
        g[v][e] *= w[e];
        dot = fmaf(g[v][e], h[e], dot);
        o[v][e] = h[e];
      }
    }
    dot = row_sum<WPR>(dot, red[parity], wr, lane);
    // rstd^3 by itself leaves fp32's range where rows are beyond 1e12 or below 1e-12
    const float k = -rk * (rk * (rk * (dot / p.n_cols)));
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int e = 0; e < 8; ++e) o[v][e] = fmaf(k, o[v][e], rk * g[v][e]);
      if (p.dsum) {
        float t[8];
        widen8(rs.v[v], t);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[v][e] += t[e];
      }
    }
    if (AHEAD && row + step < p.rows) load(row + step);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (n[v] == 0) continue;
      Raw8<DT> q;
      narrow8(q, o[v]);
      store8(p.dx, row * p.ld_dx + 8 * (v * 64 * WPR + li), q, n[v]);
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
// workgroup, 16 sub-lanes per column over contiguous ranges of partials.
constexpr int kDwCols = 32, kDwSplit = 16;
__global__ void __launch_bounds__(kDwCols * kDwSplit) rmsnorm_dw(const float* parts, int64_t nparts, int64_t cols,
                                                                 float* out) {
  __shared__ double red[kDwSplit][kDwCols];
  const int c = threadIdx.x % kDwCols, q = threadIdx.x / kDwCols;
  const int64_t col = (int64_t)blockIdx.x * kDwCols + c;
  const int64_t per = (nparts + kDwSplit - 1) / kDwSplit;
  const int64_t k0 = q * per, k1 = k0 + per < nparts ? k0 + per : nparts;
  double t = 0.0;
  if (col < cols) {
#pragma unroll 16
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

template <int DT, bool W32, int WPR, int NV, int NT>
static void launch_norm_one(const NormArgs& p, int64_t most_blocks, hipStream_t st) {
  constexpr int RPB = NT / 64 / WPR;
  int64_t blocks = cdiv(p.rows, RPB);
  if (blocks > most_blocks) blocks = most_blocks;
  if (blocks < 1) blocks = 1;
  hipLaunchKernelGGL((rmsnorm_kernel<DT, W32, WPR, NV, NT>), dim3((unsigned)blocks), dim3(NT), 0, st, p);
}

// Waves per row: one while the rows alone give the chip its waves and a row
// fits 6 vectors per lane; else four (rows of at most 8192 columns) or
// sixteen (at most kNormMaxCols).
// (Three vectors a lane for 4097 .. 6144 columns instead of four with idle ones:
// 4096 x 5120 with sum and ring 37.4 -> 35.6 us, its gradient 58.0 -> 54.6.)
template <int DT, bool W32> static hipError_t launch_norm(const NormArgs& p, hipStream_t st) {
  const int64_t ncu = device_cu_count();
  // an explicit scale with amax_out: every workgroup's maximum goes to the
  // caller's one word and these atomics serialise (about 12 ns each), so few
  // workgroups of several rows (1000 x 1535 fp16: 16.3 -> 11.5 us in graph replay)
  const bool word = !p.row_scaled && !p.ring && p.amax_out;
  const int64_t most = word ? ncu : 8 * ncu;
  const int64_t v1 = cdiv(p.cols, 512), v4 = cdiv(p.cols, 2048), v16 = cdiv(p.cols, 8192);
  if (v1 <= 1 || (v1 <= 6 && p.rows >= (word ? ncu / 2 : 4 * ncu))) {
    switch (v1) {
      case 0:
      case 1: launch_norm_one<DT, W32, 1, 1, 256>(p, most, st); break;
      case 2: launch_norm_one<DT, W32, 1, 2, 256>(p, most, st); break;
      case 3: launch_norm_one<DT, W32, 1, 3, 256>(p, most, st); break;
      case 4: launch_norm_one<DT, W32, 1, 4, 256>(p, most, st); break;
      default: launch_norm_one<DT, W32, 1, 6, 256>(p, most, st); break;
    }
  } else if (v4 <= 4) {
    switch (v4) {
      case 1: launch_norm_one<DT, W32, 4, 1, 256>(p, most, st); break;
      case 2: launch_norm_one<DT, W32, 4, 2, 256>(p, most, st); break;
      case 3: launch_norm_one<DT, W32, 4, 3, 256>(p, most, st); break;
      default: launch_norm_one<DT, W32, 4, 4, 256>(p, most, st); break;
    }
  } else {
    if (v16 <= 2) launch_norm_one<DT, W32, 16, 2, 1024>(p, most, st);
    else launch_norm_one<DT, W32, 16, 4, 1024>(p, most, st);
  }
  return hipGetLastError();
}

// No weight reads as fp32 ones.
static bool weight_32(const void* weight, int dt) { return !weight || dt == kF32; }

hipError_t launch_rmsnorm(const NormArgs& p, int dt, hipStream_t st) {
  if (p.row_scaled && p.rows == 0) return hipSuccess;
  if (!p.row_scaled && !p.ring && p.amax_out) {
    const hipError_t e = launch_zero_word(p.amax_out, st);
    if (e != hipSuccess) return e;
  }
  if (weight_32(p.weight, p.weight_dt)) {
    switch (dt) {
      case kF32: return launch_norm<kF32, true>(p, st);
      case kF16: return launch_norm<kF16, true>(p, st);
      default: return launch_norm<kBF16, true>(p, st);
    }
  }
  switch (dt) {
    case kF32: return launch_norm<kF32, false>(p, st);
    case kF16: return launch_norm<kF16, false>(p, st);
    default: return launch_norm<kBF16, false>(p, st);
  }
}

// Workgroups of the gradient's main pass (one partial row of the weight's
// gradient each).  One wave per row: 8 rows a workgroup, one workgroup per CU
// (its registers allow no second).  Four waves: one to four per CU, so that
// each has 8 rows -- the partial rows are written and read once more (1024 x
// 8192: 45 us with 1024 of them, 29.5 with 512).  Sixteen waves: one per CU.
constexpr int64_t kGradBlocks1 = 256, kGradBlocks4 = 1024, kGradBlocks16 = 256;
static bool grad_one_wave(int64_t rows, int64_t cols) { return cols <= 512 || (cols <= 2048 && rows >= 2048); }
static int64_t grad_blocks(int64_t rows, int64_t cols) {
  const bool one = grad_one_wave(rows, cols);
  const int64_t b = one ? cdiv(rows, 8) : rows;
  int64_t most = one ? kGradBlocks1 : (cols <= 8192 ? kGradBlocks4 : kGradBlocks16);
  if (!one && most > rows / 8) most = rows / 8 > 256 ? rows / 8 : 256;
  return b > most ? most : b;
}
// Few rows: the weight gradient comes from the same launch (dw_direct).  A
// second launch costs about 4.5 us, the second read of 512 rows less.
constexpr int64_t kDirectRows = 512;

int64_t rmsnorm_grad_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  return grad_blocks(rows, cols) * cols * (int64_t)sizeof(float);
}

template <int DT, bool W32> static void launch_norm_grad(const NormGradArgs& p, unsigned nb, hipStream_t st) {
  const int64_t v1 = cdiv(p.cols, 512), v4 = cdiv(p.cols, 2048), v16 = cdiv(p.cols, 8192);
  const dim3 g(nb);
  if (grad_one_wave(p.rows, p.cols)) {
    switch (v1) {
      case 1: hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, W32, 1, 1, 512>), g, dim3(512), 0, st, p); break;
      case 2: hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, W32, 1, 2, 512>), g, dim3(512), 0, st, p); break;
      case 3: hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, W32, 1, 3, 512>), g, dim3(512), 0, st, p); break;
      default: hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, W32, 1, 4, 512>), g, dim3(512), 0, st, p); break;
    }
  } else if (v4 <= 4) {
    switch (v4) {
      case 1: hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, W32, 4, 1, 256>), g, dim3(256), 0, st, p); break;
      case 2: hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, W32, 4, 2, 256>), g, dim3(256), 0, st, p); break;
      case 3: hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, W32, 4, 3, 256>), g, dim3(256), 0, st, p); break;
      default: hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, W32, 4, 4, 256>), g, dim3(256), 0, st, p); break;
    }
  } else {
    if (v16 <= 2) hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, W32, 16, 2, 1024>), g, dim3(1024), 0, st, p);
    else hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, W32, 16, 4, 1024>), g, dim3(1024), 0, st, p);
  }
}

hipError_t launch_rmsnorm_grad(const NormGradArgs& p0, int dt, float* dweight, void* workspace, hipStream_t st) {
  if (p0.cols == 0) return hipSuccess;
  const int64_t nb = p0.rows > 0 ? grad_blocks(p0.rows, p0.cols) : 0;
  NormGradArgs p = p0;
  const bool direct = dweight && nb > 0 && p0.rows <= kDirectRows;
  p.dw_direct = direct ? dweight : nullptr;
  p.parts = dweight && !direct ? static_cast<float*>(workspace) : nullptr;
  const bool w32 = weight_32(p.weight, p.weight_dt);
  auto launch = [&](int64_t row_blocks, int64_t dw_blocks) {
    p.row_blocks = row_blocks;
    const unsigned grid = (unsigned)(row_blocks + dw_blocks);
    switch (dt) {
      case kF32: w32 ? launch_norm_grad<kF32, true>(p, grid, st) : launch_norm_grad<kF32, false>(p, grid, st); break;
      case kF16: w32 ? launch_norm_grad<kF16, true>(p, grid, st) : launch_norm_grad<kF16, false>(p, grid, st); break;
      default: w32 ? launch_norm_grad<kBF16, true>(p, grid, st) : launch_norm_grad<kBF16, false>(p, grid, st); break;
    }
    return hipGetLastError();
  };
  hipError_t e = hipSuccess;
  if (direct) {
    const int64_t db = cdiv(p.cols, kDirectCols);
    if (p.dx == p.dy || p.dx == p.h) {  // the rows' results overwrite what dw_direct reads: one after the other
      e = launch(0, db);
      if (e == hipSuccess) e = launch(nb, 0);
    } else {
      e = launch(nb, db);
    }
  } else if (nb > 0) {
    e = launch(nb, 0);
  }
  if (e != hipSuccess) return e;
  if (dweight && !direct)
    hipLaunchKernelGGL(rmsnorm_dw, dim3((unsigned)cdiv(p.cols, kDwCols)), dim3(kDwCols * kDwSplit), 0, st,
                       static_cast<const float*>(workspace), nb, p.cols, dweight);
  return hipGetLastError();
}

}  // namespace fp8mi
