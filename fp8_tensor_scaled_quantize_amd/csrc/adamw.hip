// AdamW over many tensors in one launch, with states in 32 or in 8 bits, and
// the norm of all gradients that its clipping needs.
//
//   g = c grad                       m = b1 m + (1 - b1) g     v = b2 v + (1 - b2) g^2
//   w = w (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// in fp32; w is the tensor's fp32 master where it has one, and the parameter is
// w rounded once.
//
// Bound by HBM: 28 bytes per element with bf16 parameters and gradients, fp32
// masters and states, 16 with 8-bit states.  The tensors' table travels in the
// kernel's arguments (no copy, nothing for a captured graph to keep alive); a
// workgroup finds its tensor by one ballot over the tensors' first workgroups.
#include "fp8mi_device.h"
#include "fp8mi_internal.h"
#include "vec_io.h"

namespace fp8mi {

namespace {

constexpr int kNT = 256;           // threads per workgroup
constexpr int kBlock = 256;        // elements of an 8-bit state that share a scale: a wave's, four per lane
constexpr int kAdamWTensors = 44, kNormTensors = 128;  // of one launch: its arguments are at most 4 KiB
// Elements per workgroup: a block per wave.  With four blocks per wave in flight
// (88 registers instead of 38) 24 small tensors took 6.9 us instead of 4.7, ragged
// 8-bit ones 26.1 instead of 24.2, and only fp32 states gained (96 -> 94); with two, the
// second read before the first is worked on (56 registers), 5.0 instead of 4.5, 30.3
// instead of 27.2, one block of fp32 states 112.6 instead of 110.4, and only eight of
// 8-bit ones gained (541 -> 517).
constexpr int kChunk = kNT / 64 * kBlock;

// ------------------------------------------------------------------ the table
template <class T, int MAX> struct Table {
  T t[MAX];
  int32_t first[MAX];  // the tensors' first workgroups
  int32_t count;
};
// The tensor that a workgroup works on (MAX <= 128: two ballots).
template <class T, int MAX> __device__ __forceinline__ int find_tensor(const Table<T, MAX>& tab, int wg) {
  const int lane = threadIdx.x & 63;
  int n = __popcll(__ballot(lane < tab.count && tab.first[lane < MAX ? lane : 0] <= wg));
  if constexpr (MAX > 64)
    n += __popcll(__ballot(lane + 64 < tab.count && tab.first[lane + 64 < MAX ? lane + 64 : 0] <= wg));
  return __builtin_amdgcn_readfirstlane(n - 1);
}

// ------------------------------------------------------------------ four elements per lane
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32_byte1 __attribute__((aligned(1)));

struct Raw4 {
  uint32_t w[4];
};
__device__ __forceinline__ Raw4 load4(const void* p, int dt, int64_t i, int n) {
  Raw4 r = {{0u, 0u, 0u, 0u}};
  if (dt == kF32) {
    const uint32_t* q = static_cast<const uint32_t*>(p) + i;
    if (n >= 4) {
      const f32x4_any v = *reinterpret_cast<const f32x4_any*>(q);
#pragma unroll
      for (int e = 0; e < 4; ++e) r.w[e] = __float_as_uint(v[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < n) r.w[e] = q[e];
    }
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
    if (n >= 4) {
      const u32x2_any v = *reinterpret_cast<const u32x2_any*>(q);
      r.w[0] = v[0];
      r.w[1] = v[1];
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < n) r.w[e / 2] |= (uint32_t)q[e] << (16 * (e & 1));
    }
  }
  return r;
}
__device__ __forceinline__ void widen4(const Raw4& r, int dt, float (&f)[4]) {
  if (dt == kF32) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(r.w[e]);
  } else if (dt == kBF16) {
    widen2<kBF16>(r.w[0], f[0], f[1]);
    widen2<kBF16>(r.w[1], f[2], f[3]);
  } else {
    widen2<kF16>(r.w[0], f[0], f[1]);
    widen2<kF16>(r.w[1], f[2], f[3]);
  }
}
__device__ __forceinline__ void store4(void* p, int dt, int64_t i, const float (&f)[4], int n) {
  if (dt == kF32) {
    float* q = static_cast<float*>(p) + i;
    if (n >= 4) {
      *reinterpret_cast<f32x4_any*>(q) = f32x4_any{f[0], f[1], f[2], f[3]};
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < n) q[e] = f[e];
    }
    return;
  }
  uint32_t w[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const f32x2 v = {f[2 * e], f[2 * e + 1]};
    w[e] = dt == kBF16 ? __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2))
                       : __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
  }
  uint16_t* q = static_cast<uint16_t*>(p) + i;
  if (n >= 4) {
    *reinterpret_cast<u32x2_any*>(q) = u32x2_any{w[0], w[1]};
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < n) q[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
  }
}
__device__ __forceinline__ uint32_t load_codes4(const uint8_t* p, int64_t i, int n) {
  if (n >= 4) return *reinterpret_cast<const u32_byte1*>(p + i);
  uint32_t w = 0u;
#pragma unroll
  for (int e = 0; e < 3; ++e)
    if (e < n) w |= (uint32_t)p[i + e] << (8 * e);
  return w;
}
__device__ __forceinline__ void store_codes4(uint8_t* p, int64_t i, uint32_t w, int n) {
  if (n >= 4) {
    *reinterpret_cast<u32_byte1*>(p + i) = w;
    return;
  }
#pragma unroll
  for (int e = 0; e < 3; ++e)
    if (e < n) p[i + e] = (uint8_t)(w >> (8 * e));
}

// ------------------------------------------------------------------ 8-bit states
// m and r = sqrt(v) are E4M3 codes of m / s and r / s, s = max / 448 over a
// block.  Rounded to nearest, a moving average stands still once its change per
// step is below half a code step (6 per cent, against (1 - b2) = 0.1 to 5 per
// cent of v): v would stop at a few gradients' squares while the bias
// correction went on.  So codes are rounded stochastically, m so that m and
// v so that v itself (not its root) is met on average.  v > 0 never becomes 0:
// a later step without a gradient would divide m by eps alone.

// Magnitudes are compared as the bits of non-negative floats, whose order theirs
// is; a NaN is above all.  Max over the wave's 64 lanes in every lane:
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
#define FP8MI_ROR(n) (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + n, 0xf, 0xf, true)
  v = umax(v, FP8MI_ROR(8));
  v = umax(v, FP8MI_ROR(4));
  v = umax(v, FP8MI_ROR(2));
  v = umax(v, FP8MI_ROR(1));
#undef FP8MI_ROR
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = umax(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return umax(b[0], b[1]);
}

// Scale word of a block whose largest magnitude is `most`.  Below 2^-100 a block
// counts as zero (its reciprocal would leave fp32): the squares of such
// gradients are 0 in fp32 already.
__device__ __forceinline__ float block_scale(float most) {
  const float s = most * (1.0f / 448.0f);
  return s < 7.8886090522101181e-31f ? 0.0f : s;  // NaN stays
}

// y >= 0 as steps of the E4M3 grid below it: whole steps k, the rest f in [0, 1),
// and the code of k.  At most 448; subnormals have the step 2^-9.
__device__ __forceinline__ uint32_t grid_steps(float y, float& k, float& f) {
  y = fminf(y, 448.0f);
  const uint32_t exp = __float_as_uint(y) & 0x7F800000u, e = exp > 0x3C800000u ? exp : 0x3C800000u;
  const float t = y * __uint_as_float((257u << 23) - e);  // y / 2^(exponent - 3), exact
  k = floorf(t);
  f = t - k;
  return (e >> 20) - 968u + (uint32_t)k;
}

// y >= 0 rounded to the grid point above with the probability of its place between
// the two: h16 / 2^16 against the 20 bits below a code's mantissa.  2^-120 takes E4M3's
// exponents, its subnormals too, to fp32's, so that a code is the bits above those 20,
// and a carry goes into the exponent as the codes' order does.  Exact from y = 2^-6 on;
// below, the product is one of fp32's subnormals and is rounded first, by 2^-30 at most, so
// that a y which is that near to its place takes the neighbouring code (44 of 10^8).
__device__ __forceinline__ uint32_t round_code(float y, uint32_t h16) {
  const uint32_t bits = __float_as_uint(fminf(y, 448.0f) * 7.52316384526264e-37f);
  return (bits + (~(16u * h16) & 0xFFFF0u) + 7u) >> 20;
}

// Correctly rounded square root of x (or 0, or one that is not finite), by comparing x with
// the products of neighbours, and quotient x / s, given r = 1 / s correctly rounded
// (Markstein's correction), for x from 2^-103 on: below, the remainders can leave fp32 and
// the results be an ulp off (a v of 2^-103 is that of gradients of 10^-15).  A code depends on
// the last bit of what it rounds, and so does the next step; with these the codes are
// the formula's, operation by operation, in IEEE arithmetic, but for what is named here.
__device__ __forceinline__ float exact_root(float x) {
  const float s = __builtin_amdgcn_sqrtf(x);  // within an ulp; at 0, infinity and NaN both comparisons are false
  const float below = __uint_as_float(__float_as_uint(s) - 1u), above = __uint_as_float(__float_as_uint(s) + 1u);
  const float r = fmaf(-below, s, x) <= 0.0f ? below : s;
  return fmaf(-above, s, x) > 0.0f ? above : r;
}
__device__ __forceinline__ float exact_quotient(float x, float s, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, s, x), r, q);
}
// Correctly rounded 1 / s for s of 2^-100 to 2^120 (compared with the division for every
// mantissa); 0 for 0.
__device__ __forceinline__ float exact_reciprocal(float s) {
  const float r = __builtin_amdgcn_rcpf(s);
  return s != 0.0f ? fmaf(fmaf(-s, r, 1.0f), r, r) : 0.0f;
}

// A 32-bit integer hash: Appleby's finaliser (two multiplications between shifts).  The
// elements after a group's first draw from it by Marsaglia's xorshift, 13, 17 and 5.
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t h) {
  h = (h ^ (h >> 16)) * 0x85EBCA6Bu;
  h = (h ^ (h >> 13)) * 0xC2B2AE35u;
  return h ^ (h >> 16);
}
__device__ __forceinline__ float unit16(uint32_t h) { return ((float)(h & 0xFFFFu) + 0.5f) * (1.0f / 65536.0f); }

}  // namespace

// ------------------------------------------------------------------ the step
struct AdamWTable {
  Table<fp8mi_adamw_tensor, kAdamWTensors> tab;
  AdamWHyper h;
  int32_t base;  // index of the first tensor in the caller's array
};
static_assert(sizeof(AdamWTable) <= 4096, "kernel arguments");

// lr, the bias corrections and the step's number, from the host or as
// adamw_advance left them on the device.
struct StepNumbers {
  float lr, step_size, root_scale;
  uint32_t t;
};
__device__ __forceinline__ StepNumbers step_numbers(const AdamWHyper& h) {
  if (h.step_words) {
    const uint32_t* w = h.step_words;
    return {__uint_as_float(w[1]), __uint_as_float(w[2]), __uint_as_float(w[3]), w[0]};
  }
  return {h.lr, h.step_size, h.root_scale, h.t};
}

// A wave's 256 elements from `at` on (below t.n).
template <bool BYTES>
__device__ __forceinline__ void adamw_block(const fp8mi_adamw_tensor& t, const AdamWHyper& h, const StepNumbers& s,
                                            float c, uint32_t key, int64_t at) {
  const int lane = threadIdx.x & 63;
  const int64_t i = at + 4 * lane, left = t.n - i;
  const int n = left < 0 ? 0 : (left < 4 ? (int)left : 4);
  const int gdt = t.grad_dtype, pdt = t.param_dtype;
  void* const wp = t.master ? static_cast<void*>(t.master) : t.param;
  const int wdt = t.master ? (int)kF32 : pdt;
  const Raw4 rg = load4(t.grad, gdt, i, n), rw = load4(wp, wdt, i, n);
  const float decay = 1.0f - s.lr * t.weight_decay, b1 = h.beta1, b2 = h.beta2, a1 = h.one_beta1, a2 = h.one_beta2;
  float g[4], w[4], m[4], v[4];
  if constexpr (BYTES) {
    uint8_t* const mp = static_cast<uint8_t*>(t.exp_avg);
    uint8_t* const vp = static_cast<uint8_t*>(t.exp_avg_sq);
    const int mc = (int)load_codes4(mp, i, n), vc = (int)load_codes4(vp, i, n);
    const float ms = t.exp_avg_scale[at / kBlock], vs = t.exp_avg_sq_scale[at / kBlock];
    widen4(rg, gdt, g);
    widen4(rw, wdt, w);
    const f32x2 m0 = __builtin_amdgcn_cvt_pk_f32_fp8(mc, false), m1 = __builtin_amdgcn_cvt_pk_f32_fp8(mc, true);
    const f32x2 r0 = __builtin_amdgcn_cvt_pk_f32_fp8(vc, false), r1 = __builtin_amdgcn_cvt_pk_f32_fp8(vc, true);
    m[0] = m0[0]; m[1] = m0[1]; m[2] = m1[0]; m[3] = m1[1];  // in units of the block's scale
    float r[4] = {r0[0], r0[1], r1[0], r1[1]};
    uint32_t mm = 0u, rr = 0u;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      {
#pragma clang fp contract(off)
        g[e] = g[e] * c;
        m[e] = b1 * (m[e] * ms) + a1 * g[e];
        const float q = r[e] * vs;
        v[e] = b2 * (q * q) + a2 * g[e] * g[e];
      }
      r[e] = exact_root(v[e]);
      w[e] = fmaf(w[e], decay, -(s.step_size * m[e]) * __builtin_amdgcn_rcpf(fmaf(r[e], s.root_scale, h.eps)));
      mm = umax(mm, __float_as_uint(fabsf(m[e])));
      rr = umax(rr, __float_as_uint(r[e]));
    }
    const float sm = block_scale(__uint_as_float(wave_umax(mm))), sr = block_scale(__uint_as_float(wave_umax(rr)));
    const float im = exact_reciprocal(sm), ir = exact_reciprocal(sr);
    const uint64_t group = (uint64_t)i >> 2;
    uint32_t x = mix32((uint32_t)group ^ key ^ mix32((uint32_t)(group >> 32))) | 1u, cm = 0u, cv = 0u;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      cm |= (round_code(exact_quotient(fabsf(m[e]), sm, im), x & 0xFFFFu) | ((__float_as_uint(m[e]) >> 24) & 0x80u)) << (8 * e);
      float k, f;
      uint32_t code = grid_steps(exact_quotient(r[e], sr, ir), k, f);
      code += unit16(x >> 16) * (2.0f * k + 1.0f) < f * (2.0f * k + f) || (k == 0.0f && f > 0.0f) ? 1u : 0u;
      cv |= code << (8 * e);
      x ^= x << 13;
      x ^= x >> 17;
      x ^= x << 5;
    }
    store_codes4(mp, i, cm, n);
    store_codes4(vp, i, cv, n);
    if (lane == 0) {
      t.exp_avg_scale[at / kBlock] = sm;
      t.exp_avg_sq_scale[at / kBlock] = sr;
    }
  } else {
    const Raw4 rm = load4(t.exp_avg, kF32, i, n), rv = load4(t.exp_avg_sq, kF32, i, n);
    widen4(rg, gdt, g);
    widen4(rw, wdt, w);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      g[e] *= c;
      m[e] = b1 * __uint_as_float(rm.w[e]) + a1 * g[e];
      v[e] = b2 * __uint_as_float(rv.w[e]) + a2 * g[e] * g[e];
      w[e] = w[e] * decay - s.step_size * m[e] / (sqrtf(v[e]) * s.root_scale + h.eps);
    }
    store4(t.exp_avg, kF32, i, m, n);
    store4(t.exp_avg_sq, kF32, i, v, n);
  }
  if (t.master) store4(t.master, kF32, i, w, n);
  store4(t.param, pdt, i, w, n);
}

__global__ void __launch_bounds__(kNT) adamw_kernel(AdamWTable a) {
  const float c = a.h.grad_scale ? *a.h.grad_scale : 1.0f;
  if (!(fabsf(c) <= 3.40282347e38f)) return;  // the step is skipped
  const int wg = (int)blockIdx.x;
  const int k = find_tensor(a.tab, wg);
  const fp8mi_adamw_tensor& t = a.tab.t[k];
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t at = (int64_t)(wg - a.tab.first[k]) * kChunk + wid * kBlock;
  if (at >= t.n) return;
  const StepNumbers s = step_numbers(a.h);
  if (t.state_bits == 8) {
    const uint32_t t32 = (uint32_t)__builtin_amdgcn_readfirstlane((int)s.t);  // scalar hashing
    const uint32_t key = mix32(mix32(mix32(a.h.seed) ^ t32) ^ (uint32_t)(a.base + k));
    adamw_block<true>(t, a.h, s, c, key, at);
  } else {
    adamw_block<false>(t, a.h, s, c, 0u, at);
  }
}

// A step counted on the device: counts it, unless it is skipped, and leaves its
// numbers for the kernel above.
__global__ void adamw_advance(AdamWHyper h, double beta1, double beta2) {
  const float c = h.grad_scale ? *h.grad_scale : 1.0f;
  if (!(fabsf(c) <= 3.40282347e38f)) return;
  const uint32_t t = h.step_words[0] + 1;
  const float lr = h.lr_word ? *h.lr_word : h.lr;
  h.step_words[0] = t;
  h.step_words[1] = __float_as_uint(lr);
  h.step_words[2] = __float_as_uint((float)((double)lr / (1.0 - pow(beta1, (double)t))));
  h.step_words[3] = __float_as_uint((float)(1.0 / sqrt(1.0 - pow(beta2, (double)t))));
}

hipError_t launch_adamw(const fp8mi_adamw_tensor* tensors, int count, const AdamWHyper& h, double beta1, double beta2,
                        hipStream_t st) {
  if (h.step_words) {
    hipLaunchKernelGGL(adamw_advance, dim3(1), dim3(1), 0, st, h, beta1, beta2);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  for (int i = 0; i < count;) {
    AdamWTable a;
    a.h = h;
    a.base = i;
    int64_t wgs = 0;
    int k = 0;
    // a launch ends where the table is full or its grid would pass 2^31 threads (a
    // grid holds fewer than 2^32); an empty tensor takes an entry and no workgroup
    for (; k < kAdamWTensors && i + k < count; ++k) {
      const int64_t need = (tensors[i + k].n + kChunk - 1) / kChunk;
      if (k > 0 && wgs + need > (1 << 23)) break;
      a.tab.t[k] = tensors[i + k];
      a.tab.first[k] = (int32_t)wgs;
      wgs += need;
    }
    a.tab.count = k;
    for (int j = k; j < kAdamWTensors; ++j) a.tab.first[j] = 0;
    if (wgs > 0) {
      hipLaunchKernelGGL(adamw_kernel, dim3((unsigned)wgs), dim3(kNT), 0, st, a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    i += k;
  }
  return hipSuccess;
}

// ------------------------------------------------------------------ the norm of all gradients
// Squares are summed in fp64 from the first addition on (an fp32 sum of squares
// leaves its range at gradients of 1e19), in an order fixed by the sizes alone.
struct NormTable {
  Table<fp8mi_norm_tensor, kNormTensors> tab;
  double* parts;
  int32_t chunk;
};
static_assert(sizeof(NormTable) <= 4096, "kernel arguments");

__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  const int nw = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = red[0];
  for (int i = 1; i < nw; ++i) s += red[i];
  return s;
}

__global__ void __launch_bounds__(kNT) grad_norm_parts(NormTable a) {
  __shared__ double red[kNT / 64];
  const int wg = (int)blockIdx.x;
  const int k = find_tensor(a.tab, wg);
  const fp8mi_norm_tensor& t = a.tab.t[k];
  const int64_t begin = (int64_t)(wg - a.tab.first[k]) * a.chunk;
  const int64_t end = begin + a.chunk < t.n ? begin + a.chunk : t.n;
  double s0 = 0.0, s1 = 0.0;
  constexpr int U = 4;
  for (int64_t i = begin + 4 * threadIdx.x; i < end; i += U * 4 * kNT) {
    Raw4 r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t left = end - (i + u * 4 * kNT);
      r[u] = load4(t.grad, t.dtype, i + u * 4 * kNT, left < 0 ? 0 : (left < 4 ? (int)left : 4));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[4];
      widen4(r[u], t.dtype, f);
      s0 = fma((double)f[0], (double)f[0], s0);
      s1 = fma((double)f[1], (double)f[1], s1);
      s0 = fma((double)f[2], (double)f[2], s0);
      s1 = fma((double)f[3], (double)f[3], s1);
    }
  }
  const double s = block_sum(s0 + s1, red);
  if (threadIdx.x == 0) a.parts[wg] = s;
}

__global__ void __launch_bounds__(1024) grad_norm_finish(const double* parts, int n, float max_norm, float* out,
                                                         float* clip) {
  __shared__ double red[16];
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += 1024) s += parts[i];
  s = block_sum(s, red);
  if (threadIdx.x != 0) return;
  const float norm = (float)sqrt(s);
  if (out) *out = norm;
  if (!clip) return;
  // NaN where the norm is not finite: the step that reads it is skipped
  const float q = max_norm >= 0.0f ? max_norm / (norm + 1e-6f) : 1.0f;
  *clip = norm <= 3.40282347e38f ? fminf(q, 1.0f) : __builtin_nanf("");
}

// Elements per workgroup: 4096 until that gives four workgroups per CU, then
// 32768 (fewer partial sums for the last launch).
static int32_t norm_chunk(int64_t total) { return total <= (int64_t)4096 * 1024 ? 4096 : 32768; }

int64_t grad_norm_workspace_bytes(const fp8mi_norm_tensor* tensors, int count) {
  int64_t total = 0, parts = 0;
  for (int i = 0; i < count; ++i) total += tensors[i].n;
  const int64_t chunk = norm_chunk(total);
  for (int i = 0; i < count; ++i) parts += (tensors[i].n + chunk - 1) / chunk;
  return 8 * parts;
}

hipError_t launch_grad_norm(const fp8mi_norm_tensor* tensors, int count, float max_norm, float* out, float* clip,
                            double* parts, hipStream_t st) {
  int64_t total = 0, done = 0;
  for (int i = 0; i < count; ++i) total += tensors[i].n;
  const int32_t chunk = norm_chunk(total);
  for (int i = 0; i < count;) {
    NormTable a;
    a.parts = parts + done;
    a.chunk = chunk;
    int64_t wgs = 0;
    int k = 0;
    for (; k < kNormTensors && i + k < count; ++k) {
      a.tab.t[k] = tensors[i + k];
      a.tab.first[k] = (int32_t)wgs;
      wgs += (tensors[i + k].n + chunk - 1) / chunk;
    }
    a.tab.count = k;
    for (int j = k; j < kNormTensors; ++j) a.tab.first[j] = 0;
    if (wgs > 0) {
      hipLaunchKernelGGL(grad_norm_parts, dim3((unsigned)wgs), dim3(kNT), 0, st, a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    done += wgs;
    i += k;
  }
  hipLaunchKernelGGL(grad_norm_finish, dim3(1), dim3(1024), 0, st, parts, (int)done, max_norm, out, clip);
  return hipGetLastError();
}

}  // namespace fp8mi
