// The products of the cross entropy over a vocabulary (cross_entropy.hip), on
// mm_tile (mm_fp8_kernel.h) with fp16 operands -- the E4M3 codes' values, which
// fp16 holds exactly -- and epilogues of their own.  The fp8 MFMA cuts products to
// 2^-13 of the largest of eight, always toward zero: 1e-4 of a logit, more than a
// loss in fp32 may lose.  fp16's products of codes are exact and their sums fp32.
//
// The logits' gradient is kept as exp(l - lse) - [target] times kGScale, without the
// rows' loss gradients (they are factors of dA's rows, and of A's rows in dB): in
// [-2^14, 2^14], so that fp16 rounds it by 2^-11 at most and entries below 2^-28 by
// 2^-39, where bf16 would round by 2^-8: a bf16 gradient is then off by its own
// rounding alone (64 x 1000 x 512: 0.0017 of its norm, with a bf16 G 0.0025).
#pragma once
#include "mm_act_kernel.h"

namespace fp8mi {

constexpr float kLn2 = 0.693147180559945309f;
constexpr int kTargetIgnored = -2, kTargetElsewhere = -1;

// Row i's target: a column of the tile [0, n), kTargetElsewhere, or ignored.
__device__ __forceinline__ int64_t load_target(const void* targets, int bits, int64_t i) {
  return bits == 64 ? static_cast<const int64_t*>(targets)[i] : static_cast<const int32_t*>(targets)[i];
}
__device__ __forceinline__ int tile_target(int64_t t, int64_t v0, int64_t n) {
  return t < 0 ? kTargetIgnored : (t >= v0 && t < v0 + n ? (int)(t - v0) : kTargetElsewhere);
}

constexpr float kGScale = 16384.0f;

// With a loss gradient per row, G^T A takes A's rows times theirs over `unit`, the power of
// two that puts the largest |dloss| of the batch into [2^6, 2^7) (448 of that is below
// fp16's 65504).  A row below 2^-14 of the unit, 2^-20 of the largest, would leave fp16's
// normal numbers: up to 2^8 of it go to A's row, and G's row is that much smaller (its
// entries' rounding, 2^-39 of 1 in all, 2^-31 at most) until dA's sums are finished.  So a
// row of 2^-28 of the largest still enters dB with 11 bits of a code of 1.  (Without either
// a row of 10^-8 of the largest was zero in dB up to codes of 4.)
__device__ __forceinline__ float row_lift(float dloss, float unit) {  // 2^0 .. 2^8
  const int e = (int)((__float_as_uint(dloss) >> 23) & 255u) - (int)(__float_as_uint(unit) >> 23);  // exponent of dloss / unit
  const int up = -14 - e;
  return __uint_as_float((uint32_t)(127 + (up < 0 ? 0 : (up > 8 ? 8 : up))) << 23);
}

// A in fp16, B's codes as they are (kOpB; or fp16): fp16 leading dimensions, and K and
// strides of A, in bytes.  Batch z takes bytes z K .. of a row-major A's rows (the last
// batch fewer), and the rows z K / 2 .. of a K-major operand's k_major_rows.
struct Mm16Args : MmArgs {
  static constexpr int kOpB = kOpCodes;
  int64_t k_total = 0, k_major_rows = 0;
  __host__ __device__ static int64_t k_bytes(const Mm16Args& p, int64_t bz) {
    const int64_t left = p.k_total - bz * p.K;
    return left < p.K ? left : p.K;
  }
  __host__ __device__ static int64_t k_rows(const Mm16Args& p, int64_t bz) {
    const int64_t left = p.k_major_rows - bz * (p.K / 2);
    return left < p.K / 2 ? left : p.K / 2;
  }
  __host__ __device__ static float out_scale(const Mm16Args&, float sab) { return sab * (1.0f / kGScale); }
};

// What the logits' epilogues share: scales, targets, the piece's first column.
struct XentArgs : Mm16Args {
  static constexpr bool kTail = true;
  int a_rows = 0, b_rows = 0;
  const void* targets = nullptr;
  int target_bits = 64;
  int64_t v0 = 0, vocab = 0;
  int64_t tile0 = 0;                // tiles of columns in the pieces before
  // statistics
  float2* parts = nullptr;          // [tiles of columns][M]: (largest, sum of exponentials), in powers of two
  float* target_logit = nullptr;    // [M], in powers of two
  // gradient
  const float* lse = nullptr;       // [M]
  uint16_t* d = nullptr;            // fp16 [M, ld_d]
  int64_t ld_d = 0;
  const float* dloss = nullptr;     // [M] where rows have their own (row_lift), else null
  const float* unit = nullptr;
  __device__ static __forceinline__ float g_scale(const XentArgs& p, int64_t row) {
    return p.dloss ? kGScale / row_lift(p.dloss[row], *p.unit) : kGScale;
  }

  struct Rows {
    float col = 1.0f, row = 1.0f, scale = kGScale;
    int target = kTargetElsewhere;
  };
  template <int BM, int BN> static constexpr int extra_bytes() { return 4 * BN + 12 * BM; }
  template <int BM, int BN, bool GRAD>
  __device__ static __forceinline__ void fetch_rows(const XentArgs& p, Rows& r, int tid, int64_t m0, int64_t n0) {
    if (p.b_scale_inv && tid < BN) r.col = p.b_scale_inv[p.b_rows ? (n0 + tid < p.N ? n0 + tid : n0) : 0];
    if (tid >= BM || m0 + tid >= p.M) return;
    const int64_t t = load_target(p.targets, p.target_bits, m0 + tid);
    r.target = tile_target(t, p.v0 + n0, p.N - n0 < BN ? p.N - n0 : BN);
    if constexpr (GRAD) {
      r.row = t < p.vocab ? p.lse[m0 + tid] * kLog2e : __builtin_nanf("");
      r.scale = g_scale(p, m0 + tid);
    } else {
      if (p.a_rows) r.row = p.a_scale_inv[m0 + tid];
    }
  }
  // extra: column scales [BN], row words [BM], targets [BM], G's scales [BM]
  template <int BM, int BN> __device__ static __forceinline__ void park(const XentArgs&, const Rows& r, int tid, uint8_t* extra) {
    float* f = reinterpret_cast<float*>(extra);
    if (tid < BN) f[tid] = r.col;
    if (tid < BM) {
      f[BN + tid] = r.row;
      reinterpret_cast<int*>(f)[BN + BM + tid] = r.target;
      f[BN + 2 * BM + tid] = r.scale;
    }
  }
};

template <int C> __device__ __forceinline__ void pack_f16(uint32_t (&w)[C / 2], const float (&f)[C]) {
#pragma unroll
  for (int e = 0; e < C; e += 2) {
    const f32x2 v = {f[e], f[e + 1]};
    w[e / 2] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
  }
}

// A logit in powers of two is acc * (sa_i sb_j log2 e).
__device__ __forceinline__ float logit_scale(const XentArgs& p) {
  return kLog2e * (p.a_scale_inv && !p.a_rows ? *p.a_scale_inv : 1.0f);
}

// Statistics of each row over the tile's columns: lanes, then waves, through LDS.
struct XentLseArgs : XentArgs {
  template <int BM, int BN>
  __device__ static __forceinline__ void fetch(const XentArgs& p, Rows& r, int tid, int64_t m0, int64_t n0) {
    fetch_rows<BM, BN, false>(p, r, tid, m0, n0);
  }
  template <int BM, int BN, int WAVES_M, int WAVES_N, int TI, int TJ>
  __device__ static __forceinline__ void tail(const XentLseArgs& p, const v4f (&acc)[TI][TJ], uint8_t* pool,
                                              const uint8_t* extra, int64_t m0, int64_t n0, int64_t) {
    constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N, PAIRS = 4 * WAVES_N, LD = PAIRS + 1;
    static_assert(BM * LD * 8 <= 64 * 1024 && BM <= 64 * WAVES_M * WAVES_N, "pairs fit the stages");
    float2* const pairs = reinterpret_cast<float2*>(pool);
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wid / WAVES_N, wn = wid % WAVES_N;
    const float* const cols = reinterpret_cast<const float*>(extra) + wn * WN;
    const float* const rows = reinterpret_cast<const float*>(extra) + BN;
    const int* const tgt = reinterpret_cast<const int*>(extra) + BN + BM;
    const float s = logit_scale(p);
    const int64_t cl = p.N - n0 - wn * WN;
    const int cols_in = cl < WN ? (int)cl : WN;
    float cs[TJ][4];
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const float4 c = *reinterpret_cast<const float4*>(cols + 16 * j + 4 * g);
      cs[j][0] = s * c.x; cs[j][1] = s * c.y; cs[j][2] = s * c.z; cs[j][3] = s * c.w;
    }
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int lr = wm * WM + 16 * i + r16;
      float t[TJ][4];
      const float ra = rows[lr];
#pragma unroll
      for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) t[j][e] = acc[i][j][e] * (ra * cs[j][e]);
      if (cols_in < WN) {
#pragma unroll
        for (int j = 0; j < TJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (16 * j + 4 * g + e >= cols_in) t[j][e] = -__builtin_inff();
      }
      const int own = tgt[lr] - wn * WN;
      if (own >= 0 && own < WN && ((own >> 2) & 3) == g) {
#pragma unroll
        for (int j = 0; j < TJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (own == 16 * j + 4 * g + e) p.target_logit[m0 + lr] = t[j][e];
      }
      float m = t[0][0];
#pragma unroll
      for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) m = fmaxf(m, t[j][e]);
      const float ref = m > -3.0e38f ? m : 0.0f;  // nothing but columns past the edge: a sum of zeros
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += __builtin_amdgcn_exp2f(t[j][e] - ref);
      pairs[lr * LD + wn * 4 + g] = make_float2(m, sum);
    }
    __syncthreads();
    if (tid < BM && m0 + tid < p.M) {
      float2 q[PAIRS];
      float m = -__builtin_inff(), sum = 0.0f;
#pragma unroll
      for (int k = 0; k < PAIRS; ++k) {
        q[k] = pairs[tid * LD + k];
        m = fmaxf(m, q[k].x);
      }
      const float ref = m > -3.0e38f ? m : 0.0f;
#pragma unroll
      for (int k = 0; k < PAIRS; ++k) sum += q[k].y * __builtin_amdgcn_exp2f(q[k].x - ref);
      p.parts[(p.tile0 + n0 / BN) * p.M + m0 + tid] = make_float2(m, sum);
    }
  }
};

// g_scale (exp(l - lse) - [target]) in fp16, rows of the gradient's two products.
struct XentGradArgs : XentArgs {
  template <int BM, int BN>
  __device__ static __forceinline__ void fetch(const XentArgs& p, Rows& r, int tid, int64_t m0, int64_t n0) {
    fetch_rows<BM, BN, true>(p, r, tid, m0, n0);
  }
  template <int BM, int BN, int WAVES_M, int WAVES_N, int TI, int TJ>
  __device__ static __forceinline__ void tail(const XentGradArgs& p, const v4f (&acc)[TI][TJ], uint8_t*,
                                              const uint8_t* extra, int64_t m0, int64_t n0, int64_t) {
    constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N, C = pair_cols(TJ), NP = strip_pairs(TJ);
    constexpr bool STREAM = BM * BN == 256 * 256;  // G is larger than the L2 there
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wid / WAVES_N, wn = wid % WAVES_N;
    const float* const rows = reinterpret_cast<const float*>(extra) + BN;
    const int* const tgt = reinterpret_cast<const int*>(extra) + BN + BM;
    const float s = logit_scale(p) * (p.b_scale_inv ? *p.b_scale_inv : 1.0f);
    // whole groups of eight columns are written: those past the vocabulary as zeros
    const int64_t cl = p.N - n0 - wn * WN;
    const int cols_in = cl < WN ? (int)cl : WN;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int lr = wm * WM + 16 * i + r16;
      const bool in = m0 + lr < p.M;
      const float lse = rows[lr], scale = rows[2 * BM + lr];
      const int own = tgt[lr] - wn * WN;
      const bool ignored = tgt[lr] == kTargetIgnored;
      uint16_t* const out = p.d + (m0 + lr) * p.ld_d + n0 + wn * WN;
#pragma unroll
      for (int c = 0; c < NP; ++c) {
        float t[C];
        lane_columns<TJ>(acc[i], c, t);
        const int at = lane_column<TJ>(g, c);
#pragma unroll
        for (int e = 0; e < C; ++e) {
          float q = __builtin_amdgcn_exp2f(fmaf(t[e], s, -lse));
          if (own == at + e) q -= 1.0f;
          t[e] = ignored ? 0.0f : q * scale;
        }
        if (cols_in < WN) {
#pragma unroll
          for (int e = 0; e < C; ++e)
            if (at + e >= cols_in) t[e] = 0.0f;
        }
        if (in && (at & ~7) < cols_in) {
          uint32_t w[C / 2];
          pack_f16<C>(w, t);
          store_words<C / 2, 2, STREAM>(reinterpret_cast<uint8_t*>(out + at), w, C);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// G^T A: both operands K-major in fp16, the plain epilogue.
struct KmArgs : Mm16Args {
  static constexpr int kOpB = kOpF16;
};

// What becomes of a gradient's sums: bf16(scale by_i / kGScale * sum), 0 in ignored rows
// (without targets there are none); with `unit` by_i are loss gradients whose rows of G
// row_lift made smaller.
struct Finish {
  uint16_t* out = nullptr;
  int64_t ld = 0;
  const float* scale = nullptr;  // one word, or none
  const float* by = nullptr;     // one word, or one per row
  const float* unit = nullptr;
  int by_rows = 0, target_bits = 0;
  const void* targets = nullptr;
};
__device__ __forceinline__ bool finish_row(const Finish& f, int64_t row, float& factor) {
  const float by = f.by[f.by_rows ? row : 0], lift = f.unit ? row_lift(by, *f.unit) : 1.0f;
  factor = (f.scale ? *f.scale : 1.0f) * (by * (lift / kGScale));
  return !f.targets || load_target(f.targets, f.target_bits, row) >= 0;
}
__device__ __forceinline__ void finish4(const Finish& f, int64_t row, int64_t col, v4f v, bool counted, float factor) {
  v = counted ? v * factor : v4f{0.0f, 0.0f, 0.0f, 0.0f};
  const uint2 w = bf16x4_rne(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<u32x2_any*>(f.out + row * f.ld + col) = u32x2_any{w.x, w.y};
}

// fp32 sums over several launches and K splits: out[z] (+)= A B^T, N % 16 == 0; without
// `sums` they are all of it and finished here.
template <int B> struct SumArgs : Mm16Args {
  static constexpr int kOpB = B;
  static constexpr bool kTail = true;
  float* sums = nullptr;  // [batch][M, N]
  int first = 0;
  Finish fin;
  template <int BM, int BN> static constexpr int extra_bytes() { return 0; }
  template <int BM, int BN> __device__ static __forceinline__ void fetch(const SumArgs&, Rows&, int, int64_t, int64_t) {}
  template <int BM, int BN> __device__ static __forceinline__ void park(const SumArgs&, const Rows&, int, uint8_t*) {}
  template <int BM, int BN, int WAVES_M, int WAVES_N, int TI, int TJ>
  __device__ static __forceinline__ void tail(const SumArgs& p, const v4f (&acc)[TI][TJ], uint8_t*, const uint8_t*,
                                              int64_t m0, int64_t n0, int64_t bz) {
    constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wid / WAVES_N, wn = wid % WAVES_N;
    const int64_t cl = p.N - n0 - wn * WN;
    const int cols_in = cl < WN ? (int)cl : WN;
    if (!p.sums) {
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        const int64_t row = m0 + wm * WM + 16 * i + r16;
        if (row >= p.M) continue;
        float factor;
        const bool counted = finish_row(p.fin, row, factor);
#pragma unroll
        for (int j = 0; j < TJ; ++j)
          if (16 * j < cols_in) finish4(p.fin, row, n0 + wn * WN + 16 * j + 4 * g, acc[i][j], counted, factor);
      }
      return;
    }
    float* const base = p.sums + bz * p.M * p.N + n0 + wn * WN + 4 * g;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int64_t row = m0 + wm * WM + 16 * i + r16;
      if (row >= p.M) continue;
      float* const out = base + row * p.N;
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        if (16 * j >= cols_in) continue;
        v4f v = acc[i][j];
        v4f* const q = reinterpret_cast<v4f*>(out + 16 * j);
        if (!p.first) v += *q;
        *q = v;
      }
    }
  }
};

using AddArgs = SumArgs<kOpCodes>;   // G by rows, the codes K-major
using KmSumArgs = SumArgs<kOpF16>;   // both K-major in fp16

template <int BM, int BN, int WM_, int WN_, int MINB, int LAY, int DEEP, class P>
static hipError_t launch_mm16_tile(const P& p0, hipStream_t st) {
  const int64_t tiles_m = (p0.M + BM - 1) / BM, tiles_n = (p0.N + BN - 1) / BN;
  P p = p0;
  // several rounds of tiles, or long sums (a K split of G B is 128 steps and more: 237 -> 214 us)
  p.early_loads = tiles_m * tiles_n * p0.batch > (int64_t)device_cu_count() || p0.K >= 64 * kBK;
  hipLaunchKernelGGL((mm_fp8_dma<kOpF16, P::kOpB, BM, BN, WM_, WN_, MINB, -1, LAY, false, DEEP, P>),
                     dim3((unsigned)(tiles_m * tiles_n), 1, (unsigned)p0.batch), dim3(64 * WM_ * WN_), 0, st, p, tiles_m,
                     tiles_n, 4);
  return hipGetLastError();
}

// Tiles as pick_tile's: 256 x 256, or 256 x 192 where that needs less time, from
// 60% of the CUs on, below that 128 x 128, then 64 x 64 (whose eight-stage form is no
// faster here: 64 x 1000 x 512 logits 7.7 against 8.0 us, G B 6.8 against 6.3).  The
// gradients' products (`narrow`) of up to 128 rows take 128 x 128 at most: G B of 6 x 21489
// x 2976 26.5 -> 22.0.
static inline int pick16(int64_t M, int64_t N, int64_t batch, bool narrow) {
  // of an MI355X, not of the current device: the workspace's size goes by the tiles
  constexpr int64_t ncu = 256;
  const int64_t tm = (M + 255) / 256;
  const int64_t t256 = tm * ((N + 255) / 256) * batch, t192 = tm * ((N + 191) / 192) * batch;
  if ((!narrow || M > 128) && (10 * t256 >= 6 * ncu || (narrow && 10 * t192 >= 6 * ncu))) {
    if (!narrow) return 256;
    return (t192 + ncu - 1) / ncu * 230 < (t256 + ncu - 1) / ncu * 256 ? 192 : 256;
  }
  return ((M + 127) / 128) * ((N + 127) / 128) * batch >= ncu / 2 ? 128 : 64;
}

// one epilogue each
hipError_t launch_xent_lse(const XentLseArgs& p, hipStream_t st);
hipError_t launch_xent_grad(const XentGradArgs& p, hipStream_t st);
// G B, and G^T A straight to its rows or, in K splits, into fp32 sums; any may be null.
hipError_t launch_mm16_grads(const AddArgs* add, const KmArgs* km, const KmSumArgs* km_sums, hipStream_t st);
int64_t xent_lse_tile(int64_t M, int64_t N);  // columns that share a row's statistics

}  // namespace fp8mi
