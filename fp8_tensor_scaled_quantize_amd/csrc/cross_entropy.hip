// Softmax cross entropy over a vocabulary from E4M3 codes, and its gradient,
// without keeping the logits.
//
//   l_ij = sa_i sb_j sum_k A_ik B_jk        lse_i = log sum_j exp l_ij
//   loss_i = lse_i - l_{i, t_i}
//   G_ij = d_i (exp(l_ij - lse_i) - [j = t_i])   dA = sb G B   dB = sa G^T A
//
// The vocabulary is taken in pieces.  Forward: a piece's codes become bf16 (their
// exact values) in the workspace, and the product's epilogue (xent_mm.h) leaves
// each row's largest logit and sum of exponentials per tile of columns; one more
// kernel joins them.  Backward: the piece's logits once more, G in bf16, then
// G B into fp32 sums and G^T A straight to its rows of dB.  So 2 M N K flop forward
// and 6 M N K backward, at bf16's rate; what is written besides is M times a
// piece's columns.
#include "xent_mm.h"

namespace fp8mi {

namespace {

constexpr int64_t kPieceElements = (int64_t)64 << 20;  // of a piece's weights or of G: 128 MiB in bf16, half the last-level cache

int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Columns of a piece, a multiple of 256: so many that neither the piece's weights
// nor (with rows) its G are above kPieceElements.
int64_t piece_columns(int64_t N, int64_t K, int64_t rows) {
  const int64_t most = kPieceElements / (K > rows ? K : rows);
  const int64_t p = most < 256 ? 256 : (most > (1 << 20) ? 1 << 20 : most / 256 * 256);
  const int64_t all = up(N, 256);
  return p < all ? p : all;
}

struct Carve {
  int64_t at = 0;
  int64_t take(int64_t bytes) {
    const int64_t r = at;
    at += up(bytes, 256);
    return r;
  }
};

struct ForwardPlan {
  int64_t cols, tile, parts, logit, a16, b16, bytes;
  ForwardPlan(int64_t M, int64_t N, int64_t K) {
    Carve c;
    cols = piece_columns(N, K, 0);
    tile = xent_lse_tile(M, N);
    parts = c.take((N + tile - 1) / tile * M * 8);
    logit = c.take(M * 4);
    a16 = c.take(M * K * 2);
    b16 = c.take(cols * K * 2);
    bytes = c.at;
  }
};

struct BackwardPlan {
  int64_t cols, splits, ld_t, a16, at16, b16, bt16, g, sums, bytes;
  BackwardPlan(int64_t M, int64_t N, int64_t K) {
    Carve c;
    cols = piece_columns(N, K, M);
    // K splits of G B: about a tile for each of 256 CUs, steps of at least 512 columns
    const int64_t tiles = (M + 255) / 256 * ((K + 191) / 192);
    splits = 256 / tiles;
    if (splits > cols / 512) splits = cols / 512;
    if (splits < 1) splits = 1;
    ld_t = up(M, 8);
    a16 = c.take(M * K * 2);
    at16 = c.take(K * ld_t * 2);
    b16 = c.take(cols * K * 2);
    bt16 = c.take(K * cols * 2);
    g = c.take(M * cols * 2);
    sums = c.take(splits * M * K * 4);
    bytes = c.at;
  }
};

// Codes [R, C] as bf16 [R, C] (or null) and transposed, [C, ld_t] (or null) with
// zeros up to a multiple of 8 rows.  A workgroup takes 64 x 64.  C % 16 == 0.
__global__ void __launch_bounds__(256) widen_codes(const uint8_t* x, int64_t ld, int64_t R, int64_t C, uint16_t* out,
                                                   uint16_t* out_t, int64_t ld_t) {
  __shared__ uint32_t tile[64][33];  // two columns per word
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const int tid = threadIdx.x, r = tid >> 2, c = 16 * (tid & 3);
  const int64_t r0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
  u32x4 v = {0u, 0u, 0u, 0u};
  const bool in = r0 + r < R && c0 + c < C;
  if (in) v = *reinterpret_cast<const u32x4*>(x + (r0 + r) * ld + c0 + c);
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    w[2 * e] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[e], 1.0f, false));
    w[2 * e + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[e], 1.0f, true));
  }
  if (out && in) {
    u32x4* q = reinterpret_cast<u32x4*>(out + (r0 + r) * C + c0 + c);
    q[0] = u32x4{w[0], w[1], w[2], w[3]};
    q[1] = u32x4{w[4], w[5], w[6], w[7]};
  }
  if (!out_t) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) tile[r][c / 2 + e] = w[e];
  __syncthreads();
  // thread: column tid / 4, rows 16 (tid % 4) .. + 15, in two groups of eight
  const int col = tid >> 2, rr = 16 * (tid & 3);
  if (c0 + col >= C) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t row = r0 + rr + 8 * h;
    if (row >= R) break;
    u32x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = tile[rr + 8 * h + 2 * e][col >> 1] >> (16 * (col & 1)) & 0xFFFFu;
      const uint32_t hi = tile[rr + 8 * h + 2 * e + 1][col >> 1] >> (16 * (col & 1)) & 0xFFFFu;
      o[e] = lo | (hi << 16);
    }
    *reinterpret_cast<u32x4*>(out_t + (c0 + col) * ld_t + row) = o;
  }
}

hipError_t launch_widen(const uint8_t* x, int64_t ld, int64_t R, int64_t C, uint16_t* out, uint16_t* out_t, int64_t ld_t,
                        hipStream_t st) {
  hipLaunchKernelGGL(widen_codes, dim3((unsigned)((C + 63) / 64), (unsigned)((R + 63) / 64)), dim3(256), 0, st, x, ld, R, C,
                     out, out_t, ld_t);
  return hipGetLastError();
}

// Joins the statistics of `tiles` column tiles: a workgroup takes RB rows, its
// threads 256 / RB segments of the tiles.
template <int RB>
__global__ void __launch_bounds__(256) xent_join(const float2* parts, int64_t tiles, int64_t M, const float* logit,
                                                 const void* targets, int bits, int64_t vocab, float* loss, float* lse) {
  constexpr int SEG = 256 / RB;
  __shared__ float2 red[SEG][RB + 1];
  const int r = threadIdx.x % RB, seg = threadIdx.x / RB;
  const int64_t row = (int64_t)blockIdx.x * RB + r;
  float m = -__builtin_inff(), s = 0.0f;
  if (row < M) {
    constexpr int U = 8;
    for (int64_t t = seg; t < tiles; t += U * SEG) {
      float2 q[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        q[u] = t + u * SEG < tiles ? parts[(t + u * SEG) * M + row] : make_float2(-__builtin_inff(), 0.0f);
      float top = m;
#pragma unroll
      for (int u = 0; u < U; ++u) top = fmaxf(top, q[u].x);
      const float ref = top > -3.0e38f ? top : 0.0f;
      s *= __builtin_amdgcn_exp2f(m - ref);
#pragma unroll
      for (int u = 0; u < U; ++u) s += q[u].y * __builtin_amdgcn_exp2f(q[u].x - ref);
      m = top;
    }
  }
  red[seg][r] = make_float2(m, s);
  __syncthreads();
  if (seg != 0 || row >= M) return;
  for (int k = 0; k < SEG; ++k) m = fmaxf(m, red[k][r].x);
  const float ref = m > -3.0e38f ? m : 0.0f;
  s = 0.0f;
  for (int k = 0; k < SEG; ++k) s += red[k][r].y * __builtin_amdgcn_exp2f(red[k][r].x - ref);
  const float l2 = ref + log2f(s);
  const int64_t t = load_target(targets, bits, row);
  lse[row] = l2 * kLn2;
  loss[row] = t < 0 ? 0.0f : (t < vocab ? (l2 - logit[row]) * kLn2 : __builtin_nanf(""));
}

// The mean over the counted rows and 1 / their number (zeros without any), in fp64
// in a fixed order.
__global__ void __launch_bounds__(1024) xent_mean(const float* loss, const void* targets, int bits, int64_t M, float* out) {
  __shared__ double sums[16];
  __shared__ int64_t counts[16];
  double s = 0.0;
  int64_t n = 0;
  for (int64_t i = threadIdx.x; i < M; i += 1024) {
    s += (double)loss[i];  // 0 where the row is ignored
    n += load_target(targets, bits, i) >= 0;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    s += __shfl_xor(s, off, 64);
    n += __shfl_xor(n, off, 64);
  }
  if ((threadIdx.x & 63) == 0) {
    sums[threadIdx.x >> 6] = s;
    counts[threadIdx.x >> 6] = n;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int k = 1; k < 16; ++k) {
    s += sums[k];
    n += counts[k];
  }
  out[0] = n > 0 ? (float)(s / (double)n) : 0.0f;
  out[1] = n > 0 ? (float)(1.0 / (double)n) : 0.0f;
}

// dA = bf16(sb * the splits' sums), in their order.  K % 16 == 0.
__global__ void __launch_bounds__(256) xent_finish_da(const float* sums, int64_t splits, int64_t M, int64_t K,
                                                      const float* sb, uint16_t* da, int64_t ld) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= M * K) return;
  v4f v = *reinterpret_cast<const v4f*>(sums + i);
  for (int64_t z = 1; z < splits; ++z) v += *reinterpret_cast<const v4f*>(sums + z * M * K + i);
  v *= sb ? *sb : 1.0f;
  const uint2 w = bf16x4_rne(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<u32x2_any*>(da + i / K * ld + i % K) = u32x2_any{w.x, w.y};
}

__global__ void __launch_bounds__(256) zero_rows(uint16_t* p, int64_t rows, int64_t cols, int64_t ld) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int64_t c = threadIdx.x; c < cols; c += 256) p[r * ld + c] = 0;
}

#define FP8MI_TRY(x)                     \
  do {                                   \
    const hipError_t e = (x);            \
    if (e != hipSuccess) return e;       \
  } while (0)

void fill_logits(XentArgs& p, const XentCall& c, const uint16_t* a16, const uint16_t* b16, int64_t v0, int64_t n) {
  p.a = reinterpret_cast<const uint8_t*>(a16);
  p.b = reinterpret_cast<const uint8_t*>(b16);
  p.lda = p.ldb = p.K = p.k_total = 2 * c.K;
  p.M = c.M; p.N = n; p.batch = 1;
  p.a_scale_inv = c.a_scale_inv; p.b_scale_inv = c.b_scale_inv && c.b_rows ? c.b_scale_inv + v0 : c.b_scale_inv;
  p.a_rows = c.a_rows; p.b_rows = c.b_rows;
  p.targets = c.targets; p.target_bits = c.target_bits; p.v0 = v0; p.vocab = c.N;
}

}  // namespace

int64_t xent_workspace_bytes(int64_t M, int64_t N, int64_t K) { return ForwardPlan(M, N, K).bytes; }
int64_t xent_grad_workspace_bytes(int64_t M, int64_t N, int64_t K) { return BackwardPlan(M, N, K).bytes; }

hipError_t launch_xent_forward(const XentCall& c, hipStream_t st) {
  if (c.M > 0) {
    const ForwardPlan plan(c.M, c.N, c.K);
    uint16_t* const a16 = reinterpret_cast<uint16_t*>(c.ws + plan.a16);
    uint16_t* const b16 = reinterpret_cast<uint16_t*>(c.ws + plan.b16);
    float2* const parts = reinterpret_cast<float2*>(c.ws + plan.parts);
    float* const logit = reinterpret_cast<float*>(c.ws + plan.logit);
    FP8MI_TRY(launch_widen(c.a, c.lda, c.M, c.K, a16, nullptr, 0, st));
    for (int64_t v0 = 0; v0 < c.N; v0 += plan.cols) {
      const int64_t n = c.N - v0 < plan.cols ? c.N - v0 : plan.cols;
      FP8MI_TRY(launch_widen(c.b + v0 * c.ldb, c.ldb, n, c.K, b16, nullptr, 0, st));
      XentLseArgs p;
      fill_logits(p, c, a16, b16, v0, n);
      p.parts = parts;
      p.target_logit = logit;
      FP8MI_TRY(launch_xent_lse(p, st));
    }
    const int64_t tiles = (c.N + plan.tile - 1) / plan.tile;
    const auto join = [&](auto kernel, int rb) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)((c.M + rb - 1) / rb)), dim3(256), 0, st, parts, tiles, c.M, logit,
                         c.targets, c.target_bits, c.N, c.loss, c.lse);
      return hipGetLastError();
    };
    // rows share a workgroup while that leaves enough workgroups
    FP8MI_TRY(c.M >= 4096 ? join(xent_join<16>, 16) : c.M >= 512 ? join(xent_join<4>, 4) : join(xent_join<1>, 1));
  }
  if (!c.mean) return hipSuccess;
  hipLaunchKernelGGL(xent_mean, dim3(1), dim3(1024), 0, st, c.loss, c.targets, c.target_bits, c.M, c.mean);
  return hipGetLastError();
}

hipError_t launch_xent_backward(const XentCall& c, hipStream_t st) {
  if (c.M == 0) {
    if (!c.db) return hipSuccess;
    hipLaunchKernelGGL(zero_rows, dim3((unsigned)(c.N < 65536 ? c.N : 65536)), dim3(256), 0, st, c.db, c.N, c.K, c.ld_db);
    return hipGetLastError();
  }
  const BackwardPlan plan(c.M, c.N, c.K);
  const auto at = [&](int64_t off) { return reinterpret_cast<uint16_t*>(c.ws + off); };
  float* const sums = reinterpret_cast<float*>(c.ws + plan.sums);
  FP8MI_TRY(launch_widen(c.a, c.lda, c.M, c.K, at(plan.a16), c.db ? at(plan.at16) : nullptr, plan.ld_t, st));
  // bytes of G's rows per K split, from the first piece (no later one is wider):
  // whole 128-byte steps, so that every split starts on a chunk
  const int64_t first_cols = up(c.N < plan.cols ? c.N : plan.cols, 8);
  const int64_t k_split = up((2 * first_cols + plan.splits - 1) / plan.splits, 128);
  const int64_t splits = (2 * first_cols + k_split - 1) / k_split;
  for (int64_t v0 = 0; v0 < c.N; v0 += plan.cols) {
    const int64_t n = c.N - v0 < plan.cols ? c.N - v0 : plan.cols;
    FP8MI_TRY(launch_widen(c.b + v0 * c.ldb, c.ldb, n, c.K, at(plan.b16), c.da ? at(plan.bt16) : nullptr, plan.cols, st));
    XentGradArgs g;
    fill_logits(g, c, at(plan.a16), at(plan.b16), v0, n);
    g.lse = c.lse;
    g.dloss = c.dloss; g.dloss_rows = c.dloss_rows;
    g.d = at(plan.g); g.ld_d = plan.cols;
    FP8MI_TRY(launch_xent_grad(g, st));
    if (c.da) {
      AddArgs p;
      p.a = reinterpret_cast<const uint8_t*>(at(plan.g));
      p.b = reinterpret_cast<const uint8_t*>(at(plan.bt16));
      p.lda = p.ldb = 2 * plan.cols;
      p.M = c.M; p.N = c.K;
      p.k_total = 2 * up(n, 8);
      p.K = k_split;
      p.batch = (p.k_total + k_split - 1) / k_split;
      p.stride_a = p.stride_b = p.K;
      p.sums = sums;
      p.first = v0 == 0;
      FP8MI_TRY(launch_mm16_add(p, st));
    }
    if (c.db) {
      Mm16KmArgs p;
      p.a = reinterpret_cast<const uint8_t*>(at(plan.g));
      p.b = reinterpret_cast<const uint8_t*>(at(plan.at16));
      p.lda = 2 * plan.cols; p.ldb = 2 * plan.ld_t;
      p.M = n; p.N = c.K; p.batch = 1;
      p.K = p.k_total = 2 * plan.ld_t;
      p.k_major_rows = c.M;
      p.a_scale_inv = c.a_scale_inv;
      p.c = c.db + v0 * c.ld_db; p.ldc = c.ld_db; p.stride_c = 0;
      FP8MI_TRY(launch_mm16_km(p, st));
    }
  }
  if (!c.da) return hipSuccess;
  hipLaunchKernelGGL(xent_finish_da, dim3((unsigned)((c.M * c.K / 4 + 255) / 256)), dim3(256), 0, st, sums, splits, c.M,
                     c.K, c.b_scale_inv, c.da, c.ld_da);
  return hipGetLastError();
}

}  // namespace fp8mi
