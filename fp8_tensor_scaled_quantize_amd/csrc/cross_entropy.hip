// Softmax cross entropy over a vocabulary from E4M3 codes, and its gradient,
// without keeping the logits.
//
//   l_ij = sa_i sb_j sum_k A_ik B_jk        lse_i = log sum_j exp l_ij
//   loss_i = lse_i - l_{i, t_i}
//   G_ij = d_i (exp(l_ij - lse_i) - [j = t_i])   dA = sb G B   dB = sa G^T A
//
// The products are fp16's: A's codes become fp16 (their exact values) in the
// workspace, B's as a tile's fragments are read from LDS (v_cvt_scalef32 beside the
// MFMAs: 4096 x 65536 x 1536 658 -> 683 us, where writing them out first took 55, and
// 333 x 50001 x 1536 76 -> 79 against 37).  Forward: the product's epilogue
// (xent_mm.h) leaves each row's largest logit and sum of exponentials per tile of
// columns, and one more kernel joins them.  Backward, the vocabulary in pieces: the
// piece's logits once more, G / d in fp16, then G B into fp32 sums and G^T A straight
// to its rows of dB.  So 2 M N K flop forward and 6 M N K backward, at 16 bits' rate;
// what is written besides is M times a piece's columns.
#include "xent_mm.h"

namespace fp8mi {

namespace {

constexpr int64_t kPieceElements = (int64_t)128 << 20;  // of G: 256 MiB

int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Leading dimension of n fp16 values: rows whose distance is a multiple of 1 KiB
// fall on few of the memory's channels, so such rows get 128 bytes more (4096 x 1536
// x 16384, G B with rows 32 KiB apart: 261 -> 237 us).
int64_t padded(int64_t n) { return n % 512 == 0 ? n + 64 : n; }

// Columns of a piece, a multiple of 256: at most `most`, in pieces of about one size.
int64_t even_pieces(int64_t N, int64_t most) {
  most = most < 256 ? 256 : (most > (1 << 20) ? 1 << 20 : most / 256 * 256);
  const int64_t pieces = (N + most - 1) / most;
  return up((N + pieces - 1) / pieces, 256);
}
// So many that a piece's codes stay within a buffer's 32-bit offsets (ldb <= 2^22).
int64_t offset_columns(int64_t ldb) { return (INT64_C(1) << 30) / ldb; }

struct Carve {
  int64_t at = 0;
  int64_t take(int64_t bytes) {
    const int64_t r = at;
    at += up(bytes, 256);
    return r;
  }
};

// Few rows, or few logits: xent_rows, 64 rows by 16 or 32 columns to a workgroup.
// Graph replay, in tiles -> xent_rows (us): 50001 x 1536 16 rows 53 -> 29, 64 rows 53 -> 53,
// 96 rows 53 -> 79; 32768 x 4096 64 rows 60 -> 60, 96 rows 60 -> 96; 8000 x 1024 96 rows 24 ->
// 23, 192 rows 25 -> 29; 4000 x 1536 192 rows 26 -> 25, 256 rows 26 -> 28; 1000 x 512 512
// rows 23 -> 19.
bool few_rows(int64_t M, int64_t N) { return M <= 64 || M * N <= (3 << 18); }
int64_t rows_tile(int64_t N) { return N >= 8192 ? 32 : 16; }

// Rows of a workgroup of the join: 16 fill the lines that it reads, fewer while there
// are few.
int join_rows(int64_t M) { return M >= 128 ? 16 : (M >= 16 ? 4 : 1); }

struct ForwardPlan {
  int64_t ld, tile, ticket, slots, parts, logit, a16, bytes;
  bool rows;
  ForwardPlan(int64_t M, int64_t N, int64_t K) {
    Carve c;
    rows = few_rows(M, N);
    ld = padded(K);
    tile = rows ? rows_tile(N) : xent_lse_tile(M, N);
    ticket = c.take(4);
    slots = c.take((M + join_rows(M) - 1) / join_rows(M) * 16);
    parts = c.take((N + tile - 1) / tile * M * 8);
    logit = c.take(M * 4);
    a16 = c.take(rows ? 0 : M * ld * 2);
    bytes = c.at;
  }
};

struct BackwardPlan {
  int64_t cols, splits, splits_db, ld, ld_g, unit, a16, a16d, g, sums, sums_db, bytes;
  BackwardPlan(int64_t M, int64_t N, int64_t K) {
    Carve c;
    cols = even_pieces(N, kPieceElements / M);
    // K splits of G B: about a tile for each of 256 CUs, steps of at least 512 columns
    const int64_t tiles = (M + 255) / 256 * ((K + 191) / 192);
    splits = 256 / tiles;
    if (splits > cols / 512) splits = cols / 512;
    // where those fill less than three quarters of the CUs, 256 tiles of 128 x 128, which
    // run beside G^T A's in one round (the gradient of 2000 x 5000 x 256 71 -> 55 us, of 5536
    // x 2680 x 192 84 -> 56)
    const int64_t tiles128 = (M + 127) / 128 * ((K + 127) / 128);
    if (tiles * splits < 192 && splits > 256 / tiles128) splits = 256 / tiles128;
    if (splits < 1) splits = 1;
    // of G^T A over many rows, where a small vocabulary gives few tiles (of 64 x 64, or of
    // 128 x 128 from 64 of those on), to 256 workgroups of at least 512 rows: 3000 x 300 x
    // 512 both products 23.9 -> 11.1 us; the whole gradient of 6000 x 60 x 1024 74 -> 34, of
    // 1500 x 1500 x 768 (144 tiles of 128 x 128 for 72) 60.8 -> 53.7
    const int64_t widest = N < cols ? N : cols, tiles_db = (widest + 63) / 64 * ((K + 63) / 64);
    const int64_t tiles_db128 = (widest + 127) / 128 * ((K + 127) / 128);
    splits_db = tiles_db < 64 ? 256 / tiles_db : (tiles_db128 < 128 ? 256 / tiles_db128 : 1);
    if (splits_db > M / 512) splits_db = M / 512;
    if (splits_db < 1) splits_db = 1;
    ld = padded(K);
    ld_g = padded(cols);
    unit = c.take(4);
    a16 = c.take(M * ld * 2);
    a16d = c.take(M * ld * 2);
    g = c.take(M * ld_g * 2);
    sums = c.take(splits * M * K * 4);
    sums_db = c.take(splits_db > 1 ? splits_db * widest * K * 4 : 0);
    bytes = c.at;
  }
};

// Codes [R, C] as fp16, 32 codes to a thread: C % 16 == 0, whole 16-byte chunks.
// With targets, the rows of ignored ones are zeros (a NaN among their codes would
// reach dB as 0 * NaN); with row factors, out_scaled receives each row times its own.
struct Widen {
  const uint8_t* x;
  uint16_t* out;
  int64_t ld, ld_out, chunks;  // of 16 codes, in all
  int32_t row_chunks;
  int target_bits;
  const void* targets;
  const float* rows;           // [R], in units of *rows_by (row_lift)
  const float* rows_by;
  uint16_t* out_scaled;
};
__device__ __forceinline__ void widen_group(const Widen& m, int64_t group) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const int64_t at = group * 512 + threadIdx.x;
  u32x4 v[2];
  int64_t out[2], row[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t i = at + 256 * u;
    row[u] = i < (1ll << 32) ? (int64_t)((uint32_t)i / (uint32_t)m.row_chunks) : i / m.row_chunks;
    const int64_t c = (i - row[u] * m.row_chunks) * 16;
    out[u] = row[u] * m.ld_out + c;
    if (i < m.chunks) v[u] = *reinterpret_cast<const u32x4*>(m.x + row[u] * m.ld + c);
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    if (at + 256 * u >= m.chunks) return;
    if (m.targets && load_target(m.targets, m.target_bits, row[u]) < 0) v[u] = u32x4{0u, 0u, 0u, 0u};
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[2 * e] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[u][e], 1.0f, false));
      w[2 * e + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[u][e], 1.0f, true));
    }
    u32x4* q = reinterpret_cast<u32x4*>(m.out + out[u]);
    q[0] = u32x4{w[0], w[1], w[2], w[3]};
    q[1] = u32x4{w[4], w[5], w[6], w[7]};
    if (m.out_scaled) {
      const bool counted = load_target(m.targets, m.target_bits, row[u]) >= 0;
      const float d = counted ? m.rows[row[u]] : 0.0f, f = d / *m.rows_by * row_lift(d, *m.rows_by);
      float t[16];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        widen2<kF16>(w[e], t[2 * e], t[2 * e + 1]);
        t[2 * e] *= f;
        t[2 * e + 1] *= f;
      }
      pack_f16<16>(w, t);
      q = reinterpret_cast<u32x4*>(m.out_scaled + out[u]);
      q[0] = u32x4{w[0], w[1], w[2], w[3]};
      q[1] = u32x4{w[4], w[5], w[6], w[7]};
    }
  }
}

__global__ void __launch_bounds__(256) widen_codes(Widen a, uint32_t* ticket) {
  if (ticket && threadIdx.x + blockIdx.x == 0) *ticket = 0u;  // for the join, two launches on
  widen_group(a, blockIdx.x);
}
int64_t widen_groups(const Widen& a) { return (a.chunks + 511) / 512; }

Widen widen(const uint8_t* x, int64_t ld, int64_t R, int64_t C, uint16_t* out, int64_t ld_out) {
  return {x, out, ld, ld_out, R * (C / 16), (int32_t)(C / 16), 0, nullptr, nullptr, nullptr, nullptr};
}
hipError_t launch_widen(const Widen& a, uint32_t* ticket, hipStream_t st) {
  hipLaunchKernelGGL(widen_codes, dim3((unsigned)widen_groups(a)), dim3(256), 0, st, a, ticket);
  return hipGetLastError();
}

// The unit of the rows' loss gradients (row_lift): the power of two that puts the largest
// |dloss| of the counted rows into [2^6, 2^7), 2^-100 at least (a smaller one would leave
// fp32 in dB's factor), 1 where the largest is not finite.
__global__ void __launch_bounds__(1024) dloss_unit(const float* dloss, const void* targets, int bits, int64_t M, float* out) {
  __shared__ float red[16];
  float m = 0.0f;
  constexpr int U = 8;  // rows in flight
  for (int64_t i = threadIdx.x; i < M; i += U * 1024) {
    int64_t t[U];
    float d[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = i + u * 1024;
      t[u] = r < M ? load_target(targets, bits, r) : -1;
      d[u] = r < M ? dloss[r] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (t[u] >= 0) m = __builtin_elementwise_maximum(m, fabsf(d[u]));  // a NaN kept
  }
  for (int off = 32; off > 0; off >>= 1) m = __builtin_elementwise_maximum(m, __shfl_xor(m, off, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int k = 1; k < 16; ++k) m = __builtin_elementwise_maximum(m, red[k]);
  const uint32_t exp = __float_as_uint(m) >> 23;
  *out = exp < 255u ? __uint_as_float((exp < 33u ? 27u : exp - 6u) << 23) : 1.0f;
}

// Few rows (scoring while serving): bound by reading the weights once.  A workgroup
// takes 16 TJ columns of the vocabulary and all rows (16 TI), its four waves every
// fourth K step of 128; the codes come straight from global memory into
// registers, U steps in flight per wave, and become fp16 there (v_cvt_scalef32, 16
// cycles for two values and a wave, is what a wider workgroup saves on the rows').
// Lane group g takes k = 16 g .. + 15 and 64 + 16 g .. + 15 of a step, A and B
// alike, so that a load instruction reads 64 contiguous bytes of a row.  The
// waves' sums meet in LDS, and wave i finishes strip i.  One row of 32768 x 1536: 12 us,
// 4.3 TB/s; 16 rows of 50001 x 1536: 20 us, 3.8 TB/s.  64 rows (45 us) wait for the loads
// of U = 2 steps twice, three waves a SIMD; held to four the compiler spills 100
// registers.
struct RowsGrad {  // what the gradient's form does besides: A in fp16, for the products after it
  static constexpr bool kGrad = true;
  Widen a;
};
struct RowsStats {
  static constexpr bool kGrad = false;
  uint32_t* ticket;
};
template <int TI, int TJ, class G>
__global__ void __launch_bounds__(256) xent_rows(XentArgs p, G extra, uint32_t col_blocks, uint32_t blocks) {
  if constexpr (G::kGrad) {
    if (blockIdx.x >= blocks) {
      widen_group(extra.a, blockIdx.x - blocks);
      return;
    }
  }
  const uint32_t row_block = blockIdx.x / col_blocks, col_block = blockIdx.x % col_blocks;
  const int64_t m0 = (int64_t)row_block * (16 * TI);
  constexpr int NW = 4, U = TI == 4 ? 2 : 3;
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  __shared__ float4 part[NW][TI][TJ][64];
  const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  if constexpr (!G::kGrad) {
    if (tid + blockIdx.x == 0) *extra.ticket = 0u;
  }
  const int64_t n0 = (int64_t)col_block * (16 * TJ);
  // raw buffers: rows past an edge and chunks past K read as zero
  const int64_t a_rows = p.M - m0 < 16 * TI ? p.M - m0 : 16 * TI;
  const int ext_a = (int)((a_rows - 1) * p.lda + p.K);
  const int64_t b_rows = p.N - n0 < 16 * TJ ? p.N - n0 : 16 * TJ;
  const int ext_b = (int)((b_rows - 1) * p.ldb + p.K);
  const auto rsa = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p.a + m0 * p.lda), 0, ext_a, 0x00020000);
  const auto rsb = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p.b + n0 * p.ldb), 0, ext_b, 0x00020000);
  const int K = (int)p.K, steps = (K + kBK - 1) / kBK;
  uint32_t oa[TI], ob[TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
    oa[i] = m0 + 16 * i + r16 < p.M ? (uint32_t)(16 * i + r16) * (uint32_t)p.lda + 16 * g : (uint32_t)ext_a;
#pragma unroll
  for (int j = 0; j < TJ; ++j)
    ob[j] = 16 * j + r16 < b_rows ? (uint32_t)(16 * j + r16) * (uint32_t)p.ldb + 16 * g : (uint32_t)ext_b;
  struct Codes {
    u32x4 h[2];
  };
  auto fetch = [&](__amdgpu_buffer_rsrc_t rs, uint32_t off, int ext, int kt) {
    const int k = kt * kBK + 16 * g;
    Codes c;
    c.h[0] = __builtin_amdgcn_raw_buffer_load_b128(rs, k < K && off < (uint32_t)ext ? off + kt * kBK : ext, 0, 0);
    c.h[1] = __builtin_amdgcn_raw_buffer_load_b128(rs, k + 64 < K && off < (uint32_t)ext ? off + kt * kBK + 64 : ext, 0, 0);
    return c;
  };
  auto widen = [](const Codes& c, v8h (&f)[4]) {  // eight k each
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t x = c.h[q >> 1][2 * (q & 1) + e];
        w[2 * e] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x, 1.0f, false));
        w[2 * e + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x, 1.0f, true));
      }
      f[q] = __builtin_bit_cast(v8h, u32x4{w[0], w[1], w[2], w[3]});
    }
  };
  v4f acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  Codes ca[U][TI], cb[U][TJ];
  auto load = [&](int kt) {  // a step past the end reads nothing (k >= K)
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int j = 0; j < TJ; ++j) cb[u][j] = fetch(rsb, ob[j], ext_b, kt + u * NW);
#pragma unroll
      for (int i = 0; i < TI; ++i) ca[u][i] = fetch(rsa, oa[i], ext_a, kt + u * NW);
    }
    __builtin_amdgcn_sched_barrier(0);  // all in flight before anything waits
  };
  load(wid);
  for (int kt = wid; kt < steps;) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v8h fb[TJ][4];
#pragma unroll
      for (int j = 0; j < TJ; ++j) widen(cb[u][j], fb[j]);
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        v8h fa[4];
        widen(ca[u][i], fa);
#pragma unroll
        for (int j = 0; j < TJ; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[j][q], fa[q], acc[i][j], 0, 0, 0);
      }
    }
    kt += U * NW;
    if (kt < steps) load(kt);
  }
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) part[wid][i][j][lane] = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
  __syncthreads();
  const int64_t row = m0 + 16 * wid + r16;
  if (wid >= TI || m0 + 16 * wid >= p.M) return;
  const bool in = row < p.M;
  const float s = logit_scale(p) * (p.a_rows && in ? p.a_scale_inv[row] : 1.0f);
  const int64_t t = in ? load_target(p.targets, p.target_bits, row) : -1;
  float x[TJ][4], m = -__builtin_inff(), sum = 0.0f;
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    float4 f = part[0][wid][j][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) {
      const float4 q = part[w][wid][j][lane];
      f.x += q.x; f.y += q.y; f.z += q.z; f.w += q.w;
    }
    const float v[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t col = n0 + 16 * j + 4 * g + e;
      const bool has = col < p.N;
      const float sb = p.b_scale_inv ? p.b_scale_inv[p.b_rows ? (has ? col : 0) : 0] : 1.0f;
      x[j][e] = has ? v[e] * (s * sb) : -__builtin_inff();
      if constexpr (!G::kGrad) {
        if (has && in && col == t) p.target_logit[row] = x[j][e];
        m = fmaxf(m, x[j][e]);
      }
    }
  }
  if constexpr (G::kGrad) {  // as XentGradArgs: groups of eight columns, those past the vocabulary as zeros
    if (!in) return;
    const float lse = t < p.vocab ? p.lse[row] * kLog2e : __builtin_nanf(""), scale = XentArgs::g_scale(p, row);
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int64_t at = n0 + 16 * j + 4 * g;
      if ((at & ~(int64_t)7) >= p.N) continue;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float q = __builtin_amdgcn_exp2f(x[j][e] - lse);
        if (p.v0 + at + e == t) q -= 1.0f;
        v[e] = t < 0 || at + e >= p.N ? 0.0f : q * scale;
      }
      uint32_t w[2];
      pack_f16<4>(w, v);
      *reinterpret_cast<uint2*>(p.d + row * p.ld_d + at) = make_uint2(w[0], w[1]);
    }
  } else {
    m = fmaxf(m, __shfl_xor(m, 16, 64));
    m = fmaxf(m, __shfl_xor(m, 32, 64));
    const float ref = m > -3.0e38f ? m : 0.0f;
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += __builtin_amdgcn_exp2f(x[j][e] - ref);
    sum += __shfl_xor(sum, 16, 64);
    sum += __shfl_xor(sum, 32, 64);
    if (g == 0 && in) p.parts[(int64_t)col_block * p.M + row] = make_float2(m, sum);
  }
}

// Joins the statistics of `tiles` column tiles: a workgroup takes RB rows, its
// threads 256 / RB segments of the tiles.  The last workgroup to end adds up the
// mean over the counted rows (and 1 / their number; zeros without any), in fp64 in
// a fixed order: workgroups leave their sums in `slots` ([2 * workgroups], 64 bits)
// by returning device-scope atomics and wait for them before they take a ticket
// (0 before the launch), as the ring's fold does.  (Plain stores behind a
// device-scope fence, whose L2 write-back every workgroup pays for: 29 us instead
// of 8.6 at 4096 rows.)
__device__ __forceinline__ uint64_t swap64(uint64_t* p, uint64_t v) {
  return __hip_atomic_exchange(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <int RB>
__global__ void __launch_bounds__(256) xent_join(const float2* parts, int64_t tiles, int64_t M, const float* logit,
                                                 const void* targets, int bits, int64_t vocab, float* loss, float* lse,
                                                 float* mean, uint32_t* ticket, uint64_t* slots) {
  constexpr int SEG = 256 / RB;
  __shared__ float2 red[SEG][RB + 1];
  const int r = threadIdx.x % RB, seg = threadIdx.x / RB;
  const int64_t row = (int64_t)blockIdx.x * RB + r;
  float m = -__builtin_inff(), s = 0.0f;
  int64_t t = -1;
  float own = 0.0f;
  if (row < M) {
    if (seg == 0) {
      t = load_target(targets, bits, row);
      if (t >= 0 && t < vocab) own = logit[row];
    }
    constexpr int U = 8;
    for (int64_t k = seg; k < tiles; k += U * SEG) {
      float2 q[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        q[u] = k + u * SEG < tiles ? parts[(k + u * SEG) * M + row] : make_float2(-__builtin_inff(), 0.0f);
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
  // halves of the segments join the others, in a fixed order
#pragma unroll
  for (int half = SEG / 2; half > 0; half >>= 1) {
    if (seg < half) {
      const float2 a = red[seg][r], b = red[seg + half][r];
      const float top = fmaxf(a.x, b.x), ref = top > -3.0e38f ? top : 0.0f;
      red[seg][r] = make_float2(top, a.y * __builtin_amdgcn_exp2f(a.x - ref) + b.y * __builtin_amdgcn_exp2f(b.x - ref));
    }
    __syncthreads();
  }
  float l = 0.0f;
  if (seg == 0 && row < M) {
    const float2 all = red[0][r];
    // the loss from the largest logit's distance to the target's, which is exact, not from
    // lse: a loss of 10^-5 beside logits of some hundreds would be lost in lse's rounding
    const float top = all.x > -3.0e38f ? all.x : 0.0f, more = log2f(all.y);
    l = t < 0 ? 0.0f : (t < vocab ? ((top - own) + more) * kLn2 : __builtin_nanf(""));
    lse[row] = (top + more) * kLn2;
    loss[row] = l;
  }
  if (!mean) return;
  __shared__ uint32_t last;
  // rows are in wave 0's first lanes (RB <= 64)
  double total = (double)l;
  uint64_t n = row < M && t >= 0 && seg == 0 ? 1u : 0u;
#pragma unroll
  for (int off = RB / 2; off > 0; off >>= 1) {
    total += __shfl_xor(total, off, 64);
    n += __shfl_xor(n, off, 64);
  }
  if (threadIdx.x == 0) {
    const uint64_t o0 = swap64(slots + 2 * blockIdx.x, __builtin_bit_cast(uint64_t, total));
    const uint64_t o1 = swap64(slots + 2 * blockIdx.x + 1, n);
    asm volatile("" ::"v"(o0), "v"(o1) : "memory");
    wait_vmem();
    last = dev_add(ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  total = 0.0;
  n = 0;
  for (uint32_t i = threadIdx.x; i < gridDim.x; i += 256) {
    total += __builtin_bit_cast(double, __hip_atomic_load(slots + 2 * i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    n += __hip_atomic_load(slots + 2 * i + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    total += __shfl_xor(total, off, 64);
    n += __shfl_xor(n, off, 64);
  }
  __shared__ double sums[4];
  __shared__ uint64_t counts[4];
  if ((threadIdx.x & 63) == 0) {
    sums[threadIdx.x >> 6] = total;
    counts[threadIdx.x >> 6] = n;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int k = 1; k < 4; ++k) {
    total += sums[k];
    n += counts[k];
  }
  mean[0] = n > 0 ? (float)(total / (double)n) : 0.0f;
  mean[1] = n > 0 ? (float)(1.0 / (double)n) : 0.0f;
}

__global__ void zero_mean(float* mean) { mean[threadIdx.x] = 0.0f; }

// Finishes the sums of `splits` K splits, in their order, for R x K elements of one
// gradient or of both (the first blocks_a workgroups take a's).  K % 16 == 0.  Eight
// splits' loads in flight: 100 x 20000 x 512, 35 splits, 11.3 -> 5.2 us.
struct SplitSums {
  const float* sums = nullptr;
  int64_t splits = 0, count = 0;  // R K
  Finish fin;
};
__device__ __forceinline__ void add_splits(const SplitSums& s, int64_t K, int64_t i) {
  if (i >= s.count) return;
  const int64_t row = i / K;
  float factor;
  const bool counted = finish_row(s.fin, row, factor);
  v4f v = *reinterpret_cast<const v4f*>(s.sums + i);
  constexpr int U = 8;
  for (int64_t z = 1; z < s.splits; z += U) {
    v4f q[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (z + u < s.splits) q[u] = *reinterpret_cast<const v4f*>(s.sums + (z + u) * s.count + i);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (z + u < s.splits) v += q[u];
  }
  finish4(s.fin, row, i - row * K, v, counted, factor);
}
__global__ void __launch_bounds__(256) xent_finish(SplitSums a, SplitSums b, int64_t K, uint32_t blocks_a) {
  const bool second = blockIdx.x >= blocks_a;
  add_splits(second ? b : a, K, ((int64_t)(blockIdx.x - (second ? blocks_a : 0u)) * 256 + threadIdx.x) * 4);
}
hipError_t launch_finish(const SplitSums& a, const SplitSums& b, int64_t K, hipStream_t st) {
  const int64_t na = (a.count / 4 + 255) / 256, nb = (b.count / 4 + 255) / 256;
  if (na + nb == 0) return hipSuccess;
  hipLaunchKernelGGL(xent_finish, dim3((unsigned)(na + nb)), dim3(256), 0, st, a, b, K, (uint32_t)na);
  return hipGetLastError();
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

// The logits of columns v0 .. v0 + n - 1, A's codes in fp16 at a16.
void fill_logits(XentArgs& p, const XentCall& c, const uint16_t* a16, int64_t ld, int64_t v0, int64_t n) {
  p.a = reinterpret_cast<const uint8_t*>(a16);
  p.b = c.b + v0 * c.ldb;
  p.lda = 2 * ld; p.ldb = c.ldb;
  p.K = p.k_total = 2 * c.K;
  p.M = c.M; p.N = n; p.batch = 1;
  p.a_scale_inv = c.a_scale_inv; p.b_scale_inv = c.b_scale_inv && c.b_rows ? c.b_scale_inv + v0 : c.b_scale_inv;
  p.a_rows = c.a_rows; p.b_rows = c.b_rows;
  p.targets = c.targets; p.target_bits = c.target_bits; p.v0 = v0; p.vocab = c.N;
}
// The same from A's codes (xent_rows).
void fill_rows(XentArgs& p, const XentCall& c, int64_t v0, int64_t n) {
  fill_logits(p, c, nullptr, 0, v0, n);
  p.a = c.a; p.lda = c.lda; p.K = c.K;
}

}  // namespace

int64_t xent_workspace_bytes(int64_t M, int64_t N, int64_t K) { return ForwardPlan(M, N, K).bytes; }
int64_t xent_grad_workspace_bytes(int64_t M, int64_t N, int64_t K) { return BackwardPlan(M, N, K).bytes; }

template <int TJ, class G>
static hipError_t launch_rows(const XentArgs& p, const G& extra, int64_t more, hipStream_t st) {
  const int64_t rows = p.M <= 16 ? 16 : (p.M <= 32 ? 32 : 64), cols = (p.N + 16 * TJ - 1) / (16 * TJ);
  const int64_t blocks = cols * ((p.M + rows - 1) / rows);
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks + more)), dim3(256), 0, st, p, extra, (uint32_t)cols, (uint32_t)blocks);
    return hipGetLastError();
  };
  return rows == 16 ? go(xent_rows<1, TJ, G>) : rows == 32 ? go(xent_rows<2, TJ, G>) : go(xent_rows<4, TJ, G>);
}
template <class G> static hipError_t launch_rows(const XentArgs& p, const G& extra, int64_t more, hipStream_t st) {
  return rows_tile(p.N) == 32 ? launch_rows<2>(p, extra, more, st) : launch_rows<1>(p, extra, more, st);
}

hipError_t launch_xent_forward(const XentCall& c, hipStream_t st) {
  if (c.M == 0) {
    if (!c.mean) return hipSuccess;
    hipLaunchKernelGGL(zero_mean, dim3(1), dim3(2), 0, st, c.mean);
    return hipGetLastError();
  }
  const ForwardPlan plan(c.M, c.N, c.K);
  uint32_t* const ticket = reinterpret_cast<uint32_t*>(c.ws + plan.ticket);
  float2* const parts = reinterpret_cast<float2*>(c.ws + plan.parts);
  float* const logit = reinterpret_cast<float*>(c.ws + plan.logit);
  const int64_t tiles = (c.N + plan.tile - 1) / plan.tile;
  if (plan.rows) {
    XentArgs p;
    fill_rows(p, c, 0, c.N);
    p.parts = parts;
    p.target_logit = logit;
    FP8MI_TRY(launch_rows(p, RowsStats{ticket}, 0, st));
  } else {
    uint16_t* const a16 = reinterpret_cast<uint16_t*>(c.ws + plan.a16);
    FP8MI_TRY(launch_widen(widen(c.a, c.lda, c.M, c.K, a16, plan.ld), ticket, st));
    // 256 x 256 tiles of 512 threads: at most 2^31 of them in a grid
    const int64_t most = offset_columns(c.ldb), grid = (INT64_C(1) << 38) / c.M;
    const int64_t cols = even_pieces(c.N, most < grid ? most : grid);  // a multiple of every tile's
    for (int64_t v0 = 0; v0 < c.N; v0 += cols) {
      XentLseArgs p;
      fill_logits(p, c, a16, plan.ld, v0, c.N - v0 < cols ? c.N - v0 : cols);
      p.tile0 = v0 / plan.tile;
      p.parts = parts;
      p.target_logit = logit;
      FP8MI_TRY(launch_xent_lse(p, st));
    }
  }
  const int rb = join_rows(c.M);
  const auto join = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)((c.M + rb - 1) / rb)), dim3(256), 0, st, parts, tiles, c.M, logit,
                       c.targets, c.target_bits, c.N, c.loss, c.lse, c.mean, ticket,
                       reinterpret_cast<uint64_t*>(c.ws + plan.slots));
    return hipGetLastError();
  };
  return rb == 16 ? join(xent_join<16>) : rb == 4 ? join(xent_join<4>) : join(xent_join<1>);
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
  // with a loss gradient per row, dB takes A's rows times theirs, and G's rows share their
  // range (dA alone too: it is the same with dB and without)
  const bool scaled = c.db && c.dloss_rows;
  float* const unit = reinterpret_cast<float*>(c.ws + plan.unit);
  if (c.dloss_rows) {
    hipLaunchKernelGGL(dloss_unit, dim3(1), dim3(1024), 0, st, c.dloss, c.targets, c.target_bits, c.M, unit);
    FP8MI_TRY(hipGetLastError());
  }
  Widen rows = widen(c.a, c.lda, c.M, c.K, at(plan.a16), plan.ld);
  rows.targets = c.targets;
  rows.target_bits = c.target_bits;
  if (scaled) {
    rows.rows = c.dloss;
    rows.rows_by = unit;
    rows.out_scaled = at(plan.a16d);
  }
  const int64_t most = offset_columns(c.ldb), cols = plan.cols <= most ? plan.cols : even_pieces(c.N, most);
  // bytes of G's rows per K split, from the first piece (no later one is wider):
  // whole 128-byte steps, so that every split starts on a chunk
  const int64_t first_cols = up(c.N < cols ? c.N : cols, 8);
  const int64_t k_split = up((2 * first_cols + plan.splits - 1) / plan.splits, 128);
  const int64_t splits = (2 * first_cols + k_split - 1) / k_split;
  const bool direct = splits == 1 && cols >= c.N;  // dA's sums are complete in one launch
  // the same of G^T A's rows
  const int64_t rows_bytes = 2 * up(c.M, 8), k_split_db = up((rows_bytes + plan.splits_db - 1) / plan.splits_db, 128);
  SplitSums sum_a, sum_b;
  sum_a.sums = sums; sum_a.splits = splits;
  sum_a.fin.out = c.da; sum_a.fin.ld = c.ld_da;
  sum_a.fin.scale = c.b_scale_inv; sum_a.fin.by = c.dloss; sum_a.fin.by_rows = c.dloss_rows;
  sum_a.fin.unit = c.dloss_rows ? unit : nullptr;
  sum_a.fin.targets = c.targets; sum_a.fin.target_bits = c.target_bits;
  // by the whole vocabulary, as in the forward pass: a narrow last piece's logits
  // then add up in the order of the others, and of those that made lse
  const bool from_codes = few_rows(c.M, c.N);
  for (int64_t v0 = 0; v0 < c.N; v0 += cols) {
    const int64_t n = c.N - v0 < cols ? c.N - v0 : cols;
    XentGradArgs g;
    g.lse = c.lse;
    g.d = at(plan.g); g.ld_d = plan.ld_g;
    g.dloss = c.dloss_rows ? c.dloss : nullptr; g.unit = unit;
    if (from_codes) {  // the logits straight from the codes, beside the widening of A
      if (v0 > 0) rows.chunks = 0;
      fill_rows(g, c, v0, n);
      FP8MI_TRY(launch_rows(g, RowsGrad{rows}, widen_groups(rows), st));
    } else {
      if (v0 == 0) FP8MI_TRY(launch_widen(rows, nullptr, st));
      fill_logits(g, c, at(plan.a16), plan.ld, v0, n);
      FP8MI_TRY(launch_xent_grad(g, st));
    }
    AddArgs add;  // G by rows, the piece's codes K-major
    add.a = reinterpret_cast<const uint8_t*>(at(plan.g));
    add.b = c.b + v0 * c.ldb;
    add.lda = 2 * plan.ld_g; add.ldb = c.ldb;
    add.M = c.M; add.N = c.K;
    add.k_total = 2 * up(n, 8);
    add.k_major_rows = n;
    add.K = k_split;
    add.batch = (add.k_total + k_split - 1) / k_split;
    add.stride_a = k_split;
    add.stride_b = k_split / 2 * c.ldb;
    add.sums = direct ? nullptr : sums;
    add.first = v0 == 0;
    add.fin = sum_a.fin;
    const auto fill_km = [&](Mm16Args& km) {  // both K-major
      km.a = reinterpret_cast<const uint8_t*>(at(plan.g));
      km.b = reinterpret_cast<const uint8_t*>(at(scaled ? plan.a16d : plan.a16));
      km.lda = 2 * plan.ld_g; km.ldb = 2 * plan.ld;
      km.M = n; km.N = c.K;
      km.k_total = rows_bytes;
      km.k_major_rows = c.M;
      km.K = k_split_db;
      km.batch = (rows_bytes + k_split_db - 1) / k_split_db;
      km.stride_a = k_split_db / 2 * km.lda;
      km.stride_b = k_split_db / 2 * km.ldb;
    };
    const bool last = v0 + cols >= c.N;
    if (last && c.da && !direct) sum_a.count = c.M * c.K;
    if (plan.splits_db > 1) {
      KmSumArgs km;
      fill_km(km);
      km.sums = reinterpret_cast<float*>(c.ws + plan.sums_db);
      km.first = 1;
      FP8MI_TRY(launch_mm16_grads(c.da ? &add : nullptr, nullptr, c.db ? &km : nullptr, st));
      if (c.db) {
        sum_b.sums = km.sums; sum_b.splits = km.batch; sum_b.count = n * c.K;
        sum_b.fin.out = c.db + v0 * c.ld_db; sum_b.fin.ld = c.ld_db;
        sum_b.fin.scale = c.a_scale_inv; sum_b.fin.by = scaled ? unit : c.dloss;
      }
    } else {
      KmArgs km;
      fill_km(km);
      km.a_scale_inv = c.a_scale_inv;
      km.b_scale_inv = scaled ? unit : c.dloss;
      km.c = c.db + v0 * c.ld_db; km.ldc = c.ld_db; km.stride_c = 0;
      FP8MI_TRY(launch_mm16_grads(c.da ? &add : nullptr, c.db ? &km : nullptr, nullptr, st));
    }
    FP8MI_TRY(launch_finish(sum_a, sum_b, c.K, st));  // what is complete after this piece
  }
  return hipSuccess;
}

}  // namespace fp8mi
