// Eight consecutive elements at a time from any element-aligned address, and
// eight or sixteen codes to any byte address.  The vector types carry the
// element's alignment; the target runs with unaligned global access enabled,
// so the compiler still emits one 16-byte (8-byte) access, and a tensor of odd
// width or with a misaligned base takes the same code as an aligned one.
#pragma once
#include "fp8mi_device.h"

namespace fp8mi {

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4_byte __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_byte __attribute__((ext_vector_type(2), aligned(1)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Stored form of eight elements: 16 bytes (bf16, fp16) or 32 (fp32).
template <int DT> struct Raw8 {
  static constexpr int kWords = 2 * In<DT>::kBytes;
  uint32_t w[kWords];
};

template <int DT> __device__ __forceinline__ void load8(Raw8<DT>& r, const void* base, int64_t idx) {
  const char* p = static_cast<const char*>(base) + idx * In<DT>::kBytes;
#pragma unroll
  for (int c = 0; c < Raw8<DT>::kWords / 4; ++c) {
    const u32x4_any v = *reinterpret_cast<const u32x4_any*>(p + 16 * c);
#pragma unroll
    for (int e = 0; e < 4; ++e) r.w[4 * c + e] = v[e];
  }
}

template <int DT> __device__ __forceinline__ void zero8(Raw8<DT>& r) {
#pragma unroll
  for (int e = 0; e < Raw8<DT>::kWords; ++e) r.w[e] = 0u;
}

// The first n (< 8) elements, the others zero.
template <int DT> __device__ __forceinline__ void load8_tail(Raw8<DT>& r, const void* base, int64_t idx, int n) {
  zero8(r);
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < n) {
      if constexpr (DT == kF32) r.w[e] = static_cast<const uint32_t*>(base)[idx + e];
      else r.w[e / 2] |= (uint32_t)static_cast<const uint16_t*>(base)[idx + e] << (16 * (e & 1));
    }
}

template <int DT> __device__ __forceinline__ void widen8(const Raw8<DT>& r, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (DT == kF32) {
      f[2 * e] = __uint_as_float(r.w[2 * e]);
      f[2 * e + 1] = __uint_as_float(r.w[2 * e + 1]);
    } else {
      widen2<DT>(r.w[e], f[2 * e], f[2 * e + 1]);
    }
  }
}

// Round to nearest even into the element type (the hardware conversions).
template <int DT> __device__ __forceinline__ void narrow8(Raw8<DT>& r, const float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (DT == kF32) {
      r.w[2 * e] = __float_as_uint(f[2 * e]);
      r.w[2 * e + 1] = __float_as_uint(f[2 * e + 1]);
    } else if constexpr (DT == kBF16) {
      const f32x2 v = {f[2 * e], f[2 * e + 1]};
      r.w[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    } else {
      const f32x2 v = {f[2 * e], f[2 * e + 1]};
      r.w[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
    }
  }
}

// Stores the first n (<= 8) elements, non-temporal: these are whole tensors that
// the L2 cannot keep beside what is still to be read (norm 8192 x 1536 with its
// sum 22.0 -> 19.8 us, gradient 25.6 -> 23.5, 4096 x 5120 39.0 -> 37.5, over three
// sets of buffers in turn; small ones no slower: 2048 x 1536 10.4 -> 9.9).
template <int DT> __device__ __forceinline__ void store8(void* base, int64_t idx, const Raw8<DT>& r, int n) {
  char* p = static_cast<char*>(base) + idx * In<DT>::kBytes;
  if (n >= 8) {
#pragma unroll
    for (int c = 0; c < Raw8<DT>::kWords / 4; ++c) {
      const u32x4_any v = {r.w[4 * c], r.w[4 * c + 1], r.w[4 * c + 2], r.w[4 * c + 3]};
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(p + 16 * c));
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < n) {
      if constexpr (DT == kF32) reinterpret_cast<uint32_t*>(p)[e] = r.w[e];
      else reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(r.w[e / 2] >> (16 * (e & 1)));
    }
}

// Eight codes (n of them when n < 8) at any byte address; STREAM: non-temporal.
template <bool STREAM = false>
__device__ __forceinline__ void store_codes8(uint8_t* p, uint32_t lo, uint32_t hi, int n) {
  if (n >= 8) {
    const u32x2_byte v = {lo, hi};
    if constexpr (STREAM) __builtin_nontemporal_store(v, reinterpret_cast<u32x2_byte*>(p));
    else *reinterpret_cast<u32x2_byte*>(p) = v;
    return;
  }
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < n) p[e] = (uint8_t)((e < 4 ? lo : hi) >> (8 * (e & 3)));
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

}  // namespace fp8mi
