// Sixteen elements of a plain matrix's row, as the quantising kernels load them.
#pragma once
#include "fp4.cuh"

namespace tpmlp {
namespace fp4 {

template <class T>
struct Raw;   // 16 elements as loaded
template <>
struct Raw<__nv_bfloat16> {
  uint32_t w[8];
  // bits of the largest |x| as fp32: magnitudes compare as whole numbers
  __device__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    return max(m << 16, m & 0xffff0000u);
  }
  __device__ void floats(float (&v)[16]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {   // bf16 is the upper half of fp32
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw<float> {
  uint32_t w[16];
  __device__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, w[i] & 0x7fffffffu);
    return m;
  }
  __device__ void floats(float (&v)[16]) const {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(w[i]);
  }
};

// LD: bytes of a load (32 and 16: every 16-element unit starts on such a
// boundary; 8192 x 5120 of bf16: 16.9 and 17.9 us).
template <int LD, int WORDS>
__device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[WORDS]) {
  if constexpr (LD == 32) {
#pragma unroll
    for (int i = 0; i < WORDS / 8; ++i)
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[8 * i]), "=r"(w[8 * i + 1]), "=r"(w[8 * i + 2]),
                     "=r"(w[8 * i + 3]), "=r"(w[8 * i + 4]), "=r"(w[8 * i + 5]),
                     "=r"(w[8 * i + 6]), "=r"(w[8 * i + 7])
                   : "l"(static_cast<const char*>(p) + 32 * i));
  } else {
#pragma unroll
    for (int i = 0; i < WORDS / 4; ++i) {
      const uint4 u = load_u32x4(static_cast<const uint4*>(p) + i);
      w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
    }
  }
}

__device__ __forceinline__ uint32_t element_bits(const __nv_bfloat16* p) {
  return load_u16(p) << 16;
}
__device__ __forceinline__ uint32_t element_bits(const float* p) {
  return load_u32(p);
}

// The bytes of a matrix, from its first to past its last element.
struct Extent {
  const char *begin, *end;
};
template <class T>
__device__ __forceinline__ Extent extent_of(const T* x, long long stride,
                                            long long rows, long long cols) {
  return {reinterpret_cast<const char*>(x),
          reinterpret_cast<const char*>(x + (rows - 1) * stride + cols)};
}

// 16 elements from p, aligned to its element: the 16-byte pieces that hold them,
// shifted.  Reads up to 14 bytes before and 16 after them.  (One by one, a matrix
// 8192 x 5120 of bf16 off its alignment took 46 us, not 23.)
template <class T, int WORDS>
__device__ __forceinline__ void load_shifted(const T* p, uint32_t (&r)[WORDS]) {
  const unsigned a = static_cast<unsigned>(reinterpret_cast<uintptr_t>(p)) & 15u;
  uint32_t w[WORDS + 4];
  load_words<16>(reinterpret_cast<const char*>(p) - a, w);
#pragma unroll
  for (int i = 0; i < WORDS + 2; ++i) w[i] = a & 8u ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < WORDS + 1; ++i) w[i] = a & 4u ? w[i + 1] : w[i];
#pragma unroll
  for (int i = 0; i < WORDS; ++i)
    r[i] = sizeof(T) == 2 && (a & 2u) ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
}

// 16 elements from p, the first n of them in the row (n may be negative: none) of
// a matrix with the extent `e`.  LD as above; 0: any alignment.
template <class T, int LD>
__device__ __forceinline__ void load16(const T* p, int n, const Extent& e,
                                       Raw<T>& r) {
  constexpr int WORDS = sizeof(r.w) / 4;
  if (n >= 16) {
    if constexpr (LD != 0) {
      load_words<LD>(p, r.w);
      return;
    } else {
      const char* q = reinterpret_cast<const char*>(p);
      if (q - 14 >= e.begin && q + 16 * sizeof(T) + 16 <= e.end) {
        load_shifted(p, r.w);
        return;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < WORDS; ++i) {
    if constexpr (sizeof(T) == 4) {
      r.w[i] = i < n ? element_bits(p + i) : 0u;
    } else {
      const uint32_t lo = 2 * i < n ? element_bits(p + 2 * i) >> 16 : 0u;
      const uint32_t hi = 2 * i + 1 < n ? element_bits(p + 2 * i + 1) : 0u;
      r.w[i] = lo | hi;
    }
  }
}

}  // namespace fp4
}  // namespace tpmlp
