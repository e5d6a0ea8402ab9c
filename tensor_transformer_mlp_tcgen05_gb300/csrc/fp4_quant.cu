// Four-bit quantisation and its inverse: HBM-bound passes over a plain matrix.
//
//   rows        one read of x, codes and scales written: (2 + 9/16) bytes an
//               element of bf16 (NV)
//   transposed  the same, through shared memory: x is read along its rows, the
//               codes of a column are consecutive
//   both        one read for the two
//   amax        the largest finite |x| of a matrix whose g is its own
//   dequantise  the values, as bf16 or fp32
//
// Measured, 5120 x 20480 bf16 NV (268 MB of traffic, 39.7 us at the copy rate):
// rows 42 us (6.4 TB/s), transposed 46 (5.8), dequantise 41 (6.5), amax 35 (6.0);
// 8192 x 15360: both 87 us (4.5 TB/s) where the two took 111.  What is left: the
// arithmetic (some 9 instructions an element one way, with 16 to 24 warps an SM to
// hide loads behind).  Rows off a 32-byte boundary are in the comments below.
#include "fp4_kernels.h"
#include "fp4_load.cuh"

namespace tpmlp {
namespace fp4 {
namespace {

constexpr int THREADS = 256;

// Block 0 clears a status word, before a product may start that writes to it.
__device__ __forceinline__ void clear_status(const Packed& p) {
  if (blockIdx.x == 0 && threadIdx.x < 4) p.head->status[threadIdx.x] = 0;
}

// 1 / g (all threads); block 0 writes g, to `also` too.
__device__ __forceinline__ float inverse_g(const Packed& p, const Gain& gain,
                                           Header* also = nullptr) {
  int e = gain.exponent;
  if (gain.slots > 0) {
    wait_for_launch_before();   // the pass before
    uint32_t top = 0;
    for (int i = threadIdx.x & 31; i < gain.slots; i += 32)
      top = max(top, p.head->amax[i]);
    e = auto_exponent(__reduce_max_sync(0xffffffffu, top));
  } else if (gain.like != nullptr) {   // a power of two
    e = static_cast<int>(__float_as_uint(gain.like->g) >> 23) - 127;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    p.head->g = exp2_of(e);
    if (also != nullptr) also->g = exp2_of(e);
  }
  return exp2_of(-e);
}

// ------------------------------------------------------------------- rows --

// A thread takes 16 elements of a row (a block of NV, half of one of MX), 16
// threads 256 columns, a block 16 rows at a time and PASSES times those.
template <class T, int FORMAT, int LD, int PASSES>
__global__ void __launch_bounds__(THREADS)
    rows_kernel(const T* x, long long stride, const Packed p,
                const Gain gain) {
  if (gain.slots == 0) wait_for_launch_before();
  clear_status(p);
  let_next_launch_start();
  const int lane = threadIdx.x & 31;
  const int unit = threadIdx.x & 15;
  const int kt = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.ktiles));
  const int chunk = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.ktiles));
  const int row0 = chunk * 16 * PASSES + static_cast<int>(threadIdx.x >> 4);
  const int col = kt * TILE_COLS + unit * 16;
  Raw<T> raw[PASSES];
  const T* src = x + row0 * stride + col;
  // (loads behind conditions wait for one another: whole tiles have none.  Any
  // alignment: those but the matrix's first and last rows', whose pieces may pass
  // its ends.)
  bool inside = (chunk + 1) * 16 * PASSES <= p.rows && (kt + 1) * TILE_COLS <= p.cols;
  if (LD == 0)
    inside = inside && chunk > 0 && (chunk + 1) * 16 * PASSES < p.rows;
  if (inside) {
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      if constexpr (LD == 0)
        load_shifted(src + 16 * i * stride, raw[i].w);
      else
        load_words<LD>(src + 16 * i * stride, raw[i].w);
    }
  } else {
    const Extent e = extent_of(x, stride, p.rows, p.cols);
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
      load16<T, LD>(src + 16 * i * stride,
                    row0 + 16 * i < p.rows ? p.cols - col : 0, e, raw[i]);
  }
  const float inv_g = inverse_g(p, gain);
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int row = row0 + 16 * i;
    float v[16];
    raw[i].floats(v);
    uint32_t amax = raw[i].amax();
    if constexpr (FORMAT == TPFP4_MX)
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    const Scale s = block_scale<FORMAT>(amax, inv_g);
    const uint2 c = codes16<FORMAT, sizeof(T) == 4>(v, s);
    // four blocks' scale bytes in one word
    uint32_t word;
    if constexpr (FORMAT == TPFP4_NV) {
      word = s.byte << (8 * (lane & 3));
      word |= __shfl_xor_sync(0xffffffffu, word, 1);
      word |= __shfl_xor_sync(0xffffffffu, word, 2);
    } else {
      word = s.byte << (8 * ((lane >> 1) & 3));
      word |= __shfl_xor_sync(0xffffffffu, word, 2);
      word |= __shfl_xor_sync(0xffffffffu, word, 4);
    }
    if (row < p.rows) {
      *reinterpret_cast<uint2*>(p.codes + code_row(row, kt, p.ktiles) +
                                code_unit(row, unit / 2) + unit % 2 * 8) = c;
      constexpr int THREADS_A_WORD = FORMAT == TPFP4_NV ? 4 : 8;
      if (unit % THREADS_A_WORD == 0)
        *reinterpret_cast<uint32_t*>(
            p.scales + scale_word(row, kt, unit / THREADS_A_WORD, p.ktiles,
                                  tile_bytes(FORMAT))) = word;
    }
  }
}

// ------------------------------------------------------------- transposed --

// Two consecutive elements from p, as loaded; n of them are in the matrix.
template <class T>
struct Two;
template <>
struct Two<__nv_bfloat16> {
  uint32_t w;
  // bits of the largest |a| and |b| of 16
  static __device__ void amax(const Two* t, uint32_t& a, uint32_t& b) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = __vmaxu2(m, t[i].w & 0x7fff7fffu);
    a = m << 16;
    b = m & 0xffff0000u;
  }
  __device__ float a() const { return __uint_as_float(w << 16); }
  __device__ float b() const { return __uint_as_float(w & 0xffff0000u); }
  __device__ void load(const __nv_bfloat16* p) {
    w = load_u32(p);
  }
  __device__ void load(const __nv_bfloat16* p, int n) {
    w = n >= 1 ? element_bits(p) >> 16 : 0u;
    if (n >= 2) w |= element_bits(p + 1);
  }
};
template <>
struct Two<float> {
  float2 w;
  static __device__ void amax(const Two* t, uint32_t& a, uint32_t& b) {
    a = b = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      a = max(a, abs_bits(t[i].w.x));
      b = max(b, abs_bits(t[i].w.y));
    }
  }
  __device__ float a() const { return w.x; }
  __device__ float b() const { return w.y; }
  __device__ void load(const float* p) {
    const uint2 u = load_u32x2(p);
    w = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
  }
  __device__ void load(const float* p, int n) {
    w.x = n >= 1 ? load_f32(p) : 0.f;
    w.y = n >= 2 ? load_f32(p + 1) : 0.f;
  }
};

constexpr int T_COLS = 64;   // columns of x a block takes

// Where 16-byte piece c of row r of a block's elements lies in shared memory: a
// lane writes two elements of a row, then reads the pieces of a unit of 16, the
// lanes of a quarter warp those of two rows by four units, from different banks.
template <class T>
__device__ __forceinline__ int staged(int r, int c) {
  constexpr int PIECES = T_COLS * sizeof(T) / 16;
  const int x = sizeof(T) == 2 ? r & 1 : (c >> 3) | ((r & 1) << 1);
  return (r * PIECES + (c ^ x)) * 16;
}

// A warp's 32 rows (from k0 on) of a block's 64 columns (from n0 on), quantised
// along the rows into p: a lane takes four units of 16.
template <class T, int FORMAT>
__device__ __forceinline__ void quantize_staged(const uint8_t* s_x, const Packed& p,
                                                int k0, int n0, float inv_g) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = lane & 3;
  const int kt = n0 / TILE_COLS, unit0 = n0 % TILE_COLS / 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2), row = k0 + r;
    Raw<T> raw;
    constexpr int PIECES = sizeof(T);   // of a unit
#pragma unroll
    for (int j = 0; j < PIECES; ++j) {
      const uint4 u = *reinterpret_cast<const uint4*>(
          s_x + staged<T>(warp * 32 + r, unit * PIECES + j));
      raw.w[4 * j] = u.x, raw.w[4 * j + 1] = u.y;
      raw.w[4 * j + 2] = u.z, raw.w[4 * j + 3] = u.w;
    }
    float v[16];
    raw.floats(v);
    uint32_t amax = raw.amax();
    if constexpr (FORMAT == TPFP4_MX)
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    const Scale s = block_scale<FORMAT>(amax, inv_g);
    const uint2 w = codes16<FORMAT, sizeof(T) == 4>(v, s);
    constexpr int UNITS = block_size(FORMAT) / 16;
    uint32_t word = s.byte << (8 * (unit / UNITS));
    word |= __shfl_xor_sync(0xffffffffu, word, UNITS);
    if constexpr (FORMAT == TPFP4_NV) word |= __shfl_xor_sync(0xffffffffu, word, 2);
    if (row >= p.rows) continue;
    const int u = unit0 + unit;
    *reinterpret_cast<uint2*>(p.codes + code_row(row, kt, p.ktiles) +
                              code_unit(row, u / 2) + u % 2 * 8) = w;
    const int block = unit0 / UNITS;   // the first of four (NV) or two (MX)
    uint8_t* to = p.scales + scale_word(row, kt, block / 4, p.ktiles,
                                        tile_bytes(FORMAT)) + block % 4;
    if (unit == 0) {
      if constexpr (FORMAT == TPFP4_NV)
        *reinterpret_cast<uint32_t*>(to) = word;
      else
        *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(word);
    }
  }
}

// A block takes 256 rows (one k-tile of the packed matrix) of 64 columns, a
// warp 32 of those rows, a lane two columns: its 32 elements of a column are
// two blocks of NV or one of MX.  Codes and scales go through shared memory,
// so that a packed row's 128 bytes of codes are written together.
// (three blocks an SM for bf16, 85 registers: 57 -> 47 us for 5120 x 20480; four
// spill.  PAIR: a lane's two columns in one load; else, 8192 x 5120 takes 33 us
// instead of 19.)
// BOTH: the elements, read once, are quantised along the rows of x into rp too.
template <class T, int FORMAT, bool PAIR, bool BOTH>
__global__ void __launch_bounds__(THREADS, sizeof(T) == 2 ? 3 : 2)
    columns_kernel(const T* x, long long stride, int x_rows, const Packed p,
                   const Gain gain, float* __restrict__ part,
                   const Packed rp) {
  if (gain.slots == 0) wait_for_launch_before();
  clear_status(p);
  if (BOTH) clear_status(rp);
  let_next_launch_start();
  // 16-byte unit u of row n at unit u ^ (n / 2 mod 8): the lanes of a warp,
  // two rows apart, write to different banks
  __shared__ uint4 s_codes[T_COLS * 8];
  __shared__ __align__(16) uint8_t s_scales[T_COLS * 16];
  __shared__ float s_sum[8][T_COLS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // (both: up to the end of rp's last k-tile, which its products read)
  const int tiles = BOTH ? rp.ktiles * (TILE_COLS / T_COLS)
                         : (p.rows + T_COLS - 1) / T_COLS;
  const int n0 = static_cast<int>(blockIdx.x % static_cast<unsigned>(tiles)) * T_COLS;
  const int kt = static_cast<int>(blockIdx.x / static_cast<unsigned>(tiles));
  const int k0 = kt * TILE_COLS + warp * 32;
  const int n = n0 + 2 * lane;
  Two<T> raw[32];
  const T* src = x + k0 * stride + n;
  if (PAIR && n0 + T_COLS <= p.rows && (kt + 1) * TILE_COLS <= x_rows) {
#pragma unroll
    for (int i = 0; i < 32; ++i) raw[i].load(src + i * stride);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      raw[i].load(src + i * stride, k0 + i < x_rows ? p.rows - n : 0);
  }
  extern __shared__ uint4 s_x[];   // both: [256][64] elements, see staged
  if constexpr (BOTH) {
    constexpr int LANES = 8 / sizeof(T);   // of a piece
#pragma unroll
    for (int i = 0; i < 32; ++i)
      *reinterpret_cast<Two<T>*>(reinterpret_cast<uint8_t*>(s_x) +
                                 staged<T>(warp * 32 + i, lane / LANES) +
                                 lane % LANES * sizeof(Two<T>)) = raw[i];
    __syncwarp();
  }
  const float inv_g = inverse_g(p, gain, BOTH ? rp.head : nullptr);
  uint32_t tops[2][2];   // [column][16 rows]
  Two<T>::amax(raw, tops[0][0], tops[1][0]);
  Two<T>::amax(raw + 16, tops[0][1], tops[1][1]);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = 2 * lane + j;
    const uint32_t* top = tops[j];
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = j == 0 ? raw[i].a() : raw[i].b();
    uint2 c0, c1;
    if constexpr (FORMAT == TPFP4_NV) {
      const Scale a = block_scale<FORMAT>(top[0], inv_g);
      const Scale b = block_scale<FORMAT>(top[1], inv_g);
      c0 = codes16<FORMAT, sizeof(T) == 4>(v, a);
      c1 = codes16<FORMAT, sizeof(T) == 4>(v + 16, b);
      *reinterpret_cast<uint16_t*>(s_scales + r * 16 + warp * 2) =
          static_cast<uint16_t>(a.byte | (b.byte << 8));
    } else {
      const Scale a = block_scale<FORMAT>(max(top[0], top[1]), inv_g);
      c0 = codes16<FORMAT, sizeof(T) == 4>(v, a);
      c1 = codes16<FORMAT, sizeof(T) == 4>(v + 16, a);
      s_scales[r * 16 + warp] = static_cast<uint8_t>(a.byte);
    }
    s_codes[r * 8 + (warp ^ (lane & 7))] = make_uint4(c0.x, c0.y, c1.x, c1.y);
    if (part != nullptr) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) sum += v[i];
      s_sum[warp][r] = sum;
    }
  }
  if constexpr (BOTH)
    quantize_staged<T, FORMAT>(reinterpret_cast<const uint8_t*>(s_x), rp, k0, n0,
                               inv_g);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < T_COLS * 8 / THREADS; ++i) {
    const int at = i * THREADS + threadIdx.x;
    const int r = at >> 3, u = at & 7;
    if (n0 + r < p.rows)
      *reinterpret_cast<uint4*>(p.codes + code_row(n0 + r, kt, p.ktiles) +
                                code_unit(n0 + r, u)) =
          s_codes[r * 8 + (u ^ ((r >> 1) & 7))];
  }
  constexpr int WORDS = TILE_COLS / block_size(FORMAT) / 4;
  if (threadIdx.x < T_COLS * WORDS) {
    const int r = threadIdx.x / WORDS, q = threadIdx.x % WORDS;
    if (n0 + r < p.rows)
      *reinterpret_cast<uint32_t*>(
          p.scales + scale_word(n0 + r, kt, q, p.ktiles, tile_bytes(FORMAT))) =
          *reinterpret_cast<const uint32_t*>(s_scales + r * 16 + q * 4);
  }
  if (part != nullptr && threadIdx.x < T_COLS &&
      n0 + static_cast<int>(threadIdx.x) < p.rows) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) sum += s_sum[w][threadIdx.x];
    part[static_cast<size_t>(kt) * p.rows + n0 + threadIdx.x] = sum;
  }
}

// ------------------------------------------------------------------- amax --

__device__ __forceinline__ uint32_t finite(uint32_t bits) {
  return bits < 0x7f800000u ? bits : 0u;
}

// An item is AMAX_UNITS units of 16 elements in a row; a block takes every
// gridDim-th item and leaves its maximum in a slot of its own: nothing to clear
// before, no atomics.
constexpr int AMAX_UNITS = 2 * THREADS;

template <class T, int LD>
__global__ void __launch_bounds__(THREADS)
    amax_kernel(const T* x, long long stride, long long rows,
                long long cols, Header* head) {
  wait_for_launch_before();
  let_next_launch_start();
  const long long segments = (cols + AMAX_UNITS * 16 - 1) / (AMAX_UNITS * 16);
  const Extent e = extent_of(x, stride, rows, cols);
  uint32_t top = 0;
  for (long long item = blockIdx.x; item < rows * segments; item += gridDim.x) {
    const long long row = item / segments;
    const long long c0 = (item - row * segments) * (AMAX_UNITS * 16);
    Raw<T> raw[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const long long c = c0 + (i * THREADS + threadIdx.x) * 16ll;
      load16<T, LD>(x + row * stride + c,
                    static_cast<int>(max(0ll, min(16ll, cols - c))), e, raw[i]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t m = raw[i].amax();
      if (m < 0x7f800000u) {
        top = max(top, m);
      } else {   // infinities or NaNs among them: the others
        float v[16];
        raw[i].floats(v);
#pragma unroll
        for (int k = 0; k < 16; ++k) top = max(top, finite(abs_bits(v[k])));
      }
    }
  }
  top = __reduce_max_sync(0xffffffffu, top);
  __shared__ uint32_t s_top[THREADS / 32];
  if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 1; i < THREADS / 32; ++i) top = max(top, s_top[i]);
    head->amax[blockIdx.x] = top;
  }
}

// ------------------------------------------------------------- dequantise --

// wide: the bytes that a unit's place is a multiple of, at most 32.
template <class T>
__device__ __forceinline__ void store16(T* p, int n, int wide,
                                        const uint32_t (&w)[sizeof(T) * 4],
                                        const float (&v)[16]) {
  constexpr int WORDS = sizeof(T) * 4;
  if (wide >= 16 && n >= 16) {
    if (wide == 32) {
#pragma unroll
      for (int i = 0; i < WORDS / 8; ++i)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                         reinterpret_cast<char*>(p) + 32 * i),
                     "r"(w[8 * i]), "r"(w[8 * i + 1]), "r"(w[8 * i + 2]),
                     "r"(w[8 * i + 3]), "r"(w[8 * i + 4]), "r"(w[8 * i + 5]),
                     "r"(w[8 * i + 6]), "r"(w[8 * i + 7])
                     : "memory");
    } else {
#pragma unroll
      for (int i = 0; i < WORDS / 4; ++i)
        reinterpret_cast<uint4*>(p)[i] =
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < n) {
      if constexpr (sizeof(T) == 2)
        p[i] = __float2bfloat16_rn(v[i]);
      else
        p[i] = v[i];
    }
}

// Elements 0 .. n - 1 (n <= 256) of a row piece in shared memory to p, by a warp, in
// 16-byte pieces or words that are aligned in memory: of bf16 off a word's boundary
// the first and the last element are stored alone.
template <class T>
__device__ __forceinline__ void store_row(T* p, int n, const uint8_t* s) {
  const int lane = threadIdx.x & 31;
  if (n == TILE_COLS && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
      reinterpret_cast<uint4*>(p)[32 * i + lane] =
          reinterpret_cast<const uint4*>(s)[32 * i + lane];
    return;
  }
  if constexpr (sizeof(T) == 4) {
    for (int i = lane; i < n; i += 32)
      reinterpret_cast<uint32_t*>(p)[i] = reinterpret_cast<const uint32_t*>(s)[i];
  } else {
    auto* out = reinterpret_cast<uint16_t*>(p);
    const auto* in = reinterpret_cast<const uint16_t*>(s);
    const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(p) >> 1 & 1u);
    const int words = (n - odd) / 2;
    for (int i = lane; i < words; i += 32) {
      const int k = 2 * i + odd;
      *reinterpret_cast<uint32_t*>(out + k) =
          in[k] | static_cast<uint32_t>(in[k + 1]) << 16;
    }
    if (lane == 0 && odd) out[0] = in[0];
    if (lane == 1 && odd + 2 * words < n) out[n - 1] = in[n - 1];
  }
}

__device__ __forceinline__ void values8(uint32_t w, float scale, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(
        static_cast<uint8_t>(w >> (8 * i)), __NV_E2M1);
    const float2 f = __half22float2(__half2(h));
    v[2 * i] = f.x * scale;
    v[2 * i + 1] = f.y * scale;
  }
}

// STAGED: a warp's two rows go through shared memory and out in consecutive pieces,
// not unit by unit.
template <class T, int FORMAT, int PASSES, bool STAGED>
__global__ void __launch_bounds__(THREADS)
    dequantize_kernel(const Packed p, T* __restrict__ out, long long stride,
                      int wide) {
  wait_for_launch_before();
  let_next_launch_start();
  __shared__ __align__(16)
      uint8_t s_rows[STAGED ? THREADS / 16 : 1][STAGED ? TILE_COLS * sizeof(T) : 16];
  const int unit = threadIdx.x & 15;
  const int kt = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.ktiles));
  const int chunk = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.ktiles));
  const int row0 = chunk * 16 * PASSES + static_cast<int>(threadIdx.x >> 4);
  const int cols = min(TILE_COLS, p.cols - kt * TILE_COLS);   // of this k-tile
  const float g = p.head->g;
  uint2 c[PASSES];
  uint32_t byte[PASSES];
  const int b = unit * 16 / block_size(FORMAT);
  const bool inside = (chunk + 1) * 16 * PASSES <= p.rows;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int row = inside ? row0 + 16 * i : min(row0 + 16 * i, p.rows - 1);
    c[i] = load_u32x2(p.codes + code_row(row, kt, p.ktiles) +
                      code_unit(row, unit / 2) + unit % 2 * 8);
    byte[i] = load_u8(p.scales + scale_word(row, kt, b / 4, p.ktiles,
                                            tile_bytes(FORMAT)) + b % 4);
  }
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int row = row0 + 16 * i;
    // code * s is exact; g is a power of two
    const float s = scale_value<FORMAT>(byte[i]);
    float v[16];
    values8(c[i].x, s, v);
    values8(c[i].y, s, v + 8);
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] *= g;
    constexpr int WORDS = sizeof(T) * 4;
    uint32_t w[WORDS];
#pragma unroll
    for (int k = 0; k < WORDS; ++k) {
      if constexpr (sizeof(T) == 2)
        w[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
      else
        w[k] = __float_as_uint(v[k]);
    }
    T* to = out + row * stride + kt * TILE_COLS;
    if constexpr (!STAGED) {
      if (row < p.rows) store16(to + unit * 16, cols - unit * 16, wide, w, v);
      continue;
    }
    const int own = threadIdx.x >> 4;
#pragma unroll
    for (int k = 0; k < WORDS / 4; ++k)
      *reinterpret_cast<uint4*>(&s_rows[own][unit * 16 * sizeof(T) + 16 * k]) =
          make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) {   // the warp's rows
      const int r = (own & ~1) + h;
      const int at = chunk * 16 * PASSES + 16 * i + r;
      if (at < p.rows)
        store_row(out + at * stride + kt * TILE_COLS, cols, s_rows[r]);
    }
    __syncwarp();
  }
}

// ---------------------------------------------------------------- launches --

bool on_boundary(const void* p, long long stride_bytes, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(stride_bytes)) %
             bytes == 0;
}

// Blocks that keep all SMs busy: with fewer, a block takes 16 rows, not 64 (1003 x
// 1000: 1.8 us, not 3.1; 1024 x 4096 2.8 and 2.7; 8192 x 5120 19.2 and 16.9).
constexpr long long FULL_GRID = 152 * 4;

// small: a grid of few loads, which needs no L1 but runs sooner where the SMs need
// not change their shared memory's size between kernels that use some and others
// (1003 x 1001 quantised and back 6.1 us, not 11.3).  Large ones do need L1 (8192 x 5120: 16.9 us, 22.5 without).
template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), unsigned grid, bool small, size_t smem,
                   cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
  attr[1].val.sharedMemCarveout = cudaSharedmemCarveoutMaxShared;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = small ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <class T, int FORMAT, int LD>
cudaError_t rows_launch(const T* x, long long stride, const Packed& p,
                        const Gain& g, cudaStream_t s) {
  const long long units = (p.rows + 15ll) / 16 * p.ktiles;
  if (units >= 4 * FULL_GRID)
    return launch(rows_kernel<T, FORMAT, LD, 4>,
                  static_cast<unsigned>((p.rows + 63ll) / 64 * p.ktiles), false, 0, s, x,
                  stride, p, g);
  const bool small = units * static_cast<long long>(sizeof(T)) < 4 * FULL_GRID;
  return launch(rows_kernel<T, FORMAT, LD, 1>, static_cast<unsigned>(units), small, 0,
                s, x, stride, p, g);
}

template <class T, int FORMAT>
cudaError_t rows_format(const T* x, long long stride, const Packed& p,
                        const Gain& g, cudaStream_t s) {
  const long long bytes = stride * static_cast<long long>(sizeof(T));
  if (on_boundary(x, bytes, 32)) return rows_launch<T, FORMAT, 32>(x, stride, p, g, s);
  if (on_boundary(x, bytes, 16)) return rows_launch<T, FORMAT, 16>(x, stride, p, g, s);
  return rows_launch<T, FORMAT, 0>(x, stride, p, g, s);
}

template <class T, int FORMAT, bool BOTH>
cudaError_t columns_launch(const T* x, long long stride, int x_rows,
                           const Packed& p, const Gain& g, float* part,
                           const Packed& rp, cudaStream_t s) {
  const long long tiles = BOTH ? rp.ktiles * static_cast<long long>(TILE_COLS / T_COLS)
                               : (p.rows + static_cast<long long>(T_COLS) - 1) / T_COLS;
  const bool pairs =
      on_boundary(x, stride * static_cast<long long>(sizeof(T)), 2 * sizeof(T));
  auto kernel = pairs ? columns_kernel<T, FORMAT, true, BOTH>
                      : columns_kernel<T, FORMAT, false, BOTH>;
  const size_t smem = BOTH ? T_COLS * TILE_COLS * sizeof(T) : 0;
  if (BOTH) {
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch(kernel, static_cast<unsigned>(tiles * p.ktiles),
                tiles * p.ktiles < FULL_GRID, smem, s, x, stride,
                x_rows, p, g, part, rp);
}

template <class T, int FORMAT>
cudaError_t columns_format(const T* x, long long stride, int x_rows,
                           const Packed& p, const Gain& g, float* part,
                           const Packed* rp, cudaStream_t s) {
  return rp != nullptr
             ? columns_launch<T, FORMAT, true>(x, stride, x_rows, p, g, part, *rp, s)
             : columns_launch<T, FORMAT, false>(x, stride, x_rows, p, g, part, p, s);
}

template <class T>
cudaError_t amax_type(const T* x, long long stride, long long rows, long long cols,
                      Header* head, int* slots, cudaStream_t s) {
  if (stride == cols) {   // one long row
    cols *= rows;
    stride = cols;
    rows = 1;
  }
  const long long items =
      (cols + AMAX_UNITS * 16 - 1) / (AMAX_UNITS * 16) * rows;
  *slots = static_cast<int>(items < AMAX_SLOTS ? items : AMAX_SLOTS);
  const long long bytes = rows == 1 ? 0 : stride * static_cast<long long>(sizeof(T));
  auto kernel = on_boundary(x, bytes, 32)   ? amax_kernel<T, 32>
                : on_boundary(x, bytes, 16) ? amax_kernel<T, 16>
                                            : amax_kernel<T, 0>;
  return launch(kernel, static_cast<unsigned>(*slots), items < AMAX_SLOTS, 0, s, x,
                stride, rows, cols,
                head);
}

template <class T>
cudaError_t dequantize_type(const Packed& p, int format, T* out, long long stride,
                            cudaStream_t s) {
  constexpr int PASSES = 4;
  const unsigned grid = static_cast<unsigned>(
      (p.rows + 16ll * PASSES - 1) / (16 * PASSES) * p.ktiles);
  const long long bytes = stride * static_cast<long long>(sizeof(T));
  const int wide =
      on_boundary(out, bytes, 32) ? 32 : on_boundary(out, bytes, 16) ? 16 : 0;
  // Through shared memory: 8192 x 5120 of bf16 on odd rows 29 us instead of 217, of
  // fp32 33 instead of 183, on 16-byte boundaries 33 instead of 49 (bf16 there: 26
  // instead of 20.5).
  const bool staged = wide == 0 || (wide == 16 && sizeof(T) == 4);
  auto kernel = format == TPFP4_NV
                    ? (staged ? dequantize_kernel<T, TPFP4_NV, PASSES, true>
                              : dequantize_kernel<T, TPFP4_NV, PASSES, false>)
                    : (staged ? dequantize_kernel<T, TPFP4_MX, PASSES, true>
                              : dequantize_kernel<T, TPFP4_MX, PASSES, false>);
  return launch(kernel, grid, grid < FULL_GRID, 0, s, p, out, stride, wide);
}

}  // namespace

cudaError_t launch_amax(bool bf16, const void* x, long long stride,
                        long long rows, long long cols, Header* head, int* slots,
                        cudaStream_t s) {
  return bf16 ? amax_type(static_cast<const __nv_bfloat16*>(x), stride, rows, cols,
                          head, slots, s)
              : amax_type(static_cast<const float*>(x), stride, rows, cols, head,
                          slots, s);
}

cudaError_t launch_quantize_rows(bool bf16, int format, const void* x,
                                 long long stride, const Packed& p,
                                 const Gain& g, cudaStream_t s) {
  if (bf16) {
    const auto* b = static_cast<const __nv_bfloat16*>(x);
    return format == TPFP4_NV
               ? rows_format<__nv_bfloat16, TPFP4_NV>(b, stride, p, g, s)
               : rows_format<__nv_bfloat16, TPFP4_MX>(b, stride, p, g, s);
  }
  const auto* f = static_cast<const float*>(x);
  return format == TPFP4_NV ? rows_format<float, TPFP4_NV>(f, stride, p, g, s)
                            : rows_format<float, TPFP4_MX>(f, stride, p, g, s);
}

cudaError_t launch_quantize_columns(bool bf16, int format, const void* x,
                                    long long stride, int x_rows,
                                    const Packed& p, const Gain& g,
                                    float* part, const Packed* rp,
                                    cudaStream_t s) {
  if (bf16) {
    const auto* b = static_cast<const __nv_bfloat16*>(x);
    return format == TPFP4_NV
               ? columns_format<__nv_bfloat16, TPFP4_NV>(b, stride, x_rows, p, g,
                                                         part, rp, s)
               : columns_format<__nv_bfloat16, TPFP4_MX>(b, stride, x_rows, p, g,
                                                         part, rp, s);
  }
  const auto* f = static_cast<const float*>(x);
  return format == TPFP4_NV
             ? columns_format<float, TPFP4_NV>(f, stride, x_rows, p, g, part, rp, s)
             : columns_format<float, TPFP4_MX>(f, stride, x_rows, p, g, part, rp, s);
}

cudaError_t launch_dequantize(const Packed& p, int format, bool bf16, void* out,
                              long long stride, cudaStream_t s) {
  return bf16 ? dequantize_type(p, format, static_cast<__nv_bfloat16*>(out), stride,
                                s)
              : dequantize_type(p, format, static_cast<float*>(out), stride, s);
}

}  // namespace fp4
}  // namespace tpmlp
