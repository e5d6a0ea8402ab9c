// Four-bit formats: the packed layout and the device code that makes codes and
// scales.  See include/tp_fp4.h for the definitions.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "tp_fp4.h"

namespace tpmlp {
namespace fp4 {

constexpr int TILE_ROWS = 128;   // rows of a tile
constexpr int TILE_COLS = 256;   // columns of a tile: 128 bytes of codes a row
constexpr int CODE_TILE = TILE_ROWS * TILE_COLS / 2;
constexpr size_t HEADER_BYTES = 4096;
constexpr int AMAX_SLOTS = 608;  // blocks of a pass for the largest |x|

__host__ __device__ constexpr int block_size(int format) {
  return format == TPFP4_NV ? 16 : 32;
}
// Bytes of the scales of a tile.
__host__ __device__ constexpr int tile_bytes(int format) {
  return TILE_ROWS * TILE_COLS / block_size(format);
}

// The first bytes of a packed matrix.  status: of the products that read it as A
// (first, as in the blocks' workspaces); amax: of a matrix quantised with its own
// g, the largest finite |x| (fp32 bits) that each block of the pass before found.
struct Header {
  int status[4];
  float g;
  int pad[59];
  unsigned int amax[AMAX_SLOTS];
};
static_assert(sizeof(Header) <= HEADER_BYTES, "header");

// One packed matrix: tile (r / 128, c / 256) is tile number (r / 128) ktiles +
// c / 256 of the codes and of the scales.  A product's copies are whole tiles, so
// that a weight is read from HBM in consecutive 16 KB.
struct Packed {
  Header* head;
  uint8_t* codes;
  uint8_t* scales;
  int rows, cols;
  int ktiles;        // tiles of a row
};

inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

inline size_t tiles_of(long long rows, long long cols) {
  return static_cast<size_t>((rows + TILE_ROWS - 1) / TILE_ROWS) *
         ((cols + TILE_COLS - 1) / TILE_COLS);
}
inline size_t scales_offset(long long rows, long long cols) {
  return HEADER_BYTES + tiles_of(rows, cols) * CODE_TILE;
}
inline size_t packed_bytes(long long rows, long long cols, int format) {
  return scales_offset(rows, cols) + tiles_of(rows, cols) * tile_bytes(format);
}
inline Packed view(const void* buffer, long long rows, long long cols) {
  char* b = static_cast<char*>(const_cast<void*>(buffer));
  Packed p;
  p.head = reinterpret_cast<Header*>(b);
  p.codes = reinterpret_cast<uint8_t*>(b + HEADER_BYTES);
  p.scales = reinterpret_cast<uint8_t*>(b + scales_offset(rows, cols));
  p.rows = static_cast<int>(rows);
  p.cols = static_cast<int>(cols);
  p.ktiles = static_cast<int>((cols + TILE_COLS - 1) / TILE_COLS);
  return p;
}

// Where row r's codes of k-tile kt lie (128 bytes), and in them those of its
// columns 32 u .. 32 u + 31: the order of shared memory's 128-byte swizzle, so that
// an operand's rows are one plain copy away from the MMA.
__device__ __forceinline__ size_t code_row(int r, int kt, int ktiles) {
  return (static_cast<size_t>(r / TILE_ROWS) * ktiles + kt) * CODE_TILE +
         (r % TILE_ROWS) * (TILE_COLS / 2);
}

__device__ __forceinline__ int code_unit(int r, int u) {
  return (u ^ (r & 7)) * 16;
}

// Where the four scale bytes of row r, blocks 4q .. 4q + 3 of k-tile kt lie.
__device__ __forceinline__ size_t scale_word(int r, int kt, int q, int ktiles,
                                             int bytes) {
  return (static_cast<size_t>(r / TILE_ROWS) * ktiles + kt) * bytes + q * 512 +
         (r % 32) * 16 + (r % TILE_ROWS) / 32 * 4;
}

// ------------------------------------------------------------- arithmetic --

// Every kernel here is launched so that it may start while the launch before it on
// the stream still runs, and lets the next one start.  Two kinds:
//   - a call's first kernel waits for the launch before it, then lets the next
//     start: what the next one finds complete is all that came before the call;
//   - a call's later kernel (the quantisation after its amax, a product after the
//     quantisation or product that makes A) lets the next one start, loads what
//     was there before the call, and waits before it reads or writes the rest.
// So none reads what an earlier call may still write, and none ends before all that
// came before it.
__device__ __forceinline__ void wait_for_launch_before() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_launch_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Loads of what the launch before may have written.  (__ldg, a const restrict pointer
// and ld.global.nc stand for memory that nothing writes as long as the kernel runs: a
// compiler may move them before the wait, and the hardware need not see the writes.
// Volatile, as the wait is, these stay behind it.)
__device__ __forceinline__ uint32_t load_u8(const void* p) {
  uint32_t v;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t load_u16(const void* p) {
  uint32_t v;
  asm volatile("ld.global.u16 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t load_u32(const void* p) {
  uint32_t v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ float load_f32(const float* p) {
  return __uint_as_float(load_u32(p));
}
__device__ __forceinline__ uint2 load_u32x2(const void* p) {
  uint2 v;
  asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 load_u32x4(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// x rounded to 14 significant bits "to odd": a value that is not one of them
// gets the neighbour whose last bit is set.  It compares with every number of
// 13 significant bits or fewer as x itself does, so codes and scales, whose
// borders have at most 7, come out as from x, and borders stand out from all
// that is not one of them by 2^-14.  (bf16 values have 8 bits: left alone.)
__device__ __forceinline__ uint32_t sticky(uint32_t u) {
  return (u & ~0x3ffu) | (((u & 0x3ffu) + 0x3ffu) & 0x400u);
}

// g of a matrix whose largest finite |x| has the bits `amax`: the exponent of
// the smallest power of two with amax <= 2688 g, 2688 = 448 * 6 = 1.3125 * 2^11.
__host__ __device__ inline int auto_exponent(uint32_t amax) {
  if (amax == 0) return 0;
  int e = static_cast<int>(amax >> 23);
  if (e == 0) return -126;   // subnormal: far below 2688 * 2^-126
  const uint32_t m = amax & 0x7fffffu;
  e = e - 127 - 11 + (m > 0x280000u ? 1 : 0);   // .3125 * 2^23
  return e < -126 ? -126 : e;
}

__device__ __forceinline__ float exp2_of(int e) {   // e from -149 to 127
  return e >= -126 ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23)
                   : __uint_as_float(1u << (e + 149));
}

// g_A g_B as factors (x, y): the product and 1, or where fp32 does not hold it,
// halves of its exponent: a sum times the one, then the other leaves fp32's range
// only where the result does.
__device__ __forceinline__ float2 gain_factors(float ga, float gb) {
  const int e = static_cast<int>(__float_as_uint(ga) >> 23) +
                static_cast<int>(__float_as_uint(gb) >> 23) - 254;
  const int h = e < -126 || e > 127 ? e >> 1 : e;
  return make_float2(exp2_of(h), exp2_of(e - h));
}

// A block's scale byte, and what its elements are multiplied by: m (a power of
// two, exact) and then r = 1 / s rounded.  `amax`: bits of the largest |x|.
struct Scale {
  uint32_t byte;
  float m, r;
};

template <int FORMAT>
__device__ __forceinline__ Scale block_scale(uint32_t amax, float inv_g) {
  Scale s;
  if constexpr (FORMAT == TPFP4_NV) {
    s.m = inv_g;
    const float a = __uint_as_float(sticky(amax)) * inv_g;
    // a / 6 rounded to 20 bits: a product with 1 / 6 is off by less than 2^-22
    // of itself, E4M3's borders (5 bits) come out as themselves, and what is not
    // one stays 2^-14 away
    const float v = __uint_as_float((__float_as_uint(a * (1.f / 6.f)) + 8u) & ~15u);
    const uint32_t byte = __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
    const float f = __half2float(
        __half(__nv_cvt_fp8_to_halfraw(static_cast<uint8_t>(byte), __NV_E4M3)));
    s.byte = byte;
    s.r = byte == 0 ? 0.f : rcp_approx(f);
    if (amax >= 0x7f800000u) s = {0x7fu, 0.f, 0.f};
  } else {
    if (amax >= 0x7f800000u) return {0xffu, 0.f, 0.f};
    if (amax == 0) return {127u, 1.f, 1.f};
    // floor(log2) of a subnormal is below -126: e is -127 then
    const int top = static_cast<int>(amax >> 23) - 127;
    const int e = top - 2 < -127 ? -127 : top - 2;
    s.byte = static_cast<uint32_t>(e + 127);
    s.m = exp2_of(-e);
    s.r = 1.f;
  }
  return s;
}

// x / (s g) of two elements for the rounding to E2M1.  NV: x m is exact, and
// (x m) r + 96 - 96 rounds the quotient to a multiple of 2^-17: the error of 1 / s
// (2^-23 of itself, 2^-20 of a quotient up to 8) cannot move it off a border that
// it is on, nor onto one that it is 2^-16 or more away from, as everything else is
// (sticky).  MX: exact.  (Packed arithmetic: each half is the IEEE operation.)
template <int FORMAT, bool WIDE>
__device__ __forceinline__ void quotient2(float x0, float x1, const Scale& s,
                                          float& q0, float& q1) {
  if constexpr (FORMAT == TPFP4_NV && WIDE) {
    x0 = __uint_as_float(sticky(__float_as_uint(x0)));
    x1 = __uint_as_float(sticky(__float_as_uint(x1)));
  }
  uint64_t t = f2_mul(f2_pack(x0, x1), f2_pack(s.m, s.m));
  if constexpr (FORMAT == TPFP4_NV) {
    t = f2_fma(t, f2_pack(s.r, s.r), f2_pack(96.f, 96.f));
    t = f2_add(t, f2_pack(-96.f, -96.f));
  }
  f2_unpack(t, q0, q1);
}

// Eight quotients to codes, the first in the lowest nibble (nearest even,
// magnitudes above 6 to 6).
__device__ __forceinline__ uint32_t codes8(const float (&q)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]),
        "f"(q[6]), "f"(q[7]));
  return w;
}

// Sixteen elements of a block to two words of codes.
template <int FORMAT, bool WIDE>
__device__ __forceinline__ uint2 codes16(const float* x, const Scale& s) {
  float q[8];
  uint2 w;
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    quotient2<FORMAT, WIDE>(x[i], x[i + 1], s, q[i], q[i + 1]);
  w.x = codes8(q);
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    quotient2<FORMAT, WIDE>(x[8 + i], x[9 + i], s, q[i], q[i + 1]);
  w.y = codes8(q);
  return w;
}

__device__ __forceinline__ uint32_t abs_bits(float x) {
  return __float_as_uint(x) & 0x7fffffffu;
}

// The value of a scale byte (0xff / 0x7f: NaN).
template <int FORMAT>
__device__ __forceinline__ float scale_value(uint32_t byte) {
  if constexpr (FORMAT == TPFP4_NV)
    return __half2float(
        __half(__nv_cvt_fp8_to_halfraw(static_cast<uint8_t>(byte), __NV_E4M3)));
  else
    return byte == 255 ? __uint_as_float(0x7fffffffu)
                       : exp2_of(static_cast<int>(byte) - 127);
}

}  // namespace fp4
}  // namespace tpmlp
