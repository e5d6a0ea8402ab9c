// Rotary positions and the per-head norm of queries and keys (tp_rope.h), one
// pass over the heads each: a head row lives in the registers of a few lanes
// from its load to its store.
//
// A row of d elements is cut into units of 2 V elements, one lane each: V pairs
// (a, b) = (i, i + r/2) or (2i, 2i + 1) that turn together; the elements past r
// follow in units of 2 V that do not turn.  A warp holds floor(32 / units) rows at
// once (one step), and a lane keeps its unit from step to step, so that what
// depends on the token and the unit only (angles, gamma, beta, the parameter
// gradients' sums) stays in registers.  The rows of the next steps are copied
// (cp.async) into a ring in shared memory, so that enough bytes are in flight
// with few registers.  Three kinds of rows:
//
//   OWN     a unit is two 16-byte vectors, one from each half of the rotated (or
//           the other) part, and a row takes 4, 8, 16 or 32 lanes: each lane copies
//           and stores its own vectors, which a row's lanes read in whole sectors;
//   PIECES  as OWN with any number of lanes: the rows of a step are copied and
//           stored as they lie in memory, in 16-byte pieces dealt to all lanes, and
//           units are read from and written to shared memory;
//   BITS    any r, d and alignment: copied in pieces of 2 to 16 bytes, read and
//           written in bits of 4, 2 or 1 elements, a unit's bits lying `units`
//           apart so that neighbouring lanes touch neighbouring bits.
//
// 8192 tokens, bf16, 201 MB in and out (floor 30 us; gradient 45 us), GB300, us:
//                              rotation   RMS norm  LayerNorm  gradients of both
//   24 + 24 heads of 128  OWN       32.8       33.5       38.5       51.4   60.0
//                      PIECES       33.2       38.1                  60.5
//                        BITS       51.0       63.2                 105.3
//   32 + 32 heads of 96 PIECES      34.8       42.8       49.8       68.6   95.1
//                        BITS       56.8       71.0                 120.1
//   40 + 40 heads of 72   BITS      46.3       60.5       72.6      101.7  129.2
//   (the last: 189 MB, floors 28 and 42)
//   (with 48 of the 96 rotated, lanes copying their own vectors, which are then
//   no whole sectors, took 43.7 for the rotation, PIECES 34.7)
//
// What bounds it: memory, where heads fill lanes exactly.  Elsewhere latency: a
// step is a chain of reads from shared memory, one or two trees of dependent
// shuffles (RMS norm, LayerNorm) and writes, and the coefficients' registers
// leave an SM 16 to 20 warps to hide it with (LayerNorm of 2047 tokens of 32 + 32
// heads of 96: 48 % of the issue slots used with 20 % of the warps, stalled on
// fixed latencies and on shared memory).  BITS predicates every bit besides.
//
// Angles: a frequency is held as turns per position in 64-bit fixed point
// (2^-64 of a turn), so position times frequency modulo one turn is one
// integer product; its upper 32 bits, as a signed fraction, go to sincospif.
// No table of cosines is read, and positions may be anything.  The lanes of a
// warp make a token's r / 2 angles once and share them through shared memory.
#pragma once
#include "common.cuh"
#include "qk_rows.cuh"

namespace tpmlp {
namespace qk {
namespace {

// ----------------------------------------------------------- arithmetic --
// On V values, two at a time (fma.rn.f32x2 and the like: two IEEE fp32
// operations per instruction, the same results).
template <int V>
__device__ __forceinline__ void mul(float (&d)[V], const float (&x)[V],
                                    const float (&y)[V]) {
#pragma unroll
  for (int j = 0; j < V; j += 2)
    f2_unpack(f2_mul(f2_pack(x[j], x[j + 1]), f2_pack(y[j], y[j + 1])), d[j],
              d[j + 1]);
}
template <int V>
__device__ __forceinline__ void mul(float (&d)[V], const float (&x)[V], float y) {
  const uint64_t yy = f2_pack(y, y);
#pragma unroll
  for (int j = 0; j < V; j += 2)
    f2_unpack(f2_mul(f2_pack(x[j], x[j + 1]), yy), d[j], d[j + 1]);
}
// d = x y + z
template <int V>
__device__ __forceinline__ void fma(float (&d)[V], const float (&x)[V],
                                    const float (&y)[V], const float (&z)[V]) {
#pragma unroll
  for (int j = 0; j < V; j += 2)
    f2_unpack(f2_fma(f2_pack(x[j], x[j + 1]), f2_pack(y[j], y[j + 1]),
                     f2_pack(z[j], z[j + 1])),
              d[j], d[j + 1]);
}
template <int V>
__device__ __forceinline__ void fma(float (&d)[V], const float (&x)[V], float y,
                                    const float (&z)[V]) {
  const uint64_t yy = f2_pack(y, y);
#pragma unroll
  for (int j = 0; j < V; j += 2)
    f2_unpack(f2_fma(f2_pack(x[j], x[j + 1]), yy, f2_pack(z[j], z[j + 1])), d[j],
              d[j + 1]);
}
template <int V>
__device__ __forceinline__ void add(float (&d)[V], const float (&x)[V]) {
#pragma unroll
  for (int j = 0; j < V; j += 2)
    f2_unpack(f2_add(f2_pack(d[j], d[j + 1]), f2_pack(x[j], x[j + 1])), d[j],
              d[j + 1]);
}
template <int V>
__device__ __forceinline__ void add(float (&d)[V], float x) {
  const uint64_t xx = f2_pack(x, x);
#pragma unroll
  for (int j = 0; j < V; j += 2)
    f2_unpack(f2_add(f2_pack(d[j], d[j + 1]), xx), d[j], d[j + 1]);
}
template <int V>
__device__ __forceinline__ float sum(const float (&x)[V]) {
  uint64_t t = f2_pack(x[0], x[1]);
#pragma unroll
  for (int j = 2; j < V; j += 2) t = f2_add(t, f2_pack(x[j], x[j + 1]));
  float lo, hi;
  f2_unpack(t, lo, hi);
  return lo + hi;
}

// A unit's V pairs.
template <int V>
struct Pairs {
  float a[V], b[V];
};
template <int V>
__device__ __forceinline__ float total(const Pairs<V>& x) {
  return sum<V>(x.a) + sum<V>(x.b);
}
template <int V>
__device__ __forceinline__ float dot(const Pairs<V>& x, const Pairs<V>& y) {
  float t[V];
  mul<V>(t, x.a, y.a);
  fma<V>(t, x.b, y.b, t);
  return sum<V>(t);
}

// ------------------------------------------------------- rows and lanes --
// The heads of one token of a view, held in registers.
template <class T>
struct HeadRows {
  T* base;
  unsigned gs, hs, group, magic;   // strides in bytes

  __device__ __forceinline__ HeadRows(const View& v, int token)
      : base(reinterpret_cast<T*>(v.p + static_cast<long long>(token) * v.ts)),
        gs(v.gs), hs(v.hs), group(v.group), magic(v.magic) {}
  __device__ __forceinline__ T* at(unsigned head) const {
    const unsigned g = __umulhi(head, magic);
    return reinterpret_cast<T*>(
        reinterpret_cast<uintptr_t>(base) +
        static_cast<unsigned long long>(g) * gs +
        static_cast<unsigned long long>(head - g * group) * hs);
  }
};

// What a lane knows of its place: the row it works on among the warp's rows,
// and its unit there.  LEN > 0: a row takes exactly LEN lanes, a power of two, and
// no lane is idle.  LEN < 0: at most 2^-LEN lanes.
struct Lane {
  int row, unit, len, first;
  bool on;
};
template <int LEN>
__device__ __forceinline__ Lane lane_place(const Args& p, int lane) {
  Lane l;
  l.len = LEN > 0 ? LEN : p.units;
  l.row = lane / l.len;
  l.unit = lane - l.row * l.len;
  l.first = l.row * l.len;
  l.on = LEN > 0 || l.row < p.rows;
  if (!l.on) l.first = 31;
  return l;
}

// Sums over the lanes of a row, the same total on every lane, in a fixed order:
// a butterfly (LEN > 0), or a tree over a row's len consecutive lanes and a
// broadcast (LEN < 0: -LEN levels).  All 32 lanes call it.
template <int LEN, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], const Lane& l) {
  if constexpr (LEN > 0) {
#pragma unroll
    for (int o = LEN / 2; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i)
        v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  } else {
#pragma unroll
    for (int o = 1 << (-LEN - 1); o > 0; o >>= 1) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float t = __shfl_down_sync(0xffffffffu, v[i], o);
        v[i] += l.unit + o < l.len ? t : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, v[i], l.first);
  }
}

// --------------------------------------------------------------- angles --
__device__ __forceinline__ long long position(const Args& p, int token) {
  if (p.pos != nullptr)
    return p.pos64 ? __ldg(static_cast<const long long*>(p.pos) + token)
                   : static_cast<long long>(
                         __ldg(static_cast<const int*>(p.pos) + token));
  const unsigned t = static_cast<unsigned>(token);
  return p.offset + (p.seq_len != 0 ? t % p.seq_len : t);
}

// A token's cosines and sines, amplitude and direction included, by one warp.
struct Trig {
  float c[MAX_PAIRS], s[MAX_PAIRS];
};
__device__ __forceinline__ void make_angles(const Args& p,
                                            const unsigned long long* freq,
                                            long long pos, int lane, Trig& t) {
  __syncwarp();   // the last token's have been read
  for (int i = lane; i < p.rot / 2; i += 32) {
    const unsigned long long ph = static_cast<unsigned long long>(pos) * freq[i];
    const int half_turns = static_cast<int>((ph + 0x80000000ull) >> 32);
    float c, s;
    sincospif(static_cast<float>(half_turns) * 0x1p-31f, &s, &c);
    t.c[i] = c * p.amp;
    t.s[i] = s * (p.amp * p.sign);
  }
  __syncwarp();
}

__device__ __forceinline__ void stage_freq(const Args& p,
                                           unsigned long long* freq) {
  for (int i = threadIdx.x; i < p.rot / 2; i += THREADS) freq[i] = p.freq[i];
  __syncthreads();
}

// ---------------------------------------------------------------- units --
// OWN and PIECES: two 16-byte vectors, at off0 and off1 of the row.  Pairs lie as
// all a, then all b, or, interleaved, as a b a b ... in either vector.
template <class T, bool INTER>
struct VectorUnit {
  static constexpr int V = 16 / static_cast<int>(sizeof(T));
  int off0, off1, unit;
  bool on, turns;

  __device__ __forceinline__ VectorUnit(const Args& p, const Lane& l)
      : unit(l.unit), on(l.on), turns(l.unit < p.rot_units) {
    if (turns) {
      off0 = V * unit;
      off1 = p.rot / 2 + off0;
    } else {
      off0 = p.rot + V * (unit - p.rot_units);
      off1 = off0 + V * (p.units - p.rot_units);
    }
  }
  // Value i (0 .. 2V - 1) of a unit in memory order, and its element.
  __device__ __forceinline__ static float& value(Pairs<V>& x, int i) {
    if constexpr (INTER) return i % 2 ? x.b[i / 2] : x.a[i / 2];
    else return i < V ? x.a[i] : x.b[i - V];
  }
  __device__ __forceinline__ int element(int i) const {
    return i < V ? off0 + i : off1 + i - V;
  }
  __device__ __forceinline__ bool has(int) const { return on; }
  __device__ __forceinline__ void centre(Pairs<V>& x, float mu) const {
    add<V>(x.a, -mu);
    add<V>(x.b, -mu);
  }
  __device__ __forceinline__ void unpack(const uint4 (&raw)[2],
                                         Pairs<V>& x) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t w[4] = {raw[h].x, raw[h].y, raw[h].z, raw[h].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
          value(x, h * V + i) = __uint_as_float(w[i]);
        } else {
          value(x, h * V + 2 * i) = __uint_as_float(w[i] << 16);
          value(x, h * V + 2 * i + 1) = __uint_as_float(w[i] & 0xffff0000u);
        }
      }
    }
  }
  __device__ __forceinline__ uint4 pack(Pairs<V>& x, int h) const {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4)
        w[i] = __float_as_uint(value(x, h * V + i));
      else
        w[i] = pack_bf16x2(value(x, h * V + 2 * i), value(x, h * V + 2 * i + 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // The unit's angles: pairs V unit ..., or, interleaved, V / 2 from each half (1
  // and 0 for a unit that does not turn).
  __device__ __forceinline__ void angles(const Args& p, const Trig& t,
                                         float (&c)[V], float (&s)[V]) const {
    constexpr int RUN = INTER ? V / 2 : V;
#pragma unroll
    for (int h = 0; h < V / RUN; ++h) {
      const int at = RUN * unit + h * (p.rot / 4);
      if constexpr (RUN % 4 == 0) {
#pragma unroll
        for (int j = 0; j < RUN; j += 4) {
          float4 x = make_float4(1.f, 1.f, 1.f, 1.f);
          float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
          if (turns) {
            x = *reinterpret_cast<const float4*>(&t.c[at + j]);
            y = *reinterpret_cast<const float4*>(&t.s[at + j]);
          }
          const int k = h * RUN + j;
          c[k] = x.x; c[k + 1] = x.y; c[k + 2] = x.z; c[k + 3] = x.w;
          s[k] = y.x; s[k + 1] = y.y; s[k + 2] = y.z; s[k + 3] = y.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < RUN; ++j) {
          c[h * RUN + j] = turns ? t.c[at + j] : 1.f;
          s[h * RUN + j] = turns ? t.s[at + j] : 0.f;
        }
      }
    }
  }
  // The unit's values of an fp32 vector [d] (null: `missing` everywhere).
  __device__ __forceinline__ void param(const Args& p, const float* g,
                                        float missing, Pairs<V>& f) const {
    const bool ok = g != nullptr && on;
    if (p.param16) {   // the vectors are 16-byte aligned
#pragma unroll
      for (int i = 0; i < 2 * V; i += 4) {
        float4 x = make_float4(missing, missing, missing, missing);
        if (ok) x = __ldg(reinterpret_cast<const float4*>(g + element(i)));
        value(f, i) = x.x;
        value(f, i + 1) = x.y;
        value(f, i + 2) = x.z;
        value(f, i + 3) = x.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2 * V; ++i)
        value(f, i) = ok ? __ldg(g + element(i)) : missing;
    }
  }
};

// BITS: 16 elements as two runs of bits of W consecutive elements, `stride` apart,
// the first at a0 and b0, of which na and nb exist: a and b, or, interleaved, the
// first and the second half of the unit's pairs a b a b ...  A bit is read in
// vectors of A elements.
template <class T, bool INTER, int A>
struct BitUnit {
  static constexpr int V = 8;
  static constexpr int W = INTER && A == 1 ? 2 : A;
  static constexpr int RUN = V / W;
  int a0, b0, stride, na, nb, d;
  bool on, turns;

  __device__ __forceinline__ BitUnit(const Args& p, const Lane& l)
      : d(p.d), on(l.on), turns(l.unit < p.rot_units) {
    const int u = turns ? l.unit : l.unit - p.rot_units;
    const int n = turns ? p.rot_units : p.units - p.rot_units;   // units
    stride = W * n;
    if (turns && !INTER) {
      const int bits = p.rot / 2 / W;
      a0 = W * u;
      b0 = p.rot / 2 + a0;
      na = nb = (bits - u + n - 1) / n;
    } else {
      const int bits = ((turns ? p.rot : p.d - p.rot) + W - 1) / W;
      const int all = (bits - u + n - 1) / n;
      a0 = (turns ? 0 : p.rot) + W * u;
      b0 = a0 + RUN * stride;
      na = min(all, RUN);
      nb = max(all - RUN, 0);
    }
    if (!on) na = nb = 0;
  }
  __device__ __forceinline__ static float& value(Pairs<V>& x, int i) {
    if constexpr (INTER) return i % 2 ? x.b[i / 2] : x.a[i / 2];
    else return i < V ? x.a[i] : x.b[i - V];
  }
  __device__ __forceinline__ int element(int i) const {
    return i < V ? a0 + i / W * stride + i % W
                 : b0 + (i - V) / W * stride + (i - V) % W;
  }
  __device__ __forceinline__ bool has(int i) const {
    const bool bit = i < V ? i / W < na : (i - V) / W < nb;
    // (a last bit of two may be one element of an odd row)
    return W > A ? bit && element(i) < d : bit;
  }
  __device__ __forceinline__ void centre(Pairs<V>& x, float mu) const {
#pragma unroll
    for (int i = 0; i < 2 * V; ++i)
      value(x, i) = has(i) ? value(x, i) - mu : 0.f;
  }
  __device__ __forceinline__ void angles(const Args&, const Trig& t,
                                         float (&c)[V], float (&s)[V]) const {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = INTER ? 2 * j : j;
      const bool ok = turns && has(i);
      const int at = INTER ? element(i) / 2 : element(i);
      c[j] = ok ? t.c[at] : 1.f;
      s[j] = ok ? t.s[at] : 0.f;
    }
  }
  __device__ __forceinline__ void param(const Args&, const float* g,
                                        float missing, Pairs<V>& f) const {
#pragma unroll
    for (int i = 0; i < 2 * V; ++i)
      value(f, i) = g != nullptr && has(i) ? __ldg(g + element(i)) : missing;
  }
  // The unit's values from a row in shared memory (zeros where it has none), and
  // back.
  __device__ __forceinline__ void read(const T* row, Pairs<V>& x) const {
#pragma unroll
    for (int i = 0; i < 2 * V; i += A) {
      if constexpr (sizeof(T) == 4 || A == 1) {
        T v[A];
        if constexpr (A == 4) {
          const float4 w = has(i)
              ? *reinterpret_cast<const float4*>(row + element(i))
              : make_float4(0.f, 0.f, 0.f, 0.f);
          v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
        } else if constexpr (A == 2) {
          const float2 w = has(i)
              ? *reinterpret_cast<const float2*>(row + element(i))
              : make_float2(0.f, 0.f);
          v[0] = w.x; v[1] = w.y;
        } else {
          v[0] = has(i) ? row[element(i)] : T(0.f);
        }
#pragma unroll
        for (int k = 0; k < A; ++k) value(x, i + k) = static_cast<float>(v[k]);
      } else {
        uint32_t w[A / 2];
        if constexpr (A == 4) {
          const uint2 v = has(i)
              ? *reinterpret_cast<const uint2*>(row + element(i))
              : make_uint2(0u, 0u);
          w[0] = v.x; w[1] = v.y;
        } else {
          w[0] = has(i) ? *reinterpret_cast<const uint32_t*>(row + element(i))
                        : 0u;
        }
#pragma unroll
        for (int k = 0; k < A / 2; ++k) {
          value(x, i + 2 * k) = __uint_as_float(w[k] << 16);
          value(x, i + 2 * k + 1) = __uint_as_float(w[k] & 0xffff0000u);
        }
      }
    }
  }
  __device__ __forceinline__ void write(T* row, Pairs<V>& y) const {
#pragma unroll
    for (int i = 0; i < 2 * V; i += A) {
      if (!has(i)) continue;
      T* to = row + element(i);
      if constexpr (sizeof(T) == 4 || A == 1) {
        if constexpr (A == 4)
          *reinterpret_cast<float4*>(to) =
              make_float4(value(y, i), value(y, i + 1), value(y, i + 2),
                          value(y, i + 3));
        else if constexpr (A == 2)
          *reinterpret_cast<float2*>(to) =
              make_float2(value(y, i), value(y, i + 1));
        else
          *to = static_cast<T>(value(y, i));
      } else if constexpr (A == 4) {
        *reinterpret_cast<uint2*>(to) =
            make_uint2(pack_bf16x2(value(y, i), value(y, i + 1)),
                       pack_bf16x2(value(y, i + 2), value(y, i + 3)));
      } else {
        *reinterpret_cast<uint32_t*>(to) =
            pack_bf16x2(value(y, i), value(y, i + 1));
      }
    }
  }
};

// ---------------------------------------------------------------- rings --
__device__ __forceinline__ void ring_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// All groups but the last `PENDING` are there.
template <int PENDING>
__device__ __forceinline__ void ring_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// BYTES from global to shared memory (zeros where not ok).
template <int BYTES>
__device__ __forceinline__ void copy_async(uint8_t* dst, const void* src,
                                           bool ok) {
  if constexpr (BYTES == 2) {   // below cp.async's sizes
    *reinterpret_cast<uint16_t*>(dst) =
        ok ? *static_cast<const uint16_t*>(src) : uint16_t(0);
  } else {
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    const int n = ok ? BYTES : 0;
    if constexpr (BYTES == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d),
                   "l"(src), "r"(n) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(d),
                   "l"(src), "n"(BYTES), "r"(n) : "memory");
  }
}

// BITS4, BITS2, BITS1: bits read in vectors of that many elements.
enum Kind : int { OWN, PIECES, BITS1, BITS2, BITS4 };
constexpr bool is_bits(Kind k) { return k >= BITS1; }
constexpr int bit_vector(Kind k) { return k == BITS4 ? 4 : k == BITS2 ? 2 : 1; }

// A warp's ring of the rows to come, STAGES steps in shared memory.
//   copy(step, rows, head, heads)  copies heads head, head + 1, ... (those below
//                                  `heads`) into the stage of `step`
//   read(step, x)                  the lane's unit (after ring_wait and sync)
//   put(step, rows, head, heads, y), then sync, then flush(...): the lane's
//                                  results to memory
// A stage is copied into again only after what was read from it has been used:
// one step later at least, with a sync between.
template <class T, bool INTER, int STAGES, Kind KIND>
struct Ring;   // defined below for BITS

// Held as [stage][vector][lane]; a lane reads only what it copied itself, so its
// own wait_group is all the waiting that is needed.
template <class T, bool INTER, int STAGES>
struct Ring<T, INTER, STAGES, OWN> {
  using Unit = VectorUnit<T, INTER>;
  static constexpr int STAGE = 2 * 32 * 16;
  static constexpr int WARP = STAGES * STAGE;
  const Unit& un;
  uint8_t* mine;
  int row;

  __device__ __forceinline__ Ring(uint8_t* warp, const Args&, const Lane& ln,
                                  const Unit& u, int lane)
      : un(u), mine(warp + lane * 16), row(ln.row) {}
  __device__ __forceinline__ void copy(int step, const HeadRows<const T>& src,
                                       int head, int heads) const {
    const bool on = head + row < heads;
    const T* from = src.at(on ? head + row : 0);
    uint8_t* st = mine + (step % STAGES) * STAGE;
    copy_async<16>(st, from + un.off0, on);
    copy_async<16>(st + 32 * 16, from + un.off1, on);
  }
  __device__ __forceinline__ void sync() const {}
  __device__ __forceinline__ void read(int step, Pairs<Unit::V>& x) const {
    const uint8_t* st = mine + (step % STAGES) * STAGE;
    const uint4 raw[2] = {*reinterpret_cast<const uint4*>(st),
                          *reinterpret_cast<const uint4*>(st + 32 * 16)};
    un.unpack(raw, x);
  }
  __device__ __forceinline__ void put(int, const HeadRows<T>& dst, int head,
                                      int heads, Pairs<Unit::V>& y) const {
    if (head + row >= heads) return;
    T* to = dst.at(head + row);
    *reinterpret_cast<uint4*>(to + un.off0) = un.pack(y, 0);
    *reinterpret_cast<uint4*>(to + un.off1) = un.pack(y, 1);
  }
  __device__ __forceinline__ void flush(int, const HeadRows<T>&, int, int) const {}
};

// A step's rows one after the other, in 16-byte pieces dealt to the lanes in two
// rounds: at most 62 (31 units of a row, 248 elements of fp32), so that piece 63
// is nobody's and idle lanes may read it.
template <class T, bool INTER, int STAGES>
struct Ring<T, INTER, STAGES, PIECES> {
  using Unit = VectorUnit<T, INTER>;
  static constexpr int STAGE = 64 * 16;
  static constexpr int WARP = STAGES * STAGE;
  const Unit& un;
  uint8_t* mine;       // this lane's first piece in stage 0
  uint8_t* at0;        // this lane's vectors in stage 0
  uint8_t* at1;
  int row[2], col[2];  // its pieces: row (past the step's rows: none), byte

  __device__ __forceinline__ Ring(uint8_t* warp, const Args& p, const Lane& ln,
                                  const Unit& u, int lane)
      : un(u), mine(warp + lane * 16) {
    const int bytes = p.d * static_cast<int>(sizeof(T)), pieces = bytes / 16;
    at0 = warp + ln.row * bytes + un.off0 * static_cast<int>(sizeof(T));
    at1 = warp + ln.row * bytes + un.off1 * static_cast<int>(sizeof(T));
    // an idle lane reads the last piece, which then holds no row's elements
    if (!un.on) at0 = at1 = warp + 63 * 16;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int i = lane + 32 * v;
      row[v] = i / pieces;
      col[v] = (i - row[v] * pieces) * 16;
      if (row[v] >= p.rows) row[v] = 1 << 20;
    }
  }
  __device__ __forceinline__ void copy(int step, const HeadRows<const T>& src,
                                       int head, int heads) const {
    uint8_t* st = mine + (step % STAGES) * STAGE;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const bool on = head + row[v] < heads;
      copy_async<16>(st + 32 * 16 * v,
                     reinterpret_cast<const uint8_t*>(
                         src.at(on ? head + row[v] : 0)) + col[v],
                     on);
    }
  }
  // Other lanes' copies are read after this (and after each lane's wait), and
  // copied over only after the next.
  __device__ __forceinline__ void sync() const { __syncwarp(); }
  __device__ __forceinline__ void read(int step, Pairs<Unit::V>& x) const {
    const int st = (step % STAGES) * STAGE;
    const uint4 raw[2] = {*reinterpret_cast<const uint4*>(at0 + st),
                          *reinterpret_cast<const uint4*>(at1 + st)};
    un.unpack(raw, x);
  }
  __device__ __forceinline__ void put(int step, const HeadRows<T>&, int, int,
                                      Pairs<Unit::V>& y) const {
    const int st = (step % STAGES) * STAGE;
    if (!un.on) return;
    *reinterpret_cast<uint4*>(at0 + st) = un.pack(y, 0);
    *reinterpret_cast<uint4*>(at1 + st) = un.pack(y, 1);
  }
  __device__ __forceinline__ void flush(int step, const HeadRows<T>& dst,
                                        int head, int heads) const {
    const uint8_t* st = mine + (step % STAGES) * STAGE;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      if (head + row[v] >= heads) continue;
      *reinterpret_cast<uint4*>(
          reinterpret_cast<uint8_t*>(dst.at(head + row[v])) + col[v]) =
          *reinterpret_cast<const uint4*>(st + 32 * 16 * v);
    }
  }
};

// The same with pieces of p.piece bytes (16, 8, 4 or 2), in as many rounds as
// they take: at most 512 elements.
template <class T, bool INTER, int STAGES, Kind KIND>
struct Ring {
  using Unit = BitUnit<T, INTER, bit_vector(KIND)>;
  static constexpr int V = Unit::V;
  static constexpr int STAGE = 512 * static_cast<int>(sizeof(T));
  static constexpr int WARP = STAGES * STAGE;
  const Unit& un;
  const Args& p;
  uint8_t* warp;
  int lane, row;

  __device__ __forceinline__ Ring(uint8_t* w, const Args& args, const Lane& ln,
                                  const Unit& u, int l)
      : un(u), p(args), warp(w), lane(l), row(un.on ? ln.row : 0) {}
  // f(piece, its row, its byte there) for the lane's pieces of the heads head,
  // head + 1, ... that exist.
  template <int BYTES, class F>
  __device__ __forceinline__ void pieces(int head, int heads, F&& f) const {
    const int n = min(p.rows, heads - head) * p.row_pieces;
    for (int i0 = lane; i0 < n; i0 += 64) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = i0 + 32 * k;
        if (i >= n) break;
        const int r = p.row_pieces == 1
                          ? i : static_cast<int>(__umulhi(i, p.row_pieces_magic));
        f(i, r, (i - r * p.row_pieces) * BYTES);
      }
    }
  }
  template <int BYTES>
  __device__ __forceinline__ void copy_pieces(uint8_t* st,
                                              const HeadRows<const T>& src,
                                              int head, int heads) const {
    pieces<BYTES>(head, heads, [&](int i, int r, int byte) {
      copy_async<BYTES>(st + i * BYTES,
                        reinterpret_cast<const uint8_t*>(src.at(head + r)) +
                            byte,
                        true);
    });
  }
  __device__ __forceinline__ void copy(int step, const HeadRows<const T>& src,
                                       int head, int heads) const {
    uint8_t* st = warp + (step % STAGES) * STAGE;
    if (p.piece == 16) copy_pieces<16>(st, src, head, heads);
    else if (p.piece == 8) copy_pieces<8>(st, src, head, heads);
    else if (p.piece == 4) copy_pieces<4>(st, src, head, heads);
    else copy_pieces<2>(st, src, head, heads);
  }
  __device__ __forceinline__ void sync() const { __syncwarp(); }
  __device__ __forceinline__ T* place(int step) const {
    return reinterpret_cast<T*>(warp + (step % STAGES) * STAGE) + row * p.d;
  }
  // (Rows past the last head hold what was there before: they are read, and
  // go nowhere but into the gradient's sums, which leave them out.)
  __device__ __forceinline__ void read(int step, Pairs<V>& x) const {
    un.read(place(step), x);
  }
  __device__ __forceinline__ void put(int step, const HeadRows<T>&, int, int,
                                      Pairs<V>& y) const {
    un.write(place(step), y);
  }
  template <class P>
  __device__ __forceinline__ void flush_pieces(const uint8_t* st,
                                               const HeadRows<T>& dst, int head,
                                               int heads) const {
    constexpr int BYTES = static_cast<int>(sizeof(P));
    pieces<BYTES>(head, heads, [&](int i, int r, int byte) {
      *reinterpret_cast<P*>(reinterpret_cast<uint8_t*>(dst.at(head + r)) +
                            byte) =
          *reinterpret_cast<const P*>(st + i * BYTES);
    });
  }
  __device__ __forceinline__ void flush(int step, const HeadRows<T>& dst,
                                        int head, int heads) const {
    const uint8_t* st = warp + (step % STAGES) * STAGE;
    if (p.piece == 16) flush_pieces<uint4>(st, dst, head, heads);
    else if (p.piece == 8) flush_pieces<uint2>(st, dst, head, heads);
    else if (p.piece == 4) flush_pieces<uint32_t>(st, dst, head, heads);
    else flush_pieces<uint16_t>(st, dst, head, heads);
  }
};

// -------------------------------------------------------------- forward --
// GPT-3-13B-shaped layer (8192 tokens, 40 + 40 heads of 128, bf16, 336 MB in and
// out): rotation 50.9 us, 6.6 TB/s; norm and rotation 52.0 us, 6.5 TB/s (61 and 71
// with a row loaded when it was needed).  Two steps at a time, to share issue
// slots, gave 50.7 and 51.8, but for the LayerNorm 35.7 instead of 33.8 (40 + 40
// heads of 64) and 55.2 instead of 51.4 (32 + 32 of 96): not kept.
//
// What a lane multiplies a row's unit by: y_a = rstd (a ca + b sb) + za, y_b =
// rstd (a sa + b cb) + zb, with gamma folded into the rotation and beta rotated.
template <int V>
struct Turn {
  float ca[V], sb[V], sa[V], cb[V];
  float za[V], zb[V];
};
template <int NORM, class U>
__device__ __forceinline__ void load_turn(const Args& p, const Side& sd,
                                          const Trig& trig, const U& un,
                                          Turn<U::V>& t) {
  constexpr int V = U::V;
  un.angles(p, trig, t.ca, t.sa);
  if constexpr (NORM == 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      t.cb[j] = t.ca[j];
      t.sb[j] = -t.sa[j];
    }
  } else {
    Pairs<V> gam;
    un.param(p, sd.gamma, 1.f, gam);
    if constexpr (NORM == TPQK_LAYERNORM) {
      Pairs<V> bet;
      un.param(p, sd.beta, 0.f, bet);
      // (a beta past r meets no other, as x does not in the loop over rows)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        t.za[j] = un.turns ? fmaf(bet.a[j], t.ca[j], -(bet.b[j] * t.sa[j]))
                           : bet.a[j];
        t.zb[j] = un.turns ? fmaf(bet.a[j], t.sa[j], bet.b[j] * t.ca[j])
                           : bet.b[j];
      }
    }
    mul<V>(t.cb, t.ca, gam.b);
#pragma unroll
    for (int j = 0; j < V; ++j) t.sb[j] = -(t.sa[j] * gam.b[j]);
    mul<V>(t.ca, t.ca, gam.a);
    mul<V>(t.sa, t.sa, gam.a);
  }
}

// Blocks an SM has to hold, and so registers a thread may take: five where that
// spills nothing (RMS norm, 8192 tokens of 24 + 24 heads of 128: 33.2 us, with four
// 34.3; of 32 + 32 heads of 96, where it spills, 61.5 and 44.6 with six and four).
constexpr int forward_blocks(Kind kind, int norm) {
  return (norm == 0 && !is_bits(kind)) || (norm == TPQK_RMSNORM && kind == OWN)
             ? 5 : 4;
}

template <class T, Kind KIND, int NORM, bool INTER, int LEN>
__global__ void __launch_bounds__(THREADS, forward_blocks(KIND, NORM))
    qk_rows_forward(const __grid_constant__ Args p) {
  // Steps ahead that are being copied, one group each (GPT-3-13B-shaped layer, RMS:
  // five 52.0 us, three 53.1; rows in PIECES are faster with three: 32 + 32 heads
  // of 96 42.9 and 44.6).
  constexpr int STAGES = KIND == OWN ? 8 : 4;
  constexpr int AHEAD = KIND == OWN ? 5 : 3;
  using R = Ring<T, INTER, STAGES, KIND>;
  using U = typename R::Unit;
  constexpr int V = U::V;
  __shared__ __align__(16) uint8_t ring_mem[WARPS * R::WARP];
  __shared__ unsigned long long freq[MAX_PAIRS];
  __shared__ __align__(16) Trig trig[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned task = blockIdx.x * WARPS + warp;
  const int token = static_cast<int>(task / static_cast<unsigned>(p.segs));
  const int mid = p.side[0].steps;   // first step of k
  int s0 = static_cast<int>(task - token * p.segs) * p.per;
  int s1 = min(s0 + p.per, mid + p.side[1].steps);
  if (token >= p.tokens) s0 = s1 = 0;
  const Lane ln = lane_place<LEN>(p, lane);
  const U un(p, ln);
  const R ring(ring_mem + warp * R::WARP, p, ln, un, lane);
  // The next step to copy, and its side's rows and first head.
  int sc = s0;
  HeadRows<const T> src(p.side[s0 >= mid].in, token);
  int src_heads = p.side[s0 >= mid].heads;
  int hc = (s0 >= mid ? s0 - mid : s0) * p.rows;
  auto copy = [&] {
    if (sc < s1) {
      if (sc == mid) {   // on to k
        src = HeadRows<const T>(p.side[1].in, token);
        src_heads = p.side[1].heads;
        hc = 0;
      }
      ring.copy(sc, src, hc, src_heads);
      hc += p.rows;
      ++sc;
    }
    ring_commit();
  };
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) copy();
  stage_freq(p, freq);
  if (s0 >= s1) return;
  make_angles(p, freq, position(p, token), lane, trig[warp]);
#pragma unroll 1
  for (int which = s0 >= mid; which < 2; ++which) {
    // this task's steps of one side
    const Side& sd = p.side[which];
    const int end = which ? s1 : min(s1, mid);
    int s = which ? max(s0, mid) : s0;
    if (s >= end) break;
    const HeadRows<T> dst(sd.out, token);
    const int heads = sd.heads;
    int h = (which ? s - mid : s) * p.rows;
    Turn<V> t;
    load_turn<NORM>(p, sd, trig[warp], un, t);
#pragma unroll 1
    for (; s < end; ++s) {
      ring_wait<AHEAD - 1>();
      ring.sync();
      Pairs<V> x;
      ring.read(s, x);
      copy();
      float scale[1];
      if constexpr (NORM == TPQK_LAYERNORM) {
        float m[1] = {total<V>(x)};
        row_sum<LEN>(m, ln);
        un.centre(x, m[0] * p.inv_d);
      }
      if constexpr (NORM != 0) {
        scale[0] = dot<V>(x, x);
        row_sum<LEN>(scale, ln);
        scale[0] = rsqrtf(fmaf(scale[0], p.inv_d, p.eps));
      }
      // The rotation does not wait for the norm's sum.  (Values that do not
      // turn have nothing to do with one another: an infinity among them must
      // not meet another's zero sine.)
      Pairs<V> y;
      if (un.turns) {
        mul<V>(y.a, x.b, t.sb);
        mul<V>(y.b, x.b, t.cb);
        fma<V>(y.a, x.a, t.ca, y.a);
        fma<V>(y.b, x.a, t.sa, y.b);
      } else {
        mul<V>(y.a, x.a, t.ca);
        mul<V>(y.b, x.b, t.cb);
      }
      if constexpr (NORM == TPQK_LAYERNORM) {
        fma<V>(y.a, y.a, scale[0], t.za);
        fma<V>(y.b, y.b, scale[0], t.zb);
      } else if constexpr (NORM != 0) {
        mul<V>(y.a, y.a, scale[0]);
        mul<V>(y.b, y.b, scale[0]);
      }
      ring.put(s, dst, h, heads, y);
      ring.sync();
      ring.flush(s, dst, h, heads);
      h += p.rows;
    }
  }
}

// ------------------------------------------------------------- backward --
// With g = R^T dy, u = g gamma and e = x - mu:
//   xh = rstd e,  dgamma += (rstd g) e,  dbeta += g,
//   dx = (rstd g) gamma - (rstd^3 sum(e u) / d) e [- rstd mean(u)].
// Persistent blocks, so that a lane sums its unit's parameter gradients over
// all its rows in registers; a block takes q's tasks or k's.  Four blocks an SM:
// with three (more registers) the LayerNorm gradient of 8192 tokens of 24 + 24
// heads of 128 takes 72 us instead of 60.  Four leave 128 registers a thread, at
// which gradients of the LayerNorm spill: OWN in bf16 4 to 12 bytes, PIECES in
// bf16 64, BITS 44 to 120 (of the RMS norm 4 to 40); OWN and PIECES in fp32, and
// the forward but for 4 bytes in one of its BITS variants, nothing.
// GPT-3-13B-shaped layer, RMS: 79.5 us with the sums, 503 MB, 6.3 TB/s (177 with
// rows loaded when they were needed).
template <class T, Kind KIND, int NORM, bool INTER, int LEN>
__global__ void __launch_bounds__(THREADS, 4)
    qk_rows_backward(const __grid_constant__ Args p) {
  constexpr int STAGES = is_bits(KIND) && sizeof(T) == 4 ? 2 : 4;
  constexpr int AHEAD = STAGES - 1;
  using R = Ring<T, INTER, STAGES, KIND>;
  using U = typename R::Unit;
  constexpr int V = U::V;
  __shared__ __align__(16) uint8_t ring_mem[2 * WARPS * R::WARP];
  __shared__ unsigned long long freq[MAX_PAIRS];
  __shared__ __align__(16) Trig trig[WARPS];
  // at the end it holds a sum for every element of every row slot
  static_assert(2 * R::WARP >= 32 * 2 * V * 4, "ring_mem is too small");
  // the blocks' sums are added by a launch that may come up meanwhile
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  stage_freq(p, freq);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int which = static_cast<int>(blockIdx.x) >= p.q_blocks;
  const Side& sd = p.side[which];
  const unsigned blocks = which ? gridDim.x - p.q_blocks : p.q_blocks;
  const unsigned block = which ? blockIdx.x - p.q_blocks : blockIdx.x;
  const unsigned segs = p.segs_side[which];
  const int per = p.per_side[which], heads = sd.heads;
  const Lane ln = lane_place<LEN>(p, lane);
  const U un(p, ln);
  Pairs<V> gam, dgam, dbet;
  un.param(p, sd.gamma, 1.f, gam);
#pragma unroll
  for (int j = 0; j < V; ++j)
    dgam.a[j] = dgam.b[j] = dbet.a[j] = dbet.b[j] = 0.f;
  const R gring(ring_mem + 2 * warp * R::WARP, p, ln, un, lane);
  const R xring(ring_mem + (2 * warp + 1) * R::WARP, p, ln, un, lane);
  const unsigned tasks = static_cast<unsigned>(p.tokens) * segs;
  for (unsigned task = block * WARPS + warp; task < tasks;
       task += blocks * WARPS) {
    const int token = static_cast<int>(task / segs);
    const int s0 = static_cast<int>(task - token * segs) * per;
    const int s1 = min(s0 + per, sd.steps);
    const HeadRows<const T> gsrc(sd.in, token), xsrc(sd.x, token);
    const HeadRows<T> dst(sd.out, token);
    int sc = s0, h = s0 * p.rows, hc = h;
    auto copy = [&] {
      if (sc < s1) {
        gring.copy(sc, gsrc, hc, heads);
        xring.copy(sc, xsrc, hc, heads);
        hc += p.rows;
        ++sc;
      }
      ring_commit();
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) copy();
    make_angles(p, freq, position(p, token), lane, trig[warp]);
    float c[V], sa[V];
    un.angles(p, trig[warp], c, sa);
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
      ring_wait<AHEAD - 1>();
      gring.sync();
      Pairs<V> g, e;
      {
        Pairs<V> dy;
        gring.read(s, dy);
        xring.read(s, e);
        copy();
        // R^T (sa carries the opposite direction's sign)
        g = dy;
        if (un.turns) {
          float t[V];
          mul<V>(t, dy.b, -1.f);
          mul<V>(g.a, t, sa);
          fma<V>(g.a, dy.a, c, g.a);
          mul<V>(g.b, dy.b, c);
          fma<V>(g.b, dy.a, sa, g.b);
        }
      }
      if constexpr (is_bits(KIND)) {   // rows past the last head
        if (h + ln.row >= heads) {
#pragma unroll
          for (int j = 0; j < V; ++j) g.a[j] = g.b[j] = e.a[j] = e.b[j] = 0.f;
        }
      }
      float mean_u = 0.f;
      if constexpr (NORM == TPQK_LAYERNORM) {
        float m[2] = {total<V>(e), dot<V>(g, gam)};
        row_sum<LEN>(m, ln);
        un.centre(e, m[0] * p.inv_d);
        mean_u = m[1] * p.inv_d;
      }
      float q[2] = {dot<V>(e, e), 0.f};
      {   // sum of e u
        float t[V], u[V];
        mul<V>(u, g.a, gam.a);
        mul<V>(t, u, e.a);
        mul<V>(u, g.b, gam.b);
        fma<V>(t, u, e.b, t);
        q[1] = sum<V>(t);
      }
      row_sum<LEN>(q, ln);
      const float rstd = rsqrtf(fmaf(q[0], p.inv_d, p.eps));
      // (in this order: rstd^2 alone may overflow where the sum is zero)
      const float k = -(q[1] * rstd * p.inv_d * rstd * rstd);
      if constexpr (NORM == TPQK_LAYERNORM) {
        add<V>(dbet.a, g.a);
        add<V>(dbet.b, g.b);
      }
      mul<V>(g.a, g.a, rstd);
      mul<V>(g.b, g.b, rstd);
      // (a row that does not exist is zero, and with eps = 0 its rstd infinite)
      if (h + p.rows <= heads || h + ln.row < heads) {
        fma<V>(dgam.a, g.a, e.a, dgam.a);
        fma<V>(dgam.b, g.b, e.b, dgam.b);
      }
      Pairs<V> dx;
      mul<V>(dx.a, e.a, k);
      mul<V>(dx.b, e.b, k);
      if constexpr (NORM == TPQK_LAYERNORM) {
        const float m = -rstd * mean_u;
        add<V>(dx.a, m);
        add<V>(dx.b, m);
      }
      fma<V>(dx.a, g.a, gam.a, dx.a);
      fma<V>(dx.b, g.b, gam.b, dx.b);
      gring.put(s, dst, h, heads, dx);
      gring.sync();
      gring.flush(s, dst, h, heads);
      h += p.rows;
    }
    // The ring is empty again: its last steps' groups hold nothing.  (Before the
    // next task's copies, every lane has left the last stage.)
    gring.sync();
  }
  if (p.part == nullptr) return;
  // the block's sums: element i of every row slot, in the order of the slots
  float* sums = reinterpret_cast<float*>(ring_mem);
  const int slots = WARPS * p.rows;
#pragma unroll
  for (int k = 0; k < (NORM == TPQK_LAYERNORM ? 2 : 1); ++k) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2 * V; ++i)
      if (un.has(i))
        sums[(warp * p.rows + ln.row) * p.d + un.element(i)] =
            U::value(k ? dbet : dgam, i);
    __syncthreads();
    for (int i = threadIdx.x; i < p.d; i += THREADS) {
      float t = 0.f;
      for (int w = 0; w < slots; ++w) t += sums[w * p.d + i];
      p.part[(static_cast<long long>(blockIdx.x) * 2 + k) * p.d + i] = t;
    }
  }
}

// ------------------------------------------------------------- dispatch --
template <class T, Kind KIND, int NORM, bool INTER, int LEN>
cudaError_t go(const Args& a, int blocks, bool backward, cudaStream_t s) {
  if (!backward) {
    qk_rows_forward<T, KIND, NORM, INTER, LEN><<<blocks, THREADS, 0, s>>>(a);
  } else if constexpr (NORM != 0) {
    qk_rows_backward<T, KIND, NORM, INTER, LEN><<<blocks, THREADS, 0, s>>>(a);
  }
  return cudaGetLastError();
}

template <class T, int NORM, bool INTER>
cudaError_t by_length(const Args& a, int bits, int blocks, bool backward,
                      cudaStream_t s) {
  constexpr int SHORT = 2 * static_cast<int>(sizeof(T));   // 64 elements
  if (bits == 4)
    return a.units <= 8 ? go<T, BITS4, NORM, INTER, -3>(a, blocks, backward, s)
                        : go<T, BITS4, NORM, INTER, -5>(a, blocks, backward, s);
  if (bits == 2)
    return a.units <= 8 ? go<T, BITS2, NORM, INTER, -3>(a, blocks, backward, s)
                        : go<T, BITS2, NORM, INTER, -5>(a, blocks, backward, s);
  if (bits == 1)
    return a.units <= 8 ? go<T, BITS1, NORM, INTER, -3>(a, blocks, backward, s)
                        : go<T, BITS1, NORM, INTER, -5>(a, blocks, backward, s);
  if (a.units == SHORT)
    return go<T, OWN, NORM, INTER, SHORT>(a, blocks, backward, s);
  if (a.units == 2 * SHORT)
    return go<T, OWN, NORM, INTER, 2 * SHORT>(a, blocks, backward, s);
  if (a.units == 4 * SHORT)
    return go<T, OWN, NORM, INTER, 4 * SHORT>(a, blocks, backward, s);
  if (a.units <= 8)
    return go<T, PIECES, NORM, INTER, -3>(a, blocks, backward, s);
  if constexpr (sizeof(T) == 4)
    if (a.units > 16)
      return go<T, PIECES, NORM, INTER, -5>(a, blocks, backward, s);
  return go<T, PIECES, NORM, INTER, -4>(a, blocks, backward, s);
}

template <class T>
cudaError_t by_norm(const Args& a, int bits, int norm, bool inter,
                    int blocks, bool backward, cudaStream_t s) {
  if (norm == TPQK_RMSNORM)
    return (inter ? by_length<T, TPQK_RMSNORM, true>
                  : by_length<T, TPQK_RMSNORM, false>)(a, bits, blocks,
                                                       backward, s);
  if (norm == TPQK_LAYERNORM)
    return (inter ? by_length<T, TPQK_LAYERNORM, true>
                  : by_length<T, TPQK_LAYERNORM, false>)(a, bits, blocks,
                                                         backward, s);
  return (inter ? by_length<T, 0, true> : by_length<T, 0, false>)(
      a, bits, blocks, backward, s);
}

}  // namespace
}  // namespace qk
}  // namespace tpmlp
