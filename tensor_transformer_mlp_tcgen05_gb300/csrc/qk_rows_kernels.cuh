// Rotary positions and the per-head norm of queries and keys (tp_rope.h), one
// pass over the heads each: a head row lives in the registers of a few lanes
// from its load to its store.
//
// A row of d elements is cut into units of 2 V elements, one lane each: V
// pairs (a, b) = (i, i + r/2) or (2i, 2i + 1) that turn together, read as two
// V-wide vectors, one from each half of the rotated part (so that the lanes of a
// row read consecutive vectors; interleaved pairs lie in one vector either way);
// the elements past r follow in units of 2 V that do not turn, again one vector
// from each half.
// A warp holds floor(32 / units) rows at once (one step), and a lane keeps its
// unit from step to step, so that what depends on the token and the unit only
// (angles, gamma, beta, the parameter gradients' sums) stays in registers.  Each
// lane copies its own units of the next steps into a ring in shared memory
// (cp.async), so that enough bytes are in flight with few registers.
//
// Angles: a frequency is held as turns per position in 64-bit fixed point
// (2^-64 of a turn), so position times frequency modulo one turn is one
// integer product; its upper 32 bits, as a signed fraction, go to sincospif.
// No table of cosines is read, and positions may be anything.  The lanes of a
// warp make a token's r / 2 angles once, one pair each, and share them through
// shared memory.
#pragma once
#include "common.cuh"
#include "qk_rows.cuh"

namespace tpmlp {
namespace qk {
namespace {

// ------------------------------------------------------------ vectors --
template <int BYTES> struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<2> { using type = uint16_t; };

template <class T, int V>
using RawT = typename Raw<V * static_cast<int>(sizeof(T))>::type;

// The two vectors of a unit as loaded.
template <class T, int V>
struct RawUnit {
  RawT<T, V> v[2];
};

// A unit's V pairs.
template <int V>
struct Pairs {
  float a[V], b[V];
};

// Element i (0 .. 2V - 1, memory order) of a unit: V pairs lie as all a, then
// all b, or, interleaved, as a b a b ...
template <int V, bool INTER>
__device__ __forceinline__ float& element(Pairs<V>& p, int i) {
  if constexpr (INTER) return i % 2 ? p.b[i / 2] : p.a[i / 2];
  else return i < V ? p.a[i] : p.b[i - V];
}

template <class T, int V, bool INTER>
__device__ __forceinline__ void unpack(const RawUnit<T, V>& raw, Pairs<V>& p) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (sizeof(T) == 4) {
      const float* w = reinterpret_cast<const float*>(&raw.v[h]);
#pragma unroll
      for (int i = 0; i < V; ++i) element<V, INTER>(p, h * V + i) = w[i];
    } else if constexpr (V == 1) {
      element<V, INTER>(p, h) =
          __uint_as_float(static_cast<uint32_t>(raw.v[h]) << 16);
    } else {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw.v[h]);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        element<V, INTER>(p, h * V + 2 * i) = __uint_as_float(w[i] << 16);
        element<V, INTER>(p, h * V + 2 * i + 1) =
            __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
}

template <class T, int V, bool INTER>
__device__ __forceinline__ RawT<T, V> pack(Pairs<V>& p, int h) {
  RawT<T, V> raw;
  if constexpr (sizeof(T) == 4) {
    float* w = reinterpret_cast<float*>(&raw);
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = element<V, INTER>(p, h * V + i);
  } else if constexpr (V == 1) {
    raw = __bfloat16_as_ushort(__float2bfloat16_rn(element<V, INTER>(p, h)));
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(&raw);
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
      w[i] = pack_bf16x2(element<V, INTER>(p, h * V + 2 * i),
                         element<V, INTER>(p, h * V + 2 * i + 1));
  }
  return raw;
}

// Arithmetic on V values, two at a time where V is even (fma.rn.f32x2 and the
// like: two IEEE fp32 operations per instruction, the same results).
template <int V>
__device__ __forceinline__ void mul(float (&d)[V], const float (&x)[V],
                                    const float (&y)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2)
      f2_unpack(f2_mul(f2_pack(x[j], x[j + 1]), f2_pack(y[j], y[j + 1])), d[j],
                d[j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] = x[j] * y[j];
  }
}
template <int V>
__device__ __forceinline__ void mul(float (&d)[V], const float (&x)[V], float y) {
  if constexpr (V % 2 == 0) {
    const uint64_t yy = f2_pack(y, y);
#pragma unroll
    for (int j = 0; j < V; j += 2)
      f2_unpack(f2_mul(f2_pack(x[j], x[j + 1]), yy), d[j], d[j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] = x[j] * y;
  }
}
// d = x y + z
template <int V>
__device__ __forceinline__ void fma(float (&d)[V], const float (&x)[V],
                                    const float (&y)[V], const float (&z)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2)
      f2_unpack(f2_fma(f2_pack(x[j], x[j + 1]), f2_pack(y[j], y[j + 1]),
                       f2_pack(z[j], z[j + 1])),
                d[j], d[j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] = fmaf(x[j], y[j], z[j]);
  }
}
template <int V>
__device__ __forceinline__ void fma(float (&d)[V], const float (&x)[V], float y,
                                    const float (&z)[V]) {
  if constexpr (V % 2 == 0) {
    const uint64_t yy = f2_pack(y, y);
#pragma unroll
    for (int j = 0; j < V; j += 2)
      f2_unpack(f2_fma(f2_pack(x[j], x[j + 1]), yy, f2_pack(z[j], z[j + 1])),
                d[j], d[j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] = fmaf(x[j], y, z[j]);
  }
}
template <int V>
__device__ __forceinline__ void add(float (&d)[V], const float (&x)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2)
      f2_unpack(f2_add(f2_pack(d[j], d[j + 1]), f2_pack(x[j], x[j + 1])), d[j],
                d[j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] += x[j];
  }
}
template <int V>
__device__ __forceinline__ void add(float (&d)[V], float x) {
  if constexpr (V % 2 == 0) {
    const uint64_t xx = f2_pack(x, x);
#pragma unroll
    for (int j = 0; j < V; j += 2)
      f2_unpack(f2_add(f2_pack(d[j], d[j + 1]), xx), d[j], d[j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] += x;
  }
}
template <int V>
__device__ __forceinline__ float sum(const float (&x)[V]) {
  if constexpr (V >= 4) {
    uint64_t t = f2_pack(x[0], x[1]);
#pragma unroll
    for (int j = 2; j < V; j += 2) t = f2_add(t, f2_pack(x[j], x[j + 1]));
    float lo, hi;
    f2_unpack(t, lo, hi);
    return lo + hi;
  } else {
    float s = x[0];
#pragma unroll
    for (int j = 1; j < V; ++j) s += x[j];
    return s;
  }
}

// sum over a lane's units of x y, over a and b.
template <int V, int NU>
__device__ __forceinline__ float dot(const Pairs<V> (&x)[NU],
                                     const Pairs<V> (&y)[NU]) {
  float t[V];
  mul<V>(t, x[0].a, y[0].a);
  fma<V>(t, x[0].b, y[0].b, t);
#pragma unroll
  for (int n = 1; n < NU; ++n) {
    fma<V>(t, x[n].a, y[n].a, t);
    fma<V>(t, x[n].b, y[n].b, t);
  }
  return sum<V>(t);
}

template <int V, int NU>
__device__ __forceinline__ float total(const Pairs<V> (&x)[NU]) {
  float t = 0.f;
#pragma unroll
  for (int n = 0; n < NU; ++n) t += sum<V>(x[n].a) + sum<V>(x[n].b);
  return t;
}

// ------------------------------------------------------ rows and units --
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

// The two vectors of a unit: element offsets and whether they exist.  WHOLE: a
// lane has one unit, with both vectors (or is idle).
struct Unit {
  int off0, off1;
  bool ok0, ok1;
};
template <int V, bool INTER, bool WHOLE>
__device__ __forceinline__ Unit unit_at(const Args& p, int u, bool lane_on) {
  Unit n;
  n.ok0 = lane_on && (WHOLE || u < p.units);
  n.ok1 = n.ok0;
  if (u < p.rot_units) {
    if constexpr (INTER && V == 1) {   // a pair is two vectors
      n.off0 = 2 * u;
      n.off1 = n.off0 + 1;
    } else {
      n.off0 = V * u;
      n.off1 = p.rot / 2 + n.off0;
    }
  } else {
    n.off0 = p.rot + V * (u - p.rot_units);
    n.off1 = n.off0 + V * (p.units - p.rot_units);
    if (!WHOLE) n.ok1 = n.ok0 && n.off1 < p.d;
  }
  if (!n.ok0) n.off0 = 0;   // (addresses only; nothing is read or written)
  if (!n.ok1) n.off1 = 0;
  return n;
}

// A unit's values of an fp32 vector [d] (null: `missing` everywhere).
template <int V, bool INTER>
__device__ __forceinline__ void load_param(const Args& p, const float* g,
                                           float missing, const Unit& n,
                                           Pairs<V>& f) {
  const bool ok0 = g != nullptr && n.ok0, ok1 = g != nullptr && n.ok1;
  if constexpr (V % 4 == 0) {
    if (p.param16) {   // the vectors are 16-byte aligned
#pragma unroll
      for (int i = 0; i < 2 * V; i += 4) {
        float4 x = make_float4(missing, missing, missing, missing);
        if (i < V ? ok0 : ok1)
          x = __ldg(reinterpret_cast<const float4*>(
              g + (i < V ? n.off0 + i : n.off1 + i - V)));
        element<V, INTER>(f, i) = x.x;
        element<V, INTER>(f, i + 1) = x.y;
        element<V, INTER>(f, i + 2) = x.z;
        element<V, INTER>(f, i + 3) = x.w;
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    element<V, INTER>(f, i) = ok0 ? __ldg(g + n.off0 + i) : missing;
    element<V, INTER>(f, V + i) = ok1 ? __ldg(g + n.off1 + i) : missing;
  }
}

// x - mu, zero where the row has no element.
template <int V, bool INTER, bool WHOLE>
__device__ __forceinline__ void centre(Pairs<V>& x, const Unit& n, float mu) {
  if constexpr (WHOLE) {
    add<V>(x.a, -mu);
    add<V>(x.b, -mu);
  } else {
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) {
      float& e = element<V, INTER>(x, i);
      e = (i < V ? n.ok0 : n.ok1) ? e - mu : 0.f;
    }
  }
}

// What a lane knows of its place: the row it works on among the warp's rows,
// and its first unit there (g; then g + 32, ...).  LEN > 0: a row takes exactly
// LEN lanes, a power of two, and no lane is idle.  LEN < 0: at most 2^-LEN lanes.
struct Lane {
  int row, g, len, first;
  bool on;
};
template <int LEN>
__device__ __forceinline__ Lane lane_place(const Args& p, int lane) {
  Lane l;
  l.len = LEN > 0 ? LEN : min(p.units, 32);
  l.row = lane / l.len;
  l.g = lane - l.row * l.len;
  l.first = l.row * l.len;
  l.on = LEN > 0 || l.row < p.rows;
  if (!l.on) l.first = 31;
  return l;
}

// Sums over the lanes of a row, the same total on every lane, in a fixed order:
// a butterfly (LEN > 0), or a tree over a row's len consecutive lanes and a
// broadcast (LEN < 0: -LEN levels).  All 32 lanes call it.  The number of levels is
// known when compiling: a loop that stopped at len cost four times as much (10
// us of 44 at 8192 tokens of 32 + 32 heads of 96).
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
        v[i] += l.g + o < l.len ? t : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, v[i], l.first);
  }
}

// ---------------------------------------------------------------- ring --
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

// A warp's ring of rows to come, STAGES steps in shared memory, and how a lane
// moves its units between it and global memory.  A stage is copied into again
// only after what was read from it has been used.
//
// LANES: each lane copies and stores its own units, held as [stage][unit]
// [vector][lane]; its own cp.async.wait_group is all the waiting that is needed.
// Right where a row's lanes cover whole 32-byte sectors.
//
// LINEAR: the rows of a step lie one after the other as in memory, and lane l
// copies 16-byte pieces l and l + 32 of them, whichever units those hold; results
// go back the same way.  For rows whose halves are not whole sectors or lines: 96-wide
// heads, 48 of them rotated, took 43.7 us by LANES and XX by LINEAR (8192 tokens,
// 32 + 32 heads).
template <class T, int V, int NU, int STAGES, bool LINEAR>
struct Ring;

template <class T, int V, int NU, int STAGES>
struct Ring<T, V, NU, STAGES, false> {
  static constexpr int BYTES = V * static_cast<int>(sizeof(T));
  static constexpr int VECTOR = 32 * BYTES;
  static constexpr int STAGE = NU * 2 * VECTOR;
  static constexpr int WARP = STAGES * STAGE;
  uint8_t* mine;   // this lane's place in stage 0
  int row;

  __device__ __forceinline__ Ring(uint8_t* warp, const Args& p, const Lane& ln,
                                  const Unit (&)[NU], int lane)
      : mine(warp + lane * BYTES), row(ln.row) {}
  // Rows head, head + 1, ... (those below `heads`) into the stage of `step`.
  __device__ __forceinline__ void copy(int step, const HeadRows<const T>& src,
                                       int head, int heads,
                                       const Unit (&un)[NU]) {
    const bool on = head + row < heads;
    const T* from = src.at(on ? head + row : 0);
    uint8_t* st = mine + (step % STAGES) * STAGE;
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      copy_async<BYTES>(st + 2 * n * VECTOR, from + un[n].off0,
                        on && un[n].ok0);
      copy_async<BYTES>(st + (2 * n + 1) * VECTOR, from + un[n].off1,
                        on && un[n].ok1);
    }
  }
  __device__ __forceinline__ void sync() const {}
  __device__ __forceinline__ void read(int step, RawUnit<T, V> (&raw)[NU]) const {
    const uint8_t* st = mine + (step % STAGES) * STAGE;
#pragma unroll
    for (int n = 0; n < NU; ++n)
#pragma unroll
      for (int v = 0; v < 2; ++v)
        raw[n].v[v] = *reinterpret_cast<const RawT<T, V>*>(
            st + (2 * n + v) * VECTOR);
  }
  // The lane's results of a step, and (LINEAR) their way to memory.
  template <bool INTER>
  __device__ __forceinline__ void put(int, const HeadRows<T>& dst, int head,
                                      int heads, const Unit (&un)[NU],
                                      Pairs<V> (&y)[NU]) const {
    const bool on = head + row < heads;
    T* to = dst.at(on ? head + row : 0);
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      if (on && un[n].ok0)
        *reinterpret_cast<RawT<T, V>*>(to + un[n].off0) =
            pack<T, V, INTER>(y[n], 0);
      if (on && un[n].ok1)
        *reinterpret_cast<RawT<T, V>*>(to + un[n].off1) =
            pack<T, V, INTER>(y[n], 1);
    }
  }
  __device__ __forceinline__ void flush(int, const HeadRows<T>&, int, int) const {}
};

template <class T, int V, int STAGES>
struct Ring<T, V, 1, STAGES, true> {
  static constexpr int STAGE = 64 * 16;
  static constexpr int WARP = STAGES * STAGE;
  uint8_t* warp;
  int lane;
  int at0, at1;        // the lane's vectors in a stage
  int row[2], col[2];  // its pieces: row (past the step's rows: none), byte

  __device__ __forceinline__ Ring(uint8_t* w, const Args& p, const Lane& ln,
                                  const Unit (&un)[1], int lane_)
      : warp(w), lane(lane_) {
    const int bytes = p.d * static_cast<int>(sizeof(T)), pieces = bytes / 16;
    at0 = ln.row * bytes + un[0].off0 * static_cast<int>(sizeof(T));
    at1 = ln.row * bytes + un[0].off1 * static_cast<int>(sizeof(T));
    // an idle lane reads the last piece, which then holds no row's elements
    if (!ln.on) at0 = at1 = 63 * 16;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int i = lane + 32 * v;
      row[v] = i / pieces;
      col[v] = (i - row[v] * pieces) * 16;
      if (row[v] >= p.rows) row[v] = 1 << 20;
    }
  }
  __device__ __forceinline__ void copy(int step, const HeadRows<const T>& src,
                                       int head, int heads, const Unit (&)[1]) {
    uint8_t* st = warp + (step % STAGES) * STAGE;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const bool on = head + row[v] < heads;
      copy_async<16>(st + (lane + 32 * v) * 16,
                     reinterpret_cast<const uint8_t*>(
                         src.at(on ? head + row[v] : 0)) + col[v],
                     on);
    }
  }
  // Other lanes' copies are read after this (and after each lane's wait), and
  // copied over only after the next.
  __device__ __forceinline__ void sync() const { __syncwarp(); }
  __device__ __forceinline__ void read(int step, RawUnit<T, V> (&raw)[1]) const {
    const uint8_t* st = warp + (step % STAGES) * STAGE;
    raw[0].v[0] = *reinterpret_cast<const RawT<T, V>*>(st + at0);
    raw[0].v[1] = *reinterpret_cast<const RawT<T, V>*>(st + at1);
  }
  template <bool INTER>
  __device__ __forceinline__ void put(int step, const HeadRows<T>&, int, int,
                                      const Unit (&un)[1],
                                      Pairs<V> (&y)[1]) const {
    uint8_t* st = warp + (step % STAGES) * STAGE;
    if (un[0].ok0) {
      *reinterpret_cast<RawT<T, V>*>(st + at0) = pack<T, V, INTER>(y[0], 0);
      *reinterpret_cast<RawT<T, V>*>(st + at1) = pack<T, V, INTER>(y[0], 1);
    }
  }
  __device__ __forceinline__ void flush(int step, const HeadRows<T>& dst,
                                        int head, int heads) const {
    const uint8_t* st = warp + (step % STAGES) * STAGE;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      if (head + row[v] >= heads) continue;
      *reinterpret_cast<uint4*>(
          reinterpret_cast<uint8_t*>(dst.at(head + row[v])) + col[v]) =
          *reinterpret_cast<const uint4*>(st + (lane + 32 * v) * 16);
    }
  }
};

// ------------------------------------------------------------- angles --
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

// A unit's V of them (1 and 0 for a unit that does not turn): pairs V u ..., or,
// interleaved, V / 2 from each half.
template <int V, bool INTER>
__device__ __forceinline__ void load_angles(const Args& p, const Trig& t, int u,
                                            float (&c)[V], float (&s)[V]) {
  constexpr int RUN = INTER && V > 1 ? V / 2 : V;
  const bool turns = u < p.rot_units;
#pragma unroll
  for (int h = 0; h < V / RUN; ++h) {
    const int at = RUN * u + h * (p.rot / 4);
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

__device__ __forceinline__ void stage_freq(const Args& p,
                                           unsigned long long* freq) {
  for (int i = threadIdx.x; i < p.rot / 2; i += THREADS) freq[i] = p.freq[i];
  __syncthreads();
}

// -------------------------------------------------------------- forward --
// What a lane multiplies a row's unit by: y_a = rstd (a ca + b sb) + za, y_b =
// rstd (a sa + b cb) + zb, with gamma folded into the rotation and beta rotated.
template <int V>
struct Turn {
  float ca[V], sb[V], sa[V], cb[V];
  float za[V], zb[V];
};
template <int V, int NORM, bool INTER>
__device__ __forceinline__ void load_turn(const Args& p, const Side& sd,
                                          const Trig& trig, int u,
                                          const Unit& un, Turn<V>& t) {
  load_angles<V, INTER>(p, trig, u, t.ca, t.sa);
  if constexpr (NORM == 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      t.cb[j] = t.ca[j];
      t.sb[j] = -t.sa[j];
    }
  } else {
    Pairs<V> gam;
    load_param<V, INTER>(p, sd.gamma, 1.f, un, gam);
    if constexpr (NORM == TPQK_LAYERNORM) {
      Pairs<V> bet;
      load_param<V, INTER>(p, sd.beta, 0.f, un, bet);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        t.za[j] = fmaf(bet.a[j], t.ca[j], -(bet.b[j] * t.sa[j]));
        t.zb[j] = fmaf(bet.a[j], t.sa[j], bet.b[j] * t.ca[j]);
      }
    }
    mul<V>(t.cb, t.ca, gam.b);
#pragma unroll
    for (int j = 0; j < V; ++j) t.sb[j] = -(t.sa[j] * gam.b[j]);
    mul<V>(t.ca, t.ca, gam.a);
    mul<V>(t.sa, t.sa, gam.a);
  }
}

// Steps ahead that are being copied (one group each), and steps computed at a
// time: two, so that two rows' chains of sums share the issue slots and the
// lane's coefficients.
constexpr int FWD_STAGES = 8, FWD_AHEAD = 5;

template <class T, int V, int NU, int NORM, bool INTER, int LEN, bool WHOLE>
__global__ void __launch_bounds__(THREADS)
    qk_rows_forward(const __grid_constant__ Args p) {
  constexpr bool LINEAR = WHOLE && LEN < 0;
  using R = Ring<T, V, NU, FWD_STAGES, LINEAR>;
  constexpr int AT_ONCE = NU == 1 ? 2 : 1;
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
  Unit un[NU];
#pragma unroll
  for (int n = 0; n < NU; ++n)
    un[n] = unit_at<V, INTER, WHOLE>(p, ln.g + 32 * n, ln.on);
  R ring(ring_mem + warp * R::WARP, p, ln, un, lane);
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
      ring.copy(sc, src, hc, src_heads, un);
      hc += p.rows;
      ++sc;
    }
    ring_commit();
  };
#pragma unroll
  for (int i = 0; i < FWD_AHEAD; ++i) copy();
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
    Turn<V> t[NU];
#pragma unroll
    for (int n = 0; n < NU; ++n)
      load_turn<V, NORM, INTER>(p, sd, trig[warp], ln.g + 32 * n, un[n], t[n]);
#pragma unroll 1
    while (s < end) {
      // (a second step past the end is computed for nothing)
      const int used = min(AT_ONCE, end - s);
      ring_wait<FWD_AHEAD - AT_ONCE>();
      ring.sync();
      Pairs<V> x[AT_ONCE][NU];
#pragma unroll
      for (int k = 0; k < AT_ONCE; ++k) {
        RawUnit<T, V> raw[NU];
        ring.read(s + k, raw);
#pragma unroll
        for (int n = 0; n < NU; ++n) unpack<T, V, INTER>(raw[n], x[k][n]);
      }
#pragma unroll
      for (int k = 0; k < AT_ONCE; ++k)
        if (k < used) copy();
      float scale[AT_ONCE];
      if constexpr (NORM == TPQK_LAYERNORM) {
        float m[AT_ONCE];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) m[k] = total<V, NU>(x[k]);
        row_sum<LEN>(m, ln);
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k)
#pragma unroll
          for (int n = 0; n < NU; ++n)
            centre<V, INTER, WHOLE>(x[k][n], un[n], m[k] * p.inv_d);
      }
      if constexpr (NORM != 0) {
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) scale[k] = dot<V, NU>(x[k], x[k]);
        row_sum<LEN>(scale, ln);
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k)
          scale[k] = rsqrtf(fmaf(scale[k], p.inv_d, p.eps));
      }
#pragma unroll
      for (int k = 0; k < AT_ONCE; ++k) {
        Pairs<V> y[NU];
#pragma unroll
        for (int n = 0; n < NU; ++n) {
          // the rotation does not wait for the norm's sum
          mul<V>(y[n].a, x[k][n].b, t[n].sb);
          mul<V>(y[n].b, x[k][n].b, t[n].cb);
          fma<V>(y[n].a, x[k][n].a, t[n].ca, y[n].a);
          fma<V>(y[n].b, x[k][n].a, t[n].sa, y[n].b);
          if constexpr (NORM == TPQK_LAYERNORM) {
            fma<V>(y[n].a, y[n].a, scale[k], t[n].za);
            fma<V>(y[n].b, y[n].b, scale[k], t[n].zb);
          } else if constexpr (NORM != 0) {
            mul<V>(y[n].a, y[n].a, scale[k]);
            mul<V>(y[n].b, y[n].b, scale[k]);
          }
        }
        if (k < used)
          ring.template put<INTER>(s + k, dst, h + k * p.rows, heads, un, y);
      }
      ring.sync();
#pragma unroll
      for (int k = 0; k < AT_ONCE; ++k)
        if (k < used) ring.flush(s + k, dst, h + k * p.rows, heads);
      h += AT_ONCE * p.rows;
      s += used;
    }
  }
}

// ------------------------------------------------------------- backward --
// With g = R^T dy, u = g gamma and e = x - mu:
//   xh = rstd e,  dgamma += (rstd g) e,  dbeta += g,
//   dx = (rstd g) gamma - (rstd^3 sum(e u) / d) e [- rstd mean(u)].
// Persistent blocks, so that a lane sums its unit's parameter gradients over
// all its rows in registers; a block takes q's tasks or k's.
constexpr int BWD_STAGES = 4, BWD_AHEAD = 3;

template <class T, int V, int NU, int NORM, bool INTER, int LEN, bool WHOLE>
__global__ void __launch_bounds__(THREADS, 4)
    qk_rows_backward(const __grid_constant__ Args p) {
  constexpr bool LINEAR = WHOLE && LEN < 0;
  using R = Ring<T, V, NU, BWD_STAGES, LINEAR>;
  constexpr int SUMS = WARPS * 32 * NU * 2 * V;   // floats
  __shared__ __align__(16) uint8_t ring_mem[2 * WARPS * R::WARP];
  __shared__ unsigned long long freq[MAX_PAIRS];
  __shared__ __align__(16) Trig trig[WARPS];
  static_assert(sizeof(ring_mem) >= SUMS * sizeof(float), "the sums reuse it");
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
  Unit un[NU];
  Pairs<V> gam[NU], dgam[NU], dbet[NU];
#pragma unroll
  for (int n = 0; n < NU; ++n) {
    un[n] = unit_at<V, INTER, WHOLE>(p, ln.g + 32 * n, ln.on);
    load_param<V, INTER>(p, sd.gamma, 1.f, un[n], gam[n]);
#pragma unroll
    for (int j = 0; j < V; ++j)
      dgam[n].a[j] = dgam[n].b[j] = dbet[n].a[j] = dbet[n].b[j] = 0.f;
  }
  R gring(ring_mem + 2 * warp * R::WARP, p, ln, un, lane);
  R xring(ring_mem + (2 * warp + 1) * R::WARP, p, ln, un, lane);
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
        gring.copy(sc, gsrc, hc, heads, un);
        xring.copy(sc, xsrc, hc, heads, un);
        hc += p.rows;
        ++sc;
      }
      ring_commit();
    };
#pragma unroll
    for (int i = 0; i < BWD_AHEAD; ++i) copy();
    make_angles(p, freq, position(p, token), lane, trig[warp]);
    float c[NU][V], sa[NU][V];
#pragma unroll
    for (int n = 0; n < NU; ++n)
      load_angles<V, INTER>(p, trig[warp], ln.g + 32 * n, c[n], sa[n]);
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
      ring_wait<BWD_AHEAD - 1>();
      gring.sync();
      Pairs<V> g[NU], e[NU];
      {
        RawUnit<T, V> graw[NU], xraw[NU];
        gring.read(s, graw);
        xring.read(s, xraw);
        copy();
#pragma unroll
        for (int n = 0; n < NU; ++n) {
          Pairs<V> dy;
          unpack<T, V, INTER>(graw[n], dy);
          unpack<T, V, INTER>(xraw[n], e[n]);
          // R^T (sa carries the opposite direction's sign)
          float t[V];
          mul<V>(t, dy.b, -1.f);
          mul<V>(g[n].a, t, sa[n]);
          fma<V>(g[n].a, dy.a, c[n], g[n].a);
          mul<V>(g[n].b, dy.b, c[n]);
          fma<V>(g[n].b, dy.a, sa[n], g[n].b);
        }
      }
      float mean_u = 0.f;
      if constexpr (NORM == TPQK_LAYERNORM) {
        float m[2] = {total<V, NU>(e), dot<V, NU>(g, gam)};
        row_sum<LEN>(m, ln);
#pragma unroll
        for (int n = 0; n < NU; ++n)
          centre<V, INTER, WHOLE>(e[n], un[n], m[0] * p.inv_d);
        mean_u = m[1] * p.inv_d;
      }
      float q[2] = {dot<V, NU>(e, e), 0.f};
#pragma unroll
      for (int n = 0; n < NU; ++n) {   // sum of e u
        float t[V], u[V];
        mul<V>(u, g[n].a, gam[n].a);
        mul<V>(t, u, e[n].a);
        mul<V>(u, g[n].b, gam[n].b);
        fma<V>(t, u, e[n].b, t);
        q[1] += sum<V>(t);
      }
      row_sum<LEN>(q, ln);
      const float rstd = rsqrtf(fmaf(q[0], p.inv_d, p.eps));
      const float k = -(rstd * rstd) * (q[1] * rstd * p.inv_d);
      const float m = -rstd * mean_u;
      Pairs<V> dx[NU];
#pragma unroll
      for (int n = 0; n < NU; ++n) {
        if constexpr (NORM == TPQK_LAYERNORM) {
          add<V>(dbet[n].a, g[n].a);
          add<V>(dbet[n].b, g[n].b);
        }
        mul<V>(g[n].a, g[n].a, rstd);
        mul<V>(g[n].b, g[n].b, rstd);
        fma<V>(dgam[n].a, g[n].a, e[n].a, dgam[n].a);
        fma<V>(dgam[n].b, g[n].b, e[n].b, dgam[n].b);
        mul<V>(dx[n].a, e[n].a, k);
        mul<V>(dx[n].b, e[n].b, k);
        if constexpr (NORM == TPQK_LAYERNORM) {
          add<V>(dx[n].a, m);
          add<V>(dx[n].b, m);
        }
        fma<V>(dx[n].a, g[n].a, gam[n].a, dx[n].a);
        fma<V>(dx[n].b, g[n].b, gam[n].b, dx[n].b);
      }
      gring.template put<INTER>(s, dst, h, heads, un, dx);
      gring.sync();
      gring.flush(s, dst, h, heads);
      h += p.rows;
    }
    // the ring is empty again: its last steps' groups hold nothing
  }
  if (p.part == nullptr) return;
  // the block's sums: element i of every row slot, in the order of the slots
  float* sums = reinterpret_cast<float*>(ring_mem);
  const int slots = WARPS * p.rows;
#pragma unroll
  for (int k = 0; k < (NORM == TPQK_LAYERNORM ? 2 : 1); ++k) {
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NU; ++n) {
#pragma unroll
      for (int i = 0; i < 2 * V; ++i) {
        const bool ok = i < V ? un[n].ok0 : un[n].ok1;
        const int at = i < V ? un[n].off0 + i : un[n].off1 + i - V;
        if (ok)
          sums[(warp * p.rows + ln.row) * p.d + at] =
              element<V, INTER>(k ? dbet[n] : dgam[n], i);
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.d; i += THREADS) {
      float t = 0.f;
      for (int w = 0; w < slots; ++w) t += sums[w * p.d + i];
      p.part[(static_cast<long long>(blockIdx.x) * 2 + k) * p.d + i] = t;
    }
  }
}

// ------------------------------------------------------------- dispatch --
template <class T, int V, int NU, int NORM, bool INTER, int LEN, bool WHOLE>
void go(const Args& a, int blocks, bool backward, cudaStream_t s) {
  if (!backward) {
    qk_rows_forward<T, V, NU, NORM, INTER, LEN, WHOLE>
        <<<blocks, THREADS, 0, s>>>(a);
  } else if constexpr (NORM != 0) {
    qk_rows_backward<T, V, NU, NORM, INTER, LEN, WHOLE>
        <<<blocks, THREADS, 0, s>>>(a);
  }
}

// Rows of 16-byte vectors without a part unit have kernels of their own, and
// those that fill 4, 8 or 16 lanes (8, 16, 32 in fp32) one each.
template <class T, int V, int NU, int NORM, bool INTER>
void by_length(const Args& a, int blocks, bool backward, cudaStream_t s) {
  if constexpr (V * sizeof(T) == 16) {
    constexpr int SHORT = 32 / V;   // 64 elements
    if (a.d == 2 * V * a.units) {
      if (a.units == SHORT)
        return go<T, V, NU, NORM, INTER, SHORT, true>(a, blocks, backward, s);
      if (a.units == 2 * SHORT)
        return go<T, V, NU, NORM, INTER, 2 * SHORT, true>(a, blocks, backward, s);
      if (a.units == 4 * SHORT)
        return go<T, V, NU, NORM, INTER, 4 * SHORT, true>(a, blocks, backward, s);
      if (a.units <= 8)
        return go<T, V, NU, NORM, INTER, -3, true>(a, blocks, backward, s);
      if (a.units <= 16)
        return go<T, V, NU, NORM, INTER, -4, true>(a, blocks, backward, s);
      if constexpr (V == 4)
        return go<T, V, NU, NORM, INTER, -5, true>(a, blocks, backward, s);
    }
  }
  go<T, V, NU, NORM, INTER, -5, false>(a, blocks, backward, s);
}

template <class T, int V, int NU>
void by_norm(const Args& a, int norm, bool inter, int blocks, bool backward,
             cudaStream_t s) {
  if (norm == TPQK_RMSNORM) {
    if (inter) by_length<T, V, NU, TPQK_RMSNORM, true>(a, blocks, backward, s);
    else by_length<T, V, NU, TPQK_RMSNORM, false>(a, blocks, backward, s);
  } else if (norm == TPQK_LAYERNORM) {
    if (inter) by_length<T, V, NU, TPQK_LAYERNORM, true>(a, blocks, backward, s);
    else by_length<T, V, NU, TPQK_LAYERNORM, false>(a, blocks, backward, s);
  } else {
    if (inter) by_length<T, V, NU, 0, true>(a, blocks, backward, s);
    else by_length<T, V, NU, 0, false>(a, blocks, backward, s);
  }
}

}  // namespace

// Units a lane may have: 256 / (2 V) / 32, at least one.
#ifdef QK_ROWS_BF16
cudaError_t launch_bf16(const Args& a, int vec, int norm, bool inter, int blocks,
                        bool backward, cudaStream_t s) {
  using T = __nv_bfloat16;
  switch (vec) {
    case 8: by_norm<T, 8, 1>(a, norm, inter, blocks, backward, s); break;
    case 4: by_norm<T, 4, 1>(a, norm, inter, blocks, backward, s); break;
    case 2: by_norm<T, 2, 2>(a, norm, inter, blocks, backward, s); break;
    case 1: by_norm<T, 1, 4>(a, norm, inter, blocks, backward, s); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}
#else
cudaError_t launch_fp32(const Args& a, int vec, int norm, bool inter, int blocks,
                        bool backward, cudaStream_t s) {
  switch (vec) {
    case 4: by_norm<float, 4, 1>(a, norm, inter, blocks, backward, s); break;
    case 2: by_norm<float, 2, 2>(a, norm, inter, blocks, backward, s); break;
    case 1: by_norm<float, 1, 4>(a, norm, inter, blocks, backward, s); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}
#endif

}  // namespace qk
}  // namespace tpmlp
