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
#include "qk_rows.cuh"

#include "common.cuh"

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
template <class T>
__device__ __forceinline__ T* head_row(T* token, const View& v, unsigned head) {
  const unsigned g = __umulhi(head, v.magic);
  return token + (static_cast<unsigned long long>(g) * v.gs +
                  static_cast<unsigned long long>(head - g * v.group) * v.hs);
}

template <class T>
__device__ __forceinline__ T* token_row(const View& v, int token) {
  return reinterpret_cast<T*>(v.p) + static_cast<long long>(token) * v.ts;
}

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

// A lane's ring of units to come: RING stages, each a step's NU units of two
// vectors, held as [stage][unit][vector][lane].  Only the lane itself reads what
// it copied, so its own wait (cp.async.wait_group) is all that is needed, and a
// stage is copied into again one step after it was read.
constexpr int RING = 4;
template <class T, int V, int NU>
struct Ring {
  static constexpr int BYTES = V * static_cast<int>(sizeof(T));
  static constexpr int VECTOR = 32 * BYTES;
  static constexpr int STAGE = NU * 2 * VECTOR;
  static constexpr int WARP = RING * STAGE;
  uint8_t* mine;   // this lane's place in stage 0

  __device__ __forceinline__ void copy_vector(uint8_t* dst, const T* src,
                                              bool ok) {
    if constexpr (BYTES == 2) {   // below cp.async's sizes
      *reinterpret_cast<uint16_t*>(dst) =
          ok ? *reinterpret_cast<const uint16_t*>(src) : uint16_t(0);
    } else {
      const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
      const int n = ok ? BYTES : 0;   // the rest is filled with zeros
      if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d),
                     "l"(src), "r"(n) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(d),
                     "l"(src), "n"(BYTES), "r"(n) : "memory");
    }
  }
  // The lane's units of `row` (on: the row exists) into the stage of `step`.
  __device__ __forceinline__ void copy(int step, const T* row, bool on,
                                       const Unit (&un)[NU]) {
    uint8_t* st = mine + (step % RING) * STAGE;
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      copy_vector(st + 2 * n * VECTOR, row + un[n].off0, on && un[n].ok0);
      copy_vector(st + (2 * n + 1) * VECTOR, row + un[n].off1, on && un[n].ok1);
    }
  }
  __device__ __forceinline__ void read(int step, RawUnit<T, V> (&raw)[NU]) {
    const uint8_t* st = mine + (step % RING) * STAGE;
#pragma unroll
    for (int n = 0; n < NU; ++n)
#pragma unroll
      for (int v = 0; v < 2; ++v)
        raw[n].v[v] = *reinterpret_cast<const RawT<T, V>*>(
            st + (2 * n + v) * VECTOR);
  }
};
__device__ __forceinline__ void ring_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// All groups but the last RING - 2 are there.
__device__ __forceinline__ void ring_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(RING - 2) : "memory");
}

template <class T, int V, bool INTER>
__device__ __forceinline__ void store_unit(T* row, const Unit& n, bool on,
                                           Pairs<V>& f) {
  if (on && n.ok0)
    *reinterpret_cast<RawT<T, V>*>(row + n.off0) = pack<T, V, INTER>(f, 0);
  if (on && n.ok1)
    *reinterpret_cast<RawT<T, V>*>(row + n.off1) = pack<T, V, INTER>(f, 1);
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
// LEN lanes, a power of two; no lane is idle.
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
// a butterfly (LEN > 0), or a tree over the first len of a row's consecutive
// lanes and a broadcast.  All 32 lanes call it.
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
    for (int o = 16; o > 0; o >>= 1) {
      if (o >= l.len) continue;   // the same on every lane
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float t = __shfl_down_sync(0xffffffffu, v[i], o);
        if (l.g + o < l.len) v[i] += t;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, v[i], l.first);
  }
}

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

template <class T, int V, int NU, int NORM, bool INTER, int LEN, bool WHOLE>
__global__ void __launch_bounds__(THREADS)
    qk_rows_forward(const __grid_constant__ Args p) {
  using R = Ring<T, V, NU>;
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
  R ring{ring_mem + warp * R::WARP + lane * R::BYTES};
  auto copy = [&](int s) {
    if (s < s1) {
      const int which = s >= mid;
      const Side& sd = p.side[which];
      const int h = (which ? s - mid : s) * p.rows + ln.row;
      const bool on = h < sd.heads;
      ring.copy(s, head_row(token_row<const T>(sd.in, token), sd.in, on ? h : 0),
                on, un);
    }
    ring_commit();
  };
#pragma unroll
  for (int i = 0; i < RING - 1; ++i) copy(s0 + i);
  stage_freq(p, freq);
  if (s0 >= s1) return;
  make_angles(p, freq, position(p, token), lane, trig[warp]);
  Turn<V> t[NU];
#pragma unroll 1
  for (int s = s0; s < s1; ++s) {
    const int which = s >= mid;
    const Side& sd = p.side[which];
    if (s == s0 || s == mid) {
#pragma unroll
      for (int n = 0; n < NU; ++n)
        load_turn<V, NORM, INTER>(p, sd, trig[warp], ln.g + 32 * n, un[n], t[n]);
    }
    ring_wait();
    Pairs<V> x[NU];
    {
      RawUnit<T, V> raw[NU];
      ring.read(s, raw);
      copy(s + RING - 1);
#pragma unroll
      for (int n = 0; n < NU; ++n) unpack<T, V, INTER>(raw[n], x[n]);
    }
    const int h = (which ? s - mid : s) * p.rows + ln.row;
    const bool on = h < sd.heads;
    float scale = 1.f;
    if constexpr (NORM == TPQK_LAYERNORM) {
      float m[1] = {total<V, NU>(x)};
      row_sum<LEN>(m, ln);
#pragma unroll
      for (int n = 0; n < NU; ++n)
        centre<V, INTER, WHOLE>(x[n], un[n], m[0] * p.inv_d);
    }
    if constexpr (NORM != 0) {
      float ss[1] = {dot<V, NU>(x, x)};
      row_sum<LEN>(ss, ln);
      scale = rsqrtf(fmaf(ss[0], p.inv_d, p.eps));
    }
    T* row = head_row(token_row<T>(sd.out, token), sd.out, on ? h : 0);
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      // the rotation does not wait for the norm's sum
      Pairs<V> y;
      mul<V>(y.a, x[n].b, t[n].sb);
      mul<V>(y.b, x[n].b, t[n].cb);
      fma<V>(y.a, x[n].a, t[n].ca, y.a);
      fma<V>(y.b, x[n].a, t[n].sa, y.b);
      if constexpr (NORM == TPQK_LAYERNORM) {
        fma<V>(y.a, y.a, scale, t[n].za);
        fma<V>(y.b, y.b, scale, t[n].zb);
      } else if constexpr (NORM != 0) {
        mul<V>(y.a, y.a, scale);
        mul<V>(y.b, y.b, scale);
      }
      store_unit<T, V, INTER>(row, un[n], on, y);
    }
  }
}

// ------------------------------------------------------------- backward --
// With g = R^T dy, u = g gamma and e = x - mu:
//   xh = rstd e,  dgamma += (rstd g) e,  dbeta += g,
//   dx = rstd u - (rstd^3 sum(e u) / d) e [- rstd mean(u)].
// Persistent blocks, so that a lane sums its unit's parameter gradients over
// all its rows in registers; a block takes q's tasks or k's.
template <class T, int V, int NU, int NORM, bool INTER, int LEN, bool WHOLE>
__global__ void __launch_bounds__(THREADS)
    qk_rows_backward(const __grid_constant__ Args p) {
  using R = Ring<T, V, NU>;
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
  const int per = p.per_side[which];
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
  R gring{ring_mem + 2 * warp * R::WARP + lane * R::BYTES};
  R xring{gring.mine + R::WARP};
  const unsigned tasks = static_cast<unsigned>(p.tokens) * segs;
  for (unsigned task = block * WARPS + warp; task < tasks;
       task += blocks * WARPS) {
    const int token = static_cast<int>(task / segs);
    const int s0 = static_cast<int>(task - token * segs) * per;
    const int s1 = min(s0 + per, sd.steps);
    auto copy = [&](int s) {
      if (s < s1) {
        const int h = s * p.rows + ln.row;
        const bool on = h < sd.heads;
        gring.copy(s, head_row(token_row<const T>(sd.in, token), sd.in,
                               on ? h : 0), on, un);
        xring.copy(s, head_row(token_row<const T>(sd.x, token), sd.x,
                               on ? h : 0), on, un);
      }
      ring_commit();
    };
#pragma unroll
    for (int i = 0; i < RING - 1; ++i) copy(s0 + i);
    make_angles(p, freq, position(p, token), lane, trig[warp]);
    float c[NU][V], sa[NU][V];
#pragma unroll
    for (int n = 0; n < NU; ++n)
      load_angles<V, INTER>(p, trig[warp], ln.g + 32 * n, c[n], sa[n]);
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
      ring_wait();
      Pairs<V> g[NU], e[NU], u[NU];
      {
        RawUnit<T, V> graw[NU], xraw[NU];
        gring.read(s, graw);
        xring.read(s, xraw);
        copy(s + RING - 1);
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
          mul<V>(u[n].a, g[n].a, gam[n].a);
          mul<V>(u[n].b, g[n].b, gam[n].b);
        }
      }
      const int h = s * p.rows + ln.row;
      const bool on = h < sd.heads;
      float mean_u = 0.f;
      if constexpr (NORM == TPQK_LAYERNORM) {
        float m[2] = {total<V, NU>(e), total<V, NU>(u)};
        row_sum<LEN>(m, ln);
#pragma unroll
        for (int n = 0; n < NU; ++n)
          centre<V, INTER, WHOLE>(e[n], un[n], m[0] * p.inv_d);
        mean_u = m[1] * p.inv_d;
      }
      float q[2] = {dot<V, NU>(e, e), dot<V, NU>(e, u)};
      row_sum<LEN>(q, ln);
      const float rstd = rsqrtf(fmaf(q[0], p.inv_d, p.eps));
      const float k = -(rstd * rstd) * (q[1] * rstd * p.inv_d);
      T* row = head_row(token_row<T>(sd.out, token), sd.out, on ? h : 0);
#pragma unroll
      for (int n = 0; n < NU; ++n) {
        float t[V];
        mul<V>(t, g[n].a, rstd);
        fma<V>(dgam[n].a, t, e[n].a, dgam[n].a);
        mul<V>(t, g[n].b, rstd);
        fma<V>(dgam[n].b, t, e[n].b, dgam[n].b);
        if constexpr (NORM == TPQK_LAYERNORM) {
          add<V>(dbet[n].a, g[n].a);
          add<V>(dbet[n].b, g[n].b);
          add<V>(u[n].a, -mean_u);
          add<V>(u[n].b, -mean_u);
        }
        mul<V>(u[n].a, u[n].a, rstd);
        mul<V>(u[n].b, u[n].b, rstd);
        fma<V>(u[n].a, e[n].a, k, u[n].a);
        fma<V>(u[n].b, e[n].b, k, u[n].b);
        store_unit<T, V, INTER>(row, un[n], on, u[n]);
      }
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

// out[o][c] = sum over the side's blocks of part[block][k][c]: 32 columns a
// block, 32 threads down the blocks, then a tree over them; fixed order.
__global__ void __launch_bounds__(1024)
    qk_param_sums(const float* part, int d, int q_blocks, int blocks,
                  float* o0, float* o1, float* o2, float* o3) {
  __shared__ float t[32][33];
  const int o = blockIdx.y;
  float* out = o == 0 ? o0 : o == 1 ? o1 : o == 2 ? o2 : o3;
  if (out == nullptr) return;
  const int b0 = o < 2 ? 0 : q_blocks, b1 = o < 2 ? q_blocks : blocks;
  const int col = blockIdx.x * 32 + threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float s = 0.f;
  if (col < d) {
#pragma unroll 8
    for (int b = b0 + threadIdx.y; b < b1; b += 32)
      s += part[(static_cast<long long>(b) * 2 + (o & 1)) * d + col];
  }
  t[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && col < d) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += t[i][threadIdx.x];
    out[col] = s;
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

// Rows of 16-byte vectors without a part unit have a kernel of their own, and
// those that fill 4, 8 or 16 lanes (8, 16, 32 in fp32) one each: no checks of
// elements, and a butterfly of known length for the sums.
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
      return go<T, V, NU, NORM, INTER, 0, true>(a, blocks, backward, s);
    }
  }
  go<T, V, NU, NORM, INTER, 0, false>(a, blocks, backward, s);
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

// Units a lane may have: 256 / (2 V) / 32, at least one.
cudaError_t launch(const Args& a, bool bf16, int vec, int norm, bool inter,
                   int blocks, bool backward, cudaStream_t s) {
  if (bf16) {
    switch (vec) {
      case 8: by_norm<__nv_bfloat16, 8, 1>(a, norm, inter, blocks, backward, s); break;
      case 4: by_norm<__nv_bfloat16, 4, 1>(a, norm, inter, blocks, backward, s); break;
      case 2: by_norm<__nv_bfloat16, 2, 2>(a, norm, inter, blocks, backward, s); break;
      case 1: by_norm<__nv_bfloat16, 1, 4>(a, norm, inter, blocks, backward, s); break;
      default: return cudaErrorInvalidValue;
    }
  } else {
    switch (vec) {
      case 4: by_norm<float, 4, 1>(a, norm, inter, blocks, backward, s); break;
      case 2: by_norm<float, 2, 2>(a, norm, inter, blocks, backward, s); break;
      case 1: by_norm<float, 1, 4>(a, norm, inter, blocks, backward, s); break;
      default: return cudaErrorInvalidValue;
    }
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_forward(const Args& a, bool bf16, int vec, int norm,
                           bool interleaved, cudaStream_t s) {
  const unsigned tasks = static_cast<unsigned>(a.tokens) * a.segs;
  return launch(a, bf16, vec, norm, interleaved,
                static_cast<int>((tasks + WARPS - 1) / WARPS), false, s);
}

cudaError_t launch_backward(const Args& a, bool bf16, int vec, int norm,
                            bool interleaved, int blocks, cudaStream_t s) {
  if (norm == 0) return cudaErrorInvalidValue;
  return launch(a, bf16, vec, norm, interleaved, blocks, true, s);
}

cudaError_t launch_param_sums(const float* part, int d, int q_blocks,
                              int blocks, float* const out[4], cudaStream_t s) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((d + 31) / 32, 4);
  cfg.blockDim = dim3(32, 32);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, qk_param_sums, part, d, q_blocks, blocks,
                            out[0], out[1], out[2], out[3]);
}

}  // namespace qk
}  // namespace tpmlp
