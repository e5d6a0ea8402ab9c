// Rotary positions and the per-head norm of queries and keys (tp_rope.h), one
// pass over the heads each: a head row lives in the registers of a few lanes
// from its load to its store.
//
// A row of d elements is cut into units of 2 V elements, one lane each: V
// pairs (i, i + r/2) or (2i, 2i + 1) that turn together, read as two V-wide
// vectors; the elements past r follow in units of 2 V that do not turn.  A
// warp holds floor(32 / units) rows at once, and a lane keeps its unit from row
// to row, so the V angles of a (token, unit) are made once for all heads of
// the task and gamma, beta and the parameter gradients' sums stay in registers.
//
// Angles: a frequency is held as turns per position in 64-bit fixed point
// (2^-64 of a turn), so position times frequency modulo one turn is one
// integer product; its upper 32 bits, as a signed fraction, go to sincospif.
// No table of cosines is read, and positions may be anything.
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

template <class T, int V>
__device__ __forceinline__ void unpack(const RawT<T, V>& raw, float* f) {
  if constexpr (sizeof(T) == 4) {
    const float* w = reinterpret_cast<const float*>(&raw);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = w[i];
  } else if constexpr (V == 1) {
    f[0] = __uint_as_float(static_cast<uint32_t>(raw) << 16);
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <class T, int V>
__device__ __forceinline__ RawT<T, V> pack(const float* f) {
  RawT<T, V> raw;
  if constexpr (sizeof(T) == 4) {
    float* w = reinterpret_cast<float*>(&raw);
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = f[i];
  } else if constexpr (V == 1) {
    raw = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(&raw);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  }
  return raw;
}

__device__ __forceinline__ long long row_offset(const View& v, long long token,
                                                unsigned head) {
  const unsigned g = static_cast<unsigned>((head * v.magic) >> 32);
  return token * v.ts + g * v.gs + (head - g * v.group) * v.hs;
}

// The two vectors of a unit: element offsets and whether they exist.
struct Unit {
  int off0, off1;
  bool ok0, ok1;
};
template <int V, bool INTER>
__device__ __forceinline__ Unit unit_at(const Args& p, int u, bool lane_on) {
  Unit n;
  n.ok0 = lane_on && u < p.units;
  if (u < p.rot_units) {
    n.off0 = INTER ? 2 * V * u : V * u;
    n.off1 = INTER ? n.off0 + V : p.rot / 2 + n.off0;
    n.ok1 = n.ok0;
  } else {
    n.off0 = p.rot + 2 * V * (u - p.rot_units);
    n.off1 = n.off0 + V;
    n.ok1 = n.ok0 && n.off1 < p.d;
  }
  return n;
}

// Elements of pair j inside a unit's 2 V values (first vector, then second).
template <int V, bool INTER>
__device__ __forceinline__ constexpr int pair_a(int j) {
  return INTER ? 2 * j : j;
}
template <int V, bool INTER>
__device__ __forceinline__ constexpr int pair_b(int j) {
  return INTER ? 2 * j + 1 : V + j;
}

template <class T, int V>
__device__ __forceinline__ void load_unit(const T* row, const Unit& n, bool on,
                                          RawT<T, V> (&raw)[2]) {
  raw[0] = RawT<T, V>{};
  raw[1] = RawT<T, V>{};
  if (on && n.ok0) raw[0] = *reinterpret_cast<const RawT<T, V>*>(row + n.off0);
  if (on && n.ok1) raw[1] = *reinterpret_cast<const RawT<T, V>*>(row + n.off1);
}

template <class T, int V>
__device__ __forceinline__ void store_unit(T* row, const Unit& n, bool on,
                                           const float (&f)[2 * V]) {
  if (on && n.ok0)
    *reinterpret_cast<RawT<T, V>*>(row + n.off0) = pack<T, V>(f);
  if (on && n.ok1)
    *reinterpret_cast<RawT<T, V>*>(row + n.off1) = pack<T, V>(f + V);
}

template <int V>
__device__ __forceinline__ void load_param(const float* g, float missing,
                                           const Unit& n, float (&f)[2 * V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    f[i] = g != nullptr && n.ok0 ? __ldg(g + n.off0 + i) : missing;
    f[V + i] = g != nullptr && n.ok1 ? __ldg(g + n.off1 + i) : missing;
  }
}

__device__ __forceinline__ long long position(const Args& p, int token) {
  if (p.pos != nullptr)
    return p.pos64 ? __ldg(static_cast<const long long*>(p.pos) + token)
                   : static_cast<long long>(
                         __ldg(static_cast<const int*>(p.pos) + token));
  const unsigned t = static_cast<unsigned>(token);
  return p.offset + (p.seq_len != 0 ? t % p.seq_len : t);
}

// cos and sin of the unit's V angles (amplitude and direction included); 1
// and 0 for a unit that does not turn.
template <int V>
__device__ __forceinline__ void angles(const Args& p,
                                       const unsigned long long* freq, int u,
                                       long long pos, float (&c)[V],
                                       float (&s)[V]) {
  const bool turns = u < p.rot_units;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const unsigned long long ph =
        turns ? static_cast<unsigned long long>(pos) * freq[V * u + j] : 0ull;
    const int half_turns = static_cast<int>((ph + 0x80000000ull) >> 32);
    float cj, sj;
    sincospif(static_cast<float>(half_turns) * 0x1p-31f, &sj, &cj);
    c[j] = turns ? cj * p.amp : 1.f;
    s[j] = turns ? sj * (p.amp * p.sign) : 0.f;
  }
}

// Sums over the lanes of a row (`len` consecutive lanes, `g` the lane's place
// among them), the same total on every lane: a tree over the first len values
// in a fixed order, then a broadcast.  All 32 lanes call it.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int g, int len,
                                        int first) {
  if (len == 1) return;
  int o = 1 << (31 - __clz(len - 1));   // largest power of two below len
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float t = __shfl_down_sync(0xffffffffu, v[i], o);
    if (g + o < len) v[i] += t;
  }
  for (o >>= 1; o > 0; o >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      v[i] += __shfl_down_sync(0xffffffffu, v[i], o);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, v[i], first);
}

// What a lane knows of its place: the row it works on among the warp's rows,
// and its units u, u + 32, ...
struct Lane {
  int row, g, len, first;
  bool on;
};
__device__ __forceinline__ Lane lane_place(const Args& p, int lane) {
  Lane l;
  l.len = min(p.units, 32);
  l.row = lane / l.len;
  l.g = lane - l.row * l.len;
  l.first = l.row * l.len;
  l.on = l.row < p.rows;
  if (!l.on) l.first = 31;
  return l;
}

__device__ __forceinline__ void stage_freq(const Args& p,
                                           unsigned long long* freq) {
  for (int i = threadIdx.x; i < p.rot / 2; i += THREADS) freq[i] = p.freq[i];
  __syncthreads();
}

template <int V, int NU>
__device__ __forceinline__ float sum_all(const float (&e)[NU][2 * V]) {
  float s = 0.f;
#pragma unroll
  for (int n = 0; n < NU; ++n)
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) s += e[n][i];
  return s;
}

// e - mu, zero where the row has no element.
template <int V, int NU>
__device__ __forceinline__ void centre(float (&e)[NU][2 * V],
                                       const Unit (&un)[NU], float mu) {
#pragma unroll
  for (int n = 0; n < NU; ++n)
#pragma unroll
    for (int i = 0; i < 2 * V; ++i)
      e[n][i] = (i < V ? un[n].ok0 : un[n].ok1) ? e[n][i] - mu : 0.f;
}

template <int V, int NU>
__device__ __forceinline__ float dot(const float (&a)[NU][2 * V],
                                     const float (&b)[NU][2 * V]) {
  float s = 0.f;
#pragma unroll
  for (int n = 0; n < NU; ++n)
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) s = fmaf(a[n][i], b[n][i], s);
  return s;
}

// -------------------------------------------------------------- forward --
// Rows in flight per lane (their loads are issued together).
constexpr int FWD_ROWS = 2;

template <class T, int V, int NU, int NORM, bool INTER>
__global__ void __launch_bounds__(THREADS)
    qk_rows_forward(const __grid_constant__ Args p) {
  __shared__ unsigned long long freq[MAX_PAIRS];
  stage_freq(p, freq);
  const int lane = threadIdx.x & 31;
  const unsigned task = blockIdx.x * WARPS + (threadIdx.x >> 5);
  const int token = static_cast<int>(task / p.segs);
  if (token >= p.tokens) return;
  int seg = static_cast<int>(task - token * p.segs);
  const int which = seg >= p.side[0].segs;
  const Side& sd = p.side[which];
  if (which) seg -= p.side[0].segs;
  const Lane ln = lane_place(p, lane);
  const long long pos = position(p, token);
  Unit un[NU];
  float c[NU][V], s[NU][V];
  float gam[NU][2 * V], bet[NU][2 * V];
#pragma unroll
  for (int n = 0; n < NU; ++n) {
    un[n] = unit_at<V, INTER>(p, ln.g + 32 * n, ln.on);
    angles<V>(p, freq, ln.g + 32 * n, pos, c[n], s[n]);
    if constexpr (NORM != 0) load_param<V>(sd.gamma, 1.f, un[n], gam[n]);
    if constexpr (NORM == TPQK_LAYERNORM)
      load_param<V>(sd.beta, 0.f, un[n], bet[n]);
  }
  const int h0 = seg * sd.heads_per_task;
  const int h1 = min(h0 + sd.heads_per_task, sd.heads);
  const T* in = reinterpret_cast<const T*>(sd.in.p);
  T* out = reinterpret_cast<T*>(sd.out.p);
  for (int hb = h0; hb < h1; hb += p.rows * FWD_ROWS) {
    RawT<T, V> raw[FWD_ROWS][NU][2];
#pragma unroll
    for (int k = 0; k < FWD_ROWS; ++k) {
      const int h = hb + k * p.rows + ln.row;
      const T* row = in + row_offset(sd.in, token, h < h1 ? h : h0);
#pragma unroll
      for (int n = 0; n < NU; ++n)
        load_unit<T, V>(row, un[n], h < h1, raw[k][n]);
    }
#pragma unroll
    for (int k = 0; k < FWD_ROWS; ++k) {
      if (hb + k * p.rows >= h1) break;   // the same on every lane
      const int h = hb + k * p.rows + ln.row;
      float e[NU][2 * V];
#pragma unroll
      for (int n = 0; n < NU; ++n) {
        unpack<T, V>(raw[k][n][0], &e[n][0]);
        unpack<T, V>(raw[k][n][1], &e[n][V]);
      }
      if constexpr (NORM == TPQK_LAYERNORM) {
        float m[1] = {sum_all<V, NU>(e)};
        row_sum(m, ln.g, ln.len, ln.first);
        centre<V, NU>(e, un, m[0] * p.inv_d);
      }
      if constexpr (NORM != 0) {
        float ss[1] = {dot<V, NU>(e, e)};
        row_sum(ss, ln.g, ln.len, ln.first);
        const float rstd = rsqrtf(fmaf(ss[0], p.inv_d, p.eps));
#pragma unroll
        for (int n = 0; n < NU; ++n)
#pragma unroll
          for (int i = 0; i < 2 * V; ++i) {
            e[n][i] *= rstd;
            if constexpr (NORM == TPQK_LAYERNORM)
              e[n][i] = fmaf(e[n][i], gam[n][i], bet[n][i]);
            else
              e[n][i] *= gam[n][i];
          }
      }
      T* row = out + row_offset(sd.out, token, h < h1 ? h : h0);
#pragma unroll
      for (int n = 0; n < NU; ++n) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float a = e[n][pair_a<V, INTER>(j)];
          const float b = e[n][pair_b<V, INTER>(j)];
          e[n][pair_a<V, INTER>(j)] = fmaf(a, c[n][j], -(b * s[n][j]));
          e[n][pair_b<V, INTER>(j)] = fmaf(a, s[n][j], b * c[n][j]);
        }
        store_unit<T, V>(row, un[n], h < h1, e[n]);
      }
    }
  }
}

// ------------------------------------------------------------- backward --
// Persistent blocks, so that a lane sums its unit's parameter gradients over
// all its rows in registers; a block takes q's tasks or k's.
template <class T, int V, int NU, int NORM, bool INTER>
__global__ void __launch_bounds__(THREADS)
    qk_rows_backward(const __grid_constant__ Args p) {
  __shared__ unsigned long long freq[MAX_PAIRS];
  __shared__ float sums[WARPS * 32 * NU * 2 * V];
  stage_freq(p, freq);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int which = static_cast<int>(blockIdx.x) >= p.q_blocks;
  const Side& sd = p.side[which];
  const int blocks =
      which ? static_cast<int>(gridDim.x) - p.q_blocks : p.q_blocks;
  const int block = static_cast<int>(blockIdx.x) - (which ? p.q_blocks : 0);
  const Lane ln = lane_place(p, lane);
  Unit un[NU];
  float gam[NU][2 * V], dgam[NU][2 * V], dbet[NU][2 * V];
#pragma unroll
  for (int n = 0; n < NU; ++n) {
    un[n] = unit_at<V, INTER>(p, ln.g + 32 * n, ln.on);
    load_param<V>(sd.gamma, 1.f, un[n], gam[n]);
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) dgam[n][i] = dbet[n][i] = 0.f;
  }
  const T* gin = reinterpret_cast<const T*>(sd.in.p);
  const T* xin = reinterpret_cast<const T*>(sd.x.p);
  T* out = reinterpret_cast<T*>(sd.out.p);
  const unsigned tasks = static_cast<unsigned>(p.tokens) * sd.segs;
  for (unsigned task = block * WARPS + warp; task < tasks;
       task += blocks * WARPS) {
    const int token = static_cast<int>(task / sd.segs);
    const int seg = static_cast<int>(task - token * sd.segs);
    const long long pos = position(p, token);
    float c[NU][V], s[NU][V];
#pragma unroll
    for (int n = 0; n < NU; ++n)
      angles<V>(p, freq, ln.g + 32 * n, pos, c[n], s[n]);
    const int h0 = seg * sd.heads_per_task;
    const int h1 = min(h0 + sd.heads_per_task, sd.heads);
    for (int hb = h0; hb < h1; hb += p.rows) {
      const int h = hb + ln.row;
      const bool on = h < h1;
      const int hh = on ? h : h0;
      const T* grow = gin + row_offset(sd.in, token, hh);
      const T* xrow = xin + row_offset(sd.x, token, hh);
      RawT<T, V> graw[NU][2], xraw[NU][2];
#pragma unroll
      for (int n = 0; n < NU; ++n) {
        load_unit<T, V>(grow, un[n], on, graw[n]);
        load_unit<T, V>(xrow, un[n], on, xraw[n]);
      }
      float g[NU][2 * V], e[NU][2 * V], u[NU][2 * V];
#pragma unroll
      for (int n = 0; n < NU; ++n) {
        unpack<T, V>(graw[n][0], &g[n][0]);
        unpack<T, V>(graw[n][1], &g[n][V]);
        unpack<T, V>(xraw[n][0], &e[n][0]);
        unpack<T, V>(xraw[n][1], &e[n][V]);
        // g = R^T dy (s carries the opposite direction's sign)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float a = g[n][pair_a<V, INTER>(j)];
          const float b = g[n][pair_b<V, INTER>(j)];
          g[n][pair_a<V, INTER>(j)] = fmaf(a, c[n][j], -(b * s[n][j]));
          g[n][pair_b<V, INTER>(j)] = fmaf(a, s[n][j], b * c[n][j]);
        }
#pragma unroll
        for (int i = 0; i < 2 * V; ++i) u[n][i] = g[n][i] * gam[n][i];
      }
      float mean_u = 0.f;
      if constexpr (NORM == TPQK_LAYERNORM) {
        float m[2] = {sum_all<V, NU>(e), sum_all<V, NU>(u)};
        row_sum(m, ln.g, ln.len, ln.first);
        centre<V, NU>(e, un, m[0] * p.inv_d);
        mean_u = m[1] * p.inv_d;
      }
      float q[2] = {dot<V, NU>(e, e), dot<V, NU>(e, u)};
      row_sum(q, ln.g, ln.len, ln.first);
      const float rstd = rsqrtf(fmaf(q[0], p.inv_d, p.eps));
      const float mean_ux = q[1] * rstd * p.inv_d;   // mean(u xh)
      T* orow = out + row_offset(sd.out, token, hh);
#pragma unroll
      for (int n = 0; n < NU; ++n) {
#pragma unroll
        for (int i = 0; i < 2 * V; ++i) {
          const float xh = e[n][i] * rstd;
          dgam[n][i] = fmaf(g[n][i], xh, dgam[n][i]);
          if constexpr (NORM == TPQK_LAYERNORM) dbet[n][i] += g[n][i];
          u[n][i] = rstd * (fmaf(-xh, mean_ux, u[n][i]) - mean_u);
        }
        store_unit<T, V>(orow, un[n], on, u[n]);
      }
    }
  }
  if (p.part == nullptr) return;
  // the block's sums: element i of every row slot, in the order of the slots
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
          sums[(warp * p.rows + ln.row) * p.d + at] = k ? dbet[n][i] : dgam[n][i];
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
  float s = 0.f;
  if (col < d) {
#pragma unroll 4
    for (int b = b0 + threadIdx.y; b < b1; b += 32)
      s += __ldg(part + (static_cast<long long>(b) * 2 + (o & 1)) * d + col);
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
template <class T, int V, int NU, int NORM, bool INTER>
void go(const Args& a, int blocks, bool backward, cudaStream_t s) {
  if (!backward) {
    qk_rows_forward<T, V, NU, NORM, INTER><<<blocks, THREADS, 0, s>>>(a);
  } else if constexpr (NORM != 0) {
    qk_rows_backward<T, V, NU, NORM, INTER><<<blocks, THREADS, 0, s>>>(a);
  }
}

template <class T, int V, int NU>
void by_norm(const Args& a, int norm, bool inter, int blocks, bool backward,
             cudaStream_t s) {
  if (norm == TPQK_RMSNORM) {
    if (inter) go<T, V, NU, TPQK_RMSNORM, true>(a, blocks, backward, s);
    else go<T, V, NU, TPQK_RMSNORM, false>(a, blocks, backward, s);
  } else if (norm == TPQK_LAYERNORM) {
    if (inter) go<T, V, NU, TPQK_LAYERNORM, true>(a, blocks, backward, s);
    else go<T, V, NU, TPQK_LAYERNORM, false>(a, blocks, backward, s);
  } else {
    if (inter) go<T, V, NU, 0, true>(a, blocks, backward, s);
    else go<T, V, NU, 0, false>(a, blocks, backward, s);
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
  qk_param_sums<<<dim3((d + 31) / 32, 4), dim3(32, 32), 0, s>>>(
      part, d, q_blocks, blocks, out[0], out[1], out[2], out[3]);
  return cudaGetLastError();
}

}  // namespace qk
}  // namespace tpmlp
