// Global L2 norm of many gradient tensors, and clipping (tp_grad.h).
//
// Three launches: sums of squares per block, their sum and the factor by one
// block, the scaling.  The first and the last are bound by memory; each thread has
// eight 16-byte loads in flight.  The last walks the chunks backwards, so that
// what the first read last is still in L2 (129 MB): gradients smaller than that
// are read from DRAM once.  Each launch comes up while its predecessor drains
// (programmatic dependent launch), and the last loads its chunks before it
// waits for the factor.
//
// Up to 512 KB in up to 64 tensors are done by one launch of one cluster of eight
// blocks, which exchange their sums through distributed shared memory: 4 KB 4.1 us
// (three launches: 5.7), 256 KB 4.8 (6.2), 500 KB 5.8 (6.7).
//
// GB300: 1.26 GB of fp32 into other tensors in 545 us (1.26 GB read for the norm at
// 7.1 TB/s, then read and written at 6.8 TB/s; the floor of one read and one write is
// 370), 50 MB in 24 us (floor 14.8), 8 MB in 7.5.
#include <algorithm>

#include "host_common.cuh"
#include "ptx.cuh"
#include "tp_grad.h"

using namespace tpmlp;
using namespace tpmlp::host;

namespace {

// 16-byte vectors a thread loads at once.
constexpr int BATCH = 8;
constexpr int THREADS = 256;
constexpr int BLOCKS = 608;            // four on each of a GB300's 152 SMs (a
                                       // constant: it orders the sums)
constexpr int CHUNK_BYTES = 16 * BATCH * THREADS;
// Tensors of one launch: the table travels as a kernel parameter (16 KB; one of
// SMALL_TABLE, 2 KB, where that is enough: 500 KB in 8 tensors 6.7 us, with the
// large one 6.9).
constexpr int TABLE = 512;

// One cluster: pieces of one warp's batch of SMALL_BATCH vectors a lane.
constexpr int SMALL_BATCH = 4;
constexpr int SMALL_THREADS = 512;
constexpr int SMALL_BLOCKS = 8;
constexpr int SMALL_WARPS = SMALL_BLOCKS * SMALL_THREADS / 32;
constexpr int SMALL_PIECE_BYTES = 16 * SMALL_BATCH * 32;
constexpr int SMALL_TABLE = 64;

struct Entry {
  const void* grad;
  void* out;
  long long numel;
  unsigned first;      // this tensor's first chunk (piece)
  int bf16;
};
template <int N>
struct Table {
  Entry e[N];
  int count;
  unsigned chunks;
};

template <int N>
__device__ __forceinline__ const Entry& entry_of(const Table<N>& t,
                                                 unsigned chunk) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.e[mid].first <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return t.e[lo];
}

// A chunk (or piece) of a tensor: n elements of it, of which the first nv 16-byte
// vectors are read as such (none where the gradient is off 16 bytes), and written
// as such where the output is not (o16).  The output has no say in how squares are
// read, so that clipping finds the very norm that the norm alone does.
struct Part {
  const char* g;
  char* o;
  int n, nv;
  bool bf16, o16;
};
template <int BYTES>
__device__ __forceinline__ Part part_of(const Entry& e, unsigned chunk) {
  Part p;
  p.bf16 = e.bf16 != 0;
  const int size = p.bf16 ? 2 : 4;
  const long long at = static_cast<long long>(chunk - e.first) * BYTES;
  p.g = static_cast<const char*>(e.grad) + at;
  p.o = static_cast<char*>(e.out) + at;
  p.n = static_cast<int>(
      min(static_cast<long long>(BYTES / size), e.numel - at / size));
  p.nv = (reinterpret_cast<uintptr_t>(p.g) & 15u) == 0 ? p.n * size / 16 : 0;
  p.o16 = (reinterpret_cast<uintptr_t>(p.o) & 15u) == 0;
  return p;
}

// Vectors first, first + STEP, ... of the part, B of them; zeros past its end.
template <int B, int STEP>
__device__ __forceinline__ void load_batch(const Part& p, int first,
                                           uint4 (&v)[B]) {
  const uint4* g = reinterpret_cast<const uint4*>(p.g);
#pragma unroll
  for (int k = 0; k < B; ++k) {
    const int i = first + k * STEP;
    v[k] = i < p.nv ? g[i] : make_uint4(0u, 0u, 0u, 0u);
  }
}

// Adds the squares of N values: to `sum` in fp32 where that is right, which is
// where theirs is between 2^-60 and 2^110 (a thread adds at most 66 of these in
// a chunk or in its pieces, and a warp's 32 threads stay below 2^122: nothing
// overflows; squares that underflowed, below 2^-126, are nothing beside it),
// else (larger, smaller but not all zero, or not a number) to `wide` in fp64.
// fp64 is kept out of the way: an SM does two such additions per cycle.
template <int N>
__device__ __forceinline__ void add_squares(const float (&x)[N], float& sum,
                                            double& wide) {
  float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < N; ++i) a[i % 4] = fmaf(x[i], x[i], a[i % 4]);
  const float s = (a[0] + a[1]) + (a[2] + a[3]);
  if (s >= 0x1p-60f && s <= 0x1p110f) {
    sum += s;
    return;
  }
  bool any = s != 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) any = any || x[i] != 0.f;
  if (any) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const double v = static_cast<double>(x[i]);
      wide += v * v;
    }
  }
}

template <int B>
__device__ __forceinline__ void batch_squares(const uint4 (&v)[B], bool bf16,
                                              float& sum, double& wide) {
  if (bf16) {
#pragma unroll
    for (int k = 0; k < B; k += 4) {
      float x[32];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        unpack_bf16x2(v[k + j].x, x[8 * j], x[8 * j + 1]);
        unpack_bf16x2(v[k + j].y, x[8 * j + 2], x[8 * j + 3]);
        unpack_bf16x2(v[k + j].z, x[8 * j + 4], x[8 * j + 5]);
        unpack_bf16x2(v[k + j].w, x[8 * j + 6], x[8 * j + 7]);
      }
      add_squares<32>(x, sum, wide);
    }
  } else {
    float x[4 * B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      x[4 * k] = __uint_as_float(v[k].x);
      x[4 * k + 1] = __uint_as_float(v[k].y);
      x[4 * k + 2] = __uint_as_float(v[k].z);
      x[4 * k + 3] = __uint_as_float(v[k].w);
    }
    add_squares<4 * B>(x, sum, wide);
  }
}

__device__ __forceinline__ float element_at(const Part& p, int i) {
  return p.bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.g)[i])
                : reinterpret_cast<const float*>(p.g)[i];
}
__device__ __forceinline__ void store_at(const Part& p, int i, float x) {
  if (p.bf16) reinterpret_cast<__nv_bfloat16*>(p.o)[i] = __float2bfloat16_rn(x);
  else reinterpret_cast<float*>(p.o)[i] = x;
}

// The elements that load_batch leaves out, by `lanes` threads.
__device__ __forceinline__ void rest_squares(const Part& p, int lane, int lanes,
                                             float& sum, double& wide) {
  for (int i = p.nv * (p.bf16 ? 8 : 4) + lane; i < p.n; i += lanes) {
    const float x[1] = {element_at(p, i)};
    add_squares<1>(x, sum, wide);
  }
}
__device__ __forceinline__ void rest_scale(const Part& p, int lane, int lanes,
                                           float c) {
  for (int i = p.nv * (p.bf16 ? 8 : 4) + lane; i < p.n; i += lanes)
    store_at(p, i, element_at(p, i) * c);
}

__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t w, float c) {
  float lo, hi;
  unpack_bf16x2(w, lo, hi);
  return pack_bf16x2(lo * c, hi * c);
}

// A vector at an address that is off 16 bytes.
__device__ __forceinline__ void store_apart(const Part& p, char* to,
                                            const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (p.bf16) {
      reinterpret_cast<uint16_t*>(to)[2 * j] = static_cast<uint16_t>(w[j]);
      reinterpret_cast<uint16_t*>(to)[2 * j + 1] =
          static_cast<uint16_t>(w[j] >> 16);
    } else {
      reinterpret_cast<uint32_t*>(to)[j] = w[j];
    }
  }
}

template <int B, int STEP>
__device__ __forceinline__ void store_batch(const Part& p, int first,
                                            const uint4 (&v)[B], float c) {
#pragma unroll
  for (int k = 0; k < B; ++k) {
    const int i = first + k * STEP;
    if (i >= p.nv) continue;
    char* to = p.o + 16LL * i;
    uint4 u;
    if (p.bf16) {
      u = make_uint4(scale_bf16x2(v[k].x, c), scale_bf16x2(v[k].y, c),
                     scale_bf16x2(v[k].z, c), scale_bf16x2(v[k].w, c));
    } else {
      u = make_uint4(__float_as_uint(__uint_as_float(v[k].x) * c),
                     __float_as_uint(__uint_as_float(v[k].y) * c),
                     __float_as_uint(__uint_as_float(v[k].z) * c),
                     __float_as_uint(__uint_as_float(v[k].w) * c));
    }
    if (p.o16) *reinterpret_cast<uint4*>(to) = u;
    else store_apart(p, to, u);
  }
}

// Sum of n values at `x` (shared or global memory) by one warp, in a fixed
// order; every lane gets it.
__device__ __forceinline__ double warp_total(const double* x, int n) {
  double t = 0.0;
#pragma unroll 8
  for (int i = threadIdx.x & 31; i < n; i += 32) t += x[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}

// Sum over the block, on the first warp's lanes.
__device__ __forceinline__ double block_total(double v) {
  __shared__ double all[THREADS];
  all[threadIdx.x] = v;
  __syncthreads();
  return threadIdx.x < 32 ? warp_total(all, THREADS) : 0.0;
}

// min(1, max_norm / (norm + eps)); 1 for a norm that is not finite as it is
// reported, in fp32.
__device__ __forceinline__ float factor(double n, double max_norm, double eps) {
  const double ratio = max_norm / (n + eps);
  return isfinite(static_cast<float>(n)) && ratio < 1.0 ? static_cast<float>(ratio) : 1.f;
}

template <int N>
__global__ void __launch_bounds__(THREADS, 4)
    grad_squares(const __grid_constant__ Table<N> t, double* part) {
  // the second pass may take the SMs' free places from here on
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  double wide = 0.0;
  for (unsigned k = blockIdx.x; k < t.chunks; k += gridDim.x) {
    const Part p = part_of<CHUNK_BYTES>(entry_of(t, k), k);
    uint4 v[BATCH];
    load_batch<BATCH, THREADS>(p, threadIdx.x, v);
    float sum = 0.f;
    batch_squares<BATCH>(v, p.bf16, sum, wide);
    rest_squares(p, threadIdx.x, THREADS, sum, wide);
    wide += static_cast<double>(sum);
  }
  wide = block_total(wide);
  if (threadIdx.x == 0) part[blockIdx.x] = wide;
}

// Waits until the sums are there, and adds them.  (Every thread loads its own few
// first: one warp alone, load after load, took 6 us for 608 of them.)
__device__ __forceinline__ double total_norm(const double* part, int slots) {
  __shared__ double norm;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int EACH = (BLOCKS + THREADS - 1) / THREADS;
  double t = 0.0;
  for (int i = 0; i < slots; i += EACH * THREADS) {
    double x[EACH];
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
      const int at = i + k * THREADS + threadIdx.x;
      x[k] = at < slots ? part[at] : 0.0;
    }
#pragma unroll
    for (int k = 0; k < EACH; ++k) t += x[k];
  }
  t = block_total(t);
  if (threadIdx.x == 0) norm = sqrt(t);
  __syncthreads();
  return norm;
}

// (c: nullable; for grad_scale.)
__global__ void __launch_bounds__(THREADS)
    grad_norm_final(const double* part, int slots, double max_norm, double eps,
                    float* norm, float* c) {
  // grad_scale's blocks may come up and load (they wait for this one's end)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const double n = total_norm(part, slots);
  if (threadIdx.x == 0) {
    *norm = static_cast<float>(n);
    if (c != nullptr) *c = factor(n, max_norm, eps);
  }
}

// One chunk a block.  (A block that stays and walks over chunks, as in
// grad_squares, reached 6.3 TB/s of reads and writes together, one block a chunk
// 6.8: 578 and 545 us for all of 1.26 GB.)
template <int N>
__global__ void __launch_bounds__(THREADS, 4)
    grad_scale(const __grid_constant__ Table<N> t, const float* factor) {
  const unsigned chunk = t.chunks - 1 - blockIdx.x;
  const Part p = part_of<CHUNK_BYTES>(entry_of(t, chunk), chunk);
  uint4 v[BATCH];
  load_batch<BATCH, THREADS>(p, threadIdx.x, v);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float c = *factor;
  if (c == 1.f && p.g == p.o) return;
  store_batch<BATCH, THREADS>(p, threadIdx.x, v, c);
  rest_scale(p, threadIdx.x, THREADS, c);
}

// Norm and (clip) scaling of at most 2 x SMALL_WARPS pieces: a warp keeps its
// pieces in registers from the squares to the scaling.
__global__ void __cluster_dims__(SMALL_BLOCKS, 1, 1)
    __launch_bounds__(SMALL_THREADS)
    grad_small(const __grid_constant__ Table<SMALL_TABLE> t, int clip,
               double max_norm, double eps, float* norm) {
  __shared__ double warps[SMALL_THREADS / 32];
  __shared__ double mine;       // this block's sum
  __shared__ float c_shared;
  const int lane = threadIdx.x & 31;
  const unsigned warp = blockIdx.x * (SMALL_THREADS / 32) + (threadIdx.x >> 5);
  uint4 v[2][SMALL_BATCH];
  Part p[2];
  float sum = 0.f;
  double wide = 0.0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const unsigned piece = warp + k * SMALL_WARPS;
    p[k].g = p[k].o = nullptr;
    p[k].n = p[k].nv = 0;
    p[k].bf16 = p[k].o16 = false;
    if (piece < t.chunks)
      p[k] = part_of<SMALL_PIECE_BYTES>(entry_of(t, piece), piece);
    load_batch<SMALL_BATCH, 32>(p[k], lane, v[k]);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    batch_squares<SMALL_BATCH>(v[k], p[k].bf16, sum, wide);
    rest_squares(p[k], lane, 32, sum, wide);
  }
  // (2 batches and 64 single elements a lane at most: see add_squares)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (__any_sync(0xffffffffu, wide != 0.0)) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      wide += __shfl_xor_sync(0xffffffffu, wide, o);
  }
  if (lane == 0) warps[threadIdx.x >> 5] = wide + static_cast<double>(sum);
  __syncthreads();
  if (threadIdx.x < 32) {
    const double b = warp_total(warps, SMALL_THREADS / 32);
    if (lane == 0) mine = b;
  }
  ptx::cluster_sync();
  if (threadIdx.x < 32) {
    double total = 0.0;
    if (lane < SMALL_BLOCKS) {
      const uint32_t remote = ptx::mapa_shared(ptx::smem_u32(&mine), lane);
      asm volatile("ld.shared::cluster.f64 %0, [%1];"
                   : "=d"(total) : "r"(remote) : "memory");
    }
#pragma unroll
    for (int o = SMALL_BLOCKS / 2; o > 0; o >>= 1)
      total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) {
      const double n = sqrt(total);
      if (blockIdx.x == 0) *norm = static_cast<float>(n);
      c_shared = factor(n, max_norm, eps);
    }
  }
  // (and no block ends while another still reads its sum)
  ptx::cluster_sync();
  const float c = c_shared;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (clip && p[k].n > 0 && (c != 1.f || p[k].g != p[k].o)) {
      store_batch<SMALL_BATCH, 32>(p[k], lane, v[k], c);
      rest_scale(p[k], lane, 32, c);
    }
  }
}

// ----------------------------------------------------------------- host --

int bad(int code, const char* msg) {
  set_detail_msg(msg);
  return code;
}

int tables(int count) { return count <= 0 ? 1 : (count + TABLE - 1) / TABLE; }

size_t item(int dtype) { return dtype == TPMLP_BF16 ? 2 : 4; }

int check_tensors(int count, const tp_grad_tensor* t, bool clip) {
  if (count < 0) return bad(TPMLP_ERR_SHAPE, "grad: negative count");
  if (count > 0 && t == nullptr) return bad(TPMLP_ERR_ARG, "grad: null tensors");
  for (int i = 0; i < count; ++i) {
    if (t[i].dtype != TPMLP_BF16 && t[i].dtype != TPMLP_FP32)
      return bad(TPMLP_ERR_ARG, "grad: dtype must be TPMLP_BF16 or TPMLP_FP32");
    if (t[i].numel < 0 || t[i].numel > (1LL << 40))
      return bad(TPMLP_ERR_SHAPE, "grad: numel must be 0 .. 2^40");
    if (t[i].numel > 0 && (t[i].grad == nullptr || (clip && t[i].out == nullptr)))
      return bad(TPMLP_ERR_ARG, "grad: null pointer");
    const size_t size = item(t[i].dtype);
    if (reinterpret_cast<uintptr_t>(t[i].grad) % size != 0 ||
        (clip && reinterpret_cast<uintptr_t>(t[i].out) % size != 0))
      return bad(TPMLP_ERR_ALIGN, "grad: a tensor is not aligned to its element");
  }
  return TPMLP_OK;
}

// Every out is its own grad or overlaps no grad and no other out: the ranges in
// the order of their starts, each compared with the furthest out and the
// furthest range before it.
struct Range {
  uintptr_t lo, hi;
  bool out;
};
bool apart(Range* r, size_t n) {
  auto before = [](const Range& a, const Range& b) { return a.lo < b.lo; };
  if (!std::is_sorted(r, r + n, before)) std::sort(r, r + n, before);
  uintptr_t out_end = 0, any_end = 0;
  for (size_t i = 0; i < n; ++i) {
    if (r[i].lo < out_end || (r[i].out && r[i].lo < any_end)) return false;
    any_end = std::max(any_end, r[i].hi);
    if (r[i].out) out_end = std::max(out_end, r[i].hi);
  }
  return true;
}
int check_apart(int count, const tp_grad_tensor* t) {
  Range few[2 * SMALL_TABLE];
  Range* r = few;
  if (count > SMALL_TABLE) {
    r = new (std::nothrow) Range[2 * static_cast<size_t>(count)];
    if (r == nullptr) return bad(TPMLP_ERR_ARG, "grad: out of host memory");
  }
  size_t n = 0;
  for (int i = 0; i < count; ++i) {
    if (t[i].numel == 0) continue;
    const size_t bytes = static_cast<size_t>(t[i].numel) * item(t[i].dtype);
    const uintptr_t g = reinterpret_cast<uintptr_t>(t[i].grad);
    const uintptr_t o = reinterpret_cast<uintptr_t>(t[i].out);
    r[n++] = {o, o + bytes, true};
    if (o != g) r[n++] = {g, g + bytes, false};
  }
  const bool ok = apart(r, n);
  if (r != few) delete[] r;
  return ok ? TPMLP_OK
            : bad(TPMLP_ERR_ARG, "grad: an out overlaps another tensor");
}

long long parts_of(const tp_grad_tensor& t, int part_bytes) {
  const long long per = part_bytes / static_cast<int>(item(t.dtype));
  return (t.numel + per - 1) / per;
}

// Tensors [at, end) as a kernel's table, in parts of part_bytes; empty ones are
// left out.
template <int N>
int fill(Table<N>* T, int at, int end, int part_bytes, const tp_grad_tensor* t,
         bool clip) {
  T->count = 0;
  long long chunks = 0;
  for (int i = at; i < end; ++i) {
    if (t[i].numel == 0) continue;
    Entry& e = T->e[T->count++];
    e.grad = t[i].grad;
    // without clipping nothing is written, and `out` only has to be aligned
    e.out = clip ? t[i].out : const_cast<void*>(t[i].grad);
    e.numel = t[i].numel;
    e.bf16 = t[i].dtype == TPMLP_BF16;
    e.first = static_cast<unsigned>(chunks);
    chunks += parts_of(t[i], part_bytes);
    if (chunks > 0x7fffffffLL)
      return bad(TPMLP_ERR_SHAPE, "grad: more than 2^46 bytes");
  }
  T->chunks = static_cast<unsigned>(chunks);
  return TPMLP_OK;
}

int cuda_rc(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return TPMLP_OK;
  set_detail(what, e);
  return TPMLP_ERR_CUDA;
}

// A launch that may begin while its predecessor in the stream ends (it waits
// for it with griddepcontrol.wait).
template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), int blocks, cudaStream_t s,
                             const A&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The three launches, with tables of N tensors.
template <int N>
int run(int count, const tp_grad_tensor* t, bool clip, double max_norm,
        double eps, float* norm, double* part, cudaStream_t s) {
  Table<N> T;
  const int launches = std::max(1, (count + N - 1) / N);
  auto table = [&](int k) {
    return fill(&T, k * N, std::min(count, (k + 1) * N), CHUNK_BYTES, t, clip);
  };
  int slots = 0;
  for (int k = 0; k < launches; ++k) {
    TRY(table(k));
    const int blocks =
        std::max(1, static_cast<int>(std::min<unsigned>(T.chunks, BLOCKS)));
    grad_squares<N><<<blocks, THREADS, 0, s>>>(T, part + slots);
    TRY(cuda_rc(cudaGetLastError(), "grad_squares"));
    slots += blocks;
  }
  float* c = reinterpret_cast<float*>(part + slots);
  TRY(cuda_rc(launch_dependent(grad_norm_final, 1, s,
                               static_cast<const double*>(part), slots, max_norm,
                               eps, norm, clip ? c : nullptr),
              "grad_norm_final"));
  if (!clip) return TPMLP_OK;
  for (int k = launches - 1; k >= 0; --k) {
    if (launches > 1) TRY(table(k));
    if (T.chunks == 0) continue;
    const float* f = c;
    if (k == launches - 1) {
      TRY(cuda_rc(launch_dependent(grad_scale<N>, static_cast<int>(T.chunks), s,
                                   T, f),
                  "grad_scale"));
    } else {   // (its predecessor does not write what this one waits for)
      grad_scale<N><<<T.chunks, THREADS, 0, s>>>(T, f);
      TRY(cuda_rc(cudaGetLastError(), "grad_scale"));
    }
  }
  return TPMLP_OK;
}

int go(int count, const tp_grad_tensor* t, bool clip, double max_norm,
       double eps, float* norm, void* workspace, size_t bytes, void* stream) {
  TRY(check_tensors(count, t, clip));
  if (norm == nullptr || workspace == nullptr)
    return bad(TPMLP_ERR_ARG, "grad: null norm or workspace");
  if (reinterpret_cast<uintptr_t>(norm) % 4 != 0 || !aligned16(workspace))
    return bad(TPMLP_ERR_ALIGN, "grad: norm or workspace is not aligned");
  if (bytes < tp_grad_workspace_bytes(count))
    return bad(TPMLP_ERR_WORKSPACE, "grad: workspace too small");
  if (clip) TRY(check_apart(count, t));
  int sms = 0;
  TRY(check_device(&sms));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(workspace);
  if (count > SMALL_TABLE)
    return run<TABLE>(count, t, clip, max_norm, eps, norm, part, s);
  // One cluster for up to 512 KB (an empty list too).
  long long pieces = 0;
  for (int i = 0; i < count && pieces <= 2 * SMALL_WARPS; ++i)
    pieces += parts_of(t[i], SMALL_PIECE_BYTES);
  if (pieces > 2 * SMALL_WARPS)
    return run<SMALL_TABLE>(count, t, clip, max_norm, eps, norm, part, s);
  Table<SMALL_TABLE> T;
  TRY(fill(&T, 0, count, SMALL_PIECE_BYTES, t, clip));
  grad_small<<<SMALL_BLOCKS, SMALL_THREADS, 0, s>>>(T, clip ? 1 : 0, max_norm,
                                                    eps, norm);
  return cuda_rc(cudaGetLastError(), "grad_small");
}

}  // namespace

extern "C" {

size_t tp_grad_workspace_bytes(int count) {
  if (count < 0) return 0;
  // the blocks' sums and the factor
  return sizeof(double) * (BLOCKS * static_cast<size_t>(tables(count)) + 2);
}

int tp_grad_norm(int count, const tp_grad_tensor* tensors, float* norm,
                 void* workspace, size_t workspace_bytes, void* stream) {
  return go(count, tensors, false, 0.0, 0.0, norm, workspace, workspace_bytes,
            stream);
}

int tp_grad_clip(int count, const tp_grad_tensor* tensors, double max_norm,
                 double eps, float* norm, void* workspace,
                 size_t workspace_bytes, void* stream) {
  if (!(max_norm >= 0.0))
    return bad(TPMLP_ERR_ARG, "grad: max_norm must be >= 0");
  if (!(eps >= 0.0) || !std::isfinite(eps))
    return bad(TPMLP_ERR_ARG, "grad: eps must be finite and >= 0");
  return go(count, tensors, true, max_norm, eps, norm, workspace,
            workspace_bytes, stream);
}

}  // extern "C"
