// Global L2 norm of many gradient tensors, and clipping (tp_grad.h).
//
// Two passes over the data: sums of squares per block, then, each block having
// added all blocks' sums in the same fixed order, the scaling.  The second pass
// walks the chunks backwards, so that what the first read last is still in L2
// (129 MB): a set of gradients smaller than that is read from DRAM once.
// Both passes are bound by memory.
#include <algorithm>

#include "host_common.cuh"
#include "tp_grad.h"

using namespace tpmlp;
using namespace tpmlp::host;

namespace {

constexpr int THREADS = 256;
constexpr int BLOCKS = 608;            // four on each of the 152 SMs
// Bytes of a tensor that a block takes at a time: 64 (bf16: 128) elements a
// thread.
constexpr int CHUNK_BYTES = 65536;
// Tensors of one launch: the table travels as a kernel parameter.
constexpr int TABLE = 512;

struct Entry {
  const void* grad;
  void* out;
  long long numel;
  unsigned first;      // this tensor's first chunk
  int bf16;
};
struct Table {
  Entry e[TABLE];
  int count;
  unsigned chunks;
};

__device__ __forceinline__ int find_entry(const Table& t, unsigned chunk) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.e[mid].first <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ bool aligned16d(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// Squares of N values into acc (fp32), or into big (fp64) when the largest of
// them is not in [2^-40, 2^55]: a square may then over- or underflow fp32, or
// is not a number.  Inside that range what underflows is below 2^-46 of the
// largest square, and the sums of 128 elements stay below 2^127.
template <int N>
__device__ __forceinline__ void add_squares(const float (&v)[N], float& acc,
                                            double& big) {
  float m = 0.f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    m = fmaxf(m, fabsf(v[i]));
    nan = nan || v[i] != v[i];
  }
  if (!nan && ((m >= 0x1p-40f && m <= 0x1p55f) || m == 0.f)) {
#pragma unroll
    for (int i = 0; i < N; ++i) acc = fmaf(v[i], v[i], acc);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      big += static_cast<double>(v[i]) * static_cast<double>(v[i]);
  }
}

__device__ __forceinline__ void unpack16(const uint4& u, float (&v)[8]) {
  unpack_bf16x2(u.x, v[0], v[1]);
  unpack_bf16x2(u.y, v[2], v[3]);
  unpack_bf16x2(u.z, v[4], v[5]);
  unpack_bf16x2(u.w, v[6], v[7]);
}

// Sum over the block, in a fixed order; every thread gets it.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double w[THREADS / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) t += w[i];
  return t;
}

__global__ void __launch_bounds__(THREADS)
    grad_squares(const __grid_constant__ Table t, double* part) {
  double total = 0.0;
  for (unsigned chunk = blockIdx.x; chunk < t.chunks; chunk += gridDim.x) {
    const Entry& e = t.e[find_entry(t, chunk)];
    const long long per = e.bf16 ? CHUNK_BYTES / 2 : CHUNK_BYTES / 4;
    const long long base = static_cast<long long>(chunk - e.first) * per;
    const int n = static_cast<int>(min(per, e.numel - base));
    float acc = 0.f;
    int done = 0;
    if (e.bf16) {
      const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(e.grad) + base;
      if (aligned16d(g)) {
        const uint4* gv = reinterpret_cast<const uint4*>(g);
        const int nv = n / 8;
#pragma unroll 4
        for (int i = threadIdx.x; i < nv; i += THREADS) {
          float v[8];
          unpack16(gv[i], v);
          add_squares<8>(v, acc, total);
        }
        done = nv * 8;
      }
      for (int i = done + threadIdx.x; i < n; i += THREADS) {
        const float v[1] = {__bfloat162float(g[i])};
        add_squares<1>(v, acc, total);
      }
    } else {
      const float* g = static_cast<const float*>(e.grad) + base;
      if (aligned16d(g)) {
        const float4* gv = reinterpret_cast<const float4*>(g);
        const int nv = n / 4;
#pragma unroll 4
        for (int i = threadIdx.x; i < nv; i += THREADS) {
          const float4 u = gv[i];
          const float v[4] = {u.x, u.y, u.z, u.w};
          add_squares<4>(v, acc, total);
        }
        done = nv * 4;
      }
      for (int i = done + threadIdx.x; i < n; i += THREADS) {
        const float v[1] = {g[i]};
        add_squares<1>(v, acc, total);
      }
    }
    total += static_cast<double>(acc);
  }
  total = block_sum(total);
  if (threadIdx.x == 0) part[blockIdx.x] = total;
}

__device__ __forceinline__ double total_norm(const double* part, int slots) {
  double s = 0.0;
  for (int i = threadIdx.x; i < slots; i += THREADS) s += part[i];
  return sqrt(block_sum(s));
}

__global__ void __launch_bounds__(THREADS)
    grad_norm_final(const double* part, int slots, float* norm) {
  const double n = total_norm(part, slots);
  if (threadIdx.x == 0) *norm = static_cast<float>(n);
}

__global__ void __launch_bounds__(THREADS)
    grad_scale(const __grid_constant__ Table t, const double* part, int slots,
               double max_norm, double eps, float* norm) {
  const double n = total_norm(part, slots);
  if (blockIdx.x == 0 && threadIdx.x == 0 && norm != nullptr)
    *norm = static_cast<float>(n);
  // a norm that is not finite scales nothing
  const double ratio = max_norm / (n + eps);
  const float c = isfinite(n) && ratio < 1.0 ? static_cast<float>(ratio) : 1.f;
  for (unsigned k = blockIdx.x; k < t.chunks; k += gridDim.x) {
    const unsigned chunk = t.chunks - 1 - k;
    const Entry& e = t.e[find_entry(t, chunk)];
    if (c == 1.f && e.out == e.grad) continue;
    const long long per = e.bf16 ? CHUNK_BYTES / 2 : CHUNK_BYTES / 4;
    const long long base = static_cast<long long>(chunk - e.first) * per;
    const int len = static_cast<int>(min(per, e.numel - base));
    int done = 0;
    if (e.bf16) {
      const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(e.grad) + base;
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(e.out) + base;
      if (aligned16d(g) && aligned16d(o)) {
        const uint4* gv = reinterpret_cast<const uint4*>(g);
        uint4* ov = reinterpret_cast<uint4*>(o);
        const int nv = len / 8;
#pragma unroll 4
        for (int i = threadIdx.x; i < nv; i += THREADS) {
          float v[8];
          unpack16(gv[i], v);
          ov[i] = make_uint4(pack_bf16x2(v[0] * c, v[1] * c),
                             pack_bf16x2(v[2] * c, v[3] * c),
                             pack_bf16x2(v[4] * c, v[5] * c),
                             pack_bf16x2(v[6] * c, v[7] * c));
        }
        done = nv * 8;
      }
      for (int i = done + threadIdx.x; i < len; i += THREADS)
        o[i] = __float2bfloat16_rn(__bfloat162float(g[i]) * c);
    } else {
      const float* g = static_cast<const float*>(e.grad) + base;
      float* o = static_cast<float*>(e.out) + base;
      if (aligned16d(g) && aligned16d(o)) {
        const float4* gv = reinterpret_cast<const float4*>(g);
        float4* ov = reinterpret_cast<float4*>(o);
        const int nv = len / 4;
#pragma unroll 4
        for (int i = threadIdx.x; i < nv; i += THREADS) {
          const float4 v = gv[i];
          ov[i] = make_float4(v.x * c, v.y * c, v.z * c, v.w * c);
        }
        done = nv * 4;
      }
      for (int i = done + threadIdx.x; i < len; i += THREADS) o[i] = g[i] * c;
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
int check_apart(int count, const tp_grad_tensor* t) {
  struct Range {
    uintptr_t lo, hi;
    bool out;
  };
  Range* r = new (std::nothrow) Range[2 * static_cast<size_t>(count) + 1];
  if (r == nullptr) return bad(TPMLP_ERR_ARG, "grad: out of host memory");
  size_t n = 0;
  for (int i = 0; i < count; ++i) {
    if (t[i].numel == 0) continue;
    const size_t bytes = static_cast<size_t>(t[i].numel) * item(t[i].dtype);
    const uintptr_t g = reinterpret_cast<uintptr_t>(t[i].grad);
    const uintptr_t o = reinterpret_cast<uintptr_t>(t[i].out);
    r[n++] = {o, o + bytes, true};
    if (o != g) r[n++] = {g, g + bytes, false};
  }
  std::sort(r, r + n, [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t out_end = 0, any_end = 0;
  bool ok = true;
  for (size_t i = 0; i < n && ok; ++i) {
    ok = r[i].lo >= out_end && (!r[i].out || r[i].lo >= any_end);
    any_end = std::max(any_end, r[i].hi);
    if (r[i].out) out_end = std::max(out_end, r[i].hi);
  }
  delete[] r;
  return ok ? TPMLP_OK
            : bad(TPMLP_ERR_ARG, "grad: an out overlaps another tensor");
}

// Tensors [at, at + TABLE) as a kernel's table; empty ones are left out.
int fill(Table* T, int at, int count, const tp_grad_tensor* t, bool clip) {
  T->count = 0;
  long long chunks = 0;
  for (int i = at; i < std::min(count, at + TABLE); ++i) {
    if (t[i].numel == 0) continue;
    Entry& e = T->e[T->count++];
    e.grad = t[i].grad;
    e.out = clip ? t[i].out : nullptr;
    e.numel = t[i].numel;
    e.bf16 = t[i].dtype == TPMLP_BF16;
    e.first = static_cast<unsigned>(chunks);
    const long long per = CHUNK_BYTES / static_cast<int>(item(t[i].dtype));
    chunks += (t[i].numel + per - 1) / per;
    if (chunks > 0x7fffffffLL)
      return bad(TPMLP_ERR_SHAPE, "grad: more than 2^47 bytes");
  }
  T->chunks = static_cast<unsigned>(chunks);
  return TPMLP_OK;
}

int cuda_rc(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return TPMLP_OK;
  set_detail(what, e);
  return TPMLP_ERR_CUDA;
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
  Table T;
  const int launches = tables(count);
  int slots = 0;
  for (int k = 0; k < launches; ++k) {
    TRY(fill(&T, k * TABLE, count, t, clip));
    const int blocks =
        std::max(1, static_cast<int>(std::min<unsigned>(T.chunks, BLOCKS)));
    grad_squares<<<blocks, THREADS, 0, s>>>(T, part + slots);
    TRY(cuda_rc(cudaGetLastError(), "grad_squares"));
    slots += blocks;
  }
  if (!clip) {
    grad_norm_final<<<1, THREADS, 0, s>>>(part, slots, norm);
    return cuda_rc(cudaGetLastError(), "grad_norm_final");
  }
  for (int k = launches - 1; k >= 0; --k) {
    if (launches > 1) TRY(fill(&T, k * TABLE, count, t, clip));
    const int blocks =
        std::max(1, static_cast<int>(std::min<unsigned>(T.chunks, BLOCKS)));
    grad_scale<<<blocks, THREADS, 0, s>>>(T, part, slots, max_norm, eps,
                                          k == 0 ? norm : nullptr);
    TRY(cuda_rc(cudaGetLastError(), "grad_scale"));
  }
  return TPMLP_OK;
}

}  // namespace

extern "C" {

size_t tp_grad_workspace_bytes(int count) {
  if (count < 0) return 0;
  return sizeof(double) * BLOCKS * static_cast<size_t>(tables(count));
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
