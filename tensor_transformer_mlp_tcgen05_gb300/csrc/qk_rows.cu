// Launchers of the query/key head-row kernels (qk_rows_kernels.cuh, compiled once
// per element type), and the sums of the parameter gradients.
#include "qk_rows.cuh"

namespace tpmlp {
namespace qk {
namespace {

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

}  // namespace

cudaError_t launch_forward(const Args& a, bool bf16, int bits, int norm,
                           bool interleaved, cudaStream_t s) {
  const unsigned tasks = static_cast<unsigned>(a.tokens) * a.segs;
  const int blocks = static_cast<int>((tasks + WARPS - 1) / WARPS);
  return (bf16 ? launch_bf16 : launch_fp32)(a, bits, norm, interleaved, blocks,
                                            false, s);
}

cudaError_t launch_backward(const Args& a, bool bf16, int bits, int norm,
                            bool interleaved, int blocks, cudaStream_t s) {
  if (norm == 0) return cudaErrorInvalidValue;
  return (bf16 ? launch_bf16 : launch_fp32)(a, bits, norm, interleaved, blocks,
                                            true, s);
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
