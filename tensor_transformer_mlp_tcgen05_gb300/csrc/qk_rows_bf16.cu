// The query/key head-row kernels for bf16.
#include "qk_rows_kernels.cuh"

namespace tpmlp {
namespace qk {

cudaError_t launch_bf16(const Args& a, int bits, int norm, bool interleaved,
                        int blocks, bool backward, cudaStream_t s) {
  return by_norm<__nv_bfloat16>(a, bits, norm, interleaved, blocks, backward, s);
}

}  // namespace qk
}  // namespace tpmlp
