// The query/key head-row kernels for fp32.
#include "qk_rows_kernels.cuh"

namespace tpmlp {
namespace qk {

cudaError_t launch_fp32(const Args& a, int bits, int norm, bool interleaved,
                        int blocks, bool backward, cudaStream_t s) {
  return by_norm<float>(a, bits, norm, interleaved, blocks, backward, s);
}

}  // namespace qk
}  // namespace tpmlp
