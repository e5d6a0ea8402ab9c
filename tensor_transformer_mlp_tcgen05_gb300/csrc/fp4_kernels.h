// Launchers of the four-bit kernels (host side).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "fp4.cuh"

namespace tpmlp {
namespace fp4 {

// Where a quantisation takes g from: 2^exponent; or another packed matrix (like);
// or the matrix's own largest |x|, left in `slots` words of its header by
// launch_amax, the launch before.
struct Gain {
  int exponent;
  int slots;
  const Header* like;
};

// The largest finite |x| of x [rows, cols], block by block; slots: the blocks.
cudaError_t launch_amax(bool bf16, const void* x, long long stride,
                        long long rows, long long cols, Header* head, int* slots,
                        cudaStream_t s);

// x [p.rows, p.cols] into p.
cudaError_t launch_quantize_rows(bool bf16, int format, const void* x,
                                 long long stride, const Packed& p,
                                 const Gain& g, cudaStream_t s);

// x [x_rows = p.cols, p.rows], transposed, into p.  part (nullable):
// [p.ktiles][p.rows] sums of x's columns over 256 rows each.  rp (nullable): x along
// its rows, in the same launch.
cudaError_t launch_quantize_columns(bool bf16, int format, const void* x,
                                    long long stride, int x_rows,
                                    const Packed& p, const Gain& g,
                                    float* part, const Packed* rp,
                                    cudaStream_t s);

cudaError_t launch_dequantize(const Packed& p, int format, bool bf16, void* out,
                              long long stride, cudaStream_t s);

// What becomes of a product's elements.
enum Epilogue4 : int {
  OUT_BF16 = 0,
  OUT_FP32 = 1,
  OUT_GELU_FP4 = 2,   // GeLU, quantised along its rows into `y`
};

// C = g_A g_B A B^T (+ bias), then the epilogue.
struct ProductArgs {
  Packed a, b;          // [M, K], [N, K]
  int M, N;
  // instead of a's codes, scales and g: the plain matrix x that the product
  // quantises itself, g = 2^x_exponent (M <= PLAIN_ROWS_*; a then has its sizes, and
  // a's status word is cleared by the product); or null
  const void* x;
  int x_bf16;
  long long x_stride;
  int x_exponent;
  int epilogue;
  void* out;            // [M, N], row stride ldo (OUT_BF16, OUT_FP32)
  long long ldo;
  const float* bias;    // [N] or null
  const void* residual; // OUT_BF16: [M, N] bf16 of row stride ldr, added before
  long long ldr;        // the rounding; or null
  Packed y;             // OUT_GELU_FP4
  int y_exponent;       // NV: y's g
  int gelu_mode;
  int* status;
  unsigned long long budget_ns;
  // 1: a call's later kernel: the launch before it makes A, and B was complete
  // before the call (see wait_for_launch_before)
  int dependent;
};

// Tiles of 256 x 256 on CTA pairs, for many rows of A and B.  ta: boxes of 128
// rows of A's codes, tb: of 64 rows of B's; tsa, tsb: scale tiles.
cudaError_t launch_product_pairs(int format, const CUtensorMap& ta,
                                 const CUtensorMap& tsa, const CUtensorMap& tb,
                                 const CUtensorMap& tsb, const CUtensorMap* to,
                                 const ProductArgs& args, int max_pairs,
                                 cudaStream_t s);

// Tiles of 128 rows of B x up to 128 rows of A, K split over a cluster, for few
// rows of A.
// Rows that the product quantises itself.
constexpr int PLAIN_ROWS_BF16 = 8, PLAIN_ROWS_FP32 = 4;
cudaError_t launch_product_split(int format, const ProductArgs& args, int sms,
                                 cudaStream_t s);
cudaError_t launch_product_plain(int format, const ProductArgs& args, int sms,
                                 cudaStream_t s);

}  // namespace fp4
}  // namespace tpmlp
