// Arguments and launchers of the query/key head-row kernels
// (qk_rows_kernels.cuh).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "tp_rope.h"

namespace tpmlp {
namespace qk {

// Threads of a block; each warp takes one task (a token's heads, or some of
// them) at a time.
constexpr int WARPS = 4;
constexpr int THREADS = 32 * WARPS;
constexpr int MAX_PAIRS = TPROPE_MAX_HEAD_DIM / 2;
// Blocks of the backward kernel (four on each of a GB300's 152 SMs; a constant,
// so that the order of the parameter gradients' sums depends on the shapes only
// and not on the device).
constexpr int BWD_BLOCKS = 608;

// tp_heads for the kernels.  A head's group is umulhi(head, magic) with magic =
// ceil(2^32 / group): exact for heads below 2^16 and groups of 2 .. 2^16 - 1 (a
// group of one head is given as one group of all heads instead).
struct View {
  char* p;
  long long ts;          // token stride, in bytes
  unsigned gs, hs;       // group and head strides, in bytes
  unsigned group, magic;
};

struct Side {
  View in;               // forward: x; backward: dy
  View x;                // backward: x
  View out;
  const float* gamma;    // nullable
  const float* beta;     // nullable
  int heads;
  int steps;             // ceil(heads / Args::rows)
};

struct Args {
  Side side[2];          // q, k
  int tokens;            // tokens * segs < 2^31
  int d;
  int rot;               // r
  int units;             // units of a head row (at most 32)
  int rot_units;         // the first of them, which are rotated
  int rows;              // head rows a warp holds at once
  // BITS: bytes of a piece, pieces of a row, ceil(2^32 / row_pieces) (0 for one)
  int piece, row_pieces;
  unsigned row_pieces_magic;
  // forward: a task takes `per` steps of a token's q and k steps (in this
  // order); backward: `per_side` steps of one side's
  int per, segs;
  int per_side[2], segs_side[2];
  const void* pos;       // nullable
  int pos64;
  long long offset;
  unsigned seq_len;      // 0: tokens are positions
  float amp, sign;       // sign: -1 turns back
  float eps, inv_d;
  int param16;           // gamma and beta are 16-byte aligned
  float* part;           // backward: [blocks][2][d] sums of dgamma, dbeta
  int q_blocks;          // backward: blocks that take q's tasks
  unsigned long long freq[MAX_PAIRS];  // turns per position, 2^-64
};

// norm: 0 (rotation only), TPQK_RMSNORM or TPQK_LAYERNORM.  bits: 0 for rows whose
// units are whole 16-byte vectors, else the elements (4, 2 or 1) that are read at
// a time (the kinds of rows in qk_rows_kernels.cuh).
cudaError_t launch_forward(const Args& a, bool bf16, int bits, int norm,
                           bool interleaved, cudaStream_t s);
cudaError_t launch_backward(const Args& a, bool bf16, int bits, int norm,
                            bool interleaved, int blocks, cudaStream_t s);
// Either of the two above, by element type.
cudaError_t launch_bf16(const Args& a, int bits, int norm, bool interleaved,
                        int blocks, bool backward, cudaStream_t s);
cudaError_t launch_fp32(const Args& a, int bits, int norm, bool interleaved,
                        int blocks, bool backward, cudaStream_t s);
// out[side][0 dgamma, 1 dbeta], each nullable, from `blocks` blocks' sums.
cudaError_t launch_param_sums(const float* part, int d, int q_blocks,
                              int blocks, float* const out[4], cudaStream_t s);

}  // namespace qk
}  // namespace tpmlp
