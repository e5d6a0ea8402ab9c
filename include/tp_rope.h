/*
 * tp_rope.h - C ABI of libtpmlp's query/key operators on one GB300 (sm_103a):
 * rotary positions, and the per-head norm of queries and keys with the
 * rotation in the same pass, each with its gradient.  Status codes,
 * tp_mlp_status_string() and tp_mlp_last_detail() are shared with tp_mlp.h;
 * tp_attn.h's attention block runs the same kernels between its QKV
 * projection and its core (tp_attn_set_rope, tp_attn_set_qk_norm).
 *
 * Rotation (Su et al., "RoFormer"): the first r = rot_dim elements of a head
 * form r / 2 pairs (a, b): elements (i, i + r/2) in the half layout, (2i,
 * 2i + 1) in the interleaved one.  At position p pair i turns by p f_i:
 *     y_a = amp (x_a cos p f_i - x_b sin p f_i)
 *     y_b = amp (x_a sin p f_i + x_b cos p f_i)
 * and the elements from r on are passed through.  Its gradient is the same
 * with -p f_i.
 *
 * Norm and rotation: per head row x of d elements, with mu = mean(x)
 * (TPQK_LAYERNORM; 0 for TPQK_RMSNORM), rstd = 1 / sqrt(mean((x - mu)^2) +
 * eps), xh = (x - mu) rstd:
 *     y = R(xh gamma + beta)
 *     gradient: g = R^T dy, dgamma = sum g xh, dbeta = sum g (over all tokens
 *     and heads), u = g gamma, dx = rstd (u - xh mean(u xh) [- mean(u)]).
 *
 * Conventions
 * -----------
 * - Element types: queries and keys bf16 (TPMLP_BF16) or fp32 (TPMLP_FP32),
 *   gamma, beta and their gradients fp32; all arithmetic fp32, one rounding
 *   to the element type.  (A row's sum of squares too: a row whose root mean
 *   square is past 1e18, or below 1e-18 with an eps of 0, leaves its range.)
 *   Angles are made in 64-bit fixed point: p f_i, f_i being the double that
 *   tp_rope_frequencies gives (up to 2^40), is within 2^-33 + |p| 2^-64 of a
 *   turn, then rounded to fp32.
 * - Pointers are DEVICE pointers the caller owns (tp_rope_config's inv_freq
 *   and the structs are host memory, read during the call only); the library
 *   never allocates device memory.  Calls only enqueue work on `stream`.
 *   Positions, parameters and workspace share no memory with an output.
 *   Data pointers need the alignment of their element type only; 16-byte
 *   aligned rows are read fastest.  Every function returns a status code and
 *   touches no output when argument validation fails.
 */
#ifndef TP_ROPE_H_
#define TP_ROPE_H_

#include <stddef.h>

#include "tp_mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TPROPE_MAX_HEAD_DIM 256

/* How the frequencies f_i are made, b_i = base^(-2i/r): */
#define TPROPE_SCALE_NONE   0  /* f_i = b_i                                   */
#define TPROPE_SCALE_LINEAR 1  /* f_i = b_i / factor                          */
#define TPROPE_SCALE_NTK    2  /* base replaced by base factor^(r/(r-2))
                                  (r = 2: as TPROPE_SCALE_NONE)               */
#define TPROPE_SCALE_YARN   3  /* by the turns n_i = original_length b_i / 2pi
                                  that a pair makes over the original context
                                  (Peng et al., "YaRN"): with the ramp k =
                                  (n_i - slow_turns) / (fast_turns -
                                  slow_turns) clamped to [0, 1], f_i =
                                  k b_i + (1 - k) b_i / factor; amp defaults
                                  to 0.1 ln(factor) + 1                       */
#define TPROPE_SCALE_CUSTOM 4  /* f_i = inv_freq[i]                           */

typedef struct tp_rope_config {
  int    head_dim;         /* d, 1 .. TPROPE_MAX_HEAD_DIM                    */
  int    rot_dim;          /* r, even, 0 .. d (0: no rotation)               */
  int    interleaved;      /* 0: half layout, 1: interleaved                 */
  int    scaling;          /* TPROPE_SCALE_*                                 */
  double base;             /* > 0 (not read for CUSTOM)                      */
  double factor;           /* > 0 (read by LINEAR, NTK and YARN)             */
  double original_length;  /* > 0 (read by YARN)                             */
  double slow_turns;       /* YARN: usually 1                                */
  double fast_turns;       /* YARN: usually 32, > slow_turns                 */
  double amplitude;        /* amp, at most 3.4e38 in magnitude; 0: the
                              default (1, for YARN above)                    */
  const double* inv_freq;  /* CUSTOM: host array of r / 2 finite values      */
} tp_rope_config;

typedef struct tp_rope_handle tp_rope_handle;

/* Validate and create a host-side handle (TPMLP_ERR_ARG / TPMLP_ERR_SHAPE;
 * no device work).  *handle is set only on success. */
int tp_rope_create(const tp_rope_config* config, tp_rope_handle** handle);
int tp_rope_destroy(tp_rope_handle* handle);

/* The handle's r / 2 frequencies (radians per position) and its amplitude;
 * either pointer may be NULL. */
int tp_rope_frequencies(const tp_rope_handle* handle, double* inv_freq,
                        double* amplitude);

/* Heads of a tensor: element c of head j of token t is at data[t *
 * token_stride + (j / group) * group_stride + (j % group) * head_stride + c]
 * (strides in elements, >= 0 and below 4 GB each; d consecutive elements per
 * head).  `group` heads lie head_stride apart and groups group_stride apart: the
 * shard-grouped columns of tp_attn.h's QKV are group = H / t, group_stride =
 * 3 h / t, head_stride = d, token_stride = 3 h; a plain [T, H, d] tensor is group
 * = H.
 * heads = 0 stands for no tensor.  An output's heads must not overlap one
 * another. */
typedef struct tp_heads {
  void*     data;
  long long token_stride;
  long long group_stride;
  long long head_stride;
  int       heads;
  int       group;
} tp_heads;

/* Position of token t: data[t] (int32, or int64 with is_int64 = 1) if data is
 * not NULL (a device pointer to `tokens` values), else offset + (t mod
 * seq_len), or offset + t with seq_len = 0.  Any integer is a position. */
typedef struct tp_positions {
  const void* data;
  int         is_int64;
  long long   offset;
  long long   seq_len;
} tp_positions;

/* Rotate the heads of q and k (inverse = 1: the gradient, by the opposite
 * angles).  Each output is either the very view of its input (in place; where
 * both q and k are, the elements from rot_dim on are not touched) or shares no
 * element with any input or other output.  k may be NULL (then k_out too).
 *   tokens  0 <= T <= 2^28 (T = 0 enqueues nothing)
 *   dtype   TPMLP_BF16 or TPMLP_FP32, of q and k
 * TPMLP_ERR_SHAPE: a head count that differs between input and output, a
 * stride out of range, a group that does not divide the heads, more than 65535
 * heads; TPMLP_ERR_ARG: a null pointer, a bad enum, outputs that overlap;
 * TPMLP_ERR_ALIGN: a pointer off its element's alignment. */
int tp_rope_apply(tp_rope_handle* handle, int tokens, int dtype, int inverse,
                  const tp_heads* q_in, const tp_heads* q_out,
                  const tp_heads* k_in, const tp_heads* k_out,
                  const tp_positions* positions, void* stream);

#define TPQK_RMSNORM   1
#define TPQK_LAYERNORM 2

/* Parameters of the per-head norm.  gamma and beta are [d] fp32 device
 * pointers shared by all heads of q (k); NULL gamma stands for ones, NULL
 * beta for zeros (TPQK_RMSNORM takes no beta: TPMLP_ERR_ARG). */
typedef struct tp_qk_norm {
  int          norm;       /* TPQK_RMSNORM or TPQK_LAYERNORM                 */
  float        eps;        /* >= 0, finite                                   */
  const float* q_gamma;
  const float* q_beta;
  const float* k_gamma;
  const float* k_beta;
} tp_qk_norm;

/* Norm and rotation of every head of q and k.  Views as tp_rope_apply. */
int tp_qk_norm_forward(tp_rope_handle* handle, int tokens, int dtype,
                       const tp_qk_norm* norm, const tp_heads* q_in,
                       const tp_heads* q_out, const tp_heads* k_in,
                       const tp_heads* k_out, const tp_positions* positions,
                       void* stream);

/* Parameter gradients, [d] fp32 each, overwritten; each may be NULL; no two
 * share memory (TPMLP_ERR_ARG). */
typedef struct tp_qk_norm_grads {
  float* q_gamma;
  float* q_beta;   /* TPQK_LAYERNORM only */
  float* k_gamma;
  float* k_beta;
} tp_qk_norm_grads;

/* Bytes of device workspace tp_qk_norm_backward needs (partial sums of the
 * parameter gradients), the same for every token count; 16-byte aligned. */
size_t tp_qk_norm_workspace_bytes(const tp_rope_handle* handle);

/* Gradient: dq_out, dk_out from dq, dk (with respect to the rotated heads) and
 * the forward's inputs q_in, k_in, whose statistics are made again.  dq_out
 * may be the very view of dq or of q_in, else it shares no element with any
 * input or other output; k likewise.  The parameter gradients are summed in a
 * fixed order that depends on the shapes only: repeated calls are
 * bit-identical.  With T = 0 they are set to zero. */
int tp_qk_norm_backward(tp_rope_handle* handle, int tokens, int dtype,
                        const tp_qk_norm* norm, const tp_heads* dq,
                        const tp_heads* q_in, const tp_heads* dq_out,
                        const tp_heads* dk, const tp_heads* k_in,
                        const tp_heads* dk_out, const tp_positions* positions,
                        const tp_qk_norm_grads* grads, void* workspace,
                        size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* TP_ROPE_H_ */
