/*
 * tp_grad.h - C ABI of libtpmlp's global gradient norm and clipping on one
 * GB300 (sm_103a).  Status codes, tp_mlp_status_string() and
 * tp_mlp_last_detail() are shared with tp_mlp.h.
 *
 *     norm = sqrt(sum over all tensors and elements of g^2)
 *     c    = min(1, max_norm / (norm + eps)),   out = c g
 *
 * A norm that is not finite in fp32 (an infinity or NaN among the gradients, or
 * a norm beyond 3.4e38) is reported as infinity or NaN and scales nothing: c =
 * 1, so that a training step can read the norm and be skipped with its
 * gradients as they were.
 *
 * Squares are summed in fp32 over at most 64 elements of a thread (a short set:
 * then over the 32 threads of a warp), beyond that in fp64, in a fixed order
 * (bit-identical repeats); runs of elements whose squares would leave fp32's
 * range are squared in fp64, so every finite gradient has its right norm
 * (rounded to fp32 once).  c is rounded to fp32, c g to the gradient's type.
 */
#ifndef TP_GRAD_H_
#define TP_GRAD_H_

#include <stddef.h>

#include "tp_mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One gradient tensor: `numel` contiguous elements (0 is allowed, the
 * pointers may then be NULL) of type `dtype` (TPMLP_BF16 or TPMLP_FP32),
 * aligned to their element.  out: where tp_grad_clip writes c g; the same
 * pointer as grad scales in place.  tp_grad_norm does not read it. */
typedef struct tp_grad_tensor {
  const void* grad;
  void*       out;
  long long   numel;
  int         dtype;
} tp_grad_tensor;

/* Bytes of device workspace either call needs for `count` tensors (16-byte
 * aligned; 0 for a negative count).  Calls that may overlap on the GPU need a
 * workspace each. */
size_t tp_grad_workspace_bytes(int count);

/* *norm = the global norm (fp32, device memory, overwritten).  `tensors` is a
 * host array, read during the call only.  count = 0 gives 0. */
int tp_grad_norm(int count, const tp_grad_tensor* tensors, float* norm,
                 void* workspace, size_t workspace_bytes, void* stream);

/* The same norm, and every tensor scaled.  Each out is either its own grad
 * or memory that overlaps no grad and no other out (TPMLP_ERR_ARG: the same
 * tensor listed twice would be scaled twice).
 *   max_norm  >= 0 (infinity: no clipping);  eps >= 0, finite
 *   norm      as tp_grad_norm (required); no part of a tensor. */
int tp_grad_clip(int count, const tp_grad_tensor* tensors, double max_norm,
                 double eps, float* norm, void* workspace,
                 size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* TP_GRAD_H_ */
