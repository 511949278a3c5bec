/*
 * syn_clip.h -- the global 2-norm of many gradient tensors, and clipping by it
 * (libsyn.so; status codes as in syn.h, element types as in syn_rope.h).
 *
 * This is the end of a training step: over the gradients that
 * syn_layer_norm_backward, syn_gated_ffn_backward, syn_qk_norm_rope_backward and
 * the projections' products give.
 *
 *   norm = sqrt(sum over all tensors' elements of x^2)
 *   y = x c,  c = min(1, max_norm / (norm + eps))          (syn_grad_clip)
 *
 * Precision: squares and short sums in fp32, scaled where they would leave its
 * range, so that every finite input has its norm (inf only above fp32's largest);
 * longer sums in fp64, in a fixed order: the same bits for the same inputs on the
 * same device.  c is computed in fp64 and rounded to fp32; a product is rounded to
 * fp32 and then to the tensor's type (one below fp32's smallest normal number once
 * more).  An element that is NaN makes the norm, c and all y
 * NaN; one that is infinite makes the norm infinite and c 0 (with
 * max_norm infinite too, NaN): the caller reads the norm to tell.
 */
#ifndef SYN_CLIP_H
#define SYN_CLIP_H

#include <stdint.h>

#include "syn.h"
#include "syn_rope.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct syn_clip_plan_s *syn_clip_plan_t; /* opaque, owned by the library */

/* n contiguous elements of type dtype (aligned to their size).  y (syn_grad_clip)
 * may be x (in place). */
typedef struct {
    const void *x;
    void *y;
    int64_t n;
    int dtype; /* SYN_DTYPE_* */
} syn_clip_tensor_t;

/* Build a plan on the current device (a workspace for partial sums).  Its calls
 * belong to that device: with another one current they are SYN_ERR_INVALID. */
int syn_clip_plan_create(syn_clip_plan_t *out);

/* Free a plan (no call of it may still be running).  NULL is a no-op. */
int syn_clip_plan_destroy(syn_clip_plan_t plan);

/* norm (fp32 on the device, overwritten) of n_tensors tensors, whose y are not
 * used; a tensor that is listed twice counts twice.  Asynchronous on `stream`;
 * the list is read before the call returns.  Calls of one plan must not overlap
 * (they share its workspace). */
int syn_grad_norm(syn_clip_plan_t plan, const syn_clip_tensor_t *tensors, int n_tensors, float *norm, void *stream);

/* The norm (nullable) and the clipped tensors.  Memory that is written may
 * overlap no other of the call's tensors, read or written, nor norm:
 * SYN_ERR_INVALID (so a tensor listed twice).  max_norm >= 0, eps >= 0. */
int syn_grad_clip(syn_clip_plan_t plan, const syn_clip_tensor_t *tensors, int n_tensors, float max_norm, float eps,
                  float *norm, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SYN_CLIP_H */
