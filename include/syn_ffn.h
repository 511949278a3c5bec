/*
 * syn_ffn.h -- the gated feed-forward block in front of a down projection: both
 * projections, the activation and the product in one kernel, and its gradient
 * (libsyn.so; status codes as in syn.h, element types as in syn_rope.h).
 *
 * Its input is what syn_layer_norm writes or an AG-GEMM gathered, its output the
 * A of syn_gemm_rs or syn_gemm_ar (a rank's shard of the weights is a call with
 * that shard's d_ff columns).
 *
 *   G = X Wg,  U = X Wu,  H = act(G) * U                      (syn_gated_ffn)
 *   dG = dH * U * act'(G),  dU = dH * act(G)
 *   dX = dG Wg^T + dU Wu^T,  dWg = X^T dG,  dWu = X^T dU      (syn_gated_ffn_backward)
 *
 *   SYN_ACT_SILU       act(g) = g / (1 + exp(-g))
 *   SYN_ACT_GELU       act(g) = g (1 + erf(g / sqrt 2)) / 2
 *   SYN_ACT_GELU_TANH  act(g) = g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2
 *
 * X [n_tokens, d], Wg and Wu [d, d_ff] (as the B of syn.h's products; the two may
 * be the halves of one matrix), G, U, H [n_tokens, d_ff].
 *
 * Precision: 16-bit inputs; products accumulate in fp32 on the tensor cores; H
 * comes from the fp32 G and U and is rounded once.  The gradient reads G and U as
 * the forward stores them, in fp32 or rounded to the plan's type (half the memory; the
 * gradients' errors are then 1.8 times a single rounding's, else 1.4); dG and dU are
 * computed in fp32 and rounded once, as results and as operands of the products;
 * dX, dWg and dWu are rounded once.  An X row that is not finite reaches its own
 * rows of G, U, H and dX, and dWg and dWu; no other row.
 */
#ifndef SYN_FFN_H
#define SYN_FFN_H

#include <stdint.h>

#include "syn.h"
#include "syn_rope.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { SYN_ACT_SILU = 0, SYN_ACT_GELU = 1, SYN_ACT_GELU_TANH = 2 };

typedef struct syn_ffn_plan_s *syn_ffn_plan_t; /* opaque, owned by the library */

typedef struct {
    int dtype;           /* SYN_DTYPE_BF16 or SYN_DTYPE_F16                        */
    int d;               /* columns of X, a multiple of 8                          */
    int d_ff;            /* columns of H, a multiple of 8                          */
    int act;             /* SYN_ACT_*                                              */
    int backward;        /* 1: the plan can run syn_gated_ffn_backward             */
    int saved_f32;       /* 1: G and U are in fp32, 0: in dtype                    */
    uint64_t timeout_ns; /* bound on every device wait (0 = SYN_TIMEOUT_NS or 2 s); one that
                            runs out is seen up to 0.2 ms later, and the call ends within
                            the bound, at least a second, after that                    */
} syn_ffn_cfg_t;

/* A matrix: element (i, j) at p + i * row + j.  p 16-byte aligned; row (where
 * there is more than one) a positive multiple of 8 elements (4 of fp32 ones), in
 * outputs no less than the columns. */
typedef struct {
    void *p;
    int64_t row;
} syn_ffn_mat_t;

/* Defaults: bf16, d 4096, d_ff 14336, SiLU, backward, G and U in dtype. */
int syn_ffn_cfg_default(syn_ffn_cfg_t *cfg);

/* Validate and build a plan on the current device (it holds 20 MB there for tiles
 * that several CTAs share, half of it without backward).  Its calls belong to that
 * device: with another one current they are SYN_ERR_INVALID.  Calls of one plan, forward
 * and backward, must not overlap (they share this workspace); one plan serves any
 * number of layers of its sizes in turn. */
int syn_ffn_plan_create(syn_ffn_plan_t *out, const syn_ffn_cfg_t *cfg);

/* Free a plan (no call of it may still be running).  NULL is a no-op. */
int syn_ffn_plan_destroy(syn_ffn_plan_t plan);

/* The parts that the longer tiles of a call's products are cut into where they are few (1:
 * whole), of syn_gated_ffn and of syn_gated_ffn_backward with dX, with dWg and dWu, or with
 * both (want: 1, 2, 3; 0: of neither).  Needs no GPU work; either result may be NULL. */
int syn_ffn_plan_parts(syn_ffn_plan_t plan, int64_t n_tokens, int want, int *forward, int *backward);

/* H (asynchronous on `stream`), and where they are not NULL the G and U that the
 * gradient needs.  Outputs overlap neither inputs nor each other.  The same bits for
 * the same inputs on the same device. */
int syn_gated_ffn(syn_ffn_plan_t plan, const syn_ffn_mat_t *X, const syn_ffn_mat_t *Wg, const syn_ffn_mat_t *Wu,
                  const syn_ffn_mat_t *H, const syn_ffn_mat_t *G, const syn_ffn_mat_t *U, int64_t n_tokens, void *stream);

/* The gradient (asynchronous): dG and dU (dG may be G or dH, dU may be U or dH,
 * with the same type and stride), then dX (NULL: not wanted), dWg and dWu (both NULL: not
 * wanted).  Outputs overlap neither inputs nor each other otherwise; one that begins
 * where another operand of the call does is SYN_ERR_INVALID, in the forward too.
 * Weight gradients are overwritten, with zeros where there is no token.
 * No atomics on values: the same bits for the same inputs on the same device. */
int syn_gated_ffn_backward(syn_ffn_plan_t plan, const syn_ffn_mat_t *dH, const syn_ffn_mat_t *X, const syn_ffn_mat_t *Wg,
                           const syn_ffn_mat_t *Wu, const syn_ffn_mat_t *G, const syn_ffn_mat_t *U,
                           const syn_ffn_mat_t *dG, const syn_ffn_mat_t *dU, const syn_ffn_mat_t *dX,
                           const syn_ffn_mat_t *dWg, const syn_ffn_mat_t *dWu, int64_t n_tokens, void *stream);

/* Synchronise `stream`, then read and clear the device error word: SYN_OK,
 * SYN_ERR_TIMEOUT or SYN_ERR_CUDA. */
int syn_ffn_sync_status(syn_ffn_plan_t plan, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SYN_FFN_H */
