/*
 * syn_rope.h -- rotary positions of query and key heads, alone or in the same
 * pass as a root-mean-square norm of each head, with their gradients
 * (libsyn.so; status codes as in syn.h).
 *
 * This is the step in front of syn_ring_attention, syn_head_attention and
 * syn_window_attention: it makes their Q and K.  A rank of a sequence-parallel
 * group passes the global position of its first token as pos0; a serving
 * step passes each sequence's position and, as `slots`, the cache rows that
 * the rotated key and the value are written to.
 *
 *   h = x                                     (syn_rope)
 *   h = x * rsqrt(mean(x^2) + eps) * w        (syn_qk_norm_rope, per head)
 *   y[a] = h[a] c_i - h[b] s_i,  y[b] = h[a] s_i + h[b] c_i
 *   c_i, s_i = attn_factor * (cos, sin)(position * f_i), 0 <= i < d_rot / 2
 *   (a, b) = (2i, 2i+1)  SYN_ROPE_INTERLEAVED,  (i, i + d_rot/2)  SYN_ROPE_HALF
 *
 * Elements d_rot .. d-1 of a head are not rotated (and not scaled).
 * f_i = base^(-2i/d_rot), changed for long contexts as `scaling` says:
 *   LINEAR  f_i / factor
 *   NTK     base replaced by base * factor^(d_rot / (d_rot - 2))
 *   LLAMA3  f_i kept where 2 pi / f_i <= original_context / high_freq_factor,
 *           f_i / factor where it is >= original_context / low_freq_factor,
 *           between them (1-t) f_i / factor + t f_i with
 *           t = (original_context f_i / 2 pi - low) / (high - low)
 *   YARN    f_i (1 - r_i) + f_i / factor r_i, r_i = clamp((i - lo) / (hi - lo), 0, 1),
 *           lo = max(floor(n(beta_fast)), 0), hi = min(ceil(n(beta_slow)), d_rot - 1),
 *           n(t) = d_rot ln(original_context / (2 pi t)) / (2 ln base)
 *           (hi - lo at least 0.001); attn_factor 0 means 0.1 ln(factor) + 1
 *
 * Precision: inputs in the plan's type, arithmetic in fp32, one
 * round-to-nearest-even to the plan's type.  position * f_i is reduced modulo
 * one turn exactly (64-bit fixed point); an angle is right to about 1e-7 radians
 * (its rounding to fp32) and 3e-16 |position| f_i (that of f_i to 53 bits): to
 * 2e-7 at positions below 2^28, 1e-6 below 2^31.  Negative positions are allowed.
 * The norm's sums are fp32.
 */
#ifndef SYN_ROPE_H
#define SYN_ROPE_H

#include <stdint.h>

#include "syn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the operators in this header and in syn_window.h. */
enum { SYN_DTYPE_BF16 = 0, SYN_DTYPE_F16 = 1, SYN_DTYPE_F32 = 2 };

enum { SYN_ROPE_HALF = 0, SYN_ROPE_INTERLEAVED = 1 };

enum {
    SYN_ROPE_SCALE_NONE = 0,
    SYN_ROPE_SCALE_LINEAR = 1,
    SYN_ROPE_SCALE_NTK = 2,
    SYN_ROPE_SCALE_LLAMA3 = 3,
    SYN_ROPE_SCALE_YARN = 4
};

typedef struct syn_rope_plan_s *syn_rope_plan_t; /* opaque, owned by the library */

typedef struct {
    int dtype;               /* SYN_DTYPE_*: heads, norm weights                     */
    int d;                   /* elements of a head, 1..256                           */
    int d_rot;               /* rotated elements, even, 0..d                         */
    int layout;              /* SYN_ROPE_HALF or SYN_ROPE_INTERLEAVED                */
    double base;             /* > 1                                                  */
    int scaling;             /* SYN_ROPE_SCALE_*                                     */
    double factor;           /* >= 1 (all scalings but NONE)                         */
    double low_freq_factor;  /* LLAMA3: 0 < low < high                               */
    double high_freq_factor;
    double original_context; /* LLAMA3, YARN: tokens of the trained context, > 0     */
    double beta_fast;        /* YARN: > beta_slow > 0                                */
    double beta_slow;
    double attn_factor;      /* factor on the rotated elements; 0 = 1, or for YARN
                                0.1 ln(factor) + 1                                   */
} syn_rope_cfg_t;

/* Rows of one tensor: element (t, h, j) at x + t * x_token + h * x_head + j
 * (strides in elements, of any sign).  Rows that are read may overlap; written
 * ones may not, and strides of y below d elements are refused where they are
 * used.  y may be x with the same strides (in place). */
typedef struct {
    const void *x;
    int64_t x_token, x_head;
    void *y;
    int64_t y_token, y_head;
    int heads;
} syn_rope_rows_t;

/* One tensor of syn_qk_norm_rope_backward: x the forward's input, dy the
 * gradient of its output, dx the gradient of x (dx may be dy or x with the
 * same strides); w the norm's weight [d] (NULL: ones); dw its gradient, fp32
 * [d], overwritten (NULL: not wanted). */
typedef struct {
    const void *x;
    int64_t x_token, x_head;
    const void *dy;
    int64_t dy_token, dy_head;
    void *dx;
    int64_t dx_token, dx_head;
    const void *w;
    float *dw;
    int heads;
} syn_rope_grad_t;

/* Defaults: bf16, d = d_rot = 128, half layout, base 10000, no scaling;
 * factor 1, low/high 1/4, original_context 8192, beta 32/1, attn_factor 0. */
int syn_rope_cfg_default(syn_rope_cfg_t *cfg);

/* Validate and build a plan on the current device (the frequency table and
 * the workspace of the weight gradients). */
int syn_rope_plan_create(syn_rope_plan_t *out, const syn_rope_cfg_t *cfg);

/* Free a plan (no call of it may still be running).  NULL is a no-op. */
int syn_rope_plan_destroy(syn_rope_plan_t plan);

/* The plan's d_rot/2 frequencies (radians per position) and the factor on the
 * rotated elements; either pointer may be NULL.  Host-side, synchronous. */
int syn_rope_plan_frequencies(syn_rope_plan_t plan, double *f, double *attn_factor);

/* Rotate q and k (either may be NULL, or have no heads) and copy v (NULL: none).
 *   positions : int64 [n_tokens] on the device; NULL: pos0 + t
 *   slots     : int64 [n_tokens] on the device: row t of k and v is written at
 *               y + slots[t] * y_token (a cache row); a slot outside
 *               [0, n_slots) writes nothing.  NULL: row t
 * Asynchronous on `stream`; calls of one plan may run on several streams. */
int syn_rope(syn_rope_plan_t plan, const syn_rope_rows_t *q, const syn_rope_rows_t *k, const syn_rope_rows_t *v,
             const int64_t *positions, int64_t pos0, const int64_t *slots, int64_t n_slots, int64_t n_tokens,
             void *stream);

/* The gradient of syn_rope: x = dy, y = dx (the inverse turn, the same factor). */
int syn_rope_backward(syn_rope_plan_t plan, const syn_rope_rows_t *dq, const syn_rope_rows_t *dk,
                      const int64_t *positions, int64_t pos0, int64_t n_tokens, void *stream);

/* Norm and rotation in one pass.  wq, wk: weights [d] of the plan's type
 * (NULL: ones).  v, positions, pos0, slots as in syn_rope. */
int syn_qk_norm_rope(syn_rope_plan_t plan, const syn_rope_rows_t *q, const void *wq, const syn_rope_rows_t *k,
                     const void *wk, float eps, const syn_rope_rows_t *v, const int64_t *positions, int64_t pos0,
                     const int64_t *slots, int64_t n_slots, int64_t n_tokens, void *stream);

/* Its gradient.  The weight gradients are summed in a fixed order (the same
 * bits for the same inputs on the same device), through the plan's workspace:
 * calls with dw on one plan must not overlap. */
int syn_qk_norm_rope_backward(syn_rope_plan_t plan, const syn_rope_grad_t *q, const syn_rope_grad_t *k, float eps,
                              const int64_t *positions, int64_t pos0, int64_t n_tokens, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SYN_ROPE_H */
