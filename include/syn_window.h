/*
 * syn_window.h -- causal attention with a sliding window and a few first
 * tokens that stay visible (sinks): over ragged sequences with its gradient,
 * and for one token per sequence over a paged cache (libsyn.so; status codes
 * as in syn.h, element types as in syn_rope.h).
 *
 * Sequence s has q_lens[s] query rows and k_lens[s] key rows; the sequences'
 * rows lie one after another in Q, O and in K, V.  Query row i of a sequence
 * is at position p = k_len - q_len + i (the queries are the last tokens of the
 * keys) and sees key j when
 *
 *   j <= p  and  (j > p - window  or  j < sinks)        (window 0: j <= p)
 *
 *   O[i][h][:] = sum_j softmax_j(scale * Q[i][h] . K[j][hk]) V[j][hk][:]
 *   hk = h / (H_q / H_kv),  lse[i][h] = log sum_j exp(scale * Q[i][h] . K[j][hk])
 *
 * over the keys that it sees.  A row that sees none (p < 0) has O = 0,
 * lse = -inf and gives no gradient.  Rows outside the sequences are neither
 * read into a result nor written.
 *
 * Precision: 16-bit inputs; the products accumulate in fp32 on the tensor
 * cores; scores, softmax statistics and lse in fp32; the probabilities (and
 * in the gradient the score gradients) are rounded to the inputs' type as
 * operands of the next product; outputs are rounded once.  A value row V[j]
 * that is not finite reaches the rows of every 128-row query tile that reads
 * its block, as 0 * inf does in a matrix product, a key or value row that is not
 * finite likewise the dQ of such tiles' rows, and a query or dO row that is not
 * finite the gradients of the keys in the tiles that its block meets; rows
 * outside a sequence (another sequence's, an unused part of a page) never do.
 */
#ifndef SYN_WINDOW_H
#define SYN_WINDOW_H

#include <stdint.h>

#include "syn.h"
#include "syn_rope.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct syn_window_plan_s *syn_window_plan_t; /* opaque, owned by the library */
typedef struct syn_decode_plan_s *syn_decode_plan_t; /* opaque, owned by the library */

typedef struct {
    int dtype;           /* SYN_DTYPE_BF16 or SYN_DTYPE_F16                        */
    int H_q, H_kv;       /* H_q % H_kv == 0, H_q <= 1024                           */
    int d;               /* head dimension: 64 or 128                              */
    int64_t window;      /* keys seen up to and with the query's own; 0 = all      */
    int sinks;           /* first keys that stay visible, >= 0                     */
    float scale;         /* 0 = 1/sqrt(d); not negative                            */
    int backward;        /* 1: the plan can run syn_window_attention_backward      */
    uint64_t timeout_ns; /* bound on every device wait (0 = SYN_TIMEOUT_NS or 2 s) */
} syn_window_cfg_t;

/* A tensor [rows, heads, d]: element (t, h, j) at p + t * token + h * head + j.
 * p 16-byte aligned, strides positive multiples of 8 elements (where the
 * tensor has more than one row or head), those of outputs d or more. */
typedef struct {
    void *p;
    int64_t token, head;
} syn_window_rows_t;

/* Plan facts. */
typedef struct {
    int n_seqs, n_items, n_bwd_items, n_parts, grid;
    int64_t q_rows, k_rows;   /* sums of the lengths                              */
    int64_t pairs;            /* (query row, visible key) pairs of one head       */
    int64_t workspace_bytes;  /* device memory the plan holds                     */
} syn_window_info_t;

/* Defaults: bf16, 1 head, d 128, window 0, no sinks, no backward. */
int syn_window_cfg_default(syn_window_cfg_t *cfg);

/* Validate the lengths and build the plan's work lists on the current device.
 * The lists give each SM about the same number of key blocks; they depend on
 * the lengths alone, so a plan serves any number of calls (layers, steps)
 * with these lengths.  Making one allocates and copies with blocking calls and
 * waits for the device, all streams of it: 0.14 ms for a token, 0.3 for 16384 rows
 * of one sequence, 0.7 for 128 sequences; with backward 0.2, 0.9 and 2.3 (32/8
 * heads).  Lists of 2^28 tiles or more, or that host memory cannot hold, are
 * SYN_ERR_UNSUPPORTED. */
int syn_window_plan_create(syn_window_plan_t *out, const syn_window_cfg_t *cfg, int n_seqs, const int64_t *q_lens,
                           const int64_t *k_lens);

/* Free a plan (no call of it may still be running).  NULL is a no-op. */
int syn_window_plan_destroy(syn_window_plan_t plan);

int syn_window_plan_query(syn_window_plan_t plan, syn_window_info_t *info);

/* The forward (asynchronous on `stream`).  Q, O [q_rows, H_q, d]; K, V [k_rows,
 * H_kv, d]; lse nullable fp32 [q_rows, H_q], contiguous. */
int syn_window_attention(syn_window_plan_t plan, const syn_window_rows_t *Q, const syn_window_rows_t *K,
                         const syn_window_rows_t *V, const syn_window_rows_t *O, float *lse, void *stream);

/* The gradient (asynchronous): dQ, dK, dV from dO, the forward's inputs, its O
 * and lse.  Every row of the sequences is written.  No atomics: the same bits
 * for the same inputs on the same device.  Calls of one plan must not overlap
 * (they share its workspace). */
int syn_window_attention_backward(syn_window_plan_t plan, const syn_window_rows_t *dO, const syn_window_rows_t *Q,
                                  const syn_window_rows_t *K, const syn_window_rows_t *V, const syn_window_rows_t *O,
                                  const float *lse, const syn_window_rows_t *dQ, const syn_window_rows_t *dK,
                                  const syn_window_rows_t *dV, void *stream);

/* Synchronise `stream`, then read and clear the device error word: SYN_OK,
 * SYN_ERR_TIMEOUT or SYN_ERR_CUDA. */
int syn_window_sync_status(syn_window_plan_t plan, void *stream);

typedef struct {
    int dtype;       /* SYN_DTYPE_BF16 or SYN_DTYPE_F16                          */
    int max_seqs;    /* sequences of a call at most                              */
    int H_q, H_kv;   /* H_q % H_kv == 0, H_q <= 1024                             */
    int d;           /* head dimension: 64 or 128                                */
    int64_t window;  /* 0 = all keys                                             */
    int sinks;
    int page_size;   /* cache rows of a page, >= 1                               */
    float scale;     /* 0 = 1/sqrt(d); not negative                              */
} syn_decode_cfg_t;

/* A cache [n_pages, page_size, H_kv, d]: element (g, t, h, j) at
 * p + g * page + t * token + h * head + j; p 16-byte aligned, strides multiples
 * of 8 elements. */
typedef struct {
    const void *p;
    int64_t page, token, head;
} syn_window_cache_t;

int syn_decode_cfg_default(syn_decode_cfg_t *cfg);
int syn_decode_plan_create(syn_decode_plan_t *out, const syn_decode_cfg_t *cfg);
int syn_decode_plan_destroy(syn_decode_plan_t plan);

/* One query token per sequence (asynchronous): row s of q attends as the last
 * of seq_lens[s] cached tokens.
 *   q, O       : [n_seqs, H_q, d]
 *   page_table : int32 [n_seqs, table_stride] on the device: key j of sequence
 *                s lies in page page_table[s][j / page_size], row j % page_size;
 *                entries of pages without a visible key are not read.  NULL:
 *                sequence s is page s (a contiguous cache)
 *   n_pages    : pages of K and V; a visible key whose page is outside them, or
 *                a length beyond the table, is left out and reported as
 *                SYN_ERR_BOUNDS by syn_decode_sync_status
 *   seq_lens   : int32 [n_seqs] on the device; 0 gives O = 0, lse = -inf
 *   lse        : nullable fp32 [n_seqs, H_q]
 * Calls of one plan must not overlap (they share its workspace). */
int syn_window_decode(syn_decode_plan_t plan, const syn_window_rows_t *q, const syn_window_cache_t *k,
                      const syn_window_cache_t *v, const int32_t *page_table, int64_t table_stride, int64_t n_pages,
                      const int32_t *seq_lens, int n_seqs, const syn_window_rows_t *O, float *lse, void *stream);

/* Synchronise `stream`, then read and clear the device error word. */
int syn_decode_sync_status(syn_decode_plan_t plan, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SYN_WINDOW_H */
