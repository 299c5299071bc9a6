/*
 * muon_block.h -- C ABI of libmuon's row operators: what a decoder block with
 * routed experts runs between the matrices that muon.h optimises, one row per
 * token, on one AMD Instinct MI355X (gfx950).
 *
 *   norm     z = r + D(x);  rstd = 1 / sqrt(mean(z^2) + eps);  y = z rstd w
 *            and its gradients; y in fp32, bf16 or 8 bits with scales;
 *   dropout  D(x), its mask recomputed from a counter and never stored;
 *   route    the experts of each row and their weights, and the gradient of
 *            the logits;
 *   order    the (row, slot) pairs grouped by expert, for the experts'
 *            products on the [E, M, N] tensors that muon_step updates, and
 *            the update of the balance bias.
 *
 * Conventions are those of muon.h.  Device memory is the caller's; nothing
 * is allocated, freed or synchronised; kernels are enqueued on `stream` (a
 * hipStream_t, NULL = the null stream) of the current device and the call
 * returns without waiting, so every call can be captured into a HIP graph.
 * Arguments are checked before anything is enqueued: on INVALID_ARG,
 * UNSUPPORTED and WORKSPACE_TOO_SMALL nothing is launched and no buffer is
 * touched.  Results are bitwise reproducible: no sum's order depends on
 * timing.  Status codes and muon_status_str are those of muon.h.
 *
 * Matrices are row-major with a row stride in elements (at least the row's
 * length; ignored for a single row).  Bases need the alignment of one
 * element only; 16-byte aligned bases and strides run fastest.  Rows and
 * columns are below 2^31 each; offsets are 64-bit.  rows = 0 is allowed and
 * writes nothing but the outputs that do not have rows (zero gradients and
 * counts).  An output must not overlap an input or another output, except
 * where a call says so; two row-strided buffers may interleave (column
 * ranges of one wider buffer).  Values are computed in fp32 and rounded to
 * nearest even once, where they are stored.
 */
#ifndef LIBMUON_MUON_BLOCK_H
#define LIBMUON_MUON_BLOCK_H

#include "muon.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MUON_BLOCK_ABI_VERSION 1
int32_t muon_block_abi_version(void);

/* Types of a norm's output: the two of muon_dtype, and the 8-bit floating
 * formats of the OCP specification (4 exponent and 3 fraction bits, largest
 * value 448, no infinity; 5 and 2, largest 57344). */
typedef enum { MUON_ROW_F32 = 0, MUON_ROW_BF16 = 1, MUON_ROW_E4M3 = 2, MUON_ROW_E5M2 = 3 } muon_row_dtype;

/* ---- dropout ---------------------------------------------------------------
 * D(x) at row r, column c is x 2^16 / (2^16 - t) where the element is kept and
 * exactly 0 (whatever x is, NaN included) where not; t = floor(2^16 p + 1/2),
 * so p is met to 2^-17 and the scale is that of the probability used.  An
 * element is kept when its 16-bit number is at least t: piece c mod 8 (low
 * half of word 0, high half of word 0, low half of word 1, ...) of
 * Philox4x32-10 with the counter (c / 8, r, offset mod 2^32, offset / 2^32)
 * and the key (seed mod 2^32, seed / 2^32) (Salmon et al., "Parallel random
 * numbers: as easy as 1, 2, 3", 2011).  The mask depends on nothing else:
 * not on the type, the strides or the launch.  The backward pass is the same
 * call on the gradient; a program gives each use of a step its own offset. */
typedef struct {
  double p;                    /* in [0, 1] */
  uint64_t seed, offset;
  const uint64_t* seed_device; /* optional device address of {seed, offset}, read when the kernels run in
                                  place of the two fields above, so that each replay of a captured graph
                                  can draw another mask.  8-byte aligned. */
} muon_dropout_spec;

/* y = D(x), [rows, cols] of `dtype`.  y may be x (same base and stride). */
muon_status muon_dropout(int64_t rows, int64_t cols, const void* x, int64_t x_stride, void* y, int64_t y_stride,
                         muon_dtype dtype, const muon_dropout_spec* spec, void* stream);

/* ---- root-mean-square norm -------------------------------------------------
 * forward: z = residual + D(x) (residual NULL: D(x); dropout NULL: x),
 * h = z rounded to `dtype` (optional: the new residual stream, which the
 * backward pass reads), rstd = 1 / sqrt(mean(z^2) + eps) (optional, fp32),
 * y = z rstd weight from the unrounded z.  h may be x or residual (same base
 * and stride).
 *
 * 8-bit y: per row, groups of `group` columns (32, 64 or 128; 0 = the whole
 * row) share a scale; scales[r * scales_stride + g] = max |y| over the group
 * times 1 / FMAX in fp32, 1 if that maximum is 0, at least 2^-126; the stored
 * value is the quotient y / scale by that scale, rounded to nearest even, at
 * most FMAX in magnitude (the fp32 quotient but for about one in a million,
 * which is an ulp off and may so be stored as the 8-bit value next to it).  A NaN
 * in y is stored as a NaN and does not enter the maximum; an infinity makes the
 * group's scale infinite and the infinite elements NaN. */
typedef struct {
  int64_t rows, cols;
  const void* x;        int64_t x_stride;
  const void* residual; int64_t residual_stride;   /* optional */
  void* h;              int64_t h_stride;          /* optional */
  void* y;              int64_t y_stride;
  const void* weight;                              /* optional [cols]; NULL = ones */
  float* scales;        int64_t scales_stride;     /* 8-bit y only (else NULL) */
  float* rstd;                                     /* optional [rows] */
  const muon_dropout_spec* dropout;                /* optional */
  int32_t dtype;                                   /* muon_dtype of x, residual and h */
  int32_t weight_dtype;                            /* muon_dtype */
  int32_t y_dtype;                                 /* muon_row_dtype */
  int32_t group;                                   /* 0, 32, 64 or 128; 0 unless y is 8-bit */
  float eps;                                       /* >= 0 */
} muon_norm_args;
muon_status muon_norm_forward(const muon_norm_args* args, void* stream);

/* backward: from dy, the stored h and rstd (and dh, the gradient that arrives
 * on the residual stream), with xh = h rstd and g = dy weight:
 *   dz = rstd (g - xh mean(g xh)) + dh
 *   dresidual = dz, dx = D(dz), dweight = sum over rows of dy xh (fp32).
 * dx and dresidual are optional and at least one output is given; dresidual
 * may be dh (same base and stride).  dweight needs a workspace of
 * muon_norm_workspace_bytes, 256-byte aligned; with rows = 0 it is zeros. */
typedef struct {
  int64_t rows, cols;
  const void* dy;       int64_t dy_stride;
  const void* h;        int64_t h_stride;
  const void* dh;       int64_t dh_stride;         /* optional */
  void* dresidual;      int64_t dresidual_stride;  /* optional */
  void* dx;             int64_t dx_stride;         /* optional */
  const float* rstd;                               /* [rows] */
  const void* weight;                              /* optional [cols]; NULL = ones */
  float* dweight;                                  /* optional [cols] */
  const muon_dropout_spec* dropout;                /* optional: the forward call's */
  int32_t dtype;                                   /* muon_dtype of dy, h, dh, dresidual and dx */
  int32_t weight_dtype;                            /* muon_dtype */
} muon_norm_grad_args;
muon_status muon_norm_backward(const muon_norm_grad_args* args, void* workspace, size_t workspace_bytes,
                               void* stream);
/* Bytes (a multiple of 256) for dweight's partial sums; a pure host computation. */
muon_status muon_norm_workspace_bytes(int64_t rows, int64_t cols, size_t* out);

/* ---- routing to experts ----------------------------------------------------
 * Each row chooses top_k of E experts by its logits.
 *   s      softmax(l) over the row's open experts, or sigmoid(l);
 *   rank   s + bias in 64 bits, or l itself where there is no bias (the same
 *          order as s); an expert whose logit is -inf or NaN is closed: its
 *          score is 0 and it is never chosen; +inf counts as the largest
 *          finite value;
 *   groups experts in `groups` equal runs; a group's value is the sum of its
 *          group_top (1 or 2) largest open s + bias; the top_groups groups of
 *          largest value stay, the others' experts are not chosen;
 *   chosen the top_k largest ranks, in descending order; ties go to the
 *          lowest index throughout.  experts[r, k] = -1 and weights[r, k] = 0
 *          where fewer than top_k experts are open, and in rows whose
 *          token_mask byte is 0;
 *   weight scale s, or with renormalise scale s / (sum of the chosen s),
 *          which holds where some s or all of them underflow: it is formed
 *          from differences of log s there.
 * The bias is finite; with a NaN or an infinity in it the chosen experts are
 * still distinct and in range, but not further specified.  Limits: E <= 1024,
 * top_k <= 32, top_k <= top_groups E / groups. */
typedef enum { MUON_SCORE_SOFTMAX = 0, MUON_SCORE_SIGMOID = 1 } muon_score;
#define MUON_ROUTE_MAX_EXPERTS 1024
#define MUON_ROUTE_MAX_TOP_K 32

typedef struct {
  int32_t score;        /* muon_score */
  int32_t top_k;
  int32_t groups;       /* 1 = no groups; divides E */
  int32_t top_groups;
  int32_t group_top;    /* 1 or 2 */
  int32_t renormalise;  /* 0 or 1 */
  float scale;          /* finite, > 0 */
} muon_route_spec;

typedef struct {
  int64_t rows, num_experts;
  const void* logits;   int64_t logits_stride;    /* [rows, E] of dtype */
  const float* bias;                              /* optional [E] */
  const uint8_t* token_mask;                      /* optional [rows], 0 = no token */
  int32_t* experts;                               /* [rows, top_k], contiguous */
  float* weights;                                 /* [rows, top_k], contiguous */
  float* scores;                                  /* optional [rows, E], contiguous: s (0 in masked rows) */
  int32_t dtype;                                  /* muon_dtype */
} muon_route_args;
muon_status muon_route_forward(const muon_route_spec* spec, const muon_route_args* args, void* stream);

/* The gradient of the logits from dweights (and dscores, where the program
 * used the scores), with the forward pass's experts and weights:
 *   a_k = w_k dw_k, less (w_k / scale) sum_j w_j dw_j with renormalise;
 *   sigmoid: dl_e = (a_e + dscores_e s_e) (1 - s_e);
 *   softmax: dl_e = a_e - s_e sum_k a_k (zero with renormalise)
 *                   + s_e (dscores_e - sum s dscores);
 * a_e = 0 for an expert that was not chosen.  A row's experts are distinct, as
 * the forward pass gives them; an entry outside [0, E) counts as none.  Closed experts and rows without
 * a chosen expert get 0.  The bias only moves the choice and has no gradient;
 * groups and group_top are not read. */
typedef struct {
  int64_t rows, num_experts;
  const void* logits;   int64_t logits_stride;
  const int32_t* experts;
  const float* weights;
  const float* dweights;                          /* [rows, top_k], contiguous */
  const float* dscores;                           /* optional [rows, E], contiguous */
  void* dlogits;        int64_t dlogits_stride;   /* [rows, E] of dtype, all of it written */
  int32_t dtype;
} muon_route_grad_args;
muon_status muon_route_backward(const muon_route_spec* spec, const muon_route_grad_args* args, void* stream);

/* The pairs p = r top_k + k of `experts` (num_pairs entries, flat) grouped by
 * expert, each group in ascending p:
 *   counts[e]    pairs of expert e;
 *   offsets[e]   sum of the counts before e, offsets[E] their total;
 *   order[i]     the pair at place i; -1 from offsets[E] on;
 *   position[p]  the place of pair p, -1 where experts[p] is -1.
 * An entry outside [0, E) counts as -1.  num_pairs < 2^31 - 2^16.  Workspace:
 * muon_route_order_workspace_bytes, 256-byte aligned. */
muon_status muon_route_order(int64_t num_pairs, int64_t num_experts, const int32_t* experts, int32_t* counts,
                             int32_t* offsets, int32_t* order, int32_t* position, void* workspace,
                             size_t workspace_bytes, void* stream);
muon_status muon_route_order_workspace_bytes(int64_t num_pairs, int64_t num_experts, size_t* out);

/* out = bias + rate sign(mean(counts) - counts), in whole numbers up to the
 * sign: the update of a balance bias, which no gradient reaches.  out may be
 * bias.  counts may be summed over calls or ranks first. */
muon_status muon_route_balance(int64_t num_experts, const int32_t* counts, const float* bias, float* out, float rate,
                               void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBMUON_MUON_BLOCK_H */
