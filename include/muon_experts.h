/*
 * muon_experts.h -- C ABI of libmuon's expert operators: what the routed
 * (row, slot) pairs of a decoder block go through between muon_route_order
 * and the residual stream, on the [E, N, K] tensors that muon_step updates,
 * on one AMD Instinct MI355X (gfx950).
 *
 *   gather    rows copied to their pairs' places in the experts' order;
 *   product   each expert's rows times its matrix, both in 8 bits with a
 *             scale for each block of 128; with the transposed matrices the
 *             gradient of the rows;
 *   gate      the gated activation between two products, and its gradient;
 *   combine   the pairs' results back to their rows with the routing
 *             weights, and the gradient of rows and weights (without weights
 *             the gradient of gather);
 *   quantise  matrices in 8 bits by blocks of 128 x 128, also transposed;
 *   weight gradient  the experts' matrices' gradient, for muon_step.
 *
 * Conventions are those of muon_block.h: the caller's device memory, no
 * allocation and no synchronisation, kernels enqueued on `stream` of the
 * current device (every call can be captured into a HIP graph), arguments
 * checked before anything is launched, row-major matrices with a row stride
 * in elements, bases aligned to one element (16-byte aligned bases and
 * strides run fastest), no output overlapping an input or another output but
 * where a call says so, bitwise reproducible results, values computed in
 * fp32 and rounded to nearest even once, where they are stored.  Rows,
 * columns, pairs and experts are at least 0 (columns and experts 1) and
 * below 2^31.
 *
 * Places: the pairs' order has a place for each pair that has an expert, the
 * experts' runs one after another as `offsets` [E + 1] of muon_route_order
 * gives them on the device.  Rows of a buffer in that order that no pair owns
 * (from offsets[E] on) are neither read nor written.  The kernels take
 * offsets within [0, rows] and treat a run that ends before it begins as
 * empty; runs that overlap leave the rows they share with either result.
 *
 * 8-bit values: groups of 128 columns of a row (rows) or blocks of 128 x 128
 * (matrices), the last ones shorter, share an fp32 scale:
 * scale = max |v| / FMAX as an fp32 quotient, 1 if that maximum is 0, at
 * least 2^-126; the stored value is the quotient v / scale, rounded to nearest
 * even.  The quotient is the fp32 one but for about one in a million, which is
 * an ulp off and may so be stored as the 8-bit value next to it.  A NaN is
 * stored as a NaN and does not enter the maximum; an infinity makes the scale
 * infinite, its finite values 0 and its infinite ones NaN.  muon_norm_forward with group = 128 writes rows of this layout.
 */
#ifndef LIBMUON_MUON_EXPERTS_H
#define LIBMUON_MUON_EXPERTS_H

#include "muon_block.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MUON_EXPERTS_ABI_VERSION 1
int32_t muon_experts_abi_version(void);

/* out[i] = x[order[i] / top_k] for the rows * top_k places i; places whose
 * order is outside [0, rows * top_k) (-1: no pair) are left as they are.
 * With scales (8-bit rows): out_scales[i] = scales[order[i] / top_k], `groups`
 * floats a row.  rows * top_k < 2^31. */
typedef struct {
  int64_t rows, cols, top_k;
  const void* x;        int64_t x_stride;
  void* out;            int64_t out_stride;          /* [rows * top_k, cols] */
  const float* scales;  int64_t scales_stride;       /* optional [rows, groups] */
  float* out_scales;    int64_t out_scales_stride;   /* with scales: [rows * top_k, groups] */
  int64_t groups;                                    /* columns of scales; 0 without */
  const int32_t* order;                              /* [rows * top_k] */
  int32_t dtype;                                     /* muon_row_dtype of x and out */
} muon_gather_args;
muon_status muon_expert_gather(const muon_gather_args* args, void* stream);

/* out[t] = base[t] + sum over k of weights[t, k] y[position[t, k]], added in
 * the order of the slots; a position outside [0, places) (-1: the slot has no
 * expert) adds nothing.  Without base from 0, without weights with ones: the
 * gradient of gather.  out may be base (same base and stride).  top_k <= 32. */
typedef struct {
  int64_t rows, cols, top_k, places;
  const int32_t* position;                           /* [rows, top_k], contiguous */
  const float* weights;                              /* optional [rows, top_k], contiguous */
  const void* y;        int64_t y_stride;            /* [places, cols] of dtype */
  const void* base;     int64_t base_stride;         /* optional [rows, cols] of out_dtype */
  void* out;            int64_t out_stride;          /* [rows, cols] of out_dtype */
  int32_t dtype;                                     /* muon_dtype */
  int32_t out_dtype;                                 /* muon_dtype */
} muon_combine_args;
muon_status muon_expert_combine(const muon_combine_args* args, void* stream);

/* The gradients of combine from dout, for each slot with a place i:
 *   dy[i] = weights[t, k] dout[t] (optional, of dtype, and optional in 8 bits
 *   with scales [places, ceil(cols / 128)]);
 *   dweights[t, k] = sum over columns of dout[t] y[i] (optional, needs y),
 * and dweights = 0 for a slot without one.  Places that no slot names are
 * left as they are.  The places are distinct, as muon_route_order gives them;
 * a place named twice holds either slot's value in each column (its 8-bit
 * values and their scale need not be of the same slot).  The gradient of base
 * is dout. */
typedef struct {
  int64_t rows, cols, top_k, places;
  const int32_t* position;                           /* [rows, top_k], contiguous */
  const float* weights;                              /* optional; NULL = ones */
  const void* dout;     int64_t dout_stride;         /* [rows, cols] of dtype */
  const void* y;        int64_t y_stride;            /* [places, cols] of dtype, with dweights */
  void* dy;             int64_t dy_stride;           /* optional [places, cols] of dtype */
  void* dy8;            int64_t dy8_stride;          /* optional [places, cols] of dy8_dtype */
  float* scales;        int64_t scales_stride;       /* with dy8 */
  float* dweights;                                   /* optional [rows, top_k], contiguous */
  int32_t dtype;                                     /* muon_dtype */
  int32_t dy8_dtype;                                 /* MUON_ROW_E4M3 or MUON_ROW_E5M2, with dy8 */
} muon_combine_grad_args;
muon_status muon_expert_combine_backward(const muon_combine_grad_args* args, void* stream);

/* Gated activation of a = [g | u], [rows, 2 cols]: y = g sigmoid(g) u, stored
 * in dtype (y) and in 8 bits with scales (y8); either or both.  sigmoid(g) is an
 * fp32 value: below g = -87 it is subnormal, with fewer digits.  `used`: an
 * optional device address of the number of rows that are in use (offsets + E);
 * rows from there on are neither read nor written. */
typedef struct {
  int64_t rows, cols;                                /* cols of y */
  const void* a;        int64_t a_stride;            /* [rows, 2 cols] of dtype */
  void* y;              int64_t y_stride;            /* optional [rows, cols] of dtype */
  void* y8;             int64_t y8_stride;           /* optional [rows, cols] of y8_dtype */
  float* scales;        int64_t scales_stride;       /* with y8: [rows, ceil(cols / 128)] */
  const int32_t* used;                               /* optional */
  int32_t dtype;                                     /* muon_dtype */
  int32_t y8_dtype;                                  /* MUON_ROW_E4M3 or MUON_ROW_E5M2, with y8 */
} muon_gate_args;
muon_status muon_gate_forward(const muon_gate_args* args, void* stream);

/* da = [dg | du] from dy, with s = sigmoid(g):
 *   dg = dy u s (1 + g (1 - s)),  du = dy g s,
 * stored in dtype (da) and in 8 bits (da8, scales [rows, 2 cols / 128]: cols a
 * multiple of 128); either or both. */
typedef struct {
  int64_t rows, cols;                                /* cols of dy */
  const void* a;        int64_t a_stride;            /* [rows, 2 cols] of dtype */
  const void* dy;       int64_t dy_stride;           /* [rows, cols] of dtype */
  void* da;             int64_t da_stride;           /* optional [rows, 2 cols] of dtype */
  void* da8;            int64_t da8_stride;          /* optional [rows, 2 cols] of da8_dtype */
  float* scales;        int64_t scales_stride;       /* with da8 */
  const int32_t* used;                               /* optional */
  int32_t dtype;                                     /* muon_dtype */
  int32_t da8_dtype;                                 /* MUON_ROW_E4M3 or MUON_ROW_E5M2, with da8 */
} muon_gate_grad_args;
muon_status muon_gate_backward(const muon_gate_grad_args* args, void* stream);

/* `batch` matrices x [rows, cols] in 8 bits by blocks of 128 x 128: q with
 * scales [batch, ceil(rows / 128), ceil(cols / 128)], and / or transposed, qt
 * [batch, cols, rows] with scales_t [batch, ceil(cols / 128),
 * ceil(rows / 128)].  Matrices are `_matrix` elements apart (ignored for one
 * matrix), at least (rows - 1) * stride + columns of inputs and outputs alike:
 * they neither repeat nor interleave.  Scales are contiguous. */
typedef struct {
  int64_t batch, rows, cols;
  const void* x;        int64_t x_stride, x_matrix;
  void* q;              int64_t q_stride, q_matrix;     /* optional */
  float* scales;                                        /* with q */
  void* qt;             int64_t qt_stride, qt_matrix;   /* optional */
  float* scales_t;                                      /* with qt */
  int32_t dtype;                                        /* muon_dtype of x */
  int32_t q_dtype;                                      /* MUON_ROW_E4M3 or MUON_ROW_E5M2 */
} muon_quantise_args;
muon_status muon_quantise_blocks(const muon_quantise_args* args, void* stream);

/* For each place i of expert e, offsets[e] <= i < offsets[e + 1]:
 *   out[i, n] = sum over blocks b of 128 columns of
 *               (a_scales[i, b] w_scales[e, n / 128, b]) sum over k in b of a[i, k] w[e, n, k].
 * The sum over a block is formed by the matrix instructions, the product of
 * the two scales and the sum over blocks in fp32 in a fixed order (a product
 * of scales outside fp32's normal range loses its digits).  With fp32 out the
 * sums over a block are fp32 sums of exact products; with bf16 out the 8-bit
 * instructions form them, which cut each of eight neighbouring products at
 * 2^-13 of the largest one's power of two: at most 7 2^-13 of the sum of the
 * products' magnitudes, 4.4e-5 of a sum of random values in the root mean
 * square, where the store rounds by up to 2^-8.  offsets NULL: one expert, all
 * rows.  w's matrices are apart as in muon_quantise_blocks.
 * num_experts <= MUON_ROUTE_MAX_EXPERTS, and fewer than 2^31 pieces of out of
 * 128 x 128 in the runs. */
typedef struct {
  int64_t rows, n, k, num_experts;
  const void* a;        int64_t a_stride;               /* [rows, k] of a_dtype */
  const float* a_scales; int64_t a_scales_stride;       /* [rows, ceil(k / 128)] */
  const void* w;        int64_t w_stride, w_matrix;     /* [num_experts, n, k] of w_dtype */
  const float* w_scales;                                /* [num_experts, ceil(n / 128), ceil(k / 128)], contiguous */
  const int32_t* offsets;                               /* [num_experts + 1] on the device */
  void* out;            int64_t out_stride;             /* [rows, n] of out_dtype */
  int32_t a_dtype, w_dtype;                             /* MUON_ROW_E4M3 or MUON_ROW_E5M2 */
  int32_t out_dtype;                                    /* muon_dtype */
} muon_product_args;
muon_status muon_expert_product(const muon_product_args* args, void* stream);

/* dw[e, n, k] = sum over the places i of expert e of dy[i, n] x[i, k], bf16
 * products summed in fp32; zeros for an expert without rows.  offsets NULL:
 * one expert, all rows.  rows = 0 writes zeros.  num_experts <=
 * MUON_ROUTE_MAX_EXPERTS.  dw's matrices are apart as in muon_quantise_blocks.
 * The workspace (256-byte aligned) is that of
 * muon_expert_weight_grad_workspace_bytes, 0 bytes where the rows are neither
 * split nor of odd widths; it serves one call at a time.  Its size goes by
 * widths alone, so n and k that are multiples of 8 have no room for copies: rows
 * of such widths at bases or strides off 16 bytes take the kernel of odd widths,
 * which takes 2 to 2.7 times as long where there is much work. */
typedef struct {
  int64_t rows, n, k, num_experts;
  const void* dy;       int64_t dy_stride;              /* [rows, n] bf16 */
  const void* x;        int64_t x_stride;               /* [rows, k] bf16 */
  const int32_t* offsets;                               /* [num_experts + 1] on the device */
  void* dw;             int64_t dw_stride, dw_matrix;   /* [num_experts, n, k] of dw_dtype */
  int32_t dw_dtype;                                     /* muon_dtype */
} muon_weight_grad_args;
muon_status muon_expert_weight_grad(const muon_weight_grad_args* args, void* workspace, size_t workspace_bytes,
                                    void* stream);
/* Bytes (a multiple of 256); a pure host computation. */
muon_status muon_expert_weight_grad_workspace_bytes(int64_t rows, int64_t num_experts, int64_t n, int64_t k,
                                                    size_t* out);

#ifdef __cplusplus
}
#endif

#endif /* LIBMUON_MUON_EXPERTS_H */
