// C ABI of the expert operators (include/muon_experts.h): argument checks and
// dispatch to the launchers.
#include "buffers.h"
#include "experts.h"
#include "internal.h"

using namespace muon;

namespace {

bool eight_bit(int d) { return d == MUON_ROW_E4M3 || d == MUON_ROW_E5M2; }
int64_t blocks_of(int64_t n) { return (n + 127) / 128; }

// rows * k below 2^31 (both checked to be below 2^31 before)
muon_status check_pairs(int64_t rows, int64_t k) {
  if (k < 1) return MUON_ERR_INVALID_ARG;
  return k > kMaxDim || (rows > 0 && k > kMaxDim / rows) ? MUON_ERR_UNSUPPORTED : MUON_OK;
}

// `batch` matrices [rows, cols], `matrix` elements apart: as one region of rows where they
// follow one another evenly, else as the whole range.
void stack(Buffers& b, const void* p, int64_t batch, int64_t rows, int64_t cols, int64_t stride, int64_t matrix,
           int64_t size, bool written) {
  if (rows <= 1) stride = cols;
  if (batch <= 1) matrix = 0;
  else if (stride < cols || stride > (int64_t(1) << 40) || matrix > (INT64_MAX / 8) / batch ||
           rows > (INT64_MAX / 8) / stride || matrix < (rows - 1) * stride + cols)
    return b.fail(MUON_ERR_INVALID_ARG);
  if (batch <= 1 || rows == 0) {
    b.matrix(p, batch ? rows : 0, cols, stride, size, written);
  } else if (matrix == rows * stride && rows <= INT64_MAX / 8 / batch) {
    b.matrix(p, batch * rows, cols, stride, size, written);
  } else {
    const int64_t span = (batch - 1) * matrix + (rows - 1) * stride + cols;
    b.matrix(p, 1, span, span, size, written);
  }
}

muon_status check_groups(int64_t experts, const int32_t* offsets) {
  if (experts < 1) return MUON_ERR_INVALID_ARG;
  if (experts > MUON_ROUTE_MAX_EXPERTS) return MUON_ERR_UNSUPPORTED;
  if (!offsets && experts != 1) return MUON_ERR_INVALID_ARG;
  return MUON_OK;
}

// Elements of a stack of contiguous matrices, at most 2^59 of them.
bool too_many(int64_t a, int64_t b, int64_t c) { return a > 0 && b > 0 && c > 0 && (b > (int64_t(1) << 59) / a || c > (int64_t(1) << 59) / (a * b)); }

}  // namespace

extern "C" {

int32_t muon_experts_abi_version(void) { return MUON_EXPERTS_ABI_VERSION; }

muon_status muon_expert_gather(const muon_gather_args* a, void* stream) {
  if (!a) return MUON_ERR_INVALID_ARG;
  muon_status st = check_dims(a->rows, a->cols);
  if (st != MUON_OK) return st;
  if ((st = check_pairs(a->rows, a->top_k)) != MUON_OK) return st;
  if (a->dtype < MUON_ROW_F32 || a->dtype > MUON_ROW_E5M2) return MUON_ERR_INVALID_ARG;
  if (a->scales ? a->groups < 1 || a->groups > kMaxDim : a->out_scales || a->groups != 0) return MUON_ERR_INVALID_ARG;
  if (a->rows == 0) return MUON_OK;
  const int64_t pairs = a->rows * a->top_k, es = size_of(a->dtype);
  Buffers b;
  b.matrix(a->x, a->rows, a->cols, a->x_stride, es, false);
  b.matrix(a->out, pairs, a->cols, a->out_stride, es, true);
  if (a->scales) {
    b.matrix(a->scales, a->rows, a->groups, a->scales_stride, 4, false);
    b.matrix(a->out_scales, pairs, a->groups, a->out_scales_stride, 4, true);
  }
  b.flat(a->order, pairs, 4, false);
  if ((st = b.check()) != MUON_OK) return st;
  return hip_status(run_gather(*a, hip_stream(stream)));
}

muon_status muon_expert_combine(const muon_combine_args* a, void* stream) {
  if (!a) return MUON_ERR_INVALID_ARG;
  muon_status st = check_dims(a->rows, a->cols);
  if (st != MUON_OK) return st;
  if ((st = check_dims(a->places, 1)) != MUON_OK) return st;
  if ((st = check_pairs(a->rows, a->top_k)) != MUON_OK) return st;
  if (a->top_k > MUON_ROUTE_MAX_TOP_K) return MUON_ERR_UNSUPPORTED;
  if (!valid_dtype(a->dtype) || !valid_dtype(a->out_dtype)) return MUON_ERR_INVALID_ARG;
  if (a->rows == 0) return MUON_OK;
  const int64_t pairs = a->rows * a->top_k;
  Buffers b;
  b.flat(a->position, pairs, 4, false);
  if (a->weights) b.flat(a->weights, pairs, 4, false);
  if (a->places > 0) b.matrix(a->y, a->places, a->cols, a->y_stride, size_of(a->dtype), false);
  const int ib = a->base ? b.matrix(a->base, a->rows, a->cols, a->base_stride, size_of(a->out_dtype), false) : -1;
  const int io = b.matrix(a->out, a->rows, a->cols, a->out_stride, size_of(a->out_dtype), true);
  if ((st = b.check({{ib, io}})) != MUON_OK) return st;
  return hip_status(run_combine(*a, hip_stream(stream)));
}

muon_status muon_expert_combine_backward(const muon_combine_grad_args* a, void* stream) {
  if (!a) return MUON_ERR_INVALID_ARG;
  muon_status st = check_dims(a->rows, a->cols);
  if (st != MUON_OK) return st;
  if ((st = check_dims(a->places, 1)) != MUON_OK) return st;
  if ((st = check_pairs(a->rows, a->top_k)) != MUON_OK) return st;
  if (a->top_k > MUON_ROUTE_MAX_TOP_K) return MUON_ERR_UNSUPPORTED;
  if (!valid_dtype(a->dtype) || (a->dy8 ? !eight_bit(a->dy8_dtype) : a->scales != nullptr)) return MUON_ERR_INVALID_ARG;
  if (!a->dy && !a->dy8 && !a->dweights) return MUON_ERR_INVALID_ARG;
  if (a->rows == 0) return MUON_OK;
  const int64_t pairs = a->rows * a->top_k, es = size_of(a->dtype);
  Buffers b;
  b.flat(a->position, pairs, 4, false);
  if (a->weights) b.flat(a->weights, pairs, 4, false);
  b.matrix(a->dout, a->rows, a->cols, a->dout_stride, es, false);
  if (a->places > 0) {
    if (a->dweights) b.matrix(a->y, a->places, a->cols, a->y_stride, es, false);
    if (a->dy) b.matrix(a->dy, a->places, a->cols, a->dy_stride, es, true);
    if (a->dy8) {
      b.matrix(a->dy8, a->places, a->cols, a->dy8_stride, 1, true);
      b.matrix(a->scales, a->places, blocks_of(a->cols), a->scales_stride, 4, true);
    }
  }
  if (a->dweights) b.flat(a->dweights, pairs, 4, true);
  if ((st = b.check()) != MUON_OK) return st;
  return hip_status(run_combine_backward(*a, hip_stream(stream)));
}

muon_status muon_gate_forward(const muon_gate_args* a, void* stream) {
  if (!a) return MUON_ERR_INVALID_ARG;
  muon_status st = check_dims(a->rows, a->cols);
  if (st != MUON_OK) return st;
  if (a->cols > kMaxDim / 2) return MUON_ERR_UNSUPPORTED;
  if (!valid_dtype(a->dtype) || (a->y8 ? !eight_bit(a->y8_dtype) : a->scales != nullptr)) return MUON_ERR_INVALID_ARG;
  if (!a->y && !a->y8) return MUON_ERR_INVALID_ARG;
  if (a->rows == 0) return MUON_OK;
  const int64_t es = size_of(a->dtype);
  Buffers b;
  b.matrix(a->a, a->rows, 2 * a->cols, a->a_stride, es, false);
  if (a->y) b.matrix(a->y, a->rows, a->cols, a->y_stride, es, true);
  if (a->y8) {
    b.matrix(a->y8, a->rows, a->cols, a->y8_stride, 1, true);
    b.matrix(a->scales, a->rows, blocks_of(a->cols), a->scales_stride, 4, true);
  }
  if (a->used) b.flat(a->used, 1, 4, false);
  if ((st = b.check()) != MUON_OK) return st;
  return hip_status(run_gate_forward(*a, hip_stream(stream)));
}

muon_status muon_gate_backward(const muon_gate_grad_args* a, void* stream) {
  if (!a) return MUON_ERR_INVALID_ARG;
  muon_status st = check_dims(a->rows, a->cols);
  if (st != MUON_OK) return st;
  if (a->cols > kMaxDim / 2) return MUON_ERR_UNSUPPORTED;
  if (!valid_dtype(a->dtype) || (a->da8 ? !eight_bit(a->da8_dtype) : a->scales != nullptr)) return MUON_ERR_INVALID_ARG;
  if (!a->da && !a->da8) return MUON_ERR_INVALID_ARG;
  if (a->da8 && a->cols % 128 != 0) return MUON_ERR_UNSUPPORTED;   // a group would hold both halves' columns
  if (a->rows == 0) return MUON_OK;
  const int64_t es = size_of(a->dtype);
  Buffers b;
  b.matrix(a->a, a->rows, 2 * a->cols, a->a_stride, es, false);
  b.matrix(a->dy, a->rows, a->cols, a->dy_stride, es, false);
  if (a->da) b.matrix(a->da, a->rows, 2 * a->cols, a->da_stride, es, true);
  if (a->da8) {
    b.matrix(a->da8, a->rows, 2 * a->cols, a->da8_stride, 1, true);
    b.matrix(a->scales, a->rows, 2 * a->cols / 128, a->scales_stride, 4, true);
  }
  if (a->used) b.flat(a->used, 1, 4, false);
  if ((st = b.check()) != MUON_OK) return st;
  return hip_status(run_gate_backward(*a, hip_stream(stream)));
}

muon_status muon_quantise_blocks(const muon_quantise_args* a, void* stream) {
  if (!a) return MUON_ERR_INVALID_ARG;
  muon_status st = check_dims(a->rows, a->cols);
  if (st != MUON_OK) return st;
  if ((st = check_dims(a->batch, 1)) != MUON_OK) return st;
  if (!valid_dtype(a->dtype) || !eight_bit(a->q_dtype)) return MUON_ERR_INVALID_ARG;
  if (!a->q && !a->qt) return MUON_ERR_INVALID_ARG;
  if ((!a->q && a->scales) || (!a->qt && a->scales_t)) return MUON_ERR_INVALID_ARG;
  if (too_many(a->batch, a->rows, a->cols)) return MUON_ERR_UNSUPPORTED;
  if (a->rows == 0 || a->batch == 0) return MUON_OK;
  const int64_t blocks = a->batch * blocks_of(a->rows) * blocks_of(a->cols);
  Buffers b;
  stack(b, a->x, a->batch, a->rows, a->cols, a->x_stride, a->x_matrix, size_of(a->dtype), false);
  if (a->q) {
    stack(b, a->q, a->batch, a->rows, a->cols, a->q_stride, a->q_matrix, 1, true);
    b.flat(a->scales, blocks, 4, true);
  }
  if (a->qt) {
    stack(b, a->qt, a->batch, a->cols, a->rows, a->qt_stride, a->qt_matrix, 1, true);
    b.flat(a->scales_t, blocks, 4, true);
  }
  if ((st = b.check()) != MUON_OK) return st;
  return hip_status(run_quantise(*a, hip_stream(stream)));
}

muon_status muon_expert_product(const muon_product_args* a, void* stream) {
  if (!a) return MUON_ERR_INVALID_ARG;
  muon_status st = check_dims(a->rows, a->k);
  if (st != MUON_OK) return st;
  if ((st = check_dims(0, a->n)) != MUON_OK) return st;
  if ((st = check_groups(a->num_experts, a->offsets)) != MUON_OK) return st;
  if (!eight_bit(a->a_dtype) || !eight_bit(a->w_dtype) || !valid_dtype(a->out_dtype)) return MUON_ERR_INVALID_ARG;
  if (too_many(a->num_experts, a->n, a->k)) return MUON_ERR_UNSUPPORTED;
  // tiles are numbered in 32 bits
  if ((a->rows / 128 + (a->num_experts < a->rows ? a->num_experts : a->rows)) * blocks_of(a->n) >= (int64_t(1) << 31))
    return MUON_ERR_UNSUPPORTED;
  if (a->rows == 0) return MUON_OK;
  const int64_t kb = blocks_of(a->k);
  Buffers b;
  b.matrix(a->a, a->rows, a->k, a->a_stride, 1, false);
  b.matrix(a->a_scales, a->rows, kb, a->a_scales_stride, 4, false);
  stack(b, a->w, a->num_experts, a->n, a->k, a->w_stride, a->w_matrix, 1, false);
  b.flat(a->w_scales, a->num_experts * blocks_of(a->n) * kb, 4, false);
  if (a->offsets) b.flat(a->offsets, a->num_experts + 1, 4, false);
  b.matrix(a->out, a->rows, a->n, a->out_stride, size_of(a->out_dtype), true);
  if ((st = b.check()) != MUON_OK) return st;
  return hip_status(run_product(*a, hip_stream(stream)));
}

muon_status muon_expert_weight_grad_workspace_bytes(int64_t rows, int64_t num_experts, int64_t n, int64_t k,
                                                    size_t* out) {
  if (!out) return MUON_ERR_INVALID_ARG;
  muon_status st = check_dims(rows, k);
  if (st != MUON_OK) return st;
  if ((st = check_dims(0, n)) != MUON_OK) return st;
  if (num_experts < 1) return MUON_ERR_INVALID_ARG;
  if (num_experts > MUON_ROUTE_MAX_EXPERTS) return MUON_ERR_UNSUPPORTED;
  if (too_many(num_experts, n, k)) return MUON_ERR_UNSUPPORTED;
  *out = align256(size_t(weight_grad_parts_bytes(rows, num_experts, n, k)) +
                  size_t(weight_grad_copy_bytes(rows, num_experts, n, k)));
  return MUON_OK;
}

muon_status muon_expert_weight_grad(const muon_weight_grad_args* a, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  if (!a) return MUON_ERR_INVALID_ARG;
  size_t need = 0;
  muon_status st = muon_expert_weight_grad_workspace_bytes(a->rows, a->num_experts, a->n, a->k, &need);
  if (st != MUON_OK) return st;
  if ((st = check_groups(a->num_experts, a->offsets)) != MUON_OK) return st;
  if (!valid_dtype(a->dw_dtype)) return MUON_ERR_INVALID_ARG;
  if (workspace_bytes < need) return MUON_ERR_WORKSPACE_TOO_SMALL;
  Buffers b;
  if (a->rows > 0) {
    b.matrix(a->dy, a->rows, a->n, a->dy_stride, 2, false);
    b.matrix(a->x, a->rows, a->k, a->x_stride, 2, false);
    if (a->offsets) b.flat(a->offsets, a->num_experts + 1, 4, false);
  }
  stack(b, a->dw, a->num_experts, a->n, a->k, a->dw_stride, a->dw_matrix, size_of(a->dw_dtype), true);
  if (need) b.flat(workspace, int64_t(need), 1, true, 256);
  if ((st = b.check()) != MUON_OK) return st;
  return hip_status(run_weight_grad(*a, workspace, hip_stream(stream)));
}

}  // extern "C"
