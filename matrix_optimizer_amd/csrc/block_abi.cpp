// C ABI of the row operators (include/muon_block.h): argument checks and
// dispatch to the launchers.
#include <cmath>

#include "block.h"
#include "internal.h"

using namespace muon;

namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxPairs = (int64_t(1) << 31) - (int64_t(1) << 16);
constexpr int kMaxRegions = 12;

bool valid_dtype(int d) { return d == MUON_F32 || d == MUON_BF16; }
int64_t size_of(int d) {
  switch (d) {
    case MUON_ROW_F32: return 4;
    case MUON_ROW_BF16: return 2;
    default: return 1;
  }
}

// rows of `width` bytes, `pitch` bytes apart.
struct Rows {
  uintptr_t base;
  int64_t pitch, width, rows;
  bool written;
  bool empty() const { return rows == 0 || width == 0; }
};

// Whether any byte belongs to both.  Equal pitches are compared row by row
// (column ranges of one buffer may interleave), others by their whole range.
bool overlap(const Rows& a, const Rows& b) {
  if (a.empty() || b.empty()) return false;
  const Rows& lo = a.base <= b.base ? a : b;
  const Rows& hi = a.base <= b.base ? b : a;
  const uint64_t d = hi.base - lo.base;
  const uint64_t lo_len = uint64_t(lo.rows - 1) * lo.pitch + lo.width;
  if (d >= lo_len) return false;
  if (lo.pitch != hi.pitch || lo.rows == 1 || hi.rows == 1) return true;
  // hi's first row starts d bytes after lo's: q rows down and r bytes along
  const uint64_t q = d / lo.pitch, r = d % lo.pitch;
  if (r < uint64_t(lo.width)) return true;                       // into lo's row q, which exists (d < lo_len)
  return q + 1 < uint64_t(lo.rows) && r + hi.width > uint64_t(lo.pitch);   // past the pitch, into lo's row q + 1
}

// A call's buffers, gathered and then compared pairwise.
struct Buffers {
  Rows r[kMaxRegions];
  int n = 0;
  muon_status st = MUON_OK;

  void fail(muon_status s) {
    if (st == MUON_OK) st = s;
  }
  // [rows, cols] elements of `size` bytes aligned to `align`, `stride`
  // elements apart; returns the index.
  int matrix(const void* p, int64_t rows, int64_t cols, int64_t stride, int64_t size, bool written, int64_t align = 0) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    if (rows <= 1) stride = cols;
    if (!p || b % uintptr_t(align ? align : size)) fail(MUON_ERR_INVALID_ARG);
    if (stride < cols || stride > (int64_t(1) << 40)) fail(MUON_ERR_INVALID_ARG);
    else if (rows > 0 && stride > (INT64_MAX / 8) / rows) fail(MUON_ERR_INVALID_ARG);
    r[n] = Rows{b, stride * size, cols * size, rows, written};
    return n++;
  }
  int flat(const void* p, int64_t count, int64_t size, bool written, int64_t align = 0) {
    return matrix(p, 1, count, count, size, written, align);
  }
  // i may be j itself: the same base and pitch.
  bool same(int i, int j) const {
    return r[i].base == r[j].base && (r[i].pitch == r[j].pitch || r[i].rows <= 1) && r[i].width == r[j].width;
  }
  // Every output apart from everything else, the listed pairs excepted where they are the same.
  muon_status check(std::initializer_list<std::pair<int, int>> may_alias = {}) {
    if (st != MUON_OK) return st;
    for (int i = 0; i < n; ++i)
      for (int j = i + 1; j < n; ++j) {
        if (!r[i].written && !r[j].written) continue;
        bool allowed = false;
        for (const auto& p : may_alias)
          if (((p.first == i && p.second == j) || (p.first == j && p.second == i)) && same(i, j)) allowed = true;
        if (!allowed && overlap(r[i], r[j])) return MUON_ERR_INVALID_ARG;
      }
    return MUON_OK;
  }
};

muon_status check_dims(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1) return MUON_ERR_INVALID_ARG;
  if (rows > kMaxDim || cols > kMaxDim) return MUON_ERR_UNSUPPORTED;
  return MUON_OK;
}

muon_status take_drop(const muon_dropout_spec* s, Drop& d) {
  if (!s) return MUON_OK;
  if (!(s->p >= 0.0 && s->p <= 1.0)) return MUON_ERR_INVALID_ARG;   // NaN too
  if (reinterpret_cast<uintptr_t>(s->seed_device) & 7u) return MUON_ERR_INVALID_ARG;
  d.t = uint32_t(std::floor(s->p * 65536.0 + 0.5));
  d.on = d.t > 0;
  d.up = d.t < 65536u ? float(65536.0 / (65536.0 - d.t)) : 0.f;
  d.seed = s->seed;
  d.offset = s->offset;
  d.dev = s->seed_device;
  return MUON_OK;
}

muon_status hip_status(hipError_t e) { return e == hipSuccess ? MUON_OK : MUON_ERR_HIP; }
hipStream_t hip_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
size_t order_bytes(int64_t pairs, int64_t experts) {
  return align256(size_t(order_tiles(pairs)) * size_t((experts + 4) & ~int64_t(3)) * 4);
}

muon_status check_route(const muon_route_spec* s, int64_t rows, int64_t experts, int dtype) {
  if (!s) return MUON_ERR_INVALID_ARG;
  muon_status st = check_dims(rows, experts);
  if (st != MUON_OK) return st;
  if (!valid_dtype(dtype)) return MUON_ERR_INVALID_ARG;
  if (s->score != MUON_SCORE_SOFTMAX && s->score != MUON_SCORE_SIGMOID) return MUON_ERR_INVALID_ARG;
  if (s->renormalise != 0 && s->renormalise != 1) return MUON_ERR_INVALID_ARG;
  if (!std::isfinite(s->scale) || !(s->scale > 0.f)) return MUON_ERR_INVALID_ARG;
  if (s->top_k < 1 || s->top_k > experts) return MUON_ERR_INVALID_ARG;
  if (experts > MUON_ROUTE_MAX_EXPERTS || s->top_k > MUON_ROUTE_MAX_TOP_K) return MUON_ERR_UNSUPPORTED;
  return MUON_OK;
}

}  // namespace

extern "C" {

int32_t muon_block_abi_version(void) { return MUON_BLOCK_ABI_VERSION; }

muon_status muon_dropout(int64_t rows, int64_t cols, const void* x, int64_t x_stride, void* y, int64_t y_stride,
                         muon_dtype dtype, const muon_dropout_spec* spec, void* stream) {
  muon_status st = check_dims(rows, cols);
  if (st != MUON_OK) return st;
  if (!valid_dtype(dtype) || !spec) return MUON_ERR_INVALID_ARG;
  Drop d;
  if ((st = take_drop(spec, d)) != MUON_OK) return st;
  if (rows == 0) return MUON_OK;
  Buffers b;
  const int ix = b.matrix(x, rows, cols, x_stride, size_of(dtype), false);
  const int iy = b.matrix(y, rows, cols, y_stride, size_of(dtype), true);
  if (d.dev) b.flat(d.dev, 2, 8, false);
  if ((st = b.check({{ix, iy}})) != MUON_OK) return st;
  return hip_status(run_dropout(rows, cols, x, x_stride, y, y_stride, dtype, d, hip_stream(stream)));
}

muon_status muon_norm_forward(const muon_norm_args* a, void* stream) {
  if (!a) return MUON_ERR_INVALID_ARG;
  muon_status st = check_dims(a->rows, a->cols);
  if (st != MUON_OK) return st;
  if (!valid_dtype(a->dtype) || !(a->eps >= 0.f) || !std::isfinite(a->eps)) return MUON_ERR_INVALID_ARG;
  if (a->weight && !valid_dtype(a->weight_dtype)) return MUON_ERR_INVALID_ARG;
  if (a->y_dtype < MUON_ROW_F32 || a->y_dtype > MUON_ROW_E5M2) return MUON_ERR_INVALID_ARG;
  const bool eight = a->y_dtype >= MUON_ROW_E4M3;
  if (eight ? a->group != 0 && a->group != 32 && a->group != 64 && a->group != 128 : a->group != 0)
    return MUON_ERR_INVALID_ARG;
  if (!eight && a->scales) return MUON_ERR_INVALID_ARG;
  Drop d;
  if ((st = take_drop(a->dropout, d)) != MUON_OK) return st;
  if (a->rows == 0) return MUON_OK;
  const int64_t es = size_of(a->dtype), groups = a->group ? (a->cols + a->group - 1) / a->group : 1;
  Buffers b;
  const int ix = b.matrix(a->x, a->rows, a->cols, a->x_stride, es, false);
  b.matrix(a->y, a->rows, a->cols, a->y_stride, size_of(a->y_dtype), true);
  const int ir = a->residual ? b.matrix(a->residual, a->rows, a->cols, a->residual_stride, es, false) : -1;
  const int ih = a->h ? b.matrix(a->h, a->rows, a->cols, a->h_stride, es, true) : -1;
  if (a->weight) b.flat(a->weight, a->cols, size_of(a->weight_dtype), false);
  if (eight) b.matrix(a->scales, a->rows, groups, a->scales_stride, 4, true);
  if (a->rstd) b.flat(a->rstd, a->rows, 4, true);
  if (d.dev) b.flat(d.dev, 2, 8, false);
  if ((st = b.check({{ix, ih}, {ir, ih}})) != MUON_OK) return st;
  return hip_status(run_norm_forward(*a, d, hip_stream(stream)));
}

muon_status muon_norm_workspace_bytes(int64_t rows, int64_t cols, size_t* out) {
  if (!out) return MUON_ERR_INVALID_ARG;
  const muon_status st = check_dims(rows, cols);
  if (st != MUON_OK) return st;
  *out = align256(size_t(norm_parts(rows, cols)) * size_t(cols) * 4);
  return MUON_OK;
}

muon_status muon_norm_backward(const muon_norm_grad_args* a, void* workspace, size_t workspace_bytes, void* stream) {
  if (!a) return MUON_ERR_INVALID_ARG;
  muon_status st = check_dims(a->rows, a->cols);
  if (st != MUON_OK) return st;
  if (!valid_dtype(a->dtype)) return MUON_ERR_INVALID_ARG;
  if (a->weight && !valid_dtype(a->weight_dtype)) return MUON_ERR_INVALID_ARG;
  if (!a->dresidual && !a->dx && !a->dweight) return MUON_ERR_INVALID_ARG;
  Drop d;
  if ((st = take_drop(a->dropout, d)) != MUON_OK) return st;
  Buffers b;
  if (a->dweight) b.flat(a->dweight, a->cols, 4, true);
  if (a->rows > 0) {
    const int64_t es = size_of(a->dtype);
    b.matrix(a->dy, a->rows, a->cols, a->dy_stride, es, false);
    b.matrix(a->h, a->rows, a->cols, a->h_stride, es, false);
    b.flat(a->rstd, a->rows, 4, false);
    if (a->weight) b.flat(a->weight, a->cols, size_of(a->weight_dtype), false);
    const int id = a->dh ? b.matrix(a->dh, a->rows, a->cols, a->dh_stride, es, false) : -1;
    const int ir = a->dresidual ? b.matrix(a->dresidual, a->rows, a->cols, a->dresidual_stride, es, true) : -1;
    if (a->dx) b.matrix(a->dx, a->rows, a->cols, a->dx_stride, es, true);
    if (d.dev) b.flat(d.dev, 2, 8, false);
    if (a->dweight) {
      size_t need = 0;
      if ((st = muon_norm_workspace_bytes(a->rows, a->cols, &need)) != MUON_OK) return st;
      if (workspace_bytes < need) return MUON_ERR_WORKSPACE_TOO_SMALL;
      b.flat(workspace, int64_t(need), 1, true, 256);
    }
    st = b.check({{id, ir}});
  } else {
    st = b.check();
  }
  if (st != MUON_OK) return st;
  if (a->rows == 0 && !a->dweight) return MUON_OK;
  return hip_status(run_norm_backward(*a, d, static_cast<float*>(workspace), hip_stream(stream)));
}

muon_status muon_route_forward(const muon_route_spec* s, const muon_route_args* a, void* stream) {
  if (!a) return MUON_ERR_INVALID_ARG;
  muon_status st = check_route(s, a->rows, a->num_experts, a->dtype);
  if (st != MUON_OK) return st;
  const int64_t E = a->num_experts;
  if (s->groups < 1 || E % s->groups || s->top_groups < 1 || s->top_groups > s->groups) return MUON_ERR_INVALID_ARG;
  if (s->group_top != 1 && s->group_top != 2) return MUON_ERR_INVALID_ARG;
  if (s->top_k > s->top_groups * (E / s->groups)) return MUON_ERR_INVALID_ARG;
  if (a->rows == 0) return MUON_OK;
  Buffers b;
  b.matrix(a->logits, a->rows, E, a->logits_stride, size_of(a->dtype), false);
  if (a->bias) b.flat(a->bias, E, 4, false);
  if (a->token_mask) b.flat(a->token_mask, a->rows, 1, false);
  b.flat(a->experts, a->rows * s->top_k, 4, true);
  b.flat(a->weights, a->rows * s->top_k, 4, true);
  if (a->scores) b.flat(a->scores, a->rows * E, 4, true);
  if ((st = b.check()) != MUON_OK) return st;
  return hip_status(run_route_forward(*s, *a, hip_stream(stream)));
}

muon_status muon_route_backward(const muon_route_spec* s, const muon_route_grad_args* a, void* stream) {
  if (!a) return MUON_ERR_INVALID_ARG;
  muon_status st = check_route(s, a->rows, a->num_experts, a->dtype);
  if (st != MUON_OK) return st;
  if (a->rows == 0) return MUON_OK;
  const int64_t E = a->num_experts;
  Buffers b;
  b.matrix(a->logits, a->rows, E, a->logits_stride, size_of(a->dtype), false);
  b.flat(a->experts, a->rows * s->top_k, 4, false);
  b.flat(a->weights, a->rows * s->top_k, 4, false);
  b.flat(a->dweights, a->rows * s->top_k, 4, false);
  if (a->dscores) b.flat(a->dscores, a->rows * E, 4, false);
  b.matrix(a->dlogits, a->rows, E, a->dlogits_stride, size_of(a->dtype), true);
  if ((st = b.check()) != MUON_OK) return st;
  return hip_status(run_route_backward(*s, *a, hip_stream(stream)));
}

muon_status muon_route_order_workspace_bytes(int64_t num_pairs, int64_t num_experts, size_t* out) {
  if (!out || num_pairs < 0 || num_experts < 1) return MUON_ERR_INVALID_ARG;
  if (num_pairs >= kMaxPairs || num_experts > MUON_ROUTE_MAX_EXPERTS) return MUON_ERR_UNSUPPORTED;
  *out = order_bytes(num_pairs, num_experts);
  return MUON_OK;
}

muon_status muon_route_order(int64_t num_pairs, int64_t num_experts, const int32_t* experts, int32_t* counts,
                             int32_t* offsets, int32_t* order, int32_t* position, void* workspace,
                             size_t workspace_bytes, void* stream) {
  size_t need = 0;
  muon_status st = muon_route_order_workspace_bytes(num_pairs, num_experts, &need);
  if (st != MUON_OK) return st;
  if (workspace_bytes < need) return MUON_ERR_WORKSPACE_TOO_SMALL;
  Buffers b;
  b.flat(counts, num_experts, 4, true);
  b.flat(offsets, num_experts + 1, 4, true);
  if (num_pairs > 0) {
    b.flat(workspace, int64_t(need), 1, true, 256);
    b.flat(experts, num_pairs, 4, false);
    b.flat(order, num_pairs, 4, true);
    b.flat(position, num_pairs, 4, true);
  }
  if ((st = b.check()) != MUON_OK) return st;
  return hip_status(run_route_order(num_pairs, num_experts, experts, counts, offsets, order, position,
                                    static_cast<int32_t*>(workspace), hip_stream(stream)));
}

muon_status muon_route_balance(int64_t num_experts, const int32_t* counts, const float* bias, float* out, float rate,
                               void* stream) {
  if (num_experts < 1 || !std::isfinite(rate)) return MUON_ERR_INVALID_ARG;
  if (num_experts > MUON_ROUTE_MAX_EXPERTS) return MUON_ERR_UNSUPPORTED;
  Buffers b;
  b.flat(counts, num_experts, 4, false);
  const int ib = b.flat(bias, num_experts, 4, false);
  const int io = b.flat(out, num_experts, 4, true);
  const muon_status st = b.check({{ib, io}});
  if (st != MUON_OK) return st;
  return hip_status(run_route_balance(num_experts, counts, bias, out, rate, hip_stream(stream)));
}

}  // extern "C"
