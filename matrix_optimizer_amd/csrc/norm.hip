// Root-mean-square norm with the residual's addition, and dropout.
//
//   z = r + D(x);  rstd = 1 / sqrt(mean(z^2) + eps);  y = z rstd w
//   dz = rstd (g - xh mean(g xh)) + dh,  g = dy w,  xh = h rstd;  dw = sum dy xh
//
// All of it is bound by memory: a few operations per element.
#include <algorithm>

#include "internal.h"
#include "rows.h"

namespace muon {
namespace {

constexpr int NT = 256;            // threads of a workgroup
constexpr int NW = NT / WAVE;
constexpr int64_t kMaxGrid = 1 << 16;

// D(x) alone: eight columns a lane.  `per_row` = chunks of eight in a row.
template <typename T>
__global__ __launch_bounds__(NT) void dropout_k(int64_t rows, int64_t cols, const T* x, int64_t xs, T* y, int64_t ys,
                                                Drop d) {
  uint64_t seed, offset;
  drop_seed(d, seed, offset);
  const int64_t per_row = (cols + 7) / 8, total = rows * per_row;
  for (int64_t i = blockIdx.x * (int64_t)NT + threadIdx.x; i < total; i += (int64_t)gridDim.x * NT) {
    const int64_t r = i / per_row, c = (i - r * per_row) * 8;
    float f[8];
    load8(x + r * xs, c, cols, f);
    if (d.on) drop8(d, seed, offset, r, c, f);
    store8(y + r * ys, c, cols, f);
  }
}

// Columns c .. c+7 of weight (ones without one).
__device__ __forceinline__ void weight8(const void* w, int dtype, int64_t c, int64_t cols, float* f) {
  if (!w) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 1.f;
  } else if (dtype == MUON_BF16) {
    load8(static_cast<const bf16_t*>(w), c, cols, f);
  } else {
    load8(static_cast<const float*>(w), c, cols, f);
  }
}

// z of columns c .. c+7 (zeros from `cols` on).
template <typename T>
__device__ __forceinline__ void z8(const muon_norm_args& a, const Drop& d, uint64_t seed, uint64_t offset, int64_t r,
                                   int64_t c, float* z) {
  load8(static_cast<const T*>(a.x) + r * a.x_stride, c, a.cols, z);
  if (d.on) drop8(d, seed, offset, r, c, z);
  if (a.residual) {
    float e[8];
    load8(static_cast<const T*>(a.residual) + r * a.residual_stride, c, a.cols, e);
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] += e[j];
  }
}

// Scale of a group whose largest magnitude is `most`.
__device__ __forceinline__ float scale_of(float most, float top) {
  return most == 0.f ? 1.f : fmaxf(most / top, 0x1p-126f);
}

// y of columns c .. c+7 at its type; an 8-bit y with the group's scale, found
// across the group's lanes unless the row's is given.
__device__ __forceinline__ void store_y(const muon_norm_args& a, int64_t r, int64_t c, float* y, float row_scale) {
  if (a.y_dtype == MUON_ROW_F32) {
    if (c < a.cols) store8(static_cast<float*>(a.y) + r * a.y_stride, c, a.cols, y);
  } else if (a.y_dtype == MUON_ROW_BF16) {
    if (c < a.cols) store8(static_cast<bf16_t*>(a.y) + r * a.y_stride, c, a.cols, y);
  } else {
    const bool e5 = a.y_dtype == MUON_ROW_E5M2;
    float scale = row_scale;
    if (a.group) {   // 4, 8 or 16 lanes hold a group
      float most = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(y[j]));
      for (int o = a.group / 16; o >= 1; o >>= 1) most = fmaxf(most, __shfl_xor(most, o, WAVE));
      scale = scale_of(most, e5 ? 57344.f : 448.f);
      if (c < a.cols && (c & (a.group - 1)) == 0) a.scales[r * a.scales_stride + c / a.group] = scale;
    }
    const float inv = 1.f / scale;
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] *= inv;
    uint8_t* row = static_cast<uint8_t*>(a.y) + r * a.y_stride;
    if (c < a.cols) {
      if (e5) store8_8bit<true>(row, c, a.cols, y);
      else store8_8bit<false>(row, c, a.cols, y);
    }
  }
}

// One workgroup a row, z formed again in each pass over it.
template <typename T>
__global__ __launch_bounds__(NT) void norm_fwd(muon_norm_args a, Drop d) {
  __shared__ float lds[NW];
  uint64_t seed, offset;
  drop_seed(d, seed, offset);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    float z[8], w[8];
    float ss = 0.f;
    for (int64_t c0 = 0; c0 < a.cols; c0 += NT * 8) {
      const int64_t c = c0 + threadIdx.x * 8;
      if (c >= a.cols) continue;
      z8<T>(a, d, seed, offset, r, c, z);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += z[j] * z[j];
    }
    ss = group_sum<NW>(ss, lds);
    const float rstd = 1.f / sqrtf(ss / (float)a.cols + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[r] = rstd;
    float row_scale = 1.f;
    if (a.y_dtype >= MUON_ROW_E4M3 && a.group == 0) {
      float most = 0.f;
      for (int64_t c0 = 0; c0 < a.cols; c0 += NT * 8) {
        const int64_t c = c0 + threadIdx.x * 8;
        if (c >= a.cols) continue;
        z8<T>(a, d, seed, offset, r, c, z);
        weight8(a.weight, a.weight_dtype, c, a.cols, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) most = fmaxf(most, c + j < a.cols ? fabsf(z[j] * rstd * w[j]) : 0.f);
      }
      most = group_max<NW>(most, lds);
      row_scale = scale_of(most, a.y_dtype == MUON_ROW_E5M2 ? 57344.f : 448.f);
      if (threadIdx.x == 0) a.scales[r * a.scales_stride] = row_scale;
    }
    for (int64_t c0 = 0; c0 < a.cols; c0 += NT * 8) {
      const int64_t c = c0 + threadIdx.x * 8;   // lanes past the row's end take part in their group's maximum
      float y[8];
      const bool in = c < a.cols;
      if (in) {
        z8<T>(a, d, seed, offset, r, c, z);
        if (a.h) store8(static_cast<T*>(a.h) + r * a.h_stride, c, a.cols, z);
        weight8(a.weight, a.weight_dtype, c, a.cols, w);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = in && c + j < a.cols ? z[j] * rstd * w[j] : 0.f;
      store_y(a, r, c, y, row_scale);
    }
  }
}

template <typename T>
__global__ __launch_bounds__(NT) void norm_bwd(muon_norm_grad_args a, Drop d) {
  __shared__ float lds[NW];
  uint64_t seed, offset;
  drop_seed(d, seed, offset);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* dy_r = static_cast<const T*>(a.dy) + r * a.dy_stride;
    const T* h_r = static_cast<const T*>(a.h) + r * a.h_stride;
    const float rstd = a.rstd[r];
    float g[8], h[8], w[8];
    float dot = 0.f;
    for (int64_t c = threadIdx.x * 8; c < a.cols; c += NT * 8) {
      load8(dy_r, c, a.cols, g);
      load8(h_r, c, a.cols, h);
      weight8(a.weight, a.weight_dtype, c, a.cols, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) dot += g[j] * w[j] * (h[j] * rstd);
    }
    const float mean = group_sum<NW>(dot, lds) / (float)a.cols;
    for (int64_t c = threadIdx.x * 8; c < a.cols; c += NT * 8) {
      load8(dy_r, c, a.cols, g);
      load8(h_r, c, a.cols, h);
      weight8(a.weight, a.weight_dtype, c, a.cols, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = rstd * (g[j] * w[j] - h[j] * rstd * mean);
      if (a.dh) {
        load8(static_cast<const T*>(a.dh) + r * a.dh_stride, c, a.cols, h);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] += h[j];
      }
      if (a.dresidual) store8(static_cast<T*>(a.dresidual) + r * a.dresidual_stride, c, a.cols, g);
      if (a.dx) {
        if (d.on) drop8(d, seed, offset, r, c, g);
        store8(static_cast<T*>(a.dx) + r * a.dx_stride, c, a.cols, g);
      }
    }
  }
}

// dweight in two launches: part p sums rows p, p + parts, ... of 256 columns,
// then a thread sums its column over the parts, both in ascending order.
template <typename T>
__global__ __launch_bounds__(NT) void norm_dw_part(muon_norm_grad_args a, float* parts) {
  const int64_t c = blockIdx.x * (int64_t)NT + threadIdx.x;
  if (c >= a.cols) return;
  float s = 0.f;
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y)
    s += ld_as_f32(static_cast<const T*>(a.dy) + r * a.dy_stride, c) *
         (ld_as_f32(static_cast<const T*>(a.h) + r * a.h_stride, c) * a.rstd[r]);
  parts[blockIdx.y * a.cols + c] = s;
}

__global__ __launch_bounds__(NT) void norm_dw_sum(int64_t cols, int64_t n, const float* parts, float* dw) {
  const int64_t c = blockIdx.x * (int64_t)NT + threadIdx.x;
  if (c >= cols) return;
  float s = 0.f;
  for (int64_t p = 0; p < n; ++p) s += parts[p * cols + c];
  dw[c] = s;
}

}  // namespace

int64_t norm_parts(int64_t rows, int64_t cols) { return rows < 512 ? rows : 512; }

hipError_t run_dropout(int64_t rows, int64_t cols, const void* x, int64_t xs, void* y, int64_t ys, int dtype,
                       const Drop& d, hipStream_t stream) {
  const int64_t chunks = rows * ((cols + 7) / 8);
  const dim3 grid((unsigned)std::min<int64_t>((chunks + NT - 1) / NT, kMaxGrid));
  if (dtype == MUON_BF16)
    MUON_LAUNCH("dropout", dropout_k<bf16_t>, grid, dim3(NT), stream, rows, cols, static_cast<const bf16_t*>(x), xs,
                static_cast<bf16_t*>(y), ys, d);
  else
    MUON_LAUNCH("dropout", dropout_k<float>, grid, dim3(NT), stream, rows, cols, static_cast<const float*>(x), xs,
                static_cast<float*>(y), ys, d);
  return hipGetLastError();
}

hipError_t run_norm_forward(const muon_norm_args& a, const Drop& d, hipStream_t stream) {
  const dim3 grid((unsigned)std::min<int64_t>(a.rows, kMaxGrid));
  if (a.dtype == MUON_BF16) MUON_LAUNCH("norm_fwd", norm_fwd<bf16_t>, grid, dim3(NT), stream, a, d);
  else MUON_LAUNCH("norm_fwd", norm_fwd<float>, grid, dim3(NT), stream, a, d);
  return hipGetLastError();
}

hipError_t run_norm_backward(const muon_norm_grad_args& a, const Drop& d, float* parts, hipStream_t stream) {
  const dim3 grid((unsigned)std::min<int64_t>(a.rows, kMaxGrid));
  if (a.dresidual || a.dx) {
    if (a.dtype == MUON_BF16) MUON_LAUNCH("norm_bwd", norm_bwd<bf16_t>, grid, dim3(NT), stream, a, d);
    else MUON_LAUNCH("norm_bwd", norm_bwd<float>, grid, dim3(NT), stream, a, d);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.dweight) {
    const int64_t n = norm_parts(a.rows, a.cols);
    const unsigned blocks = (unsigned)((a.cols + NT - 1) / NT);
    if (n > 0) {
      const dim3 g2(blocks, (unsigned)n);
      if (a.dtype == MUON_BF16) MUON_LAUNCH("norm_dw_part", norm_dw_part<bf16_t>, g2, dim3(NT), stream, a, parts);
      else MUON_LAUNCH("norm_dw_part", norm_dw_part<float>, g2, dim3(NT), stream, a, parts);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    MUON_LAUNCH("norm_dw_sum", norm_dw_sum, dim3(blocks), dim3(NT), stream, a.cols, n, parts, a.dweight);
  }
  return hipGetLastError();
}

}  // namespace muon
