// Root-mean-square norm with the residual's addition, and dropout.
//
//   z = r + D(x);  rstd = 1 / sqrt(mean(z^2) + eps);  y = z rstd w
//   dz = rstd (g - xh mean(g xh)) + dh,  g = dy w,  xh = h rstd;  dw = sum dy xh
//
// All of it is bound by memory: a few operations per element, one pass over
// each input and output.  A copy of 1 GiB reaches 5.1 TB/s on this card.
#include <algorithm>

#include "internal.h"
#include "rows.h"

namespace muon {
namespace {

constexpr int NT = 256;            // threads of a workgroup
constexpr int64_t kMaxGrid = 1 << 16;

// D(x) alone: eight columns a lane, which share one Philox block, 16 bits an
// element.  [8192, 28672] bf16: 162 us a call among others, 5.8 TB/s, the vector
// units busy 75 % of it with one block; 32 bits an element would need two.
// WHOLE: a width of whole chunks, which spares the tests for the last one
// ([16384, 4096] bf16 48 us, 52 with them; 4095 columns 57).
template <typename T, bool WHOLE>
__global__ __launch_bounds__(NT) void dropout_k(int64_t rows, int64_t cols, const T* x, int64_t xs, T* y, int64_t ys,
                                                Drop d) {
  uint64_t seed, offset;
  drop_seed(d, seed, offset);
  const int64_t per_row = (cols + 7) / 8, total = rows * per_row;
  const uint32_t n = (uint32_t)cols;   // below 2^31
  for (int64_t i = blockIdx.x * (int64_t)NT + threadIdx.x; i < total; i += (int64_t)gridDim.x * NT) {
    const int64_t r = total <= UINT32_MAX ? (uint32_t)i / (uint32_t)per_row : i / per_row;
    const uint32_t c = (uint32_t)(i - r * per_row) * 8, end = WHOLE ? c + 8 : n;
    float f[8];
    load8(x + r * xs, c, end, f);
    if (d.on) drop8(d, seed, offset, r, c, f);
    store8(y + r * ys, c, end, f);
  }
}

// Columns c .. c+7 of weight (ones without one).
template <class I>
__device__ __forceinline__ void weight8(const void* w, int dtype, I c, I cols, float* f) {
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
__device__ __forceinline__ float scale_of(float most, int y_dtype) {
  const float unit = y_dtype == MUON_ROW_E5M2 ? 1.f / 57344.f : 1.f / 448.f;
  return most == 0.f ? 1.f : fmaxf(most * unit, 0x1p-126f);
}

// y of columns c .. c+7 at its type; an 8-bit y with the group's scale, found
// across the group's lanes unless the row's is given.  LPR: lanes of a row if
// fewer than a wave (a group then ends with the row).
template <int LPR, class I>
__device__ __forceinline__ void store_y(const muon_norm_args& a, int64_t r, I c, I cols, float* y, float row_scale) {
  if (a.y_dtype == MUON_ROW_F32) {
    if (c < cols) store8(static_cast<float*>(a.y) + r * a.y_stride, c, cols, y);
  } else if (a.y_dtype == MUON_ROW_BF16) {
    if (c < cols) store8(static_cast<bf16_t*>(a.y) + r * a.y_stride, c, cols, y);
  } else {
    const bool e5 = a.y_dtype == MUON_ROW_E5M2;
    float scale = row_scale;
    if (a.group) {   // 4, 8 or 16 lanes hold a group
      float most = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(y[j]));
      most = fmaxf(most, dpp<0xB1>(most));
      most = fmaxf(most, dpp<0x4E>(most));
      if (a.group > 32) most = fmaxf(most, dpp<0x141>(most));
      if (LPR != 8 && a.group > 64) most = fmaxf(most, dpp<0x140>(most));
      scale = scale_of(most, a.y_dtype);
      if (c < cols && (c & (a.group - 1)) == 0) a.scales[r * a.scales_stride + c / a.group] = scale;
    }
    // y / scale as fp32 divides (but for one in a million, an ulp off): 1 / scale
    // in two floats, the first a little too small so that the second is positive
    // and -0 keeps its sign.  2^-126 <= scale < 2^120, or infinite: then finite
    // elements become 0 and infinite ones NaN.  One multiplication more an
    // element than by the reciprocal alone, which moves a few in a million by an
    // 8-bit step: [4096, 8192] 45.6 us against 45.4, [32768, 1024] by groups of 32
    // 24.2 against 23.6.
    const float inv = __builtin_amdgcn_rcpf(scale) * (1.f - 0x1p-22f);
    const float rest = scale < HUGE_VALF ? __builtin_fmaf(-scale, inv, 1.f) * inv : 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = __builtin_fmaf(y[j], inv, y[j] * rest);
    uint8_t* row = static_cast<uint8_t*>(a.y) + r * a.y_stride;
    if (c < cols) {
      if (e5) store8_8bit<true>(row, c, cols, y);
      else store8_8bit<false>(row, c, cols, y);
    }
  }
}

// The 8-bit scale of a whole row is one more reduction.
__device__ __forceinline__ bool row_scaled(const muon_norm_args& a) {
  return a.y_dtype >= MUON_ROW_E4M3 && a.group == 0;
}

// Where a lane stands: `lanes` lanes share a row, this is the t-th of them;
// rows r, r + step, ... are theirs.
template <int LPR>
struct RowLanes {
  int lanes, t;
  int64_t r, step;
  __device__ __forceinline__ RowLanes() {
    lanes = LPR ? LPR : (int)blockDim.x;
    t = LPR ? threadIdx.x & (LPR - 1) : threadIdx.x;
    constexpr int rows = LPR ? NT / (LPR ? LPR : 1) : 1;   // of a workgroup at a time
    r = blockIdx.x * (int64_t)rows + (LPR ? threadIdx.x / (LPR ? LPR : 1) : 0);
    step = (int64_t)gridDim.x * rows;
  }
};

// The row in registers: every lane keeps NC chunks of eight columns, `lanes`
// chunks apart, so each input is read once.  LPR = 8 .. 64 lanes a row and no
// barriers up to 1024 columns, else (LPR = 0) a workgroup of up to 512 lanes a
// row.  The workgroups stay and step over the rows; the next row's loads are
// issued before this row's reduction and stores, so that memory is busy
// meanwhile.  Measured: [16384, 4096] bf16 with residual and p = 0.1 98 us,
// 5.5 TB/s (two passes over the row 135); [4096, 8192] to e4m3 with a scale per
// 128 columns 45.6 us, 5.2 TB/s; [65536, 128] 12.5 us; fp32 [8192, 4096] 97 us,
// [4096, 16384] bf16 103 us; one row of 4096 3.2 us, less than the call.
template <typename T, int NC, int LPR>
__global__ __launch_bounds__(LPR ? NT : 512) void norm_fwd(muon_norm_args a, Drop d) {
  __shared__ GroupRed sums, maxima;
  if constexpr (LPR == 0) {
    red_init(sums);
    red_init(maxima);
  }
  const RowLanes<LPR> at;
  const int cols = (int)a.cols;
  const int lanes = at.lanes, t = at.t;
  const int64_t step = at.step;
  int64_t r = at.r;
  uint64_t seed, offset;
  drop_seed(d, seed, offset);
  const float per_col = 1.f / (float)cols;
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.residual);
  float w[NC][8];
  Chunk<T> cx[NC], cr[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (i * lanes + t) * 8;
    weight8(a.weight, a.weight_dtype, c, cols, w[i]);
    if (r < a.rows) {
      cx[i].load(x + r * a.x_stride, c, cols);
      if (res) cr[i].load(res + r * a.residual_stride, c, cols);
    }
  }
  for (int turn = 0; r < a.rows; r += step, turn ^= 1) {
    float z[NC][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (i * lanes + t) * 8;
      cx[i].get(z[i], c, cols);
      if (d.on) drop8(d, seed, offset, r, c, z[i]);
      if (res) {
        float e[8];
        cr[i].get(e, c, cols);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[i][j] += e[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += z[i][j] * z[i][j];
    }
    if (r + step < a.rows) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = (i * lanes + t) * 8;
        cx[i].load(x + (r + step) * a.x_stride, c, cols);
        if (res) cr[i].load(res + (r + step) * a.residual_stride, c, cols);
      }
    }
    ss = LPR ? over_row<LPR ? LPR : WAVE>(ss, add_f) : group_sum(ss, sums, turn);
    const float rstd = 1.f / sqrtf(ss * per_col + a.eps);
    if (a.rstd && t == 0) a.rstd[r] = rstd;
    if (a.h) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = (i * lanes + t) * 8;
        if (c < cols) store8(static_cast<T*>(a.h) + r * a.h_stride, c, cols, z[i]);
      }
    }
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        z[i][j] = z[i][j] * rstd * w[i][j];   // past the row's end 0, or NaN with rstd: fmaxf passes over it
        most = fmaxf(most, fabsf(z[i][j]));
      }
    float row_scale = 1.f;
    if (row_scaled(a)) {
      most = LPR ? over_row<LPR ? LPR : WAVE>(most, max_f) : group_max(most, maxima, turn);
      row_scale = scale_of(most, a.y_dtype);
      if (t == 0) a.scales[r * a.scales_stride] = row_scale;
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) store_y<LPR>(a, r, (i * lanes + t) * 8, cols, z[i], row_scale);
  }
}

// Rows longer than the registers hold: z is formed again in each pass over
// the row, which the caches mostly hold by then.  [2048, 28672] bf16 with
// residual 133 us, 3.5 TB/s: the second pass is not free.
template <typename T>
__global__ __launch_bounds__(512) void norm_fwd_long(muon_norm_args a, Drop d) {
  __shared__ GroupRed sums, maxima;
  red_init(sums);
  red_init(maxima);
  uint64_t seed, offset;
  drop_seed(d, seed, offset);
  const int64_t pass = (int64_t)blockDim.x * 8;
  int turn = 0;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, turn ^= 1) {
    float z[8], w[8];
    float ss = 0.f;
    for (int64_t c = threadIdx.x * 8; c < a.cols; c += pass) {
      z8<T>(a, d, seed, offset, r, c, z);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += z[j] * z[j];
    }
    ss = group_sum(ss, sums, turn);
    const float rstd = 1.f / sqrtf(ss / (float)a.cols + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[r] = rstd;
    float row_scale = 1.f;
    if (row_scaled(a)) {
      float most = 0.f;
      for (int64_t c = threadIdx.x * 8; c < a.cols; c += pass) {
        z8<T>(a, d, seed, offset, r, c, z);
        weight8(a.weight, a.weight_dtype, c, a.cols, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) most = fmaxf(most, c + j < a.cols ? fabsf(z[j] * rstd * w[j]) : 0.f);
      }
      most = group_max(most, maxima, turn);
      row_scale = scale_of(most, a.y_dtype);
      if (threadIdx.x == 0) a.scales[r * a.scales_stride] = row_scale;
    }
    for (int64_t c0 = 0; c0 < a.cols; c0 += pass) {
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
      store_y<0>(a, r, c, a.cols, y, row_scale);
    }
  }
}

// Backward, the row in registers as in norm_fwd.  dweight's sums stay in the
// lanes' registers over all of a workgroup's rows; each workgroup leaves one
// row of partial sums (or the result, if it is the only one).  [16384, 4096]
// bf16 with dropout and dh: 128 us and 5 for norm_dw_sum, 5.0 TB/s of the
// bytes without the partial sums (passes of their own for dz and dweight 346);
// fp32 [8192, 4096] 73 + 5, bf16 [4096, 8200] 51 + 5 and [4096, 16384] 81 + 5
// (four chunks a lane and no loads ahead: 4.7 TB/s); [777, 2051] fp32 in a
// wider buffer 11 + 4 us, the latency of four rows in a row and of two launches.
template <typename T, int NC, int LPR>
__global__ __launch_bounds__(LPR ? NT : 512) void norm_bwd(muon_norm_grad_args a, Drop d, float* parts) {
  __shared__ GroupRed sums;
  if constexpr (LPR == 0) red_init(sums);
  const RowLanes<LPR> at;
  const int cols = (int)a.cols;
  const int lanes = at.lanes, t = at.t;
  const int64_t step = at.step;
  int64_t r = at.r;
  uint64_t seed, offset;
  drop_seed(d, seed, offset);
  const float per_col = 1.f / (float)cols;
  const T* dy = static_cast<const T*>(a.dy);
  const T* h = static_cast<const T*>(a.h);
  const T* dh = static_cast<const T*>(a.dh);
  float w[NC][8], dw[NC][8];
  // four chunks a lane leave no registers for the next row's
  constexpr bool AHEAD = NC <= 2;
  Chunk<T> cg[NC], ch[NC], cd[NC];
  float rstd = 0.f;
  auto fetch = [&](int64_t row) {
    rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (i * lanes + t) * 8;
      cg[i].load(dy + row * a.dy_stride, c, cols);
      ch[i].load(h + row * a.h_stride, c, cols);
      if (dh) cd[i].load(dh + row * a.dh_stride, c, cols);
    }
  };
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    weight8(a.weight, a.weight_dtype, (i * lanes + t) * 8, cols, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  }
  if (AHEAD && r < a.rows) fetch(r);
  for (int turn = 0; r < a.rows; r += step, turn ^= 1) {
    if (!AHEAD) fetch(r);
    float g[NC][8], xh[NC][8];
    Chunk<T> e[NC];
    float dot = 0.f;
    const float rs = rstd;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (i * lanes + t) * 8;
      cg[i].get(g[i], c, cols);
      ch[i].get(xh[i], c, cols);
      e[i] = cd[i];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[i][j] *= rs;
        dw[i][j] += g[i][j] * xh[i][j];
        g[i][j] *= w[i][j];
        dot += g[i][j] * xh[i][j];
      }
    }
    if (AHEAD && r + step < a.rows) fetch(r + step);
    const float mean = (LPR ? over_row<LPR ? LPR : WAVE>(dot, add_f) : group_sum(dot, sums, turn)) * per_col;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (i * lanes + t) * 8;
      if (c >= cols) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) g[i][j] = rs * (g[i][j] - xh[i][j] * mean);
      if (dh) {
        float f[8];
        e[i].get(f, c, cols);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[i][j] += f[j];
      }
      if (a.dresidual) store8(static_cast<T*>(a.dresidual) + r * a.dresidual_stride, c, cols, g[i]);
      if (a.dx) {
        if (d.on) drop8(d, seed, offset, r, c, g[i]);
        store8(static_cast<T*>(a.dx) + r * a.dx_stride, c, cols, g[i]);
      }
    }
  }
  if (!a.dweight) return;
  float* out = gridDim.x == 1 ? a.dweight : parts + blockIdx.x * (int64_t)cols;
  if constexpr (LPR != 0) {
    // the rows a workgroup worked on side by side, added in their order
    constexpr int rows = NT / (LPR ? LPR : 1);
    __shared__ float all[rows][NC * 8][LPR];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) all[threadIdx.x / LPR][i * 8 + j][t] = dw[i][j];
    __syncthreads();
    for (int q = threadIdx.x; q < NC * 8 * LPR; q += NT) {
      const int k = q / LPR, lane = q % LPR;   // chunk k / 8 of that lane, its column k % 8
      const int c = ((k / 8) * LPR + lane) * 8 + k % 8;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < rows; ++w) v += all[w][k][lane];
      if (c < cols) out[c] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (i * lanes + t) * 8;
      if (c < cols) store8(out, c, cols, dw[i]);
    }
  }
}

// Rows longer than the registers hold: two passes over the row, and dweight's
// partial sums (a row of `parts` for each workgroup, its own lanes' columns) in
// memory.  [2048, 28672] bf16 171 + 6 us, 2.0 TB/s of the bytes.
template <typename T>
__global__ __launch_bounds__(512) void norm_bwd_long(muon_norm_grad_args a, Drop d, float* parts) {
  __shared__ GroupRed sums;
  red_init(sums);
  uint64_t seed, offset;
  drop_seed(d, seed, offset);
  const int64_t pass = (int64_t)blockDim.x * 8;
  float* out = gridDim.x == 1 ? a.dweight : parts + blockIdx.x * a.cols;
  int turn = 0;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, turn ^= 1) {
    const T* dy_r = static_cast<const T*>(a.dy) + r * a.dy_stride;
    const T* h_r = static_cast<const T*>(a.h) + r * a.h_stride;
    const float rstd = a.rstd[r];
    float g[8], h[8], w[8];
    float dot = 0.f;
    for (int64_t c = threadIdx.x * 8; c < a.cols; c += pass) {
      load8(dy_r, c, a.cols, g);
      load8(h_r, c, a.cols, h);
      weight8(a.weight, a.weight_dtype, c, a.cols, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[j] *= rstd;
        dot += g[j] * w[j] * h[j];
      }
      if (a.dweight) {
        float s[8];
        if (r == (int64_t)blockIdx.x) {
#pragma unroll
          for (int j = 0; j < 8; ++j) s[j] = 0.f;
        } else {
          load8(out, c, a.cols, s);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] += g[j] * h[j];
        store8(out, c, a.cols, s);
      }
    }
    const float mean = group_sum(dot, sums, turn) / (float)a.cols;
    for (int64_t c = threadIdx.x * 8; c < a.cols; c += pass) {
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

// dweight from the partial sums: a workgroup 32 columns, 32 lanes a column,
// each every 32nd part in ascending order, then the 32 sums in order.
constexpr int DWC = 32, DWL = 32;
__global__ __launch_bounds__(DWC* DWL) void norm_dw_sum(int64_t cols, int64_t n, const float* parts, float* dw) {
  __shared__ float s[DWL][DWC + 1];
  const int cc = threadIdx.x % DWC, k = threadIdx.x / DWC;
  for (int64_t c0 = blockIdx.x * (int64_t)DWC; c0 < cols; c0 += (int64_t)gridDim.x * DWC) {
    const int64_t c = c0 + cc;
    float v = 0.f;
    if (c < cols) {
      int64_t p = k;
      for (; p + 7 * DWL < n; p += 8 * DWL) {   // eight loads in flight
        float e[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) e[q] = parts[(p + q * DWL) * cols + c];
#pragma unroll
        for (int q = 0; q < 8; ++q) v += e[q];
      }
      for (; p < n; p += DWL) v += parts[p * cols + c];
    }
    s[k][cc] = v;
    __syncthreads();
    if (k == 0 && c < cols) {
      v = 0.f;
#pragma unroll
      for (int q = 0; q < DWL; ++q) v += s[q][cc];
      dw[c] = v;
    }
    __syncthreads();
  }
}

}  // namespace

namespace {

// How a row is laid over lanes: up to 1024 columns 8 to 64 lanes, up to 16384
// a workgroup of as many waves as its chunks fill, longer rows in passes.
struct RowShape {
  int lpr;             // lanes a row; 0: the workgroup
  int nc;              // chunks a lane keeps; 0: in passes
  unsigned threads;
  int64_t per_group;   // rows a workgroup works on at once
};
RowShape row_shape(int64_t cols) {
  const int64_t chunks = (cols + 7) / 8;
  if (chunks <= 2 * WAVE) {
    const int lpr = chunks <= 8 ? 8 : chunks <= 16 ? 16 : chunks <= 32 ? 32 : 64;
    return {lpr, chunks <= WAVE ? 1 : 2, NT, NT / lpr};
  }
  const int nc = chunks <= 512 ? 1 : chunks <= 1024 ? 2 : chunks <= 2048 ? 4 : 0;
  if (nc == 0) return {0, 0, 512, 1};
  return {0, nc, (unsigned)round_up((chunks + nc - 1) / nc, WAVE), 1};
}

// Workgroups for `groups` of rows, at most `most` and all with as many rows as
// the others but the last few.
int64_t even(int64_t groups, int64_t most) {
  if (groups < 1) return 0;
  const int64_t each = (groups + most - 1) / most;
  return (groups + each - 1) / each;
}

// Forward: workgroups that stay on the GPU, at least 1024 lanes on each of 256
// CUs where a lane keeps one chunk, two workgroups where it keeps more.
// [16384, 4096] bf16 with p = 0.1: half as many 6 % slower, twice as many 3 %
// (the last round of workgroups is then part empty); [3777, 2880] by three
// workgroups of 384 lanes 20 us a call, by two or four 24 (a fourth does not fit
// the SIMD that holds two waves of each; 17 us of it are the kernel's).
int64_t resident(const RowShape& s) { return 256 * (s.nc == 1 ? (1024 + s.threads - 1) / s.threads : 1024 / s.threads); }

}  // namespace

// Backward: each workgroup leaves a row of partial sums, written and read
// again, which costs as much as parts / rows of the whole.  As many as keep
// the memory busy, 1024 lanes a CU ([12010, 1728] bf16 with dh: 39 us, 53 by
// half), as long as each has 12 rows; one a CU where a lane keeps more chunks
// ([4096, 8192]: 44 us, two 48; it leaves a CU five waves just past 4096 columns,
// [16384, 4097] 115 us where 4096 take 78); up to 4 rows in a row a single one,
// which needs no second launch.
int64_t norm_parts(int64_t rows, int64_t cols) {
  const RowShape s = row_shape(cols);
  const int64_t groups = (rows + s.per_group - 1) / s.per_group;
  if (groups <= 4) return std::min<int64_t>(groups, 1);
  return even(groups, s.nc == 1 ? std::min(resident(s), std::max<int64_t>(256, rows / 12)) : 256);
}

template <typename T>
static void launch_dropout(int64_t rows, int64_t cols, const void* x, int64_t xs, void* y, int64_t ys, const Drop& d,
                           hipStream_t stream) {
  const int64_t chunks = rows * ((cols + 7) / 8);
  const dim3 grid((unsigned)std::min<int64_t>((chunks + NT - 1) / NT, kMaxGrid));
  const T* in = static_cast<const T*>(x);
  T* out = static_cast<T*>(y);
  if (cols % 8 == 0) MUON_LAUNCH("dropout", (dropout_k<T, true>), grid, dim3(NT), stream, rows, cols, in, xs, out, ys, d);
  else MUON_LAUNCH("dropout", (dropout_k<T, false>), grid, dim3(NT), stream, rows, cols, in, xs, out, ys, d);
}

hipError_t run_dropout(int64_t rows, int64_t cols, const void* x, int64_t xs, void* y, int64_t ys, int dtype,
                       const Drop& d, hipStream_t stream) {
  if (dtype == MUON_BF16) launch_dropout<bf16_t>(rows, cols, x, xs, y, ys, d, stream);
  else launch_dropout<float>(rows, cols, x, xs, y, ys, d, stream);
  return hipGetLastError();
}

template <typename T>
static void launch_forward(const muon_norm_args& a, const Drop& d, hipStream_t stream) {
  const RowShape s = row_shape(a.cols);
  const int64_t groups = (a.rows + s.per_group - 1) / s.per_group;
  const dim3 grid((unsigned)even(groups, resident(s))), block(s.threads);
  if (s.lpr == 8) MUON_LAUNCH("norm_fwd", (norm_fwd<T, 1, 8>), grid, block, stream, a, d);
  else if (s.lpr == 16) MUON_LAUNCH("norm_fwd", (norm_fwd<T, 1, 16>), grid, block, stream, a, d);
  else if (s.lpr == 32) MUON_LAUNCH("norm_fwd", (norm_fwd<T, 1, 32>), grid, block, stream, a, d);
  else if (s.lpr == 64 && s.nc == 1) MUON_LAUNCH("norm_fwd", (norm_fwd<T, 1, 64>), grid, block, stream, a, d);
  else if (s.lpr == 64) MUON_LAUNCH("norm_fwd", (norm_fwd<T, 2, 64>), grid, block, stream, a, d);
  else if (s.nc == 1) MUON_LAUNCH("norm_fwd", (norm_fwd<T, 1, 0>), grid, block, stream, a, d);
  else if (s.nc == 2) MUON_LAUNCH("norm_fwd", (norm_fwd<T, 2, 0>), grid, block, stream, a, d);
  else if (s.nc == 4) MUON_LAUNCH("norm_fwd", (norm_fwd<T, 4, 0>), grid, block, stream, a, d);
  else MUON_LAUNCH("norm_fwd_long", norm_fwd_long<T>, grid, block, stream, a, d);
}

hipError_t run_norm_forward(const muon_norm_args& a, const Drop& d, hipStream_t stream) {
  if (a.dtype == MUON_BF16) launch_forward<bf16_t>(a, d, stream);
  else launch_forward<float>(a, d, stream);
  return hipGetLastError();
}

template <typename T>
static void launch_backward(const muon_norm_grad_args& a, const Drop& d, float* parts, hipStream_t stream) {
  const RowShape s = row_shape(a.cols);
  const int64_t groups = (a.rows + s.per_group - 1) / s.per_group;
  const dim3 grid((unsigned)(a.dweight ? norm_parts(a.rows, a.cols) : even(groups, resident(s))));
  const dim3 block(s.threads);
  if (s.lpr == 8) MUON_LAUNCH("norm_bwd", (norm_bwd<T, 1, 8>), grid, block, stream, a, d, parts);
  else if (s.lpr == 16) MUON_LAUNCH("norm_bwd", (norm_bwd<T, 1, 16>), grid, block, stream, a, d, parts);
  else if (s.lpr == 32) MUON_LAUNCH("norm_bwd", (norm_bwd<T, 1, 32>), grid, block, stream, a, d, parts);
  else if (s.lpr == 64 && s.nc == 1) MUON_LAUNCH("norm_bwd", (norm_bwd<T, 1, 64>), grid, block, stream, a, d, parts);
  else if (s.lpr == 64) MUON_LAUNCH("norm_bwd", (norm_bwd<T, 2, 64>), grid, block, stream, a, d, parts);
  else if (s.nc == 1) MUON_LAUNCH("norm_bwd", (norm_bwd<T, 1, 0>), grid, block, stream, a, d, parts);
  else if (s.nc == 2) MUON_LAUNCH("norm_bwd", (norm_bwd<T, 2, 0>), grid, block, stream, a, d, parts);
  else if (s.nc == 4) MUON_LAUNCH("norm_bwd", (norm_bwd<T, 4, 0>), grid, block, stream, a, d, parts);
  else MUON_LAUNCH("norm_bwd_long", norm_bwd_long<T>, grid, block, stream, a, d, parts);
}

hipError_t run_norm_backward(const muon_norm_grad_args& a, const Drop& d, float* parts, hipStream_t stream) {
  if (a.rows > 0) {
    if (a.dtype == MUON_BF16) launch_backward<bf16_t>(a, d, parts, stream);
    else launch_backward<float>(a, d, parts, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t n = norm_parts(a.rows, a.cols);
  if (a.dweight && n != 1)   // n = 0: zeros
    MUON_LAUNCH("norm_dw_sum", norm_dw_sum, dim3((unsigned)std::min<int64_t>((a.cols + DWC - 1) / DWC, kMaxGrid)), dim3(DWC * DWL), stream, a.cols, n,
                parts, a.dweight);
  return hipGetLastError();
}

}  // namespace muon
