// Rows to the experts' order and back (gfx950): gather, combine and combine's
// gradients.  All three move bytes and compute next to nothing.
#include "experts_rows.h"

namespace muon {
namespace {

// ---------------------------------------------------------------------------
// gather: out[i] = x[order[i] / top_k], any type as bytes.
// ---------------------------------------------------------------------------
// 16 bytes a lane and step at any alignment; a row's last chunk is its last 16
// bytes (some of them written twice with the same values).
__device__ __forceinline__ void copy_row(const uint8_t* src, uint8_t* dst, int64_t width, int lane, int lanes,
                                         int64_t first, int64_t step) {
  if (width < 16) {
    if (first == 0 && lane < width) dst[lane] = src[lane];
    return;
  }
  const int64_t n = (width + 15) >> 4;
  for (int64_t c = first + lane; c < n; c += 8 * step) {
    u32x4_any v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t o = (c + j * step) * 16;
      if (c + j * step < n) v[j] = *reinterpret_cast<const u32x4_any*>(src + (o + 16 <= width ? o : width - 16));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t o = (c + j * step) * 16;
      if (c + j * step < n) *reinterpret_cast<u32x4_any*>(dst + (o + 16 <= width ? o : width - 16)) = v[j];
    }
  }
}

__global__ void __launch_bounds__(256)
ex_gather(muon_gather_args a, int64_t es, int log_lanes) {
  const int lanes = 1 << log_lanes, lane = threadIdx.x & (lanes - 1), per = 256 >> log_lanes;
  const int64_t pairs = a.rows * a.top_k, first = (int64_t)blockIdx.y * lanes, step = (int64_t)gridDim.y * lanes;
  for (int64_t i = (int64_t)blockIdx.x * per + (threadIdx.x >> log_lanes); i < pairs; i += (int64_t)gridDim.x * per) {
    const int32_t p = a.order[i];
    if (p < 0 || p >= pairs) continue;
    const int64_t r = (uint32_t)p / (uint32_t)a.top_k;
    copy_row(static_cast<const uint8_t*>(a.x) + r * a.x_stride * es, static_cast<uint8_t*>(a.out) + i * a.out_stride * es,
             a.cols * es, lane, lanes, first, step);
    if (a.scales)
      copy_row(reinterpret_cast<const uint8_t*>(a.scales + r * a.scales_stride),
               reinterpret_cast<uint8_t*>(a.out_scales + i * a.out_scales_stride), a.groups * 4, lane, lanes, first, step);
  }
}

// ---------------------------------------------------------------------------
// combine: out[t] = base[t] + sum_k w[t, k] y[position[t, k]], four slots' rows
// on their way together.  8192 rows of 7168 bf16 with six slots and base 200 us,
// 4.7 TB/s; 16 rows 4.5 us.  Bound by memory.
// ---------------------------------------------------------------------------
template <typename T, typename O>
__global__ void __launch_bounds__(256)
ex_combine(muon_combine_args a, int log_lanes) {
  const int lanes = 1 << log_lanes, lane = threadIdx.x & (lanes - 1), per = 256 >> log_lanes;
  const int64_t step = (int64_t)gridDim.y * lanes * 8;
  const int K = (int)a.top_k;
  for (int64_t t = (int64_t)blockIdx.x * per + (threadIdx.x >> log_lanes); t < a.rows; t += (int64_t)gridDim.x * per) {
    const int32_t* pos = a.position + t * K;
    const float* w = a.weights ? a.weights + t * K : nullptr;
    for (int64_t c = ((int64_t)blockIdx.y * lanes + lane) * 8; c < a.cols; c += step) {
      float s[8] = {};
      if (a.base) load8(static_cast<const O*>(a.base) + t * a.base_stride, c, a.cols, s);
      for (int k0 = 0; k0 < K; k0 += 4) {
        Chunk<T> v[4];
        float wk[4];
        bool ok[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = k0 + j < K ? k0 + j : K - 1;
          const int64_t i = pos[k];
          ok[j] = k0 + j < K && i >= 0 && i < a.places;
          wk[j] = w ? w[k] : 1.f;
          if (ok[j]) v[j].load(static_cast<const T*>(a.y) + i * a.y_stride, c, a.cols);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (!ok[j]) continue;
          float f[8];
          v[j].get(f, c, a.cols);
#pragma unroll
          for (int e = 0; e < 8; ++e) s[e] = __builtin_fmaf(wk[j], f[e], s[e]);
        }
      }
      store8(static_cast<O*>(a.out) + t * a.out_stride, c, a.cols, s);
    }
  }
}

// ---------------------------------------------------------------------------
// combine's gradients, LANES lanes for each row of dout, four slots at a time:
// their rows of y are on their way together, and dout is read once for them.
// Few rows have their slots dealt to several workgroups (grid.y).  8192 rows of
// 7168 bf16 with six slots, in bf16 and e4m3 387 us, 4.9 TB/s (a slot at a time
// 414); bound by memory.
// ---------------------------------------------------------------------------
template <typename T, int LANES>
__global__ void __launch_bounds__(256)
ex_combine_backward(muon_combine_grad_args a) {
  constexpr int PER = 256 / LANES, SLOTS = 4;
  __shared__ float dots[4][SLOTS];
  const int lane = threadIdx.x & (LANES - 1), wave = threadIdx.x / WAVE;
  const int K = (int)a.top_k;
  const bool e5 = a.dy8_dtype == MUON_ROW_E5M2;
  const int64_t steps = (a.cols + LANES * 8 - 1) / (LANES * 8);
  for (int64_t t0 = (int64_t)blockIdx.x * PER; t0 < a.rows; t0 += (int64_t)gridDim.x * PER) {
    const int64_t t = t0 + threadIdx.x / LANES;
    for (int k0 = blockIdx.y * SLOTS; k0 < K; k0 += gridDim.y * SLOTS) {
      float dot[SLOTS] = {};
      if (t < a.rows) {
        const T* dout = static_cast<const T*>(a.dout) + t * a.dout_stride;
        int64_t at[SLOTS];
        float w[SLOTS];
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
          const int64_t p = t * K + min(k0 + j, K - 1), i = a.position[p];
          at[j] = k0 + j < K && i >= 0 && i < a.places ? i : -1;
          w[j] = a.weights ? a.weights[p] : 1.f;
        }
        for (int64_t s = 0; s < steps; ++s) {
          const int64_t c = (s * LANES + lane) * 8;   // may pass the row's end: a group's lanes stay together
          float d[8], f[8];
          Chunk<T> y[SLOTS], x;
          x.load(dout, c, a.cols);
          if (a.dweights) {
#pragma unroll
            for (int j = 0; j < SLOTS; ++j)
              if (at[j] >= 0) y[j].load(static_cast<const T*>(a.y) + at[j] * a.y_stride, c, a.cols);
          }
          x.get(d, c, a.cols);
          // the group's largest |w d| is |w| times its largest |d|: rounding keeps the order
          const float most = a.dy8 ? over_row<16>(most8(d), max_f) : 0.f;
#pragma unroll
          for (int j = 0; j < SLOTS; ++j) {
            if (at[j] < 0) continue;
            if (a.dweights) {
              y[j].get(f, c, a.cols);
#pragma unroll
              for (int e = 0; e < 8; ++e) dot[j] = __builtin_fmaf(d[e], f[e], dot[j]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = d[e] * w[j];
            if (a.dy && c < a.cols) store8(static_cast<T*>(a.dy) + at[j] * a.dy_stride, c, a.cols, f);
            if (a.dy8 && c < a.cols) {
              const float scale = group_scale(fmaxf(most * fabsf(w[j]), 0.f), e5);   // NaN: no product but NaN, or zeros
              if ((c & 127) == 0) a.scales[at[j] * a.scales_stride + (c >> 7)] = scale;
              store_eight(static_cast<uint8_t*>(a.dy8) + at[j] * a.dy8_stride, c, a.cols, f, scale, e5);
            }
          }
        }
        if (a.dweights) {
#pragma unroll
          for (int j = 0; j < SLOTS; ++j) {
            dot[j] = over_row<(LANES < WAVE ? LANES : WAVE)>(dot[j], add_f);
            if (LANES <= WAVE && lane == 0 && k0 + j < K) a.dweights[t * K + k0 + j] = dot[j];
          }
        }
      }
      if (LANES > WAVE && a.dweights) {   // t is the workgroup's
        if ((threadIdx.x & (WAVE - 1)) == 0) {
#pragma unroll
          for (int j = 0; j < SLOTS; ++j) dots[wave][j] = dot[j];
        }
        __syncthreads();
        const int j = threadIdx.x;
        if (j < SLOTS && k0 + j < K) a.dweights[t * K + k0 + j] = (dots[0][j] + dots[1][j]) + (dots[2][j] + dots[3][j]);
        __syncthreads();
      }
    }
  }
}

template <typename T>
hipError_t combine_to(const muon_combine_args& a, const RowLayout& l, hipStream_t stream) {
  if (a.out_dtype == MUON_F32) ex_combine<T, float><<<dim3(l.gx, l.gy), 256, 0, stream>>>(a, l.log_lanes);
  else ex_combine<T, bf16_t><<<dim3(l.gx, l.gy), 256, 0, stream>>>(a, l.log_lanes);
  return hipGetLastError();
}

template <typename T, int LANES>
hipError_t launch_backward(const muon_combine_grad_args& a, hipStream_t stream) {
  constexpr int PER = 256 / LANES;
  const int64_t groups = (a.rows + PER - 1) / PER, most = 1 << 20, sets = (a.top_k + 3) / 4;
  const int64_t y = groups >= 512 ? 1 : sets;
  ex_combine_backward<T, LANES><<<dim3(unsigned(groups < most ? groups : most), unsigned(y)), 256, 0, stream>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t combine_backward_of(const muon_combine_grad_args& a, hipStream_t stream) {
  if (a.cols <= 256) return launch_backward<T, 32>(a, stream);
  return a.cols <= 1024 ? launch_backward<T, 64>(a, stream) : launch_backward<T, 256>(a, stream);
}

}  // namespace

hipError_t run_gather(const muon_gather_args& a, hipStream_t stream) {
  const int64_t es = a.dtype == MUON_ROW_F32 ? 4 : a.dtype == MUON_ROW_BF16 ? 2 : 1;
  // Many rows: at most a wave each, with up to eight pieces a lane on their way (49152 rows of 7168 bytes
  // and their scales 111 us; a workgroup each 122).
  const int64_t pairs = a.rows * a.top_k, chunks = (a.cols * es + 15) / 16;
  const RowLayout l = row_layout(pairs, pairs >= 4096 && chunks > 64 ? 64 : chunks);
  ex_gather<<<dim3(l.gx, l.gy), 256, 0, stream>>>(a, es, l.log_lanes);
  return hipGetLastError();
}

hipError_t run_combine(const muon_combine_args& a, hipStream_t stream) {
  const RowLayout l = row_layout(a.rows, (a.cols + 7) / 8);
  return a.dtype == MUON_F32 ? combine_to<float>(a, l, stream) : combine_to<bf16_t>(a, l, stream);
}

hipError_t run_combine_backward(const muon_combine_grad_args& a, hipStream_t stream) {
  return a.dtype == MUON_F32 ? combine_backward_of<float>(a, stream) : combine_backward_of<bf16_t>(a, stream);
}

}  // namespace muon
