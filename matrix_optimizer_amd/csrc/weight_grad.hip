// The gradient of the experts' matrices (gfx950): dw[e] = dy_e^T x_e over the
// expert's rows, bf16 products summed in fp32.
#include "experts_tiles.h"
#include "lds.h"

namespace muon {
namespace {

// Columns c .. c+7 of a bf16 row, zeros from `cols` on.
__device__ __forceinline__ u32x4 load8_bf16(const bf16_t* row, int64_t c, int64_t cols) {
  return load16(reinterpret_cast<const uint8_t*>(row), c * 2, cols * 2);
}

// 128 x 128 of one expert's matrix a workgroup, 64 x 64 a wave, 32 rows a
// step: both operands lie with the rows of the sum along the slow axis, so
// their fragments are read transposed.  Any size, stride and alignment.
template <typename O>
__global__ void __launch_bounds__(256)
ex_weight_grad(muon_weight_grad_args p, int64_t tn, int64_t tk) {
  constexpr int BK = 32;
  __shared__ u32x4 lds[2][BK][16];   // rows of 128 columns of dy and of x
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, wn = w & 1, wk = w >> 1;
  for (int64_t index = blockIdx.x; index < p.num_experts * tn * tk; index += gridDim.x) {
    const int64_t jk = index % tk, jn = index / tk % tn;
    const int e = (int)(index / (tk * tn));
    const int64_t n0 = jn * 128, k0 = jk * 128;
    int lo, hi;
    run_of(p.offsets, e, (int)p.rows, lo, hi);
    f32x16 acc[2][2] = {};
    for (int64_t r0 = lo; r0 < hi; r0 += BK) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = (t >> 4) + 16 * i, c = t & 15;
        u32x4 a = {}, b = {};
        if (r0 + r < hi) {
          a = load8_bf16(static_cast<const bf16_t*>(p.dy) + (r0 + r) * p.dy_stride, n0 + c * 8, p.n);
          b = load8_bf16(static_cast<const bf16_t*>(p.x) + (r0 + r) * p.x_stride, k0 + c * 8, p.k);
        }
        lds[0][r][c] = a;
        lds[1][r][c] = b;
      }
      __syncthreads();
      const bf16_t* A = reinterpret_cast<const bf16_t*>(lds[0]);
      const bf16_t* B = reinterpret_cast<const bf16_t*>(lds[1]);
      const int G = lane >> 4, s4 = lane & 15;
#pragma unroll
      for (int kk = 0; kk < BK / 16; ++kk) {
        bf16x8 f[2][2];
#pragma unroll
        for (int op = 0; op < 2; ++op)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            bf16x4 h[2];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const int row = 16 * kk + 8 * (G >> 1) + 4 * hh + (s4 >> 2);
              const int col = (op ? wk : wn) * 64 + i * 32 + 16 * (G & 1) + 4 * (s4 & 3);
              h[hh] = lds_read_tr16((op ? B : A) + row * 128 + col);
            }
            f[op][i] = __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7);
          }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[0][i], f[1][j], acc[i][j], 0, 0, 0);
      }
    }
    O* out = static_cast<O*>(p.dw) + e * p.dw_matrix;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int64_t n = n0 + wn * 64 + i * 32 + mfma32_row(lane, r), k = k0 + wk * 64 + j * 32 + mfma32_col(lane);
          if (n < p.n && k < p.k) st_from_f32(out, n * p.dw_stride + k, acc[i][j][r]);
        }
  }
}

}  // namespace

int64_t weight_grad_parts(int64_t, int64_t, int64_t, int64_t) { return 1; }

hipError_t run_weight_grad(const muon_weight_grad_args& p, float*, hipStream_t stream) {
  const int64_t tn = (p.n + 127) / 128, tk = (p.k + 127) / 128, tiles = p.num_experts * tn * tk;
  const unsigned grid = unsigned(tiles < (1 << 20) ? tiles : 1 << 20);
  if (p.dw_dtype == MUON_F32) ex_weight_grad<float><<<grid, 256, 0, stream>>>(p, tn, tk);
  else ex_weight_grad<bf16_t><<<grid, 256, 0, stream>>>(p, tn, tk);
  return hipGetLastError();
}

}  // namespace muon
