// The experts' 8-bit products (gfx950): out[i, n] = sum_b s_b sum_{k in b}
// a[i, k] w[e, n, k] with a scale for each block of 128 of k.
#include "experts_tiles.h"

namespace muon {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// 16 x 16 products over the 128 columns of one scale block, 32 of them a lane
// on each side; which 32 does not matter as long as both sides agree.
//
// The 8-bit matrix instruction brings the eight products that a lane's eight
// neighbouring bytes form to the largest one's exponent and cuts what lies
// 2^-13 below it (measured; so do the 8-bit instructions of 32 columns), and
// adds the rest in fp32: sums of random values are 4.4e-5 off in the root mean
// square, a fortieth of a bf16 output's rounding.  An fp32 output takes the
// operands as bf16, which holds them exactly, through the bf16 instruction
// (2.6e-8) at half the rate.
template <int FW, int FA, typename O>
struct Block;
template <int FW, int FA>
struct Block<FW, FA, bf16_t> {
  typedef i32x8 Frag;
  template <int F>
  static __device__ __forceinline__ Frag make(const i32x8& v) { return v; }
  static __device__ __forceinline__ f32x4 mfma(const Frag& w, const Frag& a) {
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, zero, FW, FA, 0, 0, 0, 0);   // no scales
  }
};
template <int FW, int FA>
struct Block<FW, FA, float> {
  struct Frag {
    bf16x8 v[4];
  };
  template <int F>
  static __device__ __forceinline__ Frag make(const i32x8& v) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    Frag f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      bf16x2 lo, hi;
      if constexpr (F) {
        lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(v[i], 1.f, false);
        hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(v[i], 1.f, true);
      } else {
        lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], 1.f, false);
        hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], 1.f, true);
      }
      f.v[i >> 1][4 * (i & 1)] = lo[0];
      f.v[i >> 1][4 * (i & 1) + 1] = lo[1];
      f.v[i >> 1][4 * (i & 1) + 2] = hi[0];
      f.v[i >> 1][4 * (i & 1) + 3] = hi[1];
    }
    return f;
  }
  static __device__ __forceinline__ f32x4 mfma(const Frag& w, const Frag& a) {
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[i], a.v[i], d, 0, 0, 0);
    return d;
  }
};

// Slot of 16-byte chunk c of a 128-byte row r: the 16 rows that a fragment
// read touches at once lie on different banks.
__device__ __forceinline__ int slot_of(int r, int c) { return c ^ ((r >> 1) & 7); }

__device__ __forceinline__ i32x8 fragment(const u32x4* rows, int r, int g) {
  const u32x4 lo = rows[r * 8 + slot_of(r, 2 * g)], hi = rows[r * 8 + slot_of(r, 2 * g + 1)];
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

template <typename O>
__device__ __forceinline__ void store4(O* row, int64_t n, int64_t N, const f32x4& v);
template <>
__device__ __forceinline__ void store4<bf16_t>(bf16_t* row, int64_t n, int64_t N, const f32x4& v) {
  if (n + 4 <= N) {
    *reinterpret_cast<u32x2_any*>(row + n) = u32x2_any{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
  } else {
#pragma unroll
    for (int r = 0; r < 3; ++r)
      if (n + r < N) row[n + r] = f2bf(v[r]);
  }
}
template <>
__device__ __forceinline__ void store4<float>(float* row, int64_t n, int64_t N, const f32x4& v) {
  if (n + 4 <= N) {
    *reinterpret_cast<u32x4_any*>(row + n) = __builtin_bit_cast(u32x4, v);
  } else {
#pragma unroll
    for (int r = 0; r < 3; ++r)
      if (n + r < N) row[n + r] = v[r];
  }
}

// 128 rows by 128 columns a workgroup, 64 x 64 a wave: any size, stride and
// alignment, through registers.  The matrices' rows are the instruction's
// first operand, so that a lane ends with four neighbouring columns of one row.
template <int FW, int FA, typename O>
__global__ void __launch_bounds__(256)
ex_product(muon_product_args p, uint32_t tiles_n) {
  typedef Block<FW, FA, O> Blk;
  constexpr int BM = 128, BN = 128;
  __shared__ u32x4 lds[(BM + BN) * 8];
  const int t = threadIdx.x, lane = t & 63, g = lane >> 4, q = lane & 15, w = t >> 6, wn = w & 1, wm = w >> 1;
  const int64_t KB = (p.k + 127) / 128, NB = (p.n + 127) / 128;
  ExpertTile tile;
  for (uint32_t index = blockIdx.x;
       find_tile(p.offsets, (int)p.num_experts, (int)p.rows, BM, tiles_n, index, tile); index += gridDim.x) {
    const int64_t n0 = (int64_t)tile.tn * BN;
    const uint8_t* W = static_cast<const uint8_t*>(p.w) + (int64_t)tile.e * p.w_matrix + n0 * p.w_stride;
    const uint8_t* A = static_cast<const uint8_t*>(p.a) + (int64_t)tile.row0 * p.a_stride;
    const float* ws = p.w_scales + ((int64_t)tile.e * NB + tile.tn) * KB;
    const float* as[4];
    bool live[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = wm * 64 + j * 16 + q;
      live[j] = r < tile.rows;
      as[j] = p.a_scales + (int64_t)(tile.row0 + (live[j] ? r : 0)) * p.a_scales_stride;
    }
    f32x4 acc[4][4] = {};
    for (int64_t b = 0; b < KB; ++b) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = (t >> 3) + 32 * i, c = t & 7;   // rows 0 .. 127 of W, then of A
        u32x4 v = {};
        if (i < 4) {
          if (n0 + r < p.n) v = load16(W + r * p.w_stride, b * 128 + c * 16, p.k);
        } else {
          if (r - BN < tile.rows) v = load16(A + (int64_t)(r - BN) * p.a_stride, b * 128 + c * 16, p.k);
        }
        lds[r * 8 + slot_of(r, c)] = v;
      }
      __syncthreads();
      const float sw = ws[b];
      typename Blk::Frag fw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) fw[i] = Blk::template make<FW>(fragment(lds, wn * 64 + i * 16 + q, g));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const typename Blk::Frag fa = Blk::template make<FA>(fragment(lds, BN + wm * 64 + j * 16 + q, g));
        const float s = live[j] ? as[j][b] * sw : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 d = Blk::mfma(fw[i], fa);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(d[r], s, acc[i][j][r]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (!live[j]) continue;
      O* row = static_cast<O*>(p.out) + (int64_t)(tile.row0 + wm * 64 + j * 16 + q) * p.out_stride;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t n = n0 + wn * 64 + i * 16 + 4 * g;
        if (n < p.n) store4<O>(row, n, p.n, acc[i][j]);
      }
    }
  }
}

template <int FW, int FA, typename O>
hipError_t launch(const muon_product_args& p, hipStream_t stream) {
  const int64_t tiles_n = (p.n + 127) / 128;
  const int64_t most = (p.rows / 128 + (p.num_experts < p.rows ? p.num_experts : p.rows)) * tiles_n;
  ex_product<FW, FA, O><<<unsigned(most < (1 << 20) ? most : 1 << 20), 256, 0, stream>>>(p, (uint32_t)tiles_n);
  return hipGetLastError();
}

template <int FW, int FA>
hipError_t launch_out(const muon_product_args& p, hipStream_t stream) {
  return p.out_dtype == MUON_F32 ? launch<FW, FA, float>(p, stream) : launch<FW, FA, bf16_t>(p, stream);
}

}  // namespace

hipError_t run_product(const muon_product_args& p, hipStream_t stream) {
  const bool w5 = p.w_dtype == MUON_ROW_E5M2, a5 = p.a_dtype == MUON_ROW_E5M2;
  if (w5) return a5 ? launch_out<1, 1>(p, stream) : launch_out<1, 0>(p, stream);
  return a5 ? launch_out<0, 1>(p, stream) : launch_out<0, 0>(p, stream);
}

}  // namespace muon
