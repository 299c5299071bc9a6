// The experts' 8-bit products (gfx950): out[i, n] = sum_b s_b sum_{k in b}
// a[i, k] w[e, n, k] with a scale for each block of 128 of k.
#include "choice.h"
#include "experts_tiles.h"
#include "lds.h"
#include "stages.h"

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
// square, a fortieth of a bf16 output's rounding, so that 1.2 % of the outputs
// round the other way than the exact sum and the error against 64 bits stays
// 1.7e-3.  An fp32 output takes the operands as bf16, which holds them exactly,
// through the bf16 instruction (2.6e-8 a block; 8e-8 in sums of 17 blocks with
// their scales) at half the rate.
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

// Slot of 16-byte chunk c of a 128-byte row r.  A 16-byte read is served for
// lanes 0-3, 12-15 and 20-27 at once, then for the others of the 32, and so on:
// with chunks g and g + 4 for lane group g they lie on different banks (with
// 2 g and 2 g + 1 the counters showed a conflict for every read, with these none).
__device__ __forceinline__ int slot_of(int r, int c) { return c ^ ((r >> 1) & 7); }

__device__ __forceinline__ i32x8 fragment(const u32x4* rows, int r, int g) {
  const u32x4 lo = rows[r * 8 + slot_of(r, g)], hi = rows[r * 8 + slot_of(r, g + 4)];
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
// alignment, through registers, a block ahead of the one multiplied.  The
// matrices' rows are the instruction's first operand, so that a lane ends with
// four neighbouring columns of one row.  3001 rows by 13 of 16 [1371, 2051] to
// fp32: 59 us, 277 TFLOP/s (144 without the loads ahead, 98 with one workgroup a
// CU); 49152 rows by 64 [2048, 4096] to fp32 671 TFLOP/s (630 with neighbouring
// tiles on different XCDs).  Bound by its two workgroups a CU and, to fp32, by the
// conversions.
template <int FW, int FA, typename O>
__global__ void __launch_bounds__(256, 2)
ex_product(muon_product_args p, uint32_t tiles_n) {
  typedef Block<FW, FA, O> Blk;
  constexpr int BM = 128, BN = 128;
  __shared__ u32x4 lds[2][(BM + BN) * 8];
  const int t = threadIdx.x, lane = t & 63, g = lane >> 4, q = lane & 15, w = t >> 6, wn = w & 1, wm = w >> 1;
  const int64_t KB = (p.k + 127) / 128, NB = (p.n + 127) / 128;
  // consecutive tiles, which share their operands, to the workgroups of one XCD (every eighth)
  const uint32_t total = count_tiles(p.offsets, (int)p.num_experts, (int)p.rows, BM, tiles_n), per = (total + 7) / 8;
  const uint32_t end = min(total, (blockIdx.x & 7) * per + per);
  ExpertTile tile;
  for (uint32_t index = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
       index < end && find_tile(p.offsets, (int)p.num_experts, (int)p.rows, BM, tiles_n, index, tile); index += gridDim.x >> 3) {
    const int64_t n0 = (int64_t)tile.tn * BN;
    const uint8_t* W = static_cast<const uint8_t*>(p.w) + (int64_t)tile.e * p.w_matrix + n0 * p.w_stride;
    const uint8_t* A = static_cast<const uint8_t*>(p.a) + (int64_t)tile.row0 * p.a_stride;
    const float* ws = p.w_scales + ((int64_t)tile.e * NB + tile.tn) * KB;
    __syncthreads();   // the tile before has been multiplied
    const float* as[4];
    bool live[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = wm * 64 + j * 16 + q;
      live[j] = r < tile.rows;
      as[j] = p.a_scales + (int64_t)(tile.row0 + (live[j] ? r : 0)) * p.a_scales_stride;
    }
    f32x4 acc[4][4] = {};
    // Rows 32 i + t / 8 of W, then of A, piece t % 8; those past the end repeat the last.
    u32x4 v[8];
    const uint8_t* from[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = (t >> 3) + 32 * (i & 3);
      from[i] = i < 4 ? W + min((int64_t)r, p.n - 1 - n0) * p.w_stride : A + (int64_t)min(r, tile.rows - 1) * p.a_stride;
    }
    auto load = [&](int64_t b) {
      const int64_t k = b * 128 + (t & 7) * 16;
      if (b * 128 + 128 <= p.k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const u32x4_any*>(from[i] + k);
      } else {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          const u32x4 x = load16(from[i], k, p.k);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (i == j) v[j] = x;
        }
      }
    };
    load(0);
    for (int64_t b = 0; b < KB; ++b) {
      // block b is written while others still multiply the one before from the other stage
      u32x4* stage = lds[b & 1];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = (t >> 3) + 32 * i, c = t & 7;
        stage[r * 8 + slot_of(r, c)] = v[i];
      }
      __syncthreads();
      if (b + 1 < KB) load(b + 1);
      const float sw = ws[b];
      typename Blk::Frag fa[4];
      float s[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        fa[j] = Blk::template make<FA>(fragment(stage, BN + wm * 64 + j * 16 + q, g));
        s[j] = as[j][b] * sw;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {   // one fragment of W at a time: as bf16 they are large
        const typename Blk::Frag fw = Blk::template make<FW>(fragment(stage, wn * 64 + i * 16 + q, g));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4 d = Blk::mfma(fw, fa[j]);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(d[r], s[j], acc[i][j][r]);
        }
        __builtin_amdgcn_sched_barrier(0);
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

// Eight columns of a bf16 row, of which `left` belong to it.  Stored past the cache, where the operands of the
// tiles to come are.
__device__ __forceinline__ void store_packed8(bf16_t* p, int left, const u32x4& v) {
  if (left >= 8) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(p));
  } else {
#pragma unroll
    for (int r = 0; r < 7; ++r)
      if (r < left) p[r] = (bf16_t)(v[r >> 1] >> (16 * (r & 1)));
  }
}

// ---------------------------------------------------------------------------
// 256 x 256 a workgroup of eight waves, 128 columns x 64 rows a wave, for
// 8-bit rows of whole 16-byte pieces and at least two blocks.
//
// Both operands come straight from global memory into one of two stages of 128
// bytes of each row.  A wave runs a block as 32 instructions of 32 cycles, in
// four parts of two of its eight column fragments by its four row fragments;
// behind each come the four multiply-adds that scale and add the result of the
// one two before, and the reads of the next part's fragments.  The one barrier of
// a block stands before its last part: then every wave has read the stage, so
// block k + 2 may be loaded into it, and every wave's loads of block k + 1, a
// whole block old, are there, so that the last part reads the first fragments of
// the next block and no wave finds itself without operands.
//
// 49152 rows by 64 [4096, 7168] 1.57-1.61 ms, 1770 TFLOP/s of useful products at
// 2.0 GHz; the matrix units are busy for 41-45 % of it.  Without any load the same
// kernel takes 1.24 ms, with all loads from the L2 and no products 0.77, with all
// loads and no products 1.57: it is bound by the time in which the 64 KB of a block
// arrive, with one block on its way a CU (whether the cache would take more lines
// at a time, only a loop with more stages could show).  Fetching lines towards the
// L2 one to six blocks ahead was slower (1.57 to 1.72 ms).  With the rows in the loads' scalar offset, which the
// hardware need not compare with a buffer's end, runs of whole tiles took 1.47 ms
// for 1.48.  Two wave groups a quarter block apart with four barriers a
// block took 1.80 ms, address arithmetic in the vector unit 1.72.
// ---------------------------------------------------------------------------
constexpr int kTile = 256, kStage = 2 * kTile * 128 + kTile * 4 + 256;

// A tile's operands, and the scales that a wave loads, as buffers from the next block to load on; they end with
// the tile's last row.
struct Operands {
  u32x4 w, a, scales;
};

__device__ __forceinline__ u32x4 lds_read16(uint32_t at) {
  return *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>((uintptr_t)at);
}
__device__ __forceinline__ float lds_read4(uint32_t at) {
  return *reinterpret_cast<const __attribute__((address_space(3))) float*>((uintptr_t)at);
}
// The kernel's first argument read anew where it is used, once a tile: held over the loop, its fields
// would take the scalar registers that the loop needs.
typedef const __attribute__((address_space(4))) muon_product_args* ArgsPtr;
__device__ __forceinline__ ArgsPtr args_again() {
  ArgsPtr a = (ArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(a));
  return a;
}

template <int FW, int FA>
__global__ void __launch_bounds__(512, 2)
ex_product_tiled(muon_product_args p, uint32_t tiles_n) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kStage];
  __shared__ int32_t runs[MUON_ROUTE_MAX_EXPERTS + 1];
  const int t = threadIdx.x, lane = t & 63, g = lane >> 4, q = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6), wn = w & 1, wm = (w >> 1) & 3;
  const int E = (int)p.num_experts, rows = (int)p.rows, K = (int)p.k, KB = (K + 127) / 128;
  const int NB = (int)((p.n + 127) / 128);
  for (int e = t; e <= E; e += 512) runs[e] = p.offsets ? p.offsets[e] : e ? rows : 0;
  __syncthreads();
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;

  // consecutive tiles, which share their operands, to the workgroups of one XCD (every eighth)
  const uint32_t total = count_tiles(runs, E, rows, kTile, tiles_n);
  const uint32_t per = (total + 7) / 8, xcd = blockIdx.x & 7, step = gridDim.x >> 3;
  const uint32_t end = min(total, xcd * per + per);
  uint32_t index = xcd * per + (blockIdx.x >> 3);
  ExpertTile tile;
  if (index >= end || !find_tile(runs, E, rows, kTile, tiles_n, index, tile)) return;

  const uint32_t w_pitch = (uint32_t)p.w_stride, a_pitch = (uint32_t)p.a_stride, s_pitch = (uint32_t)p.a_scales_stride * 4u;
  auto operands = [&](const ExpertTile& x) {
    const ArgsPtr p = args_again();
    const int64_t n0 = (int64_t)x.tn * kTile;
    const uint32_t wr = (uint32_t)min((int64_t)kTile, p->n - n0), ar = x.rows;
    return Operands{
        buffer_of(static_cast<const uint8_t*>(p->w) + (int64_t)x.e * p->w_matrix + n0 * p->w_stride, product_bytes(wr, w_pitch, K, 0)),
        buffer_of(static_cast<const uint8_t*>(p->a) + (int64_t)x.row0 * p->a_stride, product_bytes(ar, a_pitch, K, 0)),
        w < 4 ? buffer_of(p->a_scales + (int64_t)x.row0 * p->a_scales_stride, product_bytes(ar, s_pitch, KB * 4, 0))
              : buffer_of(p->w_scales + ((int64_t)x.e * NB + 2 * x.tn) * KB, product_bytes(wr > 128 ? 2 : 1, KB * 4, KB * 4, 0))};
  };
  // The next block of a tile to a stage, load `part` of nine: this wave's 32 rows of each operand, eight a
  // load, 16-byte piece c of row r in slot slot_of(r, c), then scales.  Pieces past the end of a row are
  // cleared by settle().
  uint32_t w_off[4], a_off[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    w_off[j] = product_offset(w, lane, j, w_pitch);
    a_off[j] = product_offset(w, lane, j, a_pitch);
  }
  const uint32_t s_off = w < 4 ? product_scale_offset(w, lane, s_pitch) : product_matrix_scale_offset(lane, KB * 4);
  auto issue = [&](const Operands& o, uint32_t stage, int part) {
    if (part < 8) {
      const int j = part >> 1;
      const uint32_t to = stage + w * 4096 + j * 1024;
      if (part & 1) lds_dma16(o.a, a_off[j], to + kTile * 128);
      else lds_dma16(o.w, w_off[j], to);
    } else if (w <= 4) {   // the matrix's behind the rows'
      lds_dma4(o.scales, s_off, stage + 2 * kTile * 128 + w * 256);
    }
  };
  auto block_on = [&](Operands& o) {
    advance(o.w, 128);
    advance(o.a, 128);
    advance(o.scales, 4);
  };
  // this wave's loads have arrived, block kb's in the given stage
  bool stores = false;
  auto settle = [&](int kb, uint32_t stage) {
    if (stores) __builtin_amdgcn_s_waitcnt(vmcnt_imm(16));   // counted in the order of issue
    else __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    stores = false;
    if (kb * 128 + 128 > K) {
      int l = lane;   // formed here: registers are short in the loop
      asm volatile("" : "+v"(l));
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (kb * 128 + (int)product_piece(l, j) >= K) {
          u32x4* to = reinterpret_cast<u32x4*>(lds + (stage - lds0) + w * 4096 + l * 16 + j * 1024);
          to[0] = u32x4{};
          to[kTile * 8] = u32x4{};
        }
    }
  };
  auto read = [&](uint32_t l, uint32_t h) {
    const u32x4 x = lds_read16(l), y = lds_read16(h);
    return i32x8{(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
  };

  Operands at = operands(tile);
  uint32_t here = lds0, there = lds0 + kStage;
#pragma unroll
  for (int x = 0; x < 9; ++x) issue(at, here, x);
  block_on(at);
#pragma unroll
  for (int x = 0; x < 9; ++x) issue(at, there, x);
  block_on(at);
  settle(0, here);
  lds_barrier();
  // this lane's addresses in a stage
  const uint32_t lo = q * 128 + slot_of(q, g) * 16, hi = q * 128 + slot_of(q, g + 4) * 16;
  const uint32_t wlo = wn * 16384 + lo, whi = wn * 16384 + hi;
  const uint32_t alo = kTile * 128 + wm * 8192 + lo, ahi = kTile * 128 + wm * 8192 + hi;
  const uint32_t sat = 2 * kTile * 128 + (wm * 64 + q) * 4, swat = 2 * kTile * 128 + kTile * 4 + wn * 4;
  i32x8 fw[2][2], fa[4];
  float sn[4], swn;
  auto first_fragments = [&](uint32_t stage) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      fa[j] = read(stage + alo + j * 2048, stage + ahi + j * 2048);
      sn[j] = lds_read4(stage + sat + j * 64);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) fw[0][i] = read(stage + wlo + i * 2048, stage + whi + i * 2048);
    swn = lds_read4(stage + swat);
  };
  first_fragments(here);

  for (bool more = true; more;) {
    ExpertTile next = tile;   // the last tile loads its own first blocks once more
    index += step;
    more = index < end && find_tile(runs, E, rows, kTile, tiles_n, index, next);
    if (wm * 64 >= tile.rows) {   // on a short last tile one wave of each SIMD only loads
      for (int kb = 0; kb < KB; ++kb) {
        settle(kb + 1 < KB ? kb + 1 : 0, there);
        lds_barrier();
        if (kb + 2 == KB) at = operands(next);
#pragma unroll
        for (int x = 0; x < 9; ++x) issue(at, here, x);
        block_on(at);
        const uint32_t x = here;
        here = there;
        there = x;
      }
      first_fragments(here);
      tile = next;
      continue;
    }
    f32x4 acc[8][4] = {};
    for (int kb = 0; kb < KB; ++kb) {
      if (kb + 2 == KB) at = operands(next);
      float s[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] = sn[j] * swn;
      f32x4 d[3];
#pragma unroll
      for (int x = 0; x < 34; ++x) {
        const int part = x >> 3, i = 2 * part + (x & 1), j = (x >> 1) & 3;
        if (x == 24) {   // the stage is read, the next one is there
          settle(kb + 1 < KB ? kb + 1 : 0, there);
          lds_barrier();
        }
        if (x < 32) d[x % 3] = Block<FW, FA, bf16_t>::mfma(fw[part & 1][x & 1], fa[j]);
        __builtin_amdgcn_sched_barrier(0);
        if (x >= 2) {
          const int y = x - 2, yi = 2 * (y >> 3) + (y & 1), yj = (y >> 1) & 3;
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[yi][yj][r] = __builtin_fmaf(d[y % 3][r], s[yj], acc[yi][yj][r]);
          asm volatile("" : "+v"(acc[yi][yj]));   // here, not where the sums are used
        }
        if (x < 24) {
          if ((x & 7) < 2) {
            const int f = 2 * (part + 1) + (x & 7);
            fw[(part + 1) & 1][x & 7] = read(here + wlo + f * 2048, here + whi + f * 2048);
          }
        } else if (x < 32) {
          if (x < 26) fw[0][x - 24] = read(there + wlo + (x - 24) * 2048, there + whi + (x - 24) * 2048);
          if (x & 1) fa[j] = read(there + alo + j * 2048, there + ahi + j * 2048);
          else sn[j] = lds_read4(there + sat + j * 64);
          issue(at, here, x - 24);
        } else if (x == 32) {
          swn = lds_read4(there + swat);
          issue(at, here, 8);
          block_on(at);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      const uint32_t x = here;
      here = there;
      there = x;
    }
    const int64_t n0 = (int64_t)tile.tn * kTile + wn * 128;
    const ArgsPtr again = args_again();
    bf16_t* out = static_cast<bf16_t*>(again->out) + (int64_t)(tile.row0 + wm * 64) * again->out_stride + n0;
    const uint32_t out_pitch = (uint32_t)again->out_stride;
    const int n_left = (int)min((int64_t)128, again->n - n0), r_left = tile.rows - wm * 64;
    int lq = lane;   // formed here: registers are short in the loop
    asm volatile("" : "+v"(lq));
    const int c0 = ((lq >> 3) & 1) * 32 + ((lq >> 4) & 1) * 16 + (lq >> 5) * 8;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        u32x4 v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // lane groups 0 and 2 take the fragment's other four columns from 1 and 3, which take theirs of the next
          const f32x4 &a = acc[i + 2 * h][j], &b = acc[i + 2 * h + 1][j];
          const auto x = __builtin_amdgcn_permlane16_swap(pack_bf16(a[0], a[1]), pack_bf16(b[0], b[1]), false, false);
          const auto y = __builtin_amdgcn_permlane16_swap(pack_bf16(a[2], a[3]), pack_bf16(b[2], b[3]), false, false);
          v[h] = u32x4{x[0], y[0], x[1], y[1]};
        }
        // lanes 8-15 of 16 take the second 32 columns of the rows of lanes 0-7, which leave them theirs: 128
        // bytes of a row side by side
        swap_lanes8(v[0], v[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = j * 16 + 8 * h + (lq & 7), n = i * 16 + c0;
          if (r < r_left) store_packed8(out + (__umul24(r, out_pitch) + n), n_left - n, v[h]);
        }
      }
    }
    // sixteen stores, and nothing else, behind the loads that settle() waits for next
    stores = n_left == 128 && r_left >= 64;
    tile = next;
  }
  // the loads that are still on their way go to this workgroup's memory
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
}

// ---------------------------------------------------------------------------
// Few rows an expert: the matrices' bytes are what counts, and each is used by
// one wave only, so that they go from memory to registers.
//
// A wave takes 16 columns (matrix rows) against up to 64 rows, 16 at a time, and
// KS waves of a workgroup share the blocks of k in groups of U; their sums are
// added in the order of the waves.  Any size, stride and alignment.  96 rows with
// 50 of 64 [4096, 7168] 275 us, 5.3 TB/s (tiles of 256: 463); bound by memory.
// Eight blocks a group, or three or four waves a SIMD at fewer registers: 317 to
// 373 us.
// ---------------------------------------------------------------------------
__device__ __forceinline__ i32x8 join(const u32x4& x, const u32x4& y) {
  return i32x8{(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
}

// U blocks from block b on: FULL: they all lie within the row.
template <int FW, int FA, typename O, int NT, int U, bool FULL>
__device__ __forceinline__ void few_blocks(const uint8_t* w, const uint8_t* const (&a)[NT], const float* ws,
                                           const float* const (&as)[NT], int64_t b, int64_t KB, int64_t K, f32x4 (&acc)[NT]) {
  typedef Block<FW, FA, O> Blk;
  const int g = (threadIdx.x & 63) >> 4;
  u32x4 wv[U][2], av[U][NT][2];
  float sw[U], sa[U][NT];
  auto get = [&](const uint8_t* row, int64_t k) {
    return FULL ? (u32x4)*reinterpret_cast<const u32x4_any*>(row + k) : load16(row, k, K);
  };
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t k = (b + u) * 128 + g * 16;
    wv[u][0] = get(w, k);
    wv[u][1] = get(w, k + 64);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t k = (b + u) * 128 + g * 16;
    const bool in = FULL || b + u < KB;
    sw[u] = in ? ws[b + u] : 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      av[u][t][0] = get(a[t], k);
      av[u][t][1] = get(a[t], k + 64);
      sa[u][t] = in ? as[t][b + u] : 0.f;
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const typename Blk::Frag fw = Blk::template make<FW>(join(wv[u][0], wv[u][1]));
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const typename Blk::Frag fa = Blk::template make<FA>(join(av[u][t][0], av[u][t][1]));
      const f32x4 d = Blk::mfma(fw, fa);
      const float s = sa[u][t] * sw[u];
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[t][r] = __builtin_fmaf(d[r], s, acc[t][r]);
    }
  }
}

// Rows row0 .. row0 + rows - 1 (at most 16 NT) of expert e by columns n0 .. n0 + 15.
template <int FW, int FA, typename O, int NT, int KS>
__device__ __forceinline__ void few_rows(const muon_product_args& p, int e, int row0, int rows, int64_t n0, int part,
                                         float (*sums)[64][16]) {
  constexpr int U = NT == 1 ? 4 : 2;
  const int lane = threadIdx.x & 63, g = lane >> 4, q = lane & 15;
  const int64_t KB = (p.k + 127) / 128, NB = (p.n + 127) / 128;
  const uint8_t* w = static_cast<const uint8_t*>(p.w) + (int64_t)e * p.w_matrix + min(n0 + q, p.n - 1) * p.w_stride;
  const float* ws = p.w_scales + ((int64_t)e * NB + n0 / 128) * KB;
  const uint8_t* a[NT];
  const float* as[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t r = row0 + min(16 * t + q, rows - 1);
    a[t] = static_cast<const uint8_t*>(p.a) + r * p.a_stride;
    as[t] = p.a_scales + r * p.a_scales_stride;
  }
  f32x4 acc[NT] = {};
  const int64_t full = p.k / (128 * U) * U;   // blocks in whole groups
  for (int64_t b = part * U; b < full; b += KS * U)
    few_blocks<FW, FA, O, NT, U, true>(w, a, ws, as, b, KB, p.k, acc);
  if (full < KB && full / U % KS == part)      // the rest is one group at most
    few_blocks<FW, FA, O, NT, U, false>(w, a, ws, as, full, KB, p.k, acc);
  if (KS > 1) {
    __syncthreads();   // the sums of the rows before have been read
    if (part > 0) {
#pragma unroll
      for (int t = 0; t < NT; ++t) *reinterpret_cast<f32x4*>(&sums[part][lane][4 * t]) = acc[t];
    }
    __syncthreads();
    if (part > 0) return;
#pragma unroll
    for (int s = 1; s < KS; ++s)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[t] += *reinterpret_cast<const f32x4*>(&sums[s][lane][4 * t]);
  }
  const int64_t n = n0 + 4 * g;
#pragma unroll
  for (int t = 0; t < NT; ++t)
    if (16 * t + q < rows && n < p.n)
      store4<O>(static_cast<O*>(p.out) + (int64_t)(row0 + 16 * t + q) * p.out_stride, n, p.n, acc[t]);
}

template <int FW, int FA, typename O, int KS>
__global__ void __launch_bounds__(KS > 4 ? 64 * KS : 256)
ex_product_few(muon_product_args p) {
  constexpr int TILES = KS > 4 ? 1 : 4 / KS;   // of 16 columns a workgroup
  __shared__ float sums[KS > 1 ? TILES * KS : 1][64][16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), tile = wave / KS, part = wave % KS;
  for (int e = blockIdx.y; e < (int)p.num_experts; e += gridDim.y) {
    int lo, hi;
    run_of(p.offsets, e, (int)p.rows, lo, hi);
    for (int64_t x = blockIdx.x; lo < hi && x * TILES * 16 < p.n; x += gridDim.x) {
      // a wave past the last column works on that column's tile again (its sums' barriers are everyone's)
      const int64_t n0 = min((x * TILES + tile) * 16, (p.n - 1) / 16 * 16);
      for (int r = lo + 64 * (int)blockIdx.z; r < hi; r += 64 * (int)gridDim.z) {
        const int rows = min(hi - r, 64);
        if (rows <= 16) few_rows<FW, FA, O, 1, KS>(p, e, r, rows, n0, part, sums + tile * KS);
        else if (rows <= 32) few_rows<FW, FA, O, 2, KS>(p, e, r, rows, n0, part, sums + tile * KS);
        else few_rows<FW, FA, O, 4, KS>(p, e, r, rows, n0, part, sums + tile * KS);
      }
    }
  }
}

template <int FW, int FA, typename O, int KS>
hipError_t launch_few(const muon_product_args& p, hipStream_t stream) {
  constexpr int TILES = KS > 4 ? 1 : 4 / KS;
  const int64_t x = (p.n + TILES * 16 - 1) / (TILES * 16);
  // A run of most of the rows goes to up to four workgroups, 64 rows each in turn: 192 rows with one of 64 [4096,
  // 7168] 141 us, 198 by one; to fp32 1024 rows with one of 128 [2048, 4096] 232 and 667.  Even runs pay for
  // workgroups that find no rows: 8 rows for each of 64 [4096, 7168] to fp32 582 and 527.  Two turns are one
  // workgroup's: 128 rows with one of eight [4096, 4096] to fp32 35 by one, 44 by two, 16 with each 60 and 70.
  const int64_t z = p.rows <= 128 ? 1 : (p.rows + 63) / 64;
  ex_product_few<FW, FA, O, KS><<<dim3(unsigned(x < (1 << 20) ? x : 1 << 20), unsigned(p.num_experts), unsigned(z < 4 ? z : 4)),
                                 KS > 4 ? 64 * KS : 256, 0, stream>>>(p);
  return hipGetLastError();
}

// Rows in 16-byte pieces at 16-byte addresses, with a tile's offsets in 32 bits.
bool whole_pieces(const muon_product_args& p) {
  auto fine = [&](const void* base, int64_t stride) {
    return reinterpret_cast<uintptr_t>(base) % 16 == 0 && stride % 16 == 0 && stride < (1 << 22);
  };
  return p.k % 16 == 0 && fine(p.a, p.rows > 1 ? p.a_stride : 0) && fine(p.w, p.n > 1 ? p.w_stride : 0) &&
         (p.num_experts == 1 || p.w_matrix % 16 == 0) && p.a_scales_stride < (1 << 20) && p.k < (1 << 30) &&
         p.rows < (1 << 30) && p.out_stride < (1 << 22) && p.rows * (p.rows > 1 ? p.a_scales_stride : 1) < (1 << 30) &&
         p.num_experts * ((p.n + 127) / 128) * ((p.k + 127) / 128) < (1 << 30);
}

template <int FW, int FA, typename O>
hipError_t launch(const muon_product_args& p, hipStream_t stream) {
  const bool pieces = whole_pieces(p), tiled = sizeof(O) == 2 && pieces && p.k > 128;
  const int64_t experts = p.num_experts < p.rows ? p.num_experts : p.rows, wide = (p.n + kTile - 1) / kTile;
  const int64_t tiles_n = (p.n + 127) / 128;
  if (p.rows <= most_rows_of_waves(experts * (tiled ? wide : tiles_n), tiled, pieces) * p.num_experts && p.rows < (1 << 30)) {
    // waves for all 1024 SIMDs four times over, or the blocks of k shared by up to eight
    const int64_t tiles = (p.n + 15) / 16 * experts, blocks = (p.k + 127) / 128;
    const int64_t share = tiles >= 4096 || blocks < 8 ? 1 : tiles >= 1024 || blocks < 32 ? 4 : 8;
    return share == 1 ? launch_few<FW, FA, O, 1>(p, stream) : share == 4 ? launch_few<FW, FA, O, 4>(p, stream)
                                                                         : launch_few<FW, FA, O, 8>(p, stream);
  }
  if constexpr (sizeof(O) == 2) {
    if (tiled) {
      ex_product_tiled<FW, FA><<<256, 512, 0, stream>>>(p, (uint32_t)wide);
      return hipGetLastError();
    }
  }
  const int64_t most = (p.rows / 128 + (p.num_experts < p.rows ? p.num_experts : p.rows)) * tiles_n;
  ex_product<FW, FA, O><<<unsigned(most < (1 << 20) ? (most + 7) / 8 * 8 : 1 << 20), 256, 0, stream>>>(p, (uint32_t)tiles_n);
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
