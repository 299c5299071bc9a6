// The gradient of the experts' matrices (gfx950): dw[e] = dy_e^T x_e over the
// expert's rows, bf16 products summed in fp32.
#include "experts_tiles.h"
#include "lds.h"
#include "stages.h"

namespace muon {
namespace {

// Where a launch writes: dw itself, or fp32 parts of it that weight_grad_join
// adds up.
struct Dest {
  void* base;
  int64_t stride, matrix, part;   // elements; part 0: one part
  int parts;
};

// Rows of part `part` of `parts` of the run [lo, hi), in whole steps of `unit` rows.
__device__ __forceinline__ void part_of(int part, int parts, int unit, int& lo, int& hi) {
  const int64_t first = lo, end = hi, steps = (end - first + unit - 1) / unit;
  lo = (int)min(end, first + steps * part / parts * unit);
  hi = (int)min(end, first + steps * (part + 1) / parts * unit);
}

// Columns c .. c+7 of a bf16 row, zeros from `cols` on.
__device__ __forceinline__ u32x4 load8_bf16(const bf16_t* row, int64_t c, int64_t cols) {
  return load16(reinterpret_cast<const uint8_t*>(row), c * 2, cols * 2);
}

// ---------------------------------------------------------------------------
// 128 x 128 of one expert's matrix a workgroup, 64 x 64 a wave, 64 rows a
// step: both operands lie with the rows of the sum along the slow axis, so
// their fragments are read transposed.  Any size, stride and alignment,
// through registers, a step ahead of the one multiplied.  777 rows of 1001 and 515
// columns for 8 experts 18-20 us, bound by latency.  Odd widths of much work have
// their rows copied for the kernel below; widths that are multiples of 8 in rows off
// 16 bytes have no workspace for that and stay here: 49152 rows of 1024 and 1024 for
// 8 experts 290 us for 140, to 64 [7168, 2048] 4.1 ms for 1.55.
// ---------------------------------------------------------------------------
template <typename O>
__global__ void __launch_bounds__(256)
ex_weight_grad(muon_weight_grad_args p, Dest d, int64_t tn, int64_t tk) {
  constexpr int BK = 64, N = BK / 16;
  __shared__ u32x4 lds[2][2][BK][16];   // twice rows of 128 columns of dy and of x, piece c of row r in slot c ^ 4 (r % 4)
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, wn = w & 1, wk = w >> 1;
  // an expert's tiles, which share their operands, dealt in eight runs to the XCDs as below
  const int64_t each = tn * tk * d.parts, xcd = blockIdx.x & 7;
  const bool deal = each >= 64;
  const int64_t from = deal ? each * xcd / 8 : 0, mine = deal ? each * (xcd + 1) / 8 - from : each;
  for (int64_t index = deal ? blockIdx.x >> 3 : blockIdx.x; index < mine * p.num_experts;
       index += deal ? gridDim.x >> 3 : gridDim.x) {
    const int e = (int)(index / mine);
    const int64_t local = from + index - e * mine, tile = local / d.parts, jk = tile % tk, jn = tile / tk;
    const int part = (int)(local % d.parts);
    const int64_t n0 = jn * 128, k0 = jk * 128;
    int lo, hi;
    run_of(p.offsets, e, (int)p.rows, lo, hi);
    part_of(part, d.parts, 64, lo, hi);
    f32x16 acc[2][2] = {};
    // the next step's pieces in registers while a step is multiplied: rows t / 16 and N - 1 times 16 more,
    // piece t % 16; rows past the run's end are zeros
    u32x4 v[2][N];
    const int r = t >> 4, c = t & 15;
    const bool whole = n0 + 128 <= p.n && k0 + 128 <= p.k;
    auto load = [&](int64_t r0) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[0][i] = v[1][i] = u32x4{};
        const int64_t at = r0 + r + 16 * i;
        if (at >= hi) continue;
        const bf16_t* dy = static_cast<const bf16_t*>(p.dy) + at * p.dy_stride;
        const bf16_t* x = static_cast<const bf16_t*>(p.x) + at * p.x_stride;
        if (whole) {
          v[0][i] = *reinterpret_cast<const u32x4_any*>(dy + n0 + c * 8);
          v[1][i] = *reinterpret_cast<const u32x4_any*>(x + k0 + c * 8);
        } else {
          v[0][i] = load8_bf16(dy, n0 + c * 8, p.n);
          v[1][i] = load8_bf16(x, k0 + c * 8, p.k);
        }
      }
    };
    load(lo);
    __syncthreads();   // the tile before has been multiplied
    int turn = 0;
    for (int64_t r0 = lo; r0 < hi; r0 += BK, turn ^= 1) {
      // written while others still multiply the step before from the other half
#pragma unroll
      for (int i = 0; i < N; ++i) {
        lds[turn][0][r + 16 * i][c ^ (4 * (r & 3))] = v[0][i];
        lds[turn][1][r + 16 * i][c ^ (4 * (r & 3))] = v[1][i];
      }
      __syncthreads();
      load(r0 + BK);
      const bf16_t* A = reinterpret_cast<const bf16_t*>(lds[turn][0]);
      const bf16_t* B = reinterpret_cast<const bf16_t*>(lds[turn][1]);
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
              h[hh] = lds_read_tr16((op ? B : A) + row * 128 + ((((col >> 3) ^ (4 * (row & 3))) << 3) | (col & 7)));
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
    O* out = static_cast<O*>(d.base) + part * d.part + e * d.matrix;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int64_t n = n0 + wn * 64 + i * 32 + mfma32_row(lane, r), k = k0 + wk * 64 + j * 32 + mfma32_col(lane);
          if (n < p.n && k < p.k) st_from_f32(out, n * d.stride + k, acc[i][j][r]);
        }
  }
}

// ---------------------------------------------------------------------------
// 256 x 256 a workgroup of eight waves, 64 (n) x 128 (k) a wave, for rows of
// whole 16-byte pieces (those of the last columns may be filled up).
//
// 64 rows of both operands at a time come straight from global memory into one
// of two stages; a wave multiplies a stage in four steps of 16 rows, eight
// instructions of 32 cycles each, and reads the next step's fragments
// (transposed) between them.  The one barrier of a stage stands before its last
// step: then every wave has read the stage, so that the one after the next may
// be loaded into it, and every wave's loads of the next stage, a whole stage old,
// are there, so that the last step reads the first fragments of the next stage.
// Stages follow one another over the tiles without a gap.  x's columns are the
// instruction's rows, so that a lane ends with runs of four along k, eight after
// one exchange with the lane 32 away.
//
// 49152 rows to 64 [7168, 2048] bf16 1.47-1.52 ms, 930 TFLOP/s; a stage takes
// 1.8 us (as in the 8-bit product the time in which 64 KB, the one stage on its way,
// arrive), the matrix units are busy for 46 % of it, and the 1.9 GB of results take
// 0.24 ms that no products hide.
// ---------------------------------------------------------------------------
constexpr int kTile = 256, kRows = 64, kStage = 2 * kRows * kTile * 2;

// A tile: its columns, its run of rows and its place in the output.
struct Tile {
  int lo, hi;
  int e, part, n0, k0;
};

__device__ __forceinline__ bf16x8 read_tr(uint32_t at) {
  const bf16x4 a = lds_read_tr16_at(at), b = lds_read_tr16_at(at + 4 * 512);
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Four 16-byte pieces a lane of 32 rows of eight pieces, those of lanes n and n + 32 alternately the pieces
// of row n, dealt anew so that each register holds eight whole rows, 128 bytes in a row at a time: row
// 8 s + lane % 8, piece 2 (lane / 8 % 4) + lane / 32.  Stored past the cache, where the operands of the
// tiles to come are: 64 [7168, 2048] from one stage each in 333 us, 467 through the cache, 499 by 32 bytes a
// row as the pieces come.
__device__ __forceinline__ void whole_rows(u32x4 (&r)[4]) {
  swap_lanes8(r[0], r[1]);
  swap_lanes8(r[2], r[3]);
  swap_lanes16(r[0], r[2]);
  swap_lanes16(r[1], r[3]);
}

// 16 bytes of a row, of which `left` elements belong to it.
__device__ __forceinline__ void store_piece(bf16_t* p, int left, const u32x4& v) {
  if (left >= 8) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(p));
  } else {
#pragma unroll
    for (int r = 0; r < 7; ++r)
      if (r < left) p[r] = (bf16_t)(v[r >> 1] >> (16 * (r & 1)));
  }
}
__device__ __forceinline__ void store_piece(float* p, int left, const u32x4& v) {
  if (left >= 4) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(p));
  } else {
#pragma unroll
    for (int r = 0; r < 3; ++r)
      if (r < left) p[r] = __uint_as_float(v[r]);
  }
}

// 32 rows of 64 (bf16) or 32 (fp32) columns from an accumulator pair or one accumulator; `k_left` columns and
// `n_left` rows belong to the matrix.
__device__ __forceinline__ void store_rows(bf16_t* out, int64_t stride, int k_left, int n_left, const f32x16& v0, const f32x16& v1) {
  const int lane = threadIdx.x & 63;
  u32x4 r[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const f32x16& v = s < 2 ? v0 : v1;
    const int q = 2 * (s & 1);
    // lanes below 32 keep run q and take its other half, the others run q + 1
    const auto a = __builtin_amdgcn_permlane32_swap(pack_bf16(v[4 * q], v[4 * q + 1]), pack_bf16(v[4 * q + 4], v[4 * q + 5]),
                                                    false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(pack_bf16(v[4 * q + 2], v[4 * q + 3]),
                                                    pack_bf16(v[4 * q + 6], v[4 * q + 7]), false, false);
    r[s] = u32x4{a[0], b[0], a[1], b[1]};
  }
  whole_rows(r);
  const int k = 8 * (2 * ((lane >> 3) & 3) + (lane >> 5));
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int n = 8 * s + (lane & 7);
    if (n < n_left) store_piece(out + n * stride + k, k_left - k, r[s]);
  }
}
__device__ __forceinline__ void store_rows(float* out, int64_t stride, int k_left, int n_left, const f32x16& v) {
  const int lane = threadIdx.x & 63;
  u32x4 r[4];
#pragma unroll
  for (int s = 0; s < 4; ++s)
    r[s] = u32x4{__float_as_uint(v[4 * s]), __float_as_uint(v[4 * s + 1]), __float_as_uint(v[4 * s + 2]), __float_as_uint(v[4 * s + 3])};
  whole_rows(r);
  const int k = 4 * (2 * ((lane >> 3) & 3) + (lane >> 5));
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int n = 8 * s + (lane & 7);
    if (n < n_left) store_piece(out + n * stride + k, k_left - k, r[s]);
  }
}

template <typename O>
__global__ void __launch_bounds__(512, 2)
ex_weight_grad_tiled(muon_weight_grad_args p, Dest d, uint32_t tn, uint32_t tk) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kStage];
  __shared__ int32_t runs[MUON_ROUTE_MAX_EXPERTS + 1];
  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6), wk = w & 1, wn = (w >> 1) & 3;
  const int rows = (int)p.rows, E = (int)p.num_experts;
  for (int e = t; e <= E; e += 512) runs[e] = p.offsets ? p.offsets[e] : e ? rows : 0;
  __syncthreads();
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;

  // An expert's tiles, which share their operands, are dealt in eight runs to the XCDs (every eighth
  // workgroup); few tiles an expert go round.
  const uint32_t each = tn * tk * d.parts, xcd = blockIdx.x & 7;
  const bool deal = each >= 64;
  const uint32_t from = deal ? (uint32_t)((uint64_t)each * xcd / 8) : 0;
  const uint32_t mine = deal ? (uint32_t)((uint64_t)each * (xcd + 1) / 8) - from : each;
  const uint32_t total = mine * (uint32_t)E, step = deal ? gridDim.x >> 3 : gridDim.x;
  uint32_t index = deal ? blockIdx.x >> 3 : blockIdx.x;
  if (index >= total) return;
  auto tile_at = [&](uint32_t i) {
    Tile x;
    const uint32_t e = i / mine, local = from + i - e * mine, part = local % d.parts, u = local / d.parts;
    x.e = (int)__builtin_amdgcn_readfirstlane(e);
    x.part = (int)__builtin_amdgcn_readfirstlane(part);
    x.n0 = (int)__builtin_amdgcn_readfirstlane(u / tk) * kTile;
    x.k0 = (int)__builtin_amdgcn_readfirstlane(u % tk) * kTile;
    int lo, hi;
    run_of(runs, x.e, rows, lo, hi);
    part_of(x.part, d.parts, kRows, lo, hi);
    x.lo = __builtin_amdgcn_readfirstlane(lo);
    x.hi = __builtin_amdgcn_readfirstlane(hi);
    return x;
  };

  // Rows first .. first + 63 to a stage: this wave's eight rows of each operand, two a load, 16-byte
  // piece c of row r in slot c ^ 4 (r % 4), so that the four rows of a transposing read lie on different
  // banks.  The buffers end with the run; rows past it are cleared by settle().
  const uint32_t d_pitch = (uint32_t)p.dy_stride * 2, x_pitch = (uint32_t)p.x_stride * 2;
  uint32_t d_off[4], x_off[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    d_off[j] = grad_offset(w, lane, j, d_pitch);
    x_off[j] = grad_offset(w, lane, j, x_pitch);
  }
  Tile load = tile_at(index);       // the tile being loaded, its next rows, whether there are any
  uint32_t load_index = index;
  int first = load.lo;
  bool live = true;
  struct Rows64 {
    u32x4 dy, x;
    int first, hi;
  };
  auto next_rows = [&]() {
    if (!live) return Rows64{buffer_of(p.dy, 0), buffer_of(p.x, 0), 0, 0};
    const int left = load.hi - first, n = left < kRows ? left : kRows;
    const Rows64 r{buffer_of(static_cast<const bf16_t*>(p.dy) + (int64_t)first * p.dy_stride + load.n0,
                             grad_bytes(n, d_pitch, (uint32_t)((p.n + 7) / 8 * 8 - load.n0) * 2)),
                   buffer_of(static_cast<const bf16_t*>(p.x) + (int64_t)first * p.x_stride + load.k0,
                             grad_bytes(n, x_pitch, (uint32_t)((p.k + 7) / 8 * 8 - load.k0) * 2)),
                   first, load.hi};
    first += kRows;
    if (first >= load.hi) {
      load_index += step;
      live = load_index < total;
      if (live) load = tile_at(load_index);
      first = load.lo;
    }
    return r;
  };
  auto issue = [&](const Rows64& r, uint32_t stage, int part) {   // load `part` of eight
    const int j = part >> 1;
    const uint32_t to = stage + w * 4096 + j * 1024;
    if (part & 1) lds_dma16(r.x, x_off[j], to + kStage / 2);
    else lds_dma16(r.dy, d_off[j], to);
  };
  constexpr int kStores = sizeof(O) == 2 ? 16 : 32;
  bool stores = false;   // a tile's stores, and nothing else, are behind the loads that settle() waits for
  auto settle = [&](int f, int hi, uint32_t stage) {
    if (stores) __builtin_amdgcn_s_waitcnt(vmcnt_imm(kStores));   // counted in the order of issue
    else __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    stores = false;
    if (f + kRows > hi) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (f + 8 * w + 2 * j + (lane >> 5) >= hi) {
          u32x4* to = reinterpret_cast<u32x4*>(lds + (stage - lds0) + w * 4096 + lane * 16 + j * 1024);
          to[0] = u32x4{};
          to[kStage / 32] = u32x4{};
        }
    }
  };

  uint32_t here = lds0, there = lds0 + kStage;
  int f1, h1;   // rows of the stage after the one being worked on
  {
    const Rows64 r0 = next_rows();
#pragma unroll
    for (int x = 0; x < 8; ++x) issue(r0, here, x);
    const Rows64 r1 = next_rows();
#pragma unroll
    for (int x = 0; x < 8; ++x) issue(r1, there, x);
    f1 = r1.first;
    h1 = r1.hi;
    settle(r0.first, r0.hi, here);
  }
  lds_barrier();
  // Of 32 columns (block b of the operand's eight) a lane reads rows 8 (G / 2) + s / 4 and four below, columns
  // 16 (G % 2) + 4 (s % 4) on, in 16-lane group G at lane s.
  const int G = lane >> 4, s4 = lane & 15;
  auto column = [&](int b) {
    return (8 * (G >> 1) + (s4 >> 2)) * 512 + (((4 * b + 2 * (G & 1) + ((s4 & 3) >> 1)) ^ (4 * (s4 >> 2))) * 16) + (s4 & 1) * 8;
  };
  uint32_t xa[4], da[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) xa[i] = column(4 * wk + i) + kStage / 2;
#pragma unroll
  for (int j = 0; j < 2; ++j) da[j] = column(2 * wn + j);
  bf16x8 fx[2][4], fd[2][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) fx[0][i] = read_tr(here + xa[i]);
#pragma unroll
  for (int j = 0; j < 2; ++j) fd[0][j] = read_tr(here + da[j]);

  for (; index < total; index += step) {
    const Tile cur = tile_at(index);
    f32x16 acc[4][2] = {};
    for (int at = cur.lo, last = 0; !last; at += kRows) {
      last = at + kRows >= cur.hi;
      const Rows64 r = next_rows();
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if (kk == 3) {   // the stage is read, the next one is there
          settle(f1, h1, there);
          lds_barrier();
        }
        const uint32_t of = kk < 3 ? here + (kk + 1) * 16 * 512 : there;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          acc[x >> 1][x & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fx[kk & 1][x >> 1], fd[kk & 1][x & 1], acc[x >> 1][x & 1], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
          if (x < 4) fx[~kk & 1][x] = read_tr(of + xa[x]);
          else if (x < 6) fd[~kk & 1][x - 4] = read_tr(of + da[x - 4]);
          if (kk == 3) issue(r, here, x);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      f1 = r.first;
      h1 = r.hi;
      const uint32_t x = here;
      here = there;
      there = x;
    }
    const int n0 = cur.n0 + wn * 64, k0 = cur.k0 + wk * 128;
    O* out = static_cast<O*>(d.base) + cur.part * d.part + cur.e * d.matrix + n0 * d.stride + k0;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        O* at = out + 32 * j * d.stride + 32 * i;
        const int k_left = (int)p.k - k0 - 32 * i, n_left = (int)p.n - n0 - 32 * j;
        if constexpr (sizeof(O) == 4) store_rows(at, d.stride, k_left, n_left, acc[i][j]);
        else if (i % 2 == 0) store_rows(at, d.stride, k_left, n_left, acc[i][j], acc[i + 1][j]);
      }
    stores = n0 + 64 <= p.n && k0 + 128 <= p.k;
  }
  // the loads that are still on their way go to this workgroup's memory
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
}

// dw = the sum of the parts, in their order.
template <typename O>
__global__ void __launch_bounds__(256)
ex_weight_grad_join(muon_weight_grad_args p, const float* parts, int n_parts, int64_t part) {
  const int64_t chunks = (p.k + 7) / 8, all = p.num_experts * p.n * chunks;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / chunks, c = (i - row * chunks) * 8, e = row / p.n, n = row - e * p.n;
    float s[8] = {}, f[8];
    for (int j = 0; j < n_parts; j += 8) {   // eight parts on their way together
      Chunk<float> v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (j + u < n_parts) v[u].load(parts + (j + u) * part + row * p.k, c, p.k);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (j + u >= n_parts) continue;
        v[u].get(f, c, p.k);
#pragma unroll
        for (int q = 0; q < 8; ++q) s[q] += f[q];
      }
    }
    store8(static_cast<O*>(p.dw) + e * p.dw_matrix + n * p.dw_stride, c, p.k, s);
  }
}

// Rows of dy (y = 0) and x (y = 1) up to the end of the runs, copied to rows of whole 16-byte pieces, zeros
// behind the last column.
__global__ void __launch_bounds__(256)
ex_weight_grad_align(muon_weight_grad_args p, bf16_t* dy, bf16_t* x) {
  const bool second = blockIdx.y != 0;
  const int64_t cols = second ? p.k : p.n, chunks = (cols + 7) / 8, stride = second ? p.x_stride : p.dy_stride;
  const bf16_t* from = static_cast<const bf16_t*>(second ? p.x : p.dy);
  bf16_t* to = second ? x : dy;
  const int64_t all = end_of_runs(p.offsets, (int)p.num_experts, (int)p.rows) * chunks;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / chunks, c = (i - r * chunks) * 8;
    Chunk<bf16_t> v;
    v.load(from + r * stride, c, cols);
    v.settle(c, cols);
    *reinterpret_cast<u32x4*>(to + i * 8) = v.v;
  }
}

// A tile's row and column numbers fit 32 bits with room for the tile.
bool numbers_fit(int64_t rows, int64_t experts, int64_t n, int64_t k, int64_t parts) {
  const int64_t most = int64_t(1) << 22;
  return rows > 0 && rows < (1 << 30) && n < most && k < most &&
         experts * ((n + kTile - 1) / kTile) * ((k + kTile - 1) / kTile) * parts < (int64_t(1) << 31);
}

// 16-byte addresses and strides, and whole pieces.
bool whole_pieces(const muon_weight_grad_args& p) {
  auto fine = [&](const void* base, int64_t stride, int64_t cols) {
    return reinterpret_cast<uintptr_t>(base) % 16 == 0 && cols % 8 == 0 && (p.rows <= 1 || stride % 8 == 0) && stride < (1 << 22);
  };
  return fine(p.dy, p.dy_stride, p.n) && fine(p.x, p.x_stride, p.k);
}

template <typename O>
hipError_t launch(const muon_weight_grad_args& p, const Dest& d, bool pieces, hipStream_t stream) {
  const int64_t tn = (p.n + kTile - 1) / kTile, tk = (p.k + kTile - 1) / kTile;
  if (pieces) {
    ex_weight_grad_tiled<O><<<256, 512, 0, stream>>>(p, d, (uint32_t)tn, (uint32_t)tk);
  } else {
    const int64_t sn = (p.n + 127) / 128, sk = (p.k + 127) / 128, tiles = p.num_experts * sn * sk * d.parts;
    ex_weight_grad<O><<<unsigned(tiles < (1 << 20) ? (tiles + 7) / 8 * 8 : 1 << 20), 256, 0, stream>>>(p, d, sn, sk);
  }
  return hipGetLastError();
}

}  // namespace

// Few tiles and many rows: the rows are split so that there are tiles for the 256 CUs, with 512 rows of
// the mean expert a part at least (eight stages, against one write and one read of the part: 4096 rows to one
// [1024, 1024] 33 us, with 256 rows 41, with 1024 39) and 32 parts at most (49152 rows to one [512, 512] 71 us
// with 48, 82 with 64).
int64_t weight_grad_parts(int64_t rows, int64_t num_experts, int64_t n, int64_t k) {
  const int64_t tiles = num_experts * ((n + kTile - 1) / kTile) * ((k + kTile - 1) / kTile);
  const int64_t want = tiles > 8 ? 256 / tiles : 32, most = rows / num_experts / 512;
  const int64_t parts = want < most ? want : most;
  return parts < 2 ? 1 : parts;
}

// Odd widths of 2^30 products or more have their rows copied to whole pieces first: 49152 rows of 1001 and 1001
// for 8 experts 230-258 us, 515 without, 4096 rows of 1001 and 515 45 and 61, 2000 of them 34 and 33, 777 24 and 15.
int64_t weight_grad_copy_bytes(int64_t rows, int64_t num_experts, int64_t n, int64_t k) {
  if (n % 8 == 0 && k % 8 == 0) return 0;
  if (!numbers_fit(rows, num_experts, n, k, weight_grad_parts(rows, num_experts, n, k)) || rows * n < (int64_t(1) << 30) / k) return 0;
  return rows * ((n + 7) / 8 + (k + 7) / 8) * 16;
}

hipError_t run_weight_grad(const muon_weight_grad_args& args, void* workspace, hipStream_t stream) {
  muon_weight_grad_args p = args;
  const int64_t n_parts = weight_grad_parts(p.rows, p.num_experts, p.n, p.k), part = p.num_experts * p.n * p.k;
  const bool f32 = p.dw_dtype == MUON_F32;
  float* parts = static_cast<float*>(workspace);
  bool pieces = numbers_fit(p.rows, p.num_experts, p.n, p.k, n_parts);
  if (weight_grad_copy_bytes(p.rows, p.num_experts, p.n, p.k)) {
    p.dy_stride = (p.n + 7) / 8 * 8;
    p.x_stride = (p.k + 7) / 8 * 8;
    bf16_t* dy = reinterpret_cast<bf16_t*>(static_cast<uint8_t*>(workspace) + weight_grad_parts_bytes(p.rows, p.num_experts, p.n, p.k));
    bf16_t* x = dy + p.rows * p.dy_stride;
    const int64_t wide = p.n > p.k ? p.n : p.k, need = (p.rows * ((wide + 7) / 8) + 255) / 256;
    ex_weight_grad_align<<<dim3(unsigned(need < (1 << 16) ? need : 1 << 16), 2), 256, 0, stream>>>(args, dy, x);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    p.dy = dy;
    p.x = x;
  } else {
    pieces = pieces && whole_pieces(p);
  }
  if (n_parts == 1) {
    const Dest d{p.dw, p.dw_stride, p.dw_matrix, 0, 1};
    return f32 ? launch<float>(p, d, pieces, stream) : launch<bf16_t>(p, d, pieces, stream);
  }
  const hipError_t err = launch<float>(p, Dest{parts, p.k, p.n * p.k, part, (int)n_parts}, pieces, stream);
  if (err != hipSuccess) return err;
  const int64_t blocks = (p.num_experts * p.n * ((p.k + 7) / 8) + 255) / 256;
  const unsigned grid = unsigned(blocks < (1 << 16) ? blocks : 1 << 16);
  if (f32) ex_weight_grad_join<float><<<grid, 256, 0, stream>>>(p, parts, (int)n_parts, part);
  else ex_weight_grad_join<bf16_t><<<grid, 256, 0, stream>>>(p, parts, (int)n_parts, part);
  return hipGetLastError();
}

}  // namespace muon
