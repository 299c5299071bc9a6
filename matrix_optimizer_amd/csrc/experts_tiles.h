// Device helpers of the experts' matrix kernels: the runs of rows that the
// offsets give, and rows of any alignment in pieces of 16 bytes.
#pragma once
#include "experts.h"
#include "rows.h"

namespace muon {

// Rows lo .. hi-1 of expert e; offsets outside the buffer are taken to its nearer end.
__device__ __forceinline__ void run_of(const int32_t* offsets, int e, int rows, int& lo, int& hi) {
  if (!offsets || rows == 0) {
    lo = 0;
    hi = rows;
    return;
  }
  lo = min(max(offsets[e], 0), rows);
  hi = min(max(offsets[e + 1], lo), rows);
}

// A product's tile: BM rows of one expert's run by BN columns.
struct ExpertTile {
  int e, row0, rows;   // the expert, the tile's first row and how many of its rows are the expert's
  int tn;              // tile along the columns
};

// Tile number `index` of the launch, or false from the last one on.  An expert's tiles are
// consecutive, those of the same columns first.  Every lane of a wave takes part; the result
// is uniform.
__device__ __forceinline__ bool find_tile(const int32_t* offsets, int experts, int rows, int bm, uint32_t tiles_n,
                                          uint32_t index, ExpertTile& t) {
  const int lane = threadIdx.x & (WAVE - 1);
  uint32_t before = 0;
  for (int e0 = 0; e0 < experts; e0 += WAVE) {
    const int e = e0 + lane;
    int lo = 0, hi = 0;
    if (e < experts) run_of(offsets, e, rows, lo, hi);
    const uint32_t tm = ((uint32_t)(hi - lo) + bm - 1) / (uint32_t)bm;
    uint32_t sum = tm * tiles_n;
#pragma unroll
    for (int d = 1; d < WAVE; d <<= 1) {
      const uint32_t o = __shfl_up(sum, d, WAVE);
      if (lane >= d) sum += o;
    }
    const uint32_t total = __builtin_amdgcn_readlane(sum, WAVE - 1);
    if (index < before + total) {
      const unsigned long long past = __ballot(index < before + sum);
      const int at = __ffsll((long long)past) - 1;
      const uint32_t own = __builtin_amdgcn_readlane(tm, at), end = __builtin_amdgcn_readlane(sum, at);
      const uint32_t local = index - (before + end - own * tiles_n);
      const uint32_t n = __builtin_amdgcn_readfirstlane(local / own), m = local - n * own;
      if (n >= tiles_n) return false;   // overlapping runs of more tiles than 32 bits number
      t.e = e0 + at;
      t.tn = (int)n;
      t.row0 = __builtin_amdgcn_readlane(lo, at) + (int)m * bm;
      t.rows = min((int)__builtin_amdgcn_readlane(hi, at) - t.row0, bm);
      return true;
    }
    before += total;
  }
  return false;
}

// Tiles of the launch; every lane of a wave takes part.
__device__ __forceinline__ uint32_t count_tiles(const int32_t* offsets, int experts, int rows, int bm, uint32_t tiles_n) {
  uint32_t sum = 0;
  for (int e = threadIdx.x & (WAVE - 1); e < experts; e += WAVE) {
    int lo, hi;
    run_of(offsets, e, rows, lo, hi);
    sum += ((uint32_t)(hi - lo) + bm - 1) / (uint32_t)bm * tiles_n;
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, WAVE);
  return __builtin_amdgcn_readfirstlane(sum);
}

// Where the last run ends: rows from there on belong to nobody.  Every lane of a wave takes part.
__device__ __forceinline__ int end_of_runs(const int32_t* offsets, int experts, int rows) {
  if (!offsets) return rows;
  int end = 0;
  for (int e = threadIdx.x & (WAVE - 1); e < experts; e += WAVE) {
    int lo, hi;
    run_of(offsets, e, rows, lo, hi);
    if (lo < hi) end = max(end, hi);
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) end = max(end, __shfl_xor(end, d, WAVE));
  return __builtin_amdgcn_readfirstlane(end);
}

// Bytes k .. k+15 of a row of K bytes, zeros from K on (k may lie past it).
__device__ __forceinline__ u32x4 load16(const uint8_t* row, int64_t k, int64_t K) {
  if (k + 16 <= K) return *reinterpret_cast<const u32x4_any*>(row + k);
  u32x4 v = {};
  if (k >= K) return v;
  uint64_t lo, hi;
  if (K >= 16) {   // the row's last 16 bytes moved down
    v = *reinterpret_cast<const u32x4_any*>(row + K - 16);
    lo = (uint64_t)v[1] << 32 | v[0];
    hi = (uint64_t)v[3] << 32 | v[2];
    const int n = (int)(k + 16 - K);   // 1 .. 15
    if (n & 8) {
      lo = hi;
      hi = 0;
    }
    const int s = (n & 7) * 8;
    lo = lo >> s | (hi << 1) << (63 - s);
    hi >>= s;
  } else {         // k is 0: the whole row
    lo = hi = 0;
#pragma unroll 1
    for (int j = (int)K - 1; j >= 0; --j) {
      hi = hi << 8 | lo >> 56;
      lo = lo << 8 | row[j];
    }
  }
  return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

}  // namespace muon
