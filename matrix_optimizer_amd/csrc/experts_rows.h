// Device helpers of the expert operators' row kernels: rows of up to 256
// lanes, eight columns a lane and step, sixteen lanes to a group of 128.
#pragma once
#include "experts.h"
#include "rows.h"

namespace muon {

// How a launch of 256 threads lays rows out: 2^log_lanes lanes a row, `split`
// workgroups along the columns (grid.y).
struct RowLayout {
  int log_lanes;
  unsigned gx, gy;
};

// Lanes enough for a row's chunks, from 16 (a group of 128 columns) to 256; few rows are split over
// workgroups along their columns as well, until there are about two for each of the 256 CUs.
inline RowLayout row_layout(int64_t rows, int64_t chunks) {
  RowLayout l{4, 1, 1};
  while (l.log_lanes < 8 && (int64_t(1) << l.log_lanes) < chunks) ++l.log_lanes;
  const int64_t per = 256 >> l.log_lanes, groups = (rows + per - 1) / per, most = 1 << 20;
  l.gx = unsigned(groups < most ? groups : most);
  const int64_t steps = (chunks + 255) / 256, want = groups >= 512 ? 1 : (512 + groups - 1) / groups;
  l.gy = unsigned(want < steps ? want : steps);
  return l;
}

// Scale of a group of 8-bit values whose largest magnitude is `most` (a quotient: it is formed once a
// group) and the values divided by it.
__device__ __forceinline__ float group_scale(float most, bool e5) {
  return most == 0.f ? 1.f : fmaxf(most / (e5 ? 57344.f : 448.f), 0x1p-126f);
}

// Largest magnitude of eight values, NaN left out.
__device__ __forceinline__ float most8(const float* f) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
  return m;
}

// v / scale of columns c .. c+7 stored in 8 bits; v is overwritten.
__device__ __forceinline__ void store_eight(uint8_t* row, int64_t c, int64_t cols, float* v, float scale, bool e5) {
  quotients8(v, scale);
  if (e5) store8_8bit<true>(row, c, cols, v);
  else store8_8bit<false>(row, c, cols, v);
}

// Rows in use: all, or as many as the device says.
__device__ __forceinline__ int64_t rows_in_use(int64_t rows, const int32_t* used) {
  if (!used) return rows;
  const int64_t u = *used;
  return u < 0 ? 0 : u < rows ? u : rows;
}

}  // namespace muon
