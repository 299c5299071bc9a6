// Host checks shared by the C ABI files of the row and expert operators: sizes,
// types, and a call's buffers compared for overlap.  Not part of the public ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>
#include <utility>

#include "../../include/muon_block.h"

namespace muon {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int kMaxRegions = 12;

inline bool valid_dtype(int d) { return d == MUON_F32 || d == MUON_BF16; }
inline int64_t size_of(int d) {
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
inline bool overlap(const Rows& a, const Rows& b) {
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

inline muon_status check_dims(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1) return MUON_ERR_INVALID_ARG;
  if (rows > kMaxDim || cols > kMaxDim) return MUON_ERR_UNSUPPORTED;
  return MUON_OK;
}

inline muon_status hip_status(hipError_t e) { return e == hipSuccess ? MUON_OK : MUON_ERR_HIP; }
inline hipStream_t hip_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace muon
