// Device helpers of the row operators (gfx950, wave64): eight consecutive
// columns of a row per lane, the dropout generator, 8-bit rounding.
#pragma once
#include "block.h"
#include "common.h"

namespace muon {

// 16- and 8-byte vectors at any element's alignment: rows of odd strides
// start anywhere, and gfx950's global loads and stores take such addresses in
// one instruction.
typedef unsigned int u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef unsigned int u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

__device__ __forceinline__ void unpack8(const u32x4& v, float* f) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[2 * q] = __uint_as_float(v[q] << 16);
    f[2 * q + 1] = __uint_as_float(v[q] & 0xffff0000u);
  }
}

// Columns c .. c+7 of a row in their stored form, zeros from column `cols` on
// (c may lie past it): 4 registers of bf16 or 8 of fp32, so that loads can be
// in flight while the row before is worked on.  The row's last chunk is the
// row's last eight columns, moved down by get() and not before, since that
// waits for them ([16384, 4095] bf16: norm forward and backward 123 and 95 us,
// 191 and 161 with a load for each column behind its own test).
typedef uint16_t u16_any __attribute__((aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));

template <typename T> struct Chunk;
template <> struct Chunk<bf16_t> {
  u32x4 v;
  // elements n .. 7 to 0 .., zeros after them; n in 1 .. 7
  __device__ __forceinline__ void down(int n) {
    uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
    lo = n & 4 ? hi : lo;
    hi = n & 4 ? 0 : hi;
    const int s = (n & 3) * 16;
    lo = lo >> s | (hi << 1) << (63 - s);
    hi >>= s;
    v = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
  }
  template <class I>
  __device__ __forceinline__ void load(const bf16_t* row, I c, I cols) {
    if (cols >= 8) {   // one load for full chunks and the last
      v = u32x4{};
      if (c < cols) v = *reinterpret_cast<const u32x4_any*>(row + (c + 8 <= cols ? c : cols - 8));
    } else {   // the whole row, its last element first
      v = u32x4{};
      if (c > 0) return;
#pragma unroll 1
      for (int j = (int)cols - 1; j >= 0; --j)
        v = u32x4{v[0] << 16 | row[j], v[1] << 16 | v[0] >> 16, v[2] << 16 | v[1] >> 16, v[3] << 16 | v[2] >> 16};
    }
  }
  template <class I>
  __device__ __forceinline__ void get(float* f, I c, I cols) {
    settle(c, cols);
    values(f);
  }
  // get() in two: the shift once, the values as often as they are needed
  template <class I>
  __device__ __forceinline__ void settle(I c, I cols) {
    if (c < cols && c + 8 > cols && cols >= 8) down((int)(c + 8 - cols));
  }
  __device__ __forceinline__ void values(float* f) const { unpack8(v, f); }
};
template <> struct Chunk<float> {
  u32x4 a, b;
  __device__ __forceinline__ void down(int n) {
    const u32x4 z = {};
    if (n & 4) {
      a = b;
      b = z;
    }
    if (n & 2) {
      a = u32x4{a[2], a[3], b[0], b[1]};
      b = u32x4{b[2], b[3], 0, 0};
    }
    if (n & 1) {
      a = u32x4{a[1], a[2], a[3], b[0]};
      b = u32x4{b[1], b[2], b[3], 0};
    }
  }
  template <class I>
  __device__ __forceinline__ void load(const float* row, I c, I cols) {
    if (cols >= 8) {
      a = u32x4{};
      b = u32x4{};
      if (c < cols) {
        const float* p = row + (c + 8 <= cols ? c : cols - 8);
        a = *reinterpret_cast<const u32x4_any*>(p);
        b = *reinterpret_cast<const u32x4_any*>(p + 4);
      }
    } else {
      a = u32x4{};
      b = u32x4{};
      if (c > 0) return;
#pragma unroll 1
      for (int j = (int)cols - 1; j >= 0; --j) {
        b = u32x4{a[3], b[0], b[1], b[2]};
        a = u32x4{__float_as_uint(row[j]), a[0], a[1], a[2]};
      }
    }
  }
  template <class I>
  __device__ __forceinline__ void get(float* f, I c, I cols) {
    settle(c, cols);
    values(f);
  }
  template <class I>
  __device__ __forceinline__ void settle(I c, I cols) {
    if (c < cols && c + 8 > cols && cols >= 8) down((int)(c + 8 - cols));
  }
  __device__ __forceinline__ void values(float* f) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] = __uint_as_float(a[j]);
      f[j + 4] = __uint_as_float(b[j]);
    }
  }
};

template <typename T, class I>
__device__ __forceinline__ void load8(const T* row, I c, I cols, float* f) {
  Chunk<T> k;
  k.load(row, c, cols);
  k.get(f, c, cols);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return (uint32_t)f2bf(lo) | ((uint32_t)f2bf(hi) << 16);
}

// The same columns rounded and stored; those from `cols` on are left alone (the
// row's last chunk goes by pieces of 4, 2 and 1).
template <class I>
__device__ __forceinline__ void store8(bf16_t* row, I c, I cols, const float* f) {
  u32x4 v;
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = pack_bf16(f[2 * q], f[2 * q + 1]);
  if (c + 8 <= cols) {
    *reinterpret_cast<u32x4_any*>(row + c) = v;
  } else if (c < cols) {
    const int n = (int)(cols - c);
    bf16_t* p = row + c;
    if (n & 4) {
      *reinterpret_cast<u32x2_any*>(p) = u32x2_any{v[0], v[1]};
      v[0] = v[2];
      v[1] = v[3];
      p += 4;
    }
    if (n & 2) {
      *reinterpret_cast<u32_any*>(p) = v[0];
      v[0] = v[1];
      p += 2;
    }
    if (n & 1) *p = (bf16_t)v[0];
  }
}
template <class I>
__device__ __forceinline__ void store8(float* row, I c, I cols, const float* f) {
  u32x4 a, b;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    a[j] = __float_as_uint(f[j]);
    b[j] = __float_as_uint(f[j + 4]);
  }
  if (c + 8 <= cols) {
    *reinterpret_cast<u32x4_any*>(row + c) = a;
    *reinterpret_cast<u32x4_any*>(row + c + 4) = b;
  } else if (c < cols) {
    const int n = (int)(cols - c);
    float* p = row + c;
    if (n & 4) {
      *reinterpret_cast<u32x4_any*>(p) = a;
      a = b;
      p += 4;
    }
    if (n & 2) {
      *reinterpret_cast<u32x2_any*>(p) = u32x2_any{a[0], a[1]};
      a[0] = a[2];
      p += 2;
    }
    if (n & 1) *p = __uint_as_float(a[0]);
  }
}

// f / scale as fp32 divides (but for one in a million, an ulp off): 1 / scale
// in two floats, the first a little too small so that the second is positive
// and -0 keeps its sign.  2^-126 <= scale < 2^120, or infinite: then finite
// elements become 0 and infinite ones NaN.  One multiplication more an
// element than by the reciprocal alone, which moves a few in a million by an
// 8-bit step: norm of [4096, 8192] to e4m3 45.6 us against 45.4, of
// [32768, 1024] by groups of 32 24.2 against 23.6.
__device__ __forceinline__ void quotients8(float* f, float scale) {
  const float inv = __builtin_amdgcn_rcpf(scale) * (1.f - 0x1p-22f);
  const float rest = scale < HUGE_VALF ? __builtin_fmaf(-scale, inv, 1.f) * inv : 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = __builtin_fmaf(f[j], inv, f[j] * rest);
}

// Eight values divided by their scale in an 8-bit format, rounded to nearest
// even.  They are at most FMAX (1 + 2^-22) in magnitude, which rounds to FMAX,
// or NaN, which stays one: there is nothing to limit.
template <bool E5M2, class I>
__device__ __forceinline__ void store8_8bit(uint8_t* row, I c, I cols, const float* f) {
  u32x2_any w;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    int p = 0;
    if constexpr (E5M2) {
      p = __builtin_amdgcn_cvt_pk_bf8_f32(f[4 * q], f[4 * q + 1], p, false);
      p = __builtin_amdgcn_cvt_pk_bf8_f32(f[4 * q + 2], f[4 * q + 3], p, true);
    } else {
      p = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * q], f[4 * q + 1], p, false);
      p = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * q + 2], f[4 * q + 3], p, true);
    }
    w[q] = (uint32_t)p;
  }
  if (c + 8 <= cols) {
    *reinterpret_cast<u32x2_any*>(row + c) = w;
  } else if (c < cols) {
    const int n = (int)(cols - c);
    uint8_t* p = row + c;
    uint32_t x = w[0];
    if (n & 4) {
      *reinterpret_cast<u32_any*>(p) = x;
      x = w[1];
      p += 4;
    }
    if (n & 2) {
      *reinterpret_cast<u16_any*>(p) = (uint16_t)x;
      x >>= 16;
      p += 2;
    }
    if (n & 1) *p = (uint8_t)x;
  }
}

// Ten rounds of Philox4x32 (Salmon et al., 2011).
__device__ __forceinline__ void philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1,
                                       uint32_t* out) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)b;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  out[0] = c0;
  out[1] = c1;
  out[2] = c2;
  out[3] = c3;
}

// Seed and offset for this launch: uniform loads where they are on the device.
__device__ __forceinline__ void drop_seed(const Drop& d, uint64_t& seed, uint64_t& offset) {
  seed = d.dev ? d.dev[0] : d.seed;
  offset = d.dev ? d.dev[1] : d.offset;
}

// D on columns c .. c+7 (c a multiple of 8) of row r, in place.
__device__ __forceinline__ void drop8(const Drop& d, uint64_t seed, uint64_t offset, int64_t r, int64_t c, float* f) {
  uint32_t w[4];
  philox((uint32_t)(c >> 3), (uint32_t)r, (uint32_t)offset, (uint32_t)(offset >> 32), (uint32_t)seed,
         (uint32_t)(seed >> 32), w);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[2 * q] = (w[q] & 0xffffu) >= d.t ? f[2 * q] * d.up : 0.f;
    f[2 * q + 1] = (w[q] >> 16) >= d.t ? f[2 * q + 1] * d.up : 0.f;
  }
}

// Value of another lane of the same row; the row's lanes are active.
template <int CTRL>
__device__ __forceinline__ int dpp(int v) { return __builtin_amdgcn_mov_dpp(v, CTRL, 0xf, 0xf, true); }
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) { return (uint32_t)dpp<CTRL>((int)v); }
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)dpp<CTRL>((uint32_t)(b >> 32)) << 32 | dpp<CTRL>((uint32_t)b));
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) { return __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(int, v))); }

// f over the LPT lanes of a row, the result in each of them: two exchanges
// within four lanes, then mirrored halves of 8 and 16 lanes, then across the
// wave.  f is commutative, so that both sides of an exchange agree.
template <int LPT, class V, class F>
__device__ __forceinline__ V over_row(V v, F f) {
  v = f(v, dpp<0xB1>(v));                              // lane ^ 1
  v = f(v, dpp<0x4E>(v));                              // lane ^ 2
  if constexpr (LPT >= 8) v = f(v, dpp<0x141>(v));     // lane 7 - l of eight
  if constexpr (LPT >= 16) v = f(v, dpp<0x140>(v));    // lane 15 - l of sixteen
  if constexpr (LPT >= 32) v = f(v, __shfl_xor(v, 16, WAVE));
  if constexpr (LPT >= 64) v = f(v, __shfl_xor(v, 32, WAVE));
  return v;
}
__device__ __forceinline__ float max_f(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float add_f(float a, float b) { return a + b; }

// Sum / maximum over a workgroup of up to 8 waves, in wave order.  `lds` holds
// two sets of 8 floats, zero at first; `turn` alternates 0 and 1 from call to
// call on the same set, so that one barrier a call is enough: a wave that
// writes a set again has passed the barrier of the call in between, and with
// it every wave its reads of that set.
struct alignas(16) GroupRed {
  float s[2][8];
};
__device__ __forceinline__ void red_init(GroupRed& g) {
  if (threadIdx.x < 16) g.s[threadIdx.x >> 3][threadIdx.x & 7] = 0.f;
  __syncthreads();
}
__device__ __forceinline__ float group_sum(float v, GroupRed& g, int turn) {
  v = over_row<WAVE>(v, add_f);
  if ((threadIdx.x & (WAVE - 1)) == 0) g.s[turn][threadIdx.x / WAVE] = v;
  __syncthreads();
  const f32x4 a = *reinterpret_cast<const f32x4*>(g.s[turn]), b = *reinterpret_cast<const f32x4*>(g.s[turn] + 4);
  return ((a[0] + a[1]) + (a[2] + a[3])) + ((b[0] + b[1]) + (b[2] + b[3]));
}
__device__ __forceinline__ float group_max(float v, GroupRed& g, int turn) {   // v >= 0
  v = over_row<WAVE>(v, max_f);
  if ((threadIdx.x & (WAVE - 1)) == 0) g.s[turn][threadIdx.x / WAVE] = v;
  __syncthreads();
  const f32x4 a = *reinterpret_cast<const f32x4*>(g.s[turn]), b = *reinterpret_cast<const f32x4*>(g.s[turn] + 4);
  return fmaxf(fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])), fmaxf(fmaxf(b[0], b[1]), fmaxf(b[2], b[3])));
}

}  // namespace muon
