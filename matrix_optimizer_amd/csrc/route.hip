// Routing to experts: the choice and its weights, the gradient of the logits,
// the order of the routed pairs, the update of the balance bias.
#include <algorithm>
#include <float.h>

#include <type_traits>

#include "internal.h"
#include "rows.h"

namespace muon {
namespace {

constexpr int RT = 256;                 // threads of a workgroup: four waves, a row each
constexpr int RW = RT / WAVE;
constexpr double kOut = -HUGE_VAL;      // rank of an expert that may not be chosen
constexpr int kNone = INT32_MIN;        // the same as an ordered key

// A row's experts over LPT lanes, NC chunks of eight to a lane: expert
// (i LPT + t) 8 + j is element 8 i + j of the t-th lane.  64 / LPT rows a wave.

__device__ __forceinline__ int max_i(int a, int b) { return a > b ? a : b; }
__device__ __forceinline__ double add_d(double a, double b) { return a + b; }
__device__ __forceinline__ double max_d(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ uint32_t min_u(uint32_t a, uint32_t b) { return a < b ? a : b; }

// Floats (no NaN) in the order of integers.
__device__ __forceinline__ int key_of(float v) {
  const int b = __builtin_bit_cast(int, v + 0.f);   // -0 and 0 are one value
  return b ^ ((b >> 31) & 0x7fffffff);
}

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, WAVE);
  return v;
}

// Logit as the definition reads it: NaN closed, +inf the largest finite value.
// fmaxf of a NaN and a number is the number.
__device__ __forceinline__ float read_logit(float l) { return fminf(fmaxf(l, -HUGE_VALF), FLT_MAX); }

// One row by the whole wave with every score in 64 bits.  It runs seldom, and
// then others wait for it: its values (E ranks, G group values, G marks) are
// in shared memory, so that it takes few of the kernel's registers.
template <typename T>
__device__ __forceinline__ void route_row_64(const muon_route_spec& s, const muon_route_args& a, int64_t r,
                                             double* rank) {
  const int lane = threadIdx.x & (WAVE - 1);
  const int E = (int)a.num_experts, K = s.top_k, G = s.groups, n = E / G;
  const bool soft = s.score == MUON_SCORE_SOFTMAX;
  double* of_l = rank + E;
  double* in_l = of_l + G;
  const T* row = static_cast<const T*>(a.logits) + r * a.logits_stride;
  float top = -HUGE_VALF;
  double total = 1.0;
  if (soft) {
#pragma unroll 4
    for (int e = lane; e < E; e += WAVE) top = fmaxf(top, read_logit(ld_as_f32(row, e)));
    top = over_row<WAVE>(top, max_f);
    total = 0.0;
#pragma unroll 1
    for (int e = lane; e < E; e += WAVE) {
      const float l = read_logit(ld_as_f32(row, e));
      if (l > -HUGE_VALF) total += exp((double)l - (double)top);
    }
    total = wave_sum64(total);
  }
  wave_sync();
#pragma unroll 1
  for (int e = lane; e < E; e += WAVE) {
    const double l = (double)read_logit(ld_as_f32(row, e));
    const double x = exp(soft ? l - (double)top : -l);
    const double v = (soft ? x / total : 1.0 / (1.0 + x)) + (a.bias ? (double)a.bias[e] : 0.0);
    rank[e] = l > kOut ? v : kOut;
  }
  wave_sync();
  if (G > 1) {
    // the lanes shared out over the groups, each over its part of a group's experts
    int share = WAVE;
    while (share > 1 && share * G > WAVE) share >>= 1;
#pragma unroll 1
    for (int g0 = 0; g0 < G; g0 += WAVE / share) {
      const int g = g0 + lane / share;
      double b1 = kOut, b2 = kOut;
      if (g < G) {
#pragma unroll 4
        for (int j = lane & (share - 1); j < n; j += share) {
          const double v = rank[g * n + j];
          b2 = fmax(b2, fmin(b1, v));
          b1 = fmax(b1, v);
        }
      }
      for (int o = share >> 1; o >= 1; o >>= 1) {
        const double o1 = __shfl_xor(b1, o, WAVE), o2 = __shfl_xor(b2, o, WAVE);
        b2 = fmax(fmin(b1, o1), fmax(b2, o2));
        b1 = fmax(b1, o1);
      }
      if (g < G && (lane & (share - 1)) == 0) of_l[g] = s.group_top == 2 && b2 > kOut ? b1 + b2 : b1;
    }
    wave_sync();
#pragma unroll 1
    for (int g = lane; g < G; g += WAVE) {   // a group stays if fewer than top_groups are before it
      const double mine = of_l[g];
      int before = 0;
#pragma unroll 4
      for (int q = 0; q < G; ++q) before += of_l[q] > mine || (of_l[q] == mine && q < g);
      in_l[g] = before < s.top_groups ? 1.0 : 0.0;
    }
    wave_sync();
  }
#pragma unroll 1
  for (int e = lane; e < E; e += WAVE) {
    if (G > 1 && in_l[e / n] == 0.0) rank[e] = kOut;
    if (!a.bias && rank[e] > kOut) rank[e] = (double)read_logit(ld_as_f32(row, e));
  }
  wave_sync();
  int chosen = -1;   // lane k: the k-th expert
#pragma unroll 1
  for (int k = 0; k < K; ++k) {
    double v = kOut;
#pragma unroll 4
    for (int e = lane; e < E; e += WAVE) v = fmax(v, rank[e]);
    v = over_row<WAVE>(v, max_d);
    if (!(v > kOut)) break;   // uniform: nothing is left
    int at = 0;               // the first expert of that rank: 64 at a time, in order
    for (int e0 = 0; e0 < E; e0 += WAVE) {
      const uint64_t m = __ballot(e0 + lane < E && rank[e0 + lane] == v);
      if (m) {
        at = e0 + __ffsll((unsigned long long)m) - 1;
        break;
      }
    }
    if (lane == k) chosen = at;
    wave_sync();
    if (lane == 0) rank[at] = kOut;
    wave_sync();
  }
  // weights from log s, lane k its own
  double ls = kOut;
  if (chosen >= 0) {
    const double lc = (double)read_logit(ld_as_f32(row, chosen));
    ls = soft ? lc - (double)top : fmin(lc, 0.0) - log1p(exp(-fabs(lc)));   // log sigmoid
  }
  double w = 0.0;
  if (s.renormalise) {
    const double m = over_row<WAVE>(ls, max_d);
    const double e = chosen >= 0 ? exp(ls - m) : 0.0;
    const double sum = wave_sum64(e);
    if (chosen >= 0) w = e / sum;
  } else if (chosen >= 0) {
    w = exp(ls) / total;
  }
  if (lane < K) {
    a.experts[r * K + lane] = chosen;
    a.weights[r * K + lane] = (float)(w * (double)s.scale);
  }
  wave_sync();
}

// A score: exp(l - top), the difference's rounding made good,
// or sigmoid(l) without loss at either end.
__device__ __forceinline__ float slot_score(float l, float top, bool soft) {
  if (soft) {
    const float d = l - top, back = d + top;
    if (!(d > -150.f)) return 0.f;   // also where l - top overflows
    const float lost = (l - back) + ((back - d) - top);   // l - top = d + lost, exactly
    return expf(d) * (1.f + lost);
  }
  const float e = expf(-fabsf(l));
  return (l < 0.f ? e : 1.f) / (1.f + e);
}

// 1 - sigmoid(l) without cancellation.
__device__ __forceinline__ float one_less_sigmoid(float l) {
  const float e = expf(-fabsf(l));
  return (l > 0.f ? e : 1.f) / (1.f + e);
}

// Load of a row's logits, -inf from E on.
template <typename T, int LPT, int NC>
__device__ __forceinline__ void load_logits(const T* row, int E, int t, float* l) {
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (i * LPT + t) * 8;
    load8(row, c, E, l + 8 * i);
#pragma unroll
    for (int j = 0; j < 8; ++j) l[8 * i + j] = read_logit(l[8 * i + j]);
  }
  if (E < LPT * NC * 8) {
#pragma unroll
    for (int i = 0; i < 8 * NC; ++i)
      if (((i / 8) * LPT + t) * 8 + i % 8 >= E) l[i] = -HUGE_VALF;
  }
}

// Experts that the choice of a row may come down to: all of up to 32, else
// the top_k (at most 32) and a few whose values are too near the last's.
template <int LPT> struct Near {
  static constexpr int CAP = LPT == 4 ? 32 : 40;
};

// Shared memory of a wave in 4-byte words: for `rows` rows side by side E
// values, G group values and G marks, later `cap` times a 64-bit value, a
// score and a place in the new order; or route_row_64's for one row.
__host__ __device__ constexpr int route_wave_words(int E, int G, int rows, int cap) {
  const int one = rows * (E + 2 * G), two = 2 * (E + 2 * G), three = rows * cap * 3;
  const int most = one > two ? one : two;
  return ((most > three ? most : three) + 1) & ~1;
}

// The experts of a row and their weights.
//
// The choice is defined on scores in 64 bits; forming and sorting them so took
// 275 us for 32768 rows of 256 experts in 8 groups, of which the bytes are 4;
// now 20 to 22 us by sigmoid with a bias (16 without groups; by softmax 27 and
// 20; 11 without bias and groups), 14.7 of them vector instructions, 1060 a wave.
// What bounds it is the instructions of the choice, and at the end the longest
// wave, so a row gets 4 to 64 lanes (16 for 256 experts, four rows a wave),
// and the choice is made in three grades, each for the rows that the one
// before leaves open:
//   1. one 32-bit number holds 22 bits of a value and the expert, so that
//      numbers differ and the next largest is the least of m - 1 - number as
//      unsigned: 1.5 instructions an expert, nothing is marked.  bf16 logits
//      fit whole; other values must differ in those bits (scores by their
//      error), which most rows' do;
//   2. the experts taken, and those after them that their bits do not set
//      apart, in 64 bits, a lane each, and put in order by counting;
//   3. route_row_64.
// Logits order themselves exactly: without bias and groups no score is needed
// to choose.
template <typename T, int LPT, int NC>
__global__ __launch_bounds__(RT, 5) void route_fwd(muon_route_spec s, muon_route_args a) {
  extern __shared__ double lds_all[];
  constexpr int V = 8 * NC, RPW = WAVE / LPT, CAP = Near<LPT>::CAP;
  __shared__ int chosen_all[RT / LPT][CAP];
  const int lane = threadIdx.x & (WAVE - 1), wave = threadIdx.x / WAVE, t = lane & (LPT - 1);
  const int E = (int)a.num_experts, K = s.top_k, G = s.groups;
  float* wave_lds = reinterpret_cast<float*>(lds_all) + (size_t)wave * route_wave_words(E, G, RPW, CAP);
  int* chosen = chosen_all[threadIdx.x / LPT];
  const bool soft = s.score == MUON_SCORE_SOFTMAX;
  const bool scored = a.bias || G > 1;                 // the choice reads scores
  const bool need_z = soft && (scored || a.scores || !s.renormalise);
  // one tile of rows a workgroup: in a loop over tiles the compiler keeps every
  // address and bias across it, 100 registers more
  const int64_t tile = blockIdx.y * (int64_t)gridDim.x + blockIdx.x;
  if (tile * RW * RPW >= a.rows) return;
  // every lane stays to the end: rows past the last repeat it and store nothing
  const int64_t want = (tile * RW + wave) * RPW + lane / LPT;
  const bool live = want < a.rows;
  const int64_t r = live ? want : a.rows - 1;
  const bool masked = a.token_mask && a.token_mask[r] == 0;
  const T* row = static_cast<const T*>(a.logits) + r * a.logits_stride;
  float l[V];
  load_logits<T, LPT, NC>(row, E, t, l);
  float top = l[0], least = l[0];
#pragma unroll
  for (int i = 1; i < V; ++i) least = fminf(least, l[i]);
  const bool shut = __any(!(least > -HUGE_VALF));   // an expert of the wave's rows is closed
  if (soft) {
#pragma unroll
    for (int i = 1; i < V; ++i) top = fmaxf(top, l[i]);
    top = over_row<LPT>(top, max_f);
  }
  float z = 1.f;
  float v[V];            // what is ranked; -inf: may not be chosen
  // Bound on the error of the difference of two scores.  Sigmoid: the fast exp
  // is off by (2 |l| + 2) 2^-24, which enters with s (1 - s), the sum and the
  // reciprocal by 3 2^-24: below 2^-22 each.  Softmax: (2 d + 2) 2^-24 e^-d for
  // the exp, so at most 16 2^-24 of the sum (the mean d is at most log E), at
  // most 20 roundings in a row in the sum, which two scores share, 3 after:
  // below 2^-18 of the largest score for the difference.
  float tol = 0x1p-21f;
  if (scored || a.scores || need_z) {
    const bool fine = a.scores || !s.renormalise;   // results, not only the choice, come of these
    if (soft) {
      z = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[i] = !(l[i] > -HUGE_VALF) ? 0.f : fine ? slot_score(l[i], top, true) : __expf(l[i] - top);
        z += v[i];
      }
      z = over_row<LPT>(z, add_f);
      const float inv = z > 0.f ? 1.f / z : 0.f;
      tol = 0x1p-18f * inv;
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] *= inv;
    } else if (a.scores) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = 1.f / (1.f + expf(-l[i]));
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = __builtin_amdgcn_rcpf(1.f + __expf(-l[i]));
    }
    if (a.scores && live) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = masked ? 0.f : v[8 * i + j];
        const int c = (i * LPT + t) * 8;
        if (c < E) store8(a.scores + r * E, c, E, o);
      }
    }
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float b[8];
        load8(a.bias, (i * LPT + t) * 8, E, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[8 * i + j] += b[j];
      }
    }
    if (shut) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = l[i] > -HUGE_VALF ? v[i] : -HUGE_VALF;
    }
  }
  bool unsure = false;   // grade 3
  bool out[NC] = {};     // whole chunks whose group does not stay
  bool single = shut;    // some v are -inf
  if (G > 1) {
    float* by_l = wave_lds + (size_t)(lane / LPT) * (E + 2 * G);
    float* of_l = by_l + E;
    int* in_l = reinterpret_cast<int*>(of_l + G);
    const int n = E / G, span = n / 8;
    float size = 0.f;   // the row's largest |b1| + |b2|, the terms of a value
    auto value = [&](float b1, float b2) {
      if (b1 > -HUGE_VALF) size = fmaxf(size, fabsf(b1) + (b2 > -HUGE_VALF ? fabsf(b2) : 0.f));
      return s.group_top == 2 && b2 > -HUGE_VALF ? b1 + b2 : b1;
    };
    // groups of 8 span experts, span a power of two up to a row's lanes: the
    // same chunk of `span` neighbouring lanes, whose two best meet by exchange
    const bool lanes = n % 8 == 0 && (span & (span - 1)) == 0 && span <= LPT;
    if (lanes) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float b1 = -HUGE_VALF, b2 = -HUGE_VALF;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          b2 = fmaxf(b2, fminf(b1, v[8 * i + j]));
          b1 = fmaxf(b1, v[8 * i + j]);
        }
        auto meet = [&](float o1, float o2) {
          b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
          b1 = fmaxf(b1, o1);
        };
        if (span > 1) meet(dpp<0xB1>(b1), dpp<0xB1>(b2));
        if (span > 2) meet(dpp<0x4E>(b1), dpp<0x4E>(b2));
        if (span > 4) meet(dpp<0x141>(b1), dpp<0x141>(b2));
        if (span > 8) meet(dpp<0x140>(b1), dpp<0x140>(b2));
        if (span > 16) meet(__shfl_xor(b1, 16, WAVE), __shfl_xor(b2, 16, WAVE));
        if (span > 32) meet(__shfl_xor(b1, 32, WAVE), __shfl_xor(b2, 32, WAVE));
        const int g = (i * LPT + t) / span;
        const float of = value(b1, b2);
        if ((t & (span - 1)) == 0 && g < G) of_l[g] = of;
      }
    } else {   // a lane a group, over its experts in shared memory
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = ((i / 8) * LPT + t) * 8 + i % 8;
        if (e < E) by_l[e] = v[i];
      }
      wave_sync();
      for (int g = t; g < G; g += LPT) {
        float b1 = -HUGE_VALF, b2 = -HUGE_VALF;
        for (int j = 0; j < n; ++j) {
          const float x = by_l[g * n + j];
          b2 = fmaxf(b2, fminf(b1, x));
          b1 = fmaxf(b1, x);
        }
        of_l[g] = value(b1, b2);
      }
    }
    wave_sync();
    // How near two values may be: their scores' part is 2 tol; a value is off by
    // 2^-24 of `size` for its sum, by as much again where a bias is added to its
    // terms, the other value likewise, and the comparison rounds once.  (Large
    // biases of opposite signs leave a small value with a large error.)
    const float far = 2.f * tol + (a.bias ? 0x1p-21f : 0x1p-22f) * over_row<LPT>(size, max_f);
    // a group is in if fewer than top_groups may be before it, out if as many
    // surely are; one without an open expert is of no matter
    for (int g = t; g < G; g += LPT) {
      const float mine = of_l[g];
      int sure = 0, may = 0;
      if (mine > -HUGE_VALF) {
        for (int q = 0; q < G; ++q) {
          const float x = of_l[q];
          sure += x > mine + far;
          may += x >= mine - far;
        }
        unsure |= may > s.top_groups && sure < s.top_groups;   // may counts the group itself
      }
      in_l[g] = sure < s.top_groups;
    }
    wave_sync();
    if (!a.bias) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = l[i];
    }
    if (lanes) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int g = (i * LPT + t) / span;
        out[i] = g < G && !in_l[g];
      }
    } else {
      single = true;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = ((i / 8) * LPT + t) * 8 + i % 8;
        if (e < E && !in_l[e / n]) v[i] = -HUGE_VALF;
      }
    }
  } else if (!a.bias) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = l[i];
  }

  // grade 1
  constexpr int kIndex = MUON_ROUTE_MAX_EXPERTS - 1, kLow = 1 - (1 << 21);
  const bool whole = !a.bias && sizeof(T) == 2;
  bool open = false;     // grade 2
  int cands = 0;         // experts in `chosen`, more than K where the last's value is not apart
  {
    int num[V];
    int m = kNone;
    // 22 bits of a value: a bf16 logit's ordered key, or steps below the
    // largest, of 2^-20 in a range of 2 for scores and of 2^-17 in 16 for
    // logits; values are in order where their steps differ, and scores where
    // these differ by `apart`
    const int low = (~t & (LPT - 1)) * 8;   // 1023 - e in bits: those of t, chunk and element reversed
    int apart = 0;
    if (whole) {
#pragma unroll
      for (int i = 0; i < V; ++i) num[i] = key_of(v[i]) & ~kIndex;
    } else {
      float most = v[0];
#pragma unroll
      for (int i = 1; i < V; ++i) most = fmaxf(most, v[i]);
      most = over_row<LPT>(most, max_f);
      const float by = a.bias ? 0x1p20f : 0x1p17f;
      if (a.bias) apart = (int)fminf(2.f + by * (tol + 0x1p-22f * (fabsf(most) + 2.f)), 0x1p22f);
#pragma unroll
      for (int i = 0; i < V; ++i)   // v - most in steps, rounded once; never above 0
        num[i] = (int)__builtin_amdgcn_fmed3f(__builtin_fmaf(v[i], by, -most * by), (float)kLow, 0.f) * (kIndex + 1);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      constexpr int upper = kIndex & ~(LPT * 8 - 1);
      num[i] = num[i] | low | ((upper - (i / 8) * LPT * 8) + (7 - i % 8));
    }
    if (single) {
#pragma unroll
      for (int i = 0; i < V; ++i) num[i] = v[i] > -HUGE_VALF ? num[i] : kNone;
    }
    if (G > 1) {
#pragma unroll
      for (int i = 0; i < V; ++i) num[i] = out[i / 8] ? kNone : num[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) m = max_i(m, num[i]);
    m = over_row<LPT>(m, max_i);
    auto next = [&](int m) {   // the largest number below m; no number stays none
      uint32_t d = ~0u;
#pragma unroll
      for (int i = 0; i < V; ++i) d = min_u(d, (uint32_t)m - 1u - (uint32_t)num[i]);
      d = over_row<LPT>(d, min_u);
      return m == kNone ? kNone : (int)((uint32_t)m - 1u - d);
    };
    int last = m;
    for (int k = 0; k < K; ++k) {
      if (t == 0) chosen[k] = m;
      last = m;
      m = next(m);
    }
    cands = K;
    if (!whole) {
      wave_sync();
      for (int k = t; k < K; k += LPT)
        open |= k > 0 && chosen[k] != kNone && (chosen[k - 1] >> 10) - (chosen[k] >> 10) <= apart;
      // experts after the last, as long as they are not apart from it
      bool more = !masked && last != kNone;
      for (int k = K;; ++k) {
        more = more && m != kNone && (last >> 10) - (m >> 10) <= apart;
        if (more && k >= CAP) {
          unsure = true;
          more = false;
        }
        if (!__any(more)) break;
        if (more) {
          if (t == 0) chosen[k] = m;
          cands = k + 1;
          open = true;
        }
        m = next(m);
      }
      open = open && !masked && live;
    }
  }
  wave_sync();
  for (int k = t; k < cands; k += LPT) {   // numbers become experts
    const int m = chosen[k];
    chosen[k] = m == kNone || masked ? -1 : kIndex - (m & kIndex);
  }
  wave_sync();

  // grade 2, for all rows of a wave that has one to do
  if (__any(open)) {
    double* val = reinterpret_cast<double*>(wave_lds) + (size_t)(lane / LPT) * CAP;
    int* fresh = reinterpret_cast<int*>(wave_lds + (size_t)RPW * CAP * 2) + (size_t)(lane / LPT) * CAP;
    double total = 0.0;
    if (a.bias && soft) {
#pragma unroll 1
      for (int i = 0; i < V; ++i) {
        const int e = ((i / 8) * LPT + t) * 8 + i % 8;
        if (e < E) total += exp((double)read_logit(ld_as_f32(row, e)) - (double)top);
      }
      total = over_row<LPT>(total, add_d);
    }
    wave_sync();
    int n = 0;   // the experts that there are
    while (n < cands && chosen[n] >= 0) ++n;
    for (int c = t; c < n; c += LPT) {
      const float lc = read_logit(ld_as_f32(row, chosen[c]));
      double x = (double)lc;
      if (a.bias) {
        x = exp(soft ? x - (double)top : -x);
        x = soft ? x / total : 1.0 / (1.0 + x);
        x += (double)a.bias[chosen[c]];
        // a NaN, which a bias may bring, is last: each expert needs a place of its own
        x = x == x ? x : kOut;
      }
      val[c] = x;
    }
    wave_sync();
    for (int c = t; c < n; c += LPT) {
      const double x = val[c];
      const int e = chosen[c];
      int before = 0;
      for (int q = 0; q < n; ++q) {
        const double y = val[q];
        before += y > x || (y == x && chosen[q] < e);
      }
      fresh[before] = e;
    }
    wave_sync();
    for (int k = t; k < min(n, K); k += LPT) chosen[k] = fresh[k];
  }
  wave_sync();
  // weights: lane t the row's slots t, t + LPT, ...
  constexpr int SLOTS = (MUON_ROUTE_MAX_TOP_K + LPT - 1) / LPT;
  int at[SLOTS];
  float p[SLOTS], sum = 0.f;
  bool tiny = false;
#pragma unroll
  for (int j = 0; j < SLOTS; ++j) {
    const int k = t + j * LPT;
    at[j] = k < K ? chosen[k] : -1;
    p[j] = 0.f;
    if (at[j] < 0) continue;
    p[j] = slot_score(read_logit(ld_as_f32(row, at[j])), top, soft);
    tiny |= p[j] < 0x1p-120f;
    sum += p[j];
  }
  sum = over_row<LPT>(sum, add_f);
  // a score near or below the normal range whose share of a small sum is not
  // small: by logarithms
  if (s.renormalise && tiny && sum < 0.5f) unsure = true;
  const float by = s.renormalise ? sum : z;
#pragma unroll
  for (int j = 0; j < SLOTS; ++j) {
    const int k = t + j * LPT;
    if (!live || k >= K) continue;
    a.experts[r * K + k] = at[j];
    a.weights[r * K + k] = at[j] < 0 ? 0.f : s.scale * (p[j] / by);
  }
  // grade 3
  uint64_t again = __ballot(unsure && live && !masked);
  wave_sync();
  while (again) {   // a row's lanes may all have set their bits
    const int which = __ffsll((unsigned long long)again) - 1;
    again &= ~((LPT < WAVE ? (uint64_t(1) << (LPT & 63)) - 1 : ~uint64_t(0)) << (which / LPT * LPT));
    route_row_64<T>(s, a, (tile * RW + wave) * RPW + which / LPT, reinterpret_cast<double*>(wave_lds));
  }
}

// A wave's rows' gradients.  The chosen experts' a_k reach their columns by
// way of shared memory; the logits are read only where a dense term needs them.
// 32768 rows of 64 experts with dscores 7.1 us, 256 experts 16 us, 4.4 TB/s
// (rows as wide as a wave with scalar loads: 31 us for 64).
template <typename T, int LPT, int NC>
__global__ __launch_bounds__(RT) void route_bwd(muon_route_spec s, muon_route_grad_args a) {
  constexpr int V = 8 * NC, RPW = WAVE / LPT;
  __shared__ float spread[RT / LPT][LPT * V];
  const int lane = threadIdx.x & (WAVE - 1), wave = threadIdx.x / WAVE, t = lane & (LPT - 1);
  const int E = (int)a.num_experts, K = s.top_k;
  float* mine = spread[threadIdx.x / LPT];
  const bool soft = s.score == MUON_SCORE_SOFTMAX;
  const bool dense = a.dscores || (soft && !s.renormalise);
  const int64_t tile = blockIdx.y * (int64_t)gridDim.x + blockIdx.x;
  if (tile * RW * RPW >= a.rows) return;
  const int64_t want = (tile * RW + wave) * RPW + lane / LPT;
  const bool live = want < a.rows;
  const int64_t r = live ? want : a.rows - 1;
  const T* row = static_cast<const T*>(a.logits) + r * a.logits_stride;
  wave_sync();
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) mine[(i * LPT + t) * 8 + j] = 0.f;
  float part = 0.f;
  int some = 0;
  for (int k = t; k < K; k += LPT) {
    const int at = a.experts[r * K + k];
    if (at < 0 || at >= E) continue;
    some = 1;
    part += a.weights[r * K + k] * a.dweights[r * K + k];
  }
  const float sum = over_row<LPT>(part, add_f);
  some = over_row<LPT>(some, max_i);
  wave_sync();
  for (int k = t; k < K; k += LPT) {
    const int at = a.experts[r * K + k];
    if (at < 0 || at >= E) continue;
    const float w = a.weights[r * K + k];
    float v = w * a.dweights[r * K + k];
    if (s.renormalise) v -= w / s.scale * sum;
    if (!soft) v *= one_less_sigmoid(read_logit(ld_as_f32(row, at)));
    mine[at] = v;
  }
  wave_sync();
  float d[V];
#pragma unroll
  for (int i = 0; i < V; ++i) d[i] = mine[((i / 8) * LPT + t) * 8 + i % 8];
  if (dense) {
    float l[V], ds[V];
    load_logits<T, LPT, NC>(row, E, t, l);
#pragma unroll
    for (int i = 0; i < V; ++i) ds[i] = 0.f;
    if (a.dscores) {
#pragma unroll
      for (int i = 0; i < NC; ++i) load8(a.dscores + r * E, (i * LPT + t) * 8, E, ds + 8 * i);
    }
    if (soft) {
      float top = l[0], z = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 1; i < V; ++i) top = fmaxf(top, l[i]);
      top = over_row<LPT>(top, max_f);
      float p[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        p[i] = l[i] > -HUGE_VALF ? slot_score(l[i], top, true) : 0.f;
        z += p[i];
      }
      z = over_row<LPT>(z, add_f);
      const float inv = z > 0.f ? 1.f / z : 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        p[i] *= inv;
        if (l[i] > -HUGE_VALF) dot += p[i] * ds[i];
      }
      dot = over_row<LPT>(dot, add_f) + (s.renormalise ? 0.f : sum);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (l[i] > -HUGE_VALF) d[i] += p[i] * (ds[i] - dot);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!(l[i] > -HUGE_VALF)) continue;
        const float e = expf(-fabsf(l[i]));   // s (1 - s) without a difference
        d[i] += ds[i] * (e / ((1.f + e) * (1.f + e)));
      }
    }
  }
  if (live) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (i * LPT + t) * 8;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = some ? d[8 * i + j] : 0.f;
      if (c < E) store8(static_cast<T*>(a.dlogits) + r * a.dlogits_stride, c, E, o);
    }
  }
}

// ---- order of the pairs ----------------------------------------------------
// A stable counting sort.  The pairs are cut into at most kMaxTiles tiles;
// order_count leaves each tile's count of every expert (and, as expert E, of
// the pairs without one), then each workgroup of order_place adds up the tiles
// before its own and places its pairs.  A wave takes 64 consecutive pairs at a
// time: lanes of one expert find each other by a ballot for each bit of the
// expert's number, and the lane's rank among them and the pairs of the wave
// before is its place among the wave's.  One tile needs order_place alone.
// 1M pairs of 256 experts: 4 to 5 + 14.5 us, of which the bytes are 2.5; what is
// left is latency, one workgroup a CU going through six steps with barriers
// between (counts one at a time 57 us, stores straight to `order` 2.5 us more).
constexpr int OT = 1024, OW = OT / WAVE;
constexpr int kChunks = 4;                           // of 64 pairs, a wave in a round
constexpr int64_t kRound = OT * kChunks;             // pairs of a workgroup's round
constexpr int64_t kMaxTiles = 256;                   // one to a CU

// Words of a tile's counts: E + 1, in whole 16-byte pieces.
__host__ __device__ constexpr int order_pitch(int E) { return (E + 4) & ~3; }

__device__ __forceinline__ int read_expert(const int32_t* experts, int64_t p, int E) {
  const int e = experts[p];
  return e >= 0 && e < E ? e : E;
}

__global__ __launch_bounds__(OT) void order_count(int64_t pairs, int64_t tile, int E, const int32_t* experts,
                                                  int32_t* hist) {
  extern __shared__ int32_t lds_i[];
  const int pitch = order_pitch(E);
  for (int e = threadIdx.x; e < pitch; e += OT) lds_i[e] = 0;
  __syncthreads();
  const int64_t from = blockIdx.x * tile, to = from + tile < pairs ? from + tile : pairs;
#pragma unroll 4
  for (int64_t p = from + threadIdx.x; p < to; p += OT) atomicAdd(&lds_i[read_expert(experts, p, E)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < pitch; e += OT) hist[blockIdx.x * (int64_t)pitch + e] = lds_i[e];
}

// Shared memory of order_place, in 4-byte words: base, tot, sub and loc of
// E + 1 each, OW wave sums, a 16-byte piece of two kinds a lane (the sums over
// the tiles, then the round's pairs and places in order), and a 16-bit count a
// wave and expert.
__host__ __device__ constexpr int order_words(int E) {
  return 4 * order_pitch(E) + OW + 2 * (int)kRound + (OW * (E + 1) + 1) / 2;
}

// Exclusive sum over the workgroup in lane order; `total` of all.
__device__ __forceinline__ int group_scan(int v, int32_t* wsum, int& total) {
  const int lane = threadIdx.x & (WAVE - 1), wave = threadIdx.x / WAVE;
  int run = v;
#pragma unroll
  for (int o = 1; o < WAVE; o <<= 1) {
    const int up = __shfl_up(run, o, WAVE);
    run += lane >= o ? up : 0;
  }
  if (lane == WAVE - 1) wsum[wave] = run;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < OW; ++w) {
    const int n = wsum[w];
    before += w < wave ? n : 0;
    total += n;
  }
  __syncthreads();
  return before + run - v;
}

__global__ __launch_bounds__(OT) void order_place(int64_t pairs, int64_t tile, int E, int tiles, const int32_t* experts,
                                                  const int32_t* hist, int32_t* counts, int32_t* offsets,
                                                  int32_t* order, int32_t* position) {
  extern __shared__ int32_t lds_i[];
  const int N = E + 1;
  const int pitch = order_pitch(E);
  int32_t* base = lds_i;             // place of the round's first pair of each expert
  int32_t* tot = base + pitch;       // all pairs of each expert
  int32_t* sub = tot + pitch;        // the round's
  int32_t* loc = sub + pitch;        // place of its first one in the round
  int32_t* wsum = loc + pitch;
  int32_t* part = wsum + OW;         // [2][slices][pitch], then the round's pairs and places
  uint16_t* cnt = reinterpret_cast<uint16_t*>(part + 2 * kRound);   // [OW][N]; at most kRound
  const int lane = threadIdx.x & (WAVE - 1), wave = threadIdx.x / WAVE;
  uint16_t* mine = cnt + (size_t)wave * N;
  // neighbouring tiles write the two halves of a cache line: on one XCD
  const int me = (blockIdx.x & 7) * (gridDim.x / 8) + blockIdx.x / 8;
  if (me >= tiles) return;
  const int64_t from = me * tile, to = from + tile < pairs ? from + tile : pairs;
  int bits = 1;
  while ((1 << bits) <= E) ++bits;

  int ex[kChunks];
  auto fetch = [&](int64_t p0) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int64_t p = p0 + (int64_t)(wave * kChunks + c) * WAVE + lane;
      ex[c] = p < to ? read_expert(experts, p, E) : -1;
    }
  };
  fetch(from);

  if (tiles > 1) {
    // pairs of each expert in the tiles before this one and in all: four
    // experts a lane, slices of the tiles side by side
    typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
    const int quads = pitch / 4, slices = OT / quads;   // at most 257 quads
    const int quad = threadIdx.x % quads, slice = threadIdx.x / quads;
    i32x4* sums = reinterpret_cast<i32x4*>(part);
    if (slice < slices) {
      i32x4 before = {}, after = {};
      const i32x4* h = reinterpret_cast<const i32x4*>(hist) + quad;
      int t = slice;
#pragma unroll 8
      for (; t < me; t += slices) before += h[t * quads];   // at most 256 tiles of 257 pieces
#pragma unroll 8
      for (; t < tiles; t += slices) after += h[t * quads];
      sums[slice * quads + quad] = before;
      sums[(slices + slice) * quads + quad] = before + after;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < N; e += OT) {
      int before = 0, all = 0;
#pragma unroll 4
      for (int q = 0; q < slices; ++q) {
        before += part[q * pitch + e];
        all += part[(slices + q) * pitch + e];
      }
      base[e] = before;
      tot[e] = all;
    }
  }

  for (int64_t p0 = from; p0 < to; p0 += kRound) {
    for (int i = threadIdx.x; i < (OW * N + 1) / 2; i += OT) reinterpret_cast<int32_t*>(cnt)[i] = 0;
    int rank[kChunks];
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const uint64_t there = __ballot(ex[c] >= 0);
      uint32_t lo = (uint32_t)there, hi = (uint32_t)(there >> 32);
      for (int b = 0; b < bits; ++b) {
        const int bit = -((ex[c] >> b) & 1);   // all ones or zero
        const uint64_t m = __ballot(bit != 0);
        lo &= ~((uint32_t)m ^ (uint32_t)bit);
        hi &= ~((uint32_t)(m >> 32) ^ (uint32_t)bit);
      }
      const uint64_t same = (uint64_t)hi << 32 | lo;
      const int before = __popcll(same & ((uint64_t(1) << lane) - 1));
      const int so_far = ex[c] >= 0 ? mine[ex[c]] : 0;
      rank[c] = so_far + before;
      wave_sync();
      if (ex[c] >= 0 && before == 0) mine[ex[c]] = (uint16_t)(so_far + __popcll(same));
      wave_sync();
    }
    __syncthreads();
    for (int e = threadIdx.x; e < N; e += OT) {   // counts of the waves become their first places
      int run = 0;
#pragma unroll
      for (int w = 0; w < OW; ++w) {
        const int n = cnt[w * N + e];
        cnt[w * N + e] = (uint16_t)run;
        run += n;
      }
      sub[e] = run;
      if (tiles == 1) {
        base[e] = 0;
        tot[e] = run;
      }
    }
    __syncthreads();
    const int e0 = threadIdx.x;   // E <= OT
    int total;
    const int inside = group_scan(e0 < E ? sub[e0] : 0, wsum, total);
    if (e0 < E) loc[e0] = inside;
    if (e0 == 0) loc[E] = total;
    if (p0 == from) {   // the experts' first places
      const int v = e0 < E ? tot[e0] : 0;
      const int first = group_scan(v, wsum, total);
      if (e0 < E) base[e0] += first;
      if (e0 == 0) base[E] += total;
      if (me == 0) {
        if (e0 < E) {
          offsets[e0] = first;
          counts[e0] = v;
        }
        if (e0 == 0) offsets[E] = total;
      }
    }
    __syncthreads();
    // pairs and places in the round's order, so that a wave's stores to
    // `order` are a few runs and not 64 lines
    int2* sorted = reinterpret_cast<int2*>(part);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int64_t p = p0 + (int64_t)(wave * kChunks + c) * WAVE + lane;
      const int e = ex[c];
      if (e < 0) continue;
      const int at = (int)mine[e] + rank[c], place = base[e] + at;
      sorted[loc[e] + at] = make_int2(e < E ? (int)p : -1, place);
      position[p] = e < E ? place : -1;
    }
    if (p0 + kRound < to) fetch(p0 + kRound);
    __syncthreads();
    const int n = (int)(to - p0 < kRound ? to - p0 : kRound);
    for (int i = threadIdx.x; i < n; i += OT) {
      const int2 x = sorted[i];
      order[x.y] = x.x;
    }
    for (int e = threadIdx.x; e < N; e += OT) base[e] += sub[e];
    __syncthreads();
  }
}

__global__ __launch_bounds__(OT) void order_none(int E, int32_t* counts, int32_t* offsets) {
  for (int e = threadIdx.x; e <= E; e += OT) {
    offsets[e] = 0;
    if (e < E) counts[e] = 0;
  }
}

__global__ __launch_bounds__(RT) void balance_k(int E, const int32_t* counts, const float* bias, float* out,
                                                float rate) {
  __shared__ int64_t part[RW];
  int64_t n = 0;
  for (int e = threadIdx.x; e < E; e += RT) n += counts[e];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) n += __shfl_xor((long long)n, o, WAVE);
  if ((threadIdx.x & (WAVE - 1)) == 0) part[threadIdx.x / WAVE] = n;
  __syncthreads();
  n = 0;
  for (int w = 0; w < RW; ++w) n += part[w];
  for (int e = threadIdx.x; e < E; e += RT) {
    const int64_t d = n - (int64_t)counts[e] * E;   // E (mean - count)
    out[e] = bias[e] + (d > 0 ? rate : d < 0 ? -rate : 0.f);
  }
}

}  // namespace

// A workgroup a tile, in two dimensions: the lanes of one are below 2^32.
static dim3 tile_grid(int64_t tiles) {
  const int64_t x = std::min<int64_t>(tiles, 1 << 20);
  return dim3((unsigned)x, (unsigned)((tiles + x - 1) / x));
}

// Lanes of a row and chunks of a lane by the number of experts: 16 lanes of
// one or two chunks for the common sizes.
template <class F>
static void by_experts(int64_t experts, F f) {
  if (experts <= 32) f(std::integral_constant<int, 4>(), std::integral_constant<int, 1>());
  else if (experts <= 64) f(std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
  else if (experts <= 128) f(std::integral_constant<int, 16>(), std::integral_constant<int, 1>());
  else if (experts <= 256) f(std::integral_constant<int, 16>(), std::integral_constant<int, 2>());
  else if (experts <= 512) f(std::integral_constant<int, 32>(), std::integral_constant<int, 2>());
  else f(std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
}

template <typename T>
static void launch_route_forward(const muon_route_spec& s, const muon_route_args& a, hipStream_t stream) {
  by_experts(a.num_experts, [&](auto lpt, auto nc) {
    constexpr int LPT = decltype(lpt)::value, NC = decltype(nc)::value, per = RW * (WAVE / LPT);
    const dim3 grid = tile_grid((a.rows + per - 1) / per);
    const size_t shm = size_t(RW) * route_wave_words((int)a.num_experts, s.groups, WAVE / LPT, Near<LPT>::CAP) * 4;
    MUON_LAUNCH_SHM("route_fwd", (route_fwd<T, LPT, NC>), grid, dim3(RT), shm, stream, s, a);
  });
}

hipError_t run_route_forward(const muon_route_spec& s, const muon_route_args& a, hipStream_t stream) {
  if (a.dtype == MUON_BF16) launch_route_forward<bf16_t>(s, a, stream);
  else launch_route_forward<float>(s, a, stream);
  return hipGetLastError();
}

template <typename T>
static void launch_route_backward(const muon_route_spec& s, const muon_route_grad_args& a, hipStream_t stream) {
  by_experts(a.num_experts, [&](auto lpt, auto nc) {
    constexpr int LPT = decltype(lpt)::value, NC = decltype(nc)::value, per = RW * (WAVE / LPT);
    const dim3 grid = tile_grid((a.rows + per - 1) / per);
    MUON_LAUNCH("route_bwd", (route_bwd<T, LPT, NC>), grid, dim3(RT), stream, s, a);
  });
}

hipError_t run_route_backward(const muon_route_spec& s, const muon_route_grad_args& a, hipStream_t stream) {
  if (a.dtype == MUON_BF16) launch_route_backward<bf16_t>(s, a, stream);
  else launch_route_backward<float>(s, a, stream);
  return hipGetLastError();
}

// Pairs of a tile: whole rounds, as many as keep the tiles to one a CU.
static int64_t order_tile(int64_t pairs) {
  const int64_t rounds = (pairs + kRound - 1) / kRound;
  return kRound * std::max<int64_t>(1, (rounds + kMaxTiles - 1) / kMaxTiles);
}
int64_t order_tiles(int64_t pairs) { return (pairs + order_tile(pairs) - 1) / order_tile(pairs); }

hipError_t run_route_order(int64_t pairs, int64_t experts_n, const int32_t* experts, int32_t* counts, int32_t* offsets,
                           int32_t* order, int32_t* position, int32_t* ws, hipStream_t stream) {
  const int E = (int)experts_n;
  const int64_t tile = order_tile(pairs), tiles = order_tiles(pairs);
  if (tiles == 0) {
    MUON_LAUNCH("order_none", order_none, dim3(1), dim3(OT), stream, E, counts, offsets);
    return hipGetLastError();
  }
  if (tiles > 1) {
    MUON_LAUNCH_SHM("order_count", order_count, dim3((unsigned)tiles), dim3(OT), size_t(order_pitch(E)) * 4, stream, pairs,
                    tile, E, experts, ws);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  MUON_LAUNCH_SHM("order_place", order_place, dim3((unsigned)(tiles + 7) / 8 * 8), dim3(OT), size_t(order_words(E)) * 4, stream, pairs,
                  tile, E, (int)tiles, experts, ws, counts, offsets, order, position);
  return hipGetLastError();
}

hipError_t run_route_balance(int64_t experts_n, const int32_t* counts, const float* bias, float* out, float rate,
                             hipStream_t stream) {
  MUON_LAUNCH("route_balance", balance_k, dim3(1), dim3(RT), stream, (int)experts_n, counts, bias, out, rate);
  return hipGetLastError();
}

}  // namespace muon
