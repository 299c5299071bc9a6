// Routing to experts: the choice and its weights, the gradient of the logits,
// the order of the routed pairs, the update of the balance bias.
#include <algorithm>
#include <float.h>

#include "internal.h"
#include "rows.h"

namespace muon {
namespace {

constexpr int RT = 256;                 // threads of a workgroup: four waves, a row each
constexpr int RW = RT / WAVE;
constexpr int64_t kMaxGrid = 1 << 16;
constexpr int EPL = MUON_ROUTE_MAX_EXPERTS / WAVE;   // experts a lane may hold
constexpr double kOut = -HUGE_VAL;      // rank of an expert that may not be chosen

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, WAVE);
  return v;
}

// Logit as the definition reads it: NaN closed, +inf the largest finite value.
__device__ __forceinline__ float read_logit(float l) { return l != l ? -HUGE_VALF : fminf(l, FLT_MAX); }

// The largest (value, then lowest index) over the wave.
__device__ __forceinline__ void wave_best(double& v, int& i) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const double v2 = __shfl_xor(v, o, WAVE);
    const int i2 = __shfl_xor(i, o, WAVE);
    if (v2 > v || (v2 == v && i2 < i)) {
      v = v2;
      i = i2;
    }
  }
}

// log sigmoid(l), l finite.
__device__ __forceinline__ double log_sigmoid(double l) { return fmin(l, 0.0) - log1p(exp(-fabs(l))); }

// A wave a row; lane l holds experts l, l + 64, ...; every score in 64 bits.
template <typename T>
__global__ __launch_bounds__(RT) void route_fwd(muon_route_spec s, muon_route_args a) {
  extern __shared__ double lds_all[];   // with groups: E values and `groups` results a wave
  const int lane = threadIdx.x & (WAVE - 1), wave = threadIdx.x / WAVE;
  const int E = (int)a.num_experts, K = s.top_k, G = s.groups;
  double* by_l = lds_all + (size_t)wave * (E + G);
  double* of_l = by_l + E;
  for (int64_t r = blockIdx.x * (int64_t)RW + wave; r < a.rows; r += (int64_t)gridDim.x * RW) {
    int32_t* idx_r = a.experts + r * K;
    float* w_r = a.weights + r * K;
    if (a.token_mask && a.token_mask[r] == 0) {
      if (lane < K) {
        idx_r[lane] = -1;
        w_r[lane] = 0.f;
      }
      if (a.scores)
        for (int e = lane; e < E; e += WAVE) a.scores[r * E + e] = 0.f;
      continue;
    }
    const T* row = static_cast<const T*>(a.logits) + r * a.logits_stride;
    float l[EPL];
    double rank[EPL];
    float top = -HUGE_VALF;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + i * WAVE;
      l[i] = e < E ? read_logit(ld_as_f32(row, e)) : -HUGE_VALF;
      top = fmaxf(top, l[i]);
    }
    top = wave_max(top);
    double total = 1.0;
    if (s.score == MUON_SCORE_SOFTMAX) {
      total = 0.0;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (l[i] > -HUGE_VALF) total += exp((double)l[i] - (double)top);
      total = wave_sum64(total);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + i * WAVE;
      rank[i] = kOut;
      if (e >= E) continue;
      double v = 0.0;
      const bool open = l[i] > -HUGE_VALF;
      if (open)
        v = s.score == MUON_SCORE_SOFTMAX ? exp((double)l[i] - (double)top) / total : 1.0 / (1.0 + exp(-(double)l[i]));
      if (a.scores) a.scores[r * E + e] = (float)v;
      if (a.bias) v += (double)a.bias[e];
      if (open) rank[i] = a.bias ? v : (double)l[i];
      if (G > 1) by_l[e] = open ? v : kOut;
    }
    if (G > 1) {
      const int n = E / G;
      wave_sync();
      for (int g = lane; g < G; g += WAVE) {
        double b1 = kOut, b2 = kOut;
        for (int j = 0; j < n; ++j) {
          const double v = by_l[g * n + j];
          b2 = fmax(b2, fmin(b1, v));
          b1 = fmax(b1, v);
        }
        of_l[g] = s.group_top == 2 && b2 > kOut ? b1 + b2 : b1;
      }
      wave_sync();
      // a group stays if fewer than top_groups are before it
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane + i * WAVE;
        if (e >= E) continue;
        const int g = e / n;
        const double mine = of_l[g];
        int before = 0;
        for (int q = 0; q < G; ++q) before += of_l[q] > mine || (of_l[q] == mine && q < g);
        if (before >= s.top_groups) rank[i] = kOut;
      }
      wave_sync();
    }
    int chosen = -1;   // lane k: the k-th expert
    for (int k = 0; k < K; ++k) {
      double v = kOut;
      int at = INT32_MAX;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (rank[i] > v) {   // ascending experts: the first of equals stays
          v = rank[i];
          at = lane + i * WAVE;
        }
      wave_best(v, at);
      if (!(v > kOut)) break;   // uniform: nothing is left
      if (lane == k) chosen = at;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (lane + i * WAVE == at) rank[i] = kOut;
    }
    // weights from log s, lane k its own
    double ls = kOut;
    if (chosen >= 0) {
      const double lc = (double)read_logit(ld_as_f32(row, chosen));
      ls = s.score == MUON_SCORE_SOFTMAX ? lc - (double)top : log_sigmoid(lc);
    }
    double w = 0.0;
    if (s.renormalise) {
      double m = ls;
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) m = fmax(m, __shfl_xor(m, o, WAVE));
      const double e = chosen >= 0 ? exp(ls - m) : 0.0;
      const double sum = wave_sum64(e);
      if (chosen >= 0) w = e / sum;
    } else if (chosen >= 0) {
      w = exp(ls) / total;
    }
    if (lane < K) {
      idx_r[lane] = chosen;
      w_r[lane] = (float)(w * (double)s.scale);
    }
  }
}

// A wave a row.  dlogits from the chosen experts' a_k, spread over the row
// through shared memory, and the dense terms.
template <typename T>
__global__ __launch_bounds__(RT) void route_bwd(muon_route_spec s, muon_route_grad_args a) {
  extern __shared__ float lds_f[];
  const int lane = threadIdx.x & (WAVE - 1), wave = threadIdx.x / WAVE;
  const int E = (int)a.num_experts, K = s.top_k;
  float* mine = lds_f + (size_t)wave * E;
  for (int64_t r = blockIdx.x * (int64_t)RW + wave; r < a.rows; r += (int64_t)gridDim.x * RW) {
    T* out = static_cast<T*>(a.dlogits) + r * a.dlogits_stride;
    const T* row = static_cast<const T*>(a.logits) + r * a.logits_stride;
    const int at = lane < K ? a.experts[r * K + lane] : -1;
    const bool on = at >= 0 && at < E;
    const bool any = __ballot(on) != 0;
    for (int e = lane; e < E; e += WAVE) mine[e] = 0.f;
    wave_sync();
    const float w = on ? a.weights[r * K + lane] : 0.f;
    float v = on ? w * a.dweights[r * K + lane] : 0.f;
    const float sum = wave_sum(v);
    if (s.renormalise) v -= w / s.scale * sum;
    if (on) mine[at] = v;
    wave_sync();
    const bool soft = s.score == MUON_SCORE_SOFTMAX;
    const float rest = soft && !s.renormalise ? sum : 0.f;
    float l[EPL], sc[EPL];
    float top = -HUGE_VALF, total = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + i * WAVE;
      l[i] = e < E ? read_logit(ld_as_f32(row, e)) : -HUGE_VALF;
      top = fmaxf(top, l[i]);
    }
    top = wave_max(top);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      sc[i] = 0.f;
      if (l[i] > -HUGE_VALF) sc[i] = soft ? expf(l[i] - top) : 1.f / (1.f + expf(-l[i]));
      total += sc[i];
    }
    if (soft) {
      total = wave_sum(total);
#pragma unroll
      for (int i = 0; i < EPL; ++i) sc[i] = sc[i] / total;
    }
    if (soft && a.dscores) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (l[i] > -HUGE_VALF) dot += sc[i] * a.dscores[r * E + lane + i * WAVE];
      dot = wave_sum(dot);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + i * WAVE;
      if (e >= E) continue;
      float d = 0.f;
      if (any && l[i] > -HUGE_VALF) {
        const float ds = a.dscores ? a.dscores[r * E + e] : 0.f;
        const float q = l[i] >= 0.f ? expf(-l[i]) * sc[i] : 1.f - sc[i];   // 1 - sigmoid without cancellation
        d = soft ? mine[e] - rest * sc[i] + (a.dscores ? sc[i] * (ds - dot) : 0.f) : (mine[e] + ds * sc[i]) * q;
      }
      st_from_f32(out, e, d);
    }
    wave_sync();
  }
}

// ---- order of the pairs ----------------------------------------------------
// A stable counting sort over tiles of pairs.  order_count leaves each tile's
// count of every expert (and of pairs without one); order_place sums the
// tiles before its own, then ranks its pairs in ascending order: a wave takes
// 64 consecutive pairs, and lanes of equal experts find each other by one
// ballot for each bit of the expert's number.
constexpr int OT = 512, OW = OT / WAVE;
constexpr int64_t kTile = 8192;         // pairs of a tile

__device__ __forceinline__ int read_expert(const int32_t* experts, int64_t p, int E) {
  const int e = experts[p];
  return e >= 0 && e < E ? e : E;
}

__global__ __launch_bounds__(OT) void order_count(int64_t pairs, int E, const int32_t* experts, int32_t* hist) {
  extern __shared__ int32_t lds_i[];
  for (int e = threadIdx.x; e <= E; e += OT) lds_i[e] = 0;
  __syncthreads();
  const int64_t from = blockIdx.x * kTile, to = from + kTile < pairs ? from + kTile : pairs;
  for (int64_t p = from + threadIdx.x; p < to; p += OT) atomicAdd(&lds_i[read_expert(experts, p, E)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += OT) hist[blockIdx.x * (int64_t)(E + 1) + e] = lds_i[e];
}

__global__ __launch_bounds__(OT) void order_place(int64_t pairs, int E, int64_t tiles, const int32_t* experts,
                                                  const int32_t* hist, int32_t* counts, int32_t* offsets,
                                                  int32_t* order, int32_t* position) {
  // next[w][e]: the place of wave w's next pair of expert e; tot[e]: all pairs of e
  extern __shared__ int32_t lds_i[];
  int32_t* next = lds_i;
  int32_t* tot = lds_i + (size_t)OW * (E + 1);
  const int lane = threadIdx.x & (WAVE - 1), wave = threadIdx.x / WAVE;
  constexpr int64_t per_wave = kTile / OW;
  const int64_t from = blockIdx.x * kTile + wave * per_wave;
  const int64_t to = from + per_wave < pairs ? from + per_wave : pairs;
  for (int i = threadIdx.x; i < OW * (E + 1); i += OT) next[i] = 0;
  __syncthreads();
  for (int64_t p = from + lane; p < to; p += WAVE) atomicAdd(&next[wave * (E + 1) + read_expert(experts, p, E)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += OT) {
    int before = 0, all = 0;
    for (int64_t t = 0; t < tiles; ++t) {
      const int n = hist[t * (E + 1) + e];
      if (t < (int64_t)blockIdx.x) before += n;
      all += n;
    }
    for (int w = 0; w < OW; ++w) {   // counts of the waves become places within the expert's group
      const int n = next[w * (E + 1) + e];
      next[w * (E + 1) + e] = before;
      before += n;
    }
    tot[e] = all;
  }
  __syncthreads();
  // exclusive sums over the experts, by one thread each (E + 1 is small)
  for (int e = threadIdx.x; e <= E; e += OT) {
    int before = 0;
    for (int q = 0; q < e; ++q) before += tot[q];
    for (int w = 0; w < OW; ++w) next[w * (E + 1) + e] += before;
    if (blockIdx.x == 0) {
      offsets[e] = before;
      if (e < E) counts[e] = tot[e];
    }
  }
  __syncthreads();
  int bits = 1;
  while ((1 << bits) <= E) ++bits;
  for (int64_t p0 = from; p0 < to; p0 += WAVE) {
    const int64_t p = p0 + lane;
    const bool in = p < to;
    const int e = in ? read_expert(experts, p, E) : 0;
    uint64_t same = __ballot(in);
    for (int b = 0; b < bits; ++b) {
      const uint64_t m = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? m : ~m;
    }
    const int before = __popcll(same & ((uint64_t(1) << lane) - 1));
    int place = 0;
    if (in) place = next[wave * (E + 1) + e] + before;
    wave_sync();
    if (in && before == 0) next[wave * (E + 1) + e] += __popcll(same);
    wave_sync();
    if (in) {
      order[place] = e < E ? (int32_t)p : -1;
      position[p] = e < E ? place : -1;
    }
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

hipError_t run_route_forward(const muon_route_spec& s, const muon_route_args& a, hipStream_t stream) {
  const dim3 grid((unsigned)std::min<int64_t>((a.rows + RW - 1) / RW, kMaxGrid));
  const size_t shm = s.groups > 1 ? size_t(RW) * size_t(a.num_experts + s.groups) * sizeof(double) : 0;
  if (a.dtype == MUON_BF16) MUON_LAUNCH_SHM("route_fwd", route_fwd<bf16_t>, grid, dim3(RT), shm, stream, s, a);
  else MUON_LAUNCH_SHM("route_fwd", route_fwd<float>, grid, dim3(RT), shm, stream, s, a);
  return hipGetLastError();
}

hipError_t run_route_backward(const muon_route_spec& s, const muon_route_grad_args& a, hipStream_t stream) {
  const dim3 grid((unsigned)std::min<int64_t>((a.rows + RW - 1) / RW, kMaxGrid));
  const size_t shm = size_t(RW) * size_t(a.num_experts) * sizeof(float);
  if (a.dtype == MUON_BF16) MUON_LAUNCH_SHM("route_bwd", route_bwd<bf16_t>, grid, dim3(RT), shm, stream, s, a);
  else MUON_LAUNCH_SHM("route_bwd", route_bwd<float>, grid, dim3(RT), shm, stream, s, a);
  return hipGetLastError();
}

int64_t order_tiles(int64_t pairs) { return (pairs + kTile - 1) / kTile; }

hipError_t run_route_order(int64_t pairs, int64_t experts_n, const int32_t* experts, int32_t* counts, int32_t* offsets,
                           int32_t* order, int32_t* position, int32_t* ws, hipStream_t stream) {
  const int E = (int)experts_n;
  const int64_t tiles = order_tiles(pairs);
  if (tiles == 0) {
    MUON_LAUNCH("order_none", order_none, dim3(1), dim3(OT), stream, E, counts, offsets);
    return hipGetLastError();
  }
  MUON_LAUNCH_SHM("order_count", order_count, dim3((unsigned)tiles), dim3(OT), size_t(E + 1) * 4, stream, pairs, E,
                  experts, ws);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  MUON_LAUNCH_SHM("order_place", order_place, dim3((unsigned)tiles), dim3(OT), size_t(OW + 1) * size_t(E + 1) * 4,
                  stream, pairs, E, tiles, experts, ws, counts, offsets, order, position);
  return hipGetLastError();
}

hipError_t run_route_balance(int64_t experts_n, const int32_t* counts, const float* bias, float* out, float rate,
                             hipStream_t stream) {
  MUON_LAUNCH("route_balance", balance_k, dim3(1), dim3(RT), stream, (int)experts_n, counts, bias, out, rate);
  return hipGetLastError();
}

}  // namespace muon
