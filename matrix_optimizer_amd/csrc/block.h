// Internal interface between the C ABI of the row operators (block_abi.cpp)
// and their launchers (norm.hip, route.hip).  Not part of the public ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/muon_block.h"

namespace muon {

// Dropout as the kernels take it.
struct Drop {
  bool on = false;
  uint32_t t = 0;               // elements whose 16-bit number is below t are dropped
  float up = 1.f;               // 2^16 / (2^16 - t); 0 if everything is dropped
  uint64_t seed = 0, offset = 0;
  const uint64_t* dev = nullptr;   // {seed, offset} on the device, or null
};

hipError_t run_dropout(int64_t rows, int64_t cols, const void* x, int64_t xs, void* y, int64_t ys, int dtype,
                       const Drop& d, hipStream_t stream);
hipError_t run_norm_forward(const muon_norm_args& a, const Drop& d, hipStream_t stream);
hipError_t run_norm_backward(const muon_norm_grad_args& a, const Drop& d, float* parts, hipStream_t stream);
// Rows of [cols] fp32 partial sums that dweight's reduction uses.
int64_t norm_parts(int64_t rows, int64_t cols);

hipError_t run_route_forward(const muon_route_spec& s, const muon_route_args& a, hipStream_t stream);
hipError_t run_route_backward(const muon_route_spec& s, const muon_route_grad_args& a, hipStream_t stream);
// Tiles of pairs (each with num_experts + 1 counts in the workspace, in whole 16-byte pieces).
int64_t order_tiles(int64_t pairs);
hipError_t run_route_order(int64_t pairs, int64_t experts_n, const int32_t* experts, int32_t* counts, int32_t* offsets,
                           int32_t* order, int32_t* position, int32_t* ws, hipStream_t stream);
hipError_t run_route_balance(int64_t experts_n, const int32_t* counts, const float* bias, float* out, float rate,
                             hipStream_t stream);

}  // namespace muon
