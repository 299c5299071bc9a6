// Internal interface between the C ABI of the expert operators
// (experts_abi.cpp) and their launchers (places.hip, gate.hip, quantise.hip,
// product.hip, weight_grad.hip).  Not part of the public ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/muon_experts.h"

namespace muon {

hipError_t run_gather(const muon_gather_args& a, hipStream_t stream);
hipError_t run_combine(const muon_combine_args& a, hipStream_t stream);
hipError_t run_combine_backward(const muon_combine_grad_args& a, hipStream_t stream);
hipError_t run_gate_forward(const muon_gate_args& a, hipStream_t stream);
hipError_t run_gate_backward(const muon_gate_grad_args& a, hipStream_t stream);
hipError_t run_quantise(const muon_quantise_args& a, hipStream_t stream);
hipError_t run_product(const muon_product_args& a, hipStream_t stream);
hipError_t run_weight_grad(const muon_weight_grad_args& a, void* workspace, hipStream_t stream);
// Parts that a weight gradient's rows are split into (1: straight to dw, no
// parts in the workspace; else that many [num_experts, n, k] fp32 tensors).
int64_t weight_grad_parts(int64_t rows, int64_t num_experts, int64_t n, int64_t k);
inline int64_t weight_grad_parts_bytes(int64_t rows, int64_t num_experts, int64_t n, int64_t k) {
  const int64_t parts = weight_grad_parts(rows, num_experts, n, k);
  return parts > 1 ? (parts * num_experts * n * k * 4 + 255) / 256 * 256 : 0;
}
// Bytes of the copies of rows of odd widths that follow the parts.
int64_t weight_grad_copy_bytes(int64_t rows, int64_t num_experts, int64_t n, int64_t k);

}  // namespace muon
