// Internal launch interface of the layer operators around the products (api_layer.hip to the
// kernel files).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nm_launch.h"

namespace nml {

struct NormArgs {
  const void* x;
  const void* r;            // residual or null
  void* sum_out;            // x + r, or null
  const float* weight;      // null: ones
  uint16_t* y;              // normed row, bf16, or null
  int8_t* q;
  float* scale;
  int64_t rows, k, ldx, ldr, lds, ldy, ldq;
  int x_bf16, r_bf16;       // types; r_bf16: of r and sum_out
  float eps;
  int n, m, ns;
};
hipError_t launch_rmsnorm_i8(const NormArgs& a, hipStream_t s);

struct RouteArgs {
  const float* logits;
  const float* bias;        // null: the choice goes by the logits
  int32_t* ids;
  float* weights;
  int64_t t, experts, ldl;
  int top, sigmoid, renormalize;
  float scale;
};
hipError_t launch_moe_route(const RouteArgs& a, hipStream_t s);

}  // namespace nml
