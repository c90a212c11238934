// Internal launch interface of the layer operators around the products (api_layer.hip to the
// kernel files).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "i8_launch.h"

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

// The experts' MLPs of a few tokens.  Weights: row o of expert e at (e rows + o) ld bytes; 2:4
// positions of an expert [ceil(k/128)][rows][16].
struct MoeArgs {
  const int8_t* x;
  const float* x_scale;
  const int32_t* ids;       // [t][top]
  const float* weights;
  const int8_t *w_gate, *w_up, *w_down;
  const float *gate_scale, *up_scale, *down_scale;
  const uint8_t *gate_meta, *up_meta, *down_meta;   // all null: dense
  const void* residual;     // of y's type, or null
  void* y;
  int64_t ldx, ldw, ldd, ldr, ldy;
  int64_t t, hidden, inter;
  int experts, top, act, bf16_out;
};
int64_t moe_workspace_bytes(int64_t t, int64_t top, int64_t inter);
hipError_t launch_moe_i8(const MoeArgs& a, void* ws, hipStream_t s);

}  // namespace nml
