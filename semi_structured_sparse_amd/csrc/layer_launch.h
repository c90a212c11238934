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

// Output side of the bf16 products: y = residual + fn(sum + bias).
struct LinEpi {
  const float* bias;        // null: none
  const void* residual;     // of y's type; null: none
  void* y;
  int64_t ldr, ldy;
  int fn, bf16_out;
};
struct LinArgs {
  const uint16_t* x;
  const uint16_t* w;        // dense [o][ldw], or the kept values of 2:4 rows [o][ldw >= k / 2]
  const uint8_t* meta;      // 2:4 positions [ceil(k/128)][o][16]; null: dense
  int64_t ldx, ldw, t, o, k;
  LinEpi epi;
  Route route;
};
// Streaming kernel: any shape.  The reduction is split across workgroups where part holds
// lin_few_part_bytes.
hipError_t launch_lin_few(const LinArgs& a, float* part, int64_t part_bytes, hipStream_t s);
int64_t lin_few_part_bytes(int64_t t, int64_t o, int64_t k, bool sparse);
// Tile kernels: 256 x 256 tiles (large), or smaller ones by shape, the reduction split across
// workgroups where part holds lin_mid_part_bytes.
bool lin_tile_eligible(const LinArgs& a);
int64_t lin_mid_part_bytes(int64_t t, int64_t o, int64_t k, bool sparse);
hipError_t launch_lin_tile(const LinArgs& a, bool large, float* part, int64_t part_bytes, hipStream_t s);
// y from `splits` partial sums part[split][t][o4], o4 = o rounded up to 4
hipError_t launch_lin_reduce(const float* part, int64_t splits, int64_t t, int64_t o, const LinEpi& e, const Route& r,
                             hipStream_t s);

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
int64_t moe_workspace_bytes(int64_t t, int64_t experts, int64_t top, int64_t hidden, int64_t inter);
hipError_t launch_moe_i8(const MoeArgs& a, void* ws, hipStream_t s);

}  // namespace nml
