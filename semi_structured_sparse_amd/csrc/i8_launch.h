// Internal launch interface of the int8 layers (api_i8.hip to the kernel files).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nm_launch.h"

namespace nml {

// Output side of the int8 products: y = (fp32(sum) * x_scale[t]) * w_scale[o] + beta_t c_o, or
// act(gate) * up from two sums.
struct I8Epi {
  const float* x_scale;
  const float* w_scale;
  const float* up_scale;    // GLU: scale of the second weight
  const float* row_shift;   // null: 1
  const float* col_shift;   // null: no term
  void* y;
  int64_t ldy;
  int bf16_out, accumulate, act;
};

struct I8Args {
  const int8_t* x;
  int64_t ldx;
  const int8_t* w;
  const int8_t* w_up;       // GLU: the second weight
  int64_t ldw;
  const uint8_t* meta;      // 2:4 positions [ceil(k/128)][o][16]; null: dense weights
  const uint8_t* up_meta;
  int64_t t, o, k;          // k: reduction positions (2:4: twice the values of a row)
  int glu;                  // 1: act(x w) * (x w_up)
  I8Epi epi;
  Route route;
};

hipError_t launch_quant_i8(const uint16_t* x, int64_t rows, int64_t k, int64_t ldx, int n, int m, int ns, int8_t* q,
                           int64_t ldq, float* scale, hipStream_t s);
hipError_t launch_meta_step_block(const uint8_t* meta, int64_t o, int64_t kc, uint8_t* out, hipStream_t s);

// Streaming kernel: any shape.  The reduction is split across workgroups where part holds
// i8_few_part_bytes.
hipError_t launch_i8_few(const I8Args& a, int32_t* part, int64_t part_bytes, hipStream_t s);
int64_t i8_few_part_bytes(int64_t t, int64_t o, int64_t k, bool sparse, bool glu);

// Tile kernels: 256 x 256 tiles (large), or smaller ones by shape, the reduction split across
// workgroups where part holds i8_mid_part_bytes.
bool i8_tile_eligible(const I8Args& a);
int64_t i8_mid_part_bytes(int64_t t, int64_t o, int64_t k, bool glu);
hipError_t launch_i8_tile(const I8Args& a, bool large, int32_t* part, int64_t part_bytes, hipStream_t s);

// y from `splits` partial sums part[split][matrix][t][o4], o4 = o rounded up to 4
hipError_t launch_i8_reduce(const int32_t* part, int64_t splits, bool glu, int64_t t, int64_t o, const I8Epi& e,
                            const Route& r, hipStream_t s);

}  // namespace nml
