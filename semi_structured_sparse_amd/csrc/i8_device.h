// Device-side pieces shared by the int8 product kernels.
#pragma once
#include "i8_launch.h"
#include "nm_device.h"

// Roundings are the ones written in these files: no product is fused into a sum unless it says
// fmaf.  (Left to the compiler, the shift's product, the scale's product or the accumulation
// could be fused in one kernel and not in another, and routes would give other bits.)
#pragma clang fp contract(off)

namespace nmk {

typedef int i32x16 __attribute__((ext_vector_type(16)));

// Sixteen readable zero bytes: where loads past the end of a row go.
static __device__ const uint4 kZero16 = {0u, 0u, 0u, 0u};

// Between a wave's writes to LDS and its reads of them as another type (either way round): LDS
// serves one wave in order, and the compiler moves or merges no access across.
__device__ __forceinline__ void wave_lds_fence() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
  asm volatile("" ::: "memory");
}

// Gate of a GLU in fp32.  silu: g / (1 + e^-g).  gelu: (1 + tanh z) / 2 = 1 / (1 + e^-2z), the
// same function without the cancellation of 1 + tanh z for negative z (2 sqrt(2/pi) =
// 1.5957691).  Where the exponential overflows the gate is its limit, -0 (g = -inf enters the
// last product as the largest finite number).  The exponent's rounding leaves the result
// |z| 2^-24 off, relative: at z = -20, where the gate is 4e-8 of the largest, 1e-6.  The
// quotient is a reciprocal (1 ulp) and a product: a correctly rounded division costs 10
// instructions more, and the gates of a 256 x 256 tile 3 us more.  Both sides carry a factor
// 1/4, so that the reciprocal, which has no subnormal results, covers every finite exponential.
__device__ __forceinline__ float glu_gate(float g, int act) {
  float z = g;
  if (act == NM_GLU_GELU_TANH) z = 1.5957691216057308f * __builtin_fmaf(0.044715f, g * g * g, g);
  const float d = 0.25f + __builtin_amdgcn_exp2f(__builtin_fmaf(z, -1.442695041f, -2.0f));
  return (0.25f * fmaxf(g, -3.402823466e38f)) * __builtin_amdgcn_rcpf(d);
}

// fp32 to bf16, to nearest even; a NaN stays one.
__device__ __forceinline__ uint16_t bf16_rne(float v) {
  const uint32_t b = __float_as_uint(v);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((b >> 16) | 0x40u);
  return (uint16_t)((b + 0x7FFFu + ((b >> 16) & 1u)) >> 16);
}

// A sum with its scales, and the shift term added to it: the steps of every epilogue.
__device__ __forceinline__ float i8_scaled(int s, float xs, float ws) { return ((float)s * xs) * ws; }
__device__ __forceinline__ float i8_shifted(float v, float rb, float cs) { return __builtin_fmaf(rb, cs, v); }

// The value of one GLU output from its sums (s1: the second weight's).
__device__ __forceinline__ float i8_gated(const nml::I8Epi& e, int s0, int s1, float xs, float ws, float us) {
  return glu_gate(i8_scaled(s0, xs, ws), e.act) * i8_scaled(s1, xs, us);
}

// One output, every address worked out (the few-token kernels and the reduction).
template <bool GLU>
__device__ __forceinline__ void i8_store(const nml::I8Epi& e, int s0, int s1, int64_t t, int64_t o) {
  const float xs = e.x_scale[t], ws = e.w_scale[o];
  float v;
  if constexpr (GLU) {
    v = i8_gated(e, s0, s1, xs, ws, e.up_scale[o]);
  } else {
    v = i8_scaled(s0, xs, ws);
    if (e.col_shift != nullptr) v = i8_shifted(v, e.row_shift != nullptr ? e.row_shift[t] : 1.f, e.col_shift[o]);
  }
  if (e.bf16_out) {
    static_cast<uint16_t*>(e.y)[t * e.ldy + o] = bf16_rne(v);
  } else {
    float* p = static_cast<float*>(e.y) + t * e.ldy + o;
    *p = e.accumulate ? *p + v : v;
  }
}

}  // namespace nmk
