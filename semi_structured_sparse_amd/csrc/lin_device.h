// Device-side pieces shared by the bf16 products with an epilogue.
#pragma once
#include "i8_device.h"
#include "layer_launch.h"

namespace nmk {

// The activation in fp32 (glu_gate: silu and gelu; a NaN stays one in every form).
__device__ __forceinline__ float lin_fn(float v, int fn) {
  if (fn == NM_FN_NONE) return v;
  if (fn == NM_FN_RELU) return v < 0.0f ? 0.0f : v;
  return glu_gate(v, fn == NM_FN_SILU ? NM_GLU_SILU : NM_GLU_GELU_TANH);
}

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// Two fp32 values as packed bf16, to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

// One output from its finished sum.
__device__ __forceinline__ void lin_store(const nml::LinEpi& e, float s, int64_t t, int64_t o) {
  if (e.bias != nullptr) s = s + e.bias[o];
  s = lin_fn(s, e.fn);
  if (e.bf16_out) {
    if (e.residual != nullptr) s = s + bf16_to_f32(static_cast<const uint16_t*>(e.residual)[t * e.ldr + o]);
    static_cast<uint16_t*>(e.y)[t * e.ldy + o] = (uint16_t)pack_bf16(s, 0.0f);
  } else {
    if (e.residual != nullptr) s = s + static_cast<const float*>(e.residual)[t * e.ldr + o];
    static_cast<float*>(e.y)[t * e.ldy + o] = s;
  }
}

// N values through the activation: one test of its kind for all of them.
template <int N>
__device__ __forceinline__ void lin_fns(float (&v)[N], int fn) {
  if (fn == NM_FN_NONE) return;
  if (fn == NM_FN_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];
  } else if (fn == NM_FN_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = glu_gate(v[i], NM_GLU_SILU);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = glu_gate(v[i], NM_GLU_GELU_TANH);
  }
}

// Four neighbouring outputs of a row, on a multiple of their size: the residual's, as loaded ...
template <bool BF16>
__device__ __forceinline__ uint4 lin_load4(const nml::LinEpi& e, int64_t t, int64_t o) {
  if constexpr (BF16) {
    const uint2 d = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(e.residual) + t * e.ldr + o);
    return make_uint4(d.x, d.y, 0u, 0u);
  }
  return *reinterpret_cast<const uint4*>(static_cast<const float*>(e.residual) + t * e.ldr + o);
}
// ... and y's, from values that have their bias and activation
__device__ __forceinline__ void lin_store4(const nml::LinEpi& e, const float* v, const uint4& r, int64_t t, int64_t o) {
  f32x4 s = {v[0], v[1], v[2], v[3]};
  if (e.bf16_out) {
    if (e.residual != nullptr) {
      s[0] = s[0] + __uint_as_float(r.x << 16);
      s[1] = s[1] + __uint_as_float(r.x & 0xFFFF0000u);
      s[2] = s[2] + __uint_as_float(r.y << 16);
      s[3] = s[3] + __uint_as_float(r.y & 0xFFFF0000u);
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(e.y) + t * e.ldy + o) =
        make_uint2(pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]));
  } else {
    if (e.residual != nullptr) {
      s[0] = s[0] + __uint_as_float(r.x);
      s[1] = s[1] + __uint_as_float(r.y);
      s[2] = s[2] + __uint_as_float(r.z);
      s[3] = s[3] + __uint_as_float(r.w);
    }
    *reinterpret_cast<f32x4*>(static_cast<float*>(e.y) + t * e.ldy + o) = s;
  }
}

// Rows of y and of the residual keep the alignment of four outputs.
__host__ __device__ inline bool lin_whole(const nml::LinEpi& e) {
  return e.ldy % 4 == 0 && (e.residual == nullptr || e.ldr % 4 == 0);
}

// The first `keep` (0 .. 8) of eight bf16 values, zeros behind.
__device__ __forceinline__ u32x4 head_of(u32x4 v, int keep) {
#pragma unroll
  for (int d = 0; d < 4; ++d) v[d] = keep >= 2 * d + 2 ? v[d] : keep == 2 * d + 1 ? (v[d] & 0xFFFFu) : 0u;
  return v;
}

}  // namespace nmk
