// The experts of a token and their weights, from the router's fp32 logits.
//
//   choice: the `top` experts of largest score, ties to the lower index; the score is the logit,
//   or with a bias (sigmoid only) 1 / (1 + e^-logit) + bias in fp64, so that experts whose scores
//   lie next to each other are told apart as the definition tells them
//   weight: e^(logit - max) / sum over all experts (softmax) or 1 / (1 + e^-logit) (sigmoid, 0 where
//   e^-logit passes fp64), over the sum of the chosen ones if renormalized, times scale
//
// A wave per token.  Lane l holds the scores of experts [NV l, NV l + NV) as unsigned keys that
// order like them, 0 for an expert that cannot be chosen (a logit of -inf or NaN).  A round finds
// the largest key of the wave by cross-lane moves (no LDS), the first lane that holds it by a
// ballot, and takes that expert out: the lowest index of equals, since a lane's own best is its
// first.  What is recorded is the expert's number; its logit is read again from the row, which is in
// the cache by then: chosen by a uniform index from the lane's values, the compiler moves those into
// LDS (8192 x 256, 8 of biased scores: 24.8 us instead of 11.3).
//
// Bound by the rounds' chains of dependent cross-lane moves, not by memory: 8192 tokens, 8 chosen,
// 64 / 256 / 512 biased experts 6.0-6.5 / 10.3-11.8 / 20-22 us, 256 by softmax 7.4-7.8 (8.9 MB: 1.5 at
// the rate of a large copy); 16 x 64 3.0-3.2 us, most of it the launch.
#include <type_traits>

#include "layer_launch.h"
#include "nm_device.h"

#pragma clang fp contract(off)

namespace {

using namespace nml;

template <int CTRL>
__device__ __forceinline__ uint32_t moved(uint32_t v) {   // lanes without a source get 0
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}

// The wave's largest key, in every lane.  Lane 63 has it after shifts by 1, 2, 4, 8 within rows of
// 16 and broadcasts of the rows' last lanes.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  uint32_t o;
#define NM_STEP(C)     \
  o = moved<C>(v);     \
  v = o > v ? o : v;
  NM_STEP(0x111) NM_STEP(0x112) NM_STEP(0x114) NM_STEP(0x118) NM_STEP(0x142) NM_STEP(0x143)
#undef NM_STEP
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
#define NM_STEP(C)                                                                       \
  {                                                                                      \
    const uint64_t o = (uint64_t)moved<C>((uint32_t)(v >> 32)) << 32 | moved<C>((uint32_t)v); \
    v = o > v ? o : v;                                                                   \
  }
  NM_STEP(0x111) NM_STEP(0x112) NM_STEP(0x114) NM_STEP(0x118) NM_STEP(0x142) NM_STEP(0x143)
#undef NM_STEP
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), 63) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, 63);
}

// Keys that order like the values (-0 below +0 is undone by adding 0), none of them 0.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return b >> 63 ? ~b : b | 1ull << 63;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// The value of a key.
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7FFFFFFFu : ~k); }

// Up to n rounds: won(j, key, lane, which) is told the j-th largest key and where it lies, the lowest
// expert of equals, and says whether to go on.
template <int NV, typename Key, typename Won>
__device__ __forceinline__ void rounds(Key (&key)[NV], int n, Won&& won) {
  const int lane = threadIdx.x & 63;
  for (int j = 0; j < n; ++j) {
    Key best = key[0];
    int at = 0;
#pragma unroll
    for (int v = 1; v < NV; ++v) {
      at = key[v] > best ? v : at;
      best = key[v] > best ? key[v] : best;
    }
    const Key m = wave_max(best);
    if (m == 0) return;   // no expert left
    const int win = __ffsll((unsigned long long)__ballot(best == m)) - 1;
    const int which = __builtin_amdgcn_readlane(at, win);
    if (!won(j, m, win, which)) return;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (lane == win && v == which) key[v] = 0;
  }
}

// NV: experts a lane; BIASED: the choice by biased sigmoid scores
template <int NV, bool BIASED>
__global__ __launch_bounds__(256) void k_moe_route(RouteArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= a.t) return;   // whole waves, and no barrier below
  const float* row = a.logits + t * a.ldl;
  const int e0 = lane * NV, E = (int)a.experts;
  float l[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) l[v] = row[e0 + v < E ? e0 + v : E - 1];
#pragma unroll
  for (int v = 0; v < NV; ++v) l[v] = e0 + v < E ? l[v] : -__builtin_inff();
  int id = -1;           // lane j: the expert of slot j
  auto take = [&](int j, int win, int which) { id = lane == j ? win * NV + which : id; };
  auto open = [&](int v) { return l[v] > -__builtin_inff(); };   // false for NaN
  if constexpr (BIASED) {
    // first in fp32, one round more than slots: the sigmoid's exponent, exponential, sum and
    // reciprocal leave it within 4 * 2^-24, the sum with the bias within 2^-24 of its size, so where
    // every score lies over 2^-20 (times the larger size, where that passes 1) above the next one,
    // the order is that of fp64.  Otherwise (two scores of 256 next to the top, in one of 1000
    // tokens) it is decided in fp64.  8192 x 256, 8 chosen: 11.3 us, all in fp64 14.7.
    float bias[NV];
    uint32_t key[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) bias[v] = a.bias[e0 + v < E ? e0 + v : E - 1];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l[v] * -1.442695041f));
      key[v] = open(v) ? key_of(s + bias[v]) : 0;
    }
    bool clear = true;
    float last = 0.0f;
    rounds<NV>(key, a.top + 1, [&](int j, uint32_t m, int win, int which) {
      const float now = value_of(m);
      if (j > 0) clear = last - now > 0x1p-20f * fmaxf(1.0f, fmaxf(__builtin_fabsf(last), __builtin_fabsf(now)));
      last = now;
      if (clear && j < a.top) take(j, win, which);
      return clear;
    });
    if (!clear) {
      uint64_t exact[NV];
#pragma unroll
      for (int v = 0; v < NV; ++v) exact[v] = open(v) ? key_of(1.0 / (1.0 + exp(-(double)l[v])) + (double)bias[v]) : 0;
      rounds<NV>(exact, a.top, [&](int j, uint64_t, int win, int which) {
        take(j, win, which);
        return true;
      });
    }
  } else {
    uint32_t key[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) key[v] = open(v) ? key_of(l[v]) : 0;
    rounds<NV>(key, a.top, [&](int j, uint32_t, int win, int which) {
      take(j, win, which);
      return true;
    });
  }
  const float logit = id < 0 ? 0.0f : row[id];
  float w, total;
  if (a.sigmoid) {
    w = id < 0 ? 0.0f : 1.0f / (1.0f + expf(-logit));
    if (a.renormalize && __any(id >= 0 && logit < -80.0f)) {
      // Below -88 the weight passes the least value of fp32, its share of the chosen ones does not: with
      // 1 / (1 + e^-l) = e^min(l, 0) / (1 + e^-|l|) all of them go over e^min(M, 0), M their largest
      // logit, so that M's is at least a half.  (-709.7827: the last l whose e^-l fp64 holds.)  A branch:
      // in every row 8192 x 64 takes 6.4 us instead of 6.0.
      const float base = fminf(value_of(wave_max(id < 0 ? 0u : key_of(logit))), 0.0f);
      const bool held = id >= 0 && logit > -709.7827f;
      w = held ? expf(fminf(logit, 0.0f) - base) / (1.0f + expf(-__builtin_fabsf(logit))) : 0.0f;
    }
    total = a.renormalize ? wave_sum(w) : 1.0f;
  } else {
    // slot 0 holds the largest logit; a difference of infinities is the largest itself
    const float mx = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(logit), 0));
    w = id < 0 ? 0.0f : logit == mx ? 1.0f : expf(logit - mx);
    total = w;
    if (!a.renormalize) {
      total = 0.0f;
#pragma unroll
      for (int v = 0; v < NV; ++v) total += l[v] > -__builtin_inff() ? (l[v] == mx ? 1.0f : expf(l[v] - mx)) : 0.0f;
    }
    total = wave_sum(total);
  }
  if (lane < a.top) {
    a.ids[t * a.top + lane] = id;
    a.weights[t * a.top + lane] = total > 0.0f ? w / total * a.scale : 0.0f;
  }
}

template <int NV>
hipError_t launch_r(const RouteArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.t + 3) / 4)), block(256);
  if (a.bias != nullptr) k_moe_route<NV, true><<<grid, block, 0, s>>>(a);
  else k_moe_route<NV, false><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

namespace nml {

hipError_t launch_moe_route(const RouteArgs& a, hipStream_t s) {
  if (a.t <= 0 || a.top <= 0) return hipSuccess;
  if (a.t > 4ll * 0xFFFFFF) return hipErrorInvalidValue;   // a grid holds under 2^32 threads
  if (a.experts <= 64) return launch_r<1>(a, s);
  if (a.experts <= 128) return launch_r<2>(a, s);
  if (a.experts <= 256) return launch_r<4>(a, s);
  if (a.experts <= 512) return launch_r<8>(a, s);
  return launch_r<16>(a, s);
}

}  // namespace nml
