// Rows of bf16 -> int8 codes with one scale per row, after an optional n:m selection or
// followed by the lift for (2N-2):2N weights (SlideSparse page, technical summary 2.B: the
// online step quantizes the activations and expands them for the lowered weights in one pass;
// Flexible (N:M) Activation Sparsity page, 2.A: the selection), and the step-blocked copy of
// 2-bit positions that the int8 products read.
//
//   amax = max |x|,  scale = fp32(amax / 127),  q = the integer nearest to 127 x / amax
//
// The quotient's rounding is exact.  x and amax have 8 significant bits, so 127 x / amax is
// either a half integer exactly or further than 2^-16, relative, from every half integer
// (numerator and denominator are integers of at most 15 and 8 bits once scaled).  One
// correctly rounded fp32 division therefore lands on the same side, and on a tie exactly:
// with y = fp32(1 / amax), q0 = a y, and one residual step q = q0 + (a - q0 amax) y in fused
// arithmetic.  amax and x are first scaled by a power of two where amax would make 1 / amax
// or the residual leave the normal range.  Adding 1.5 * 2^23 then rounds to an integer, ties
// to even, whose low byte is the code.
//
// One pass: a row's values stay in registers between the maximum and the codes (the lift
// with N != 4 passes the codes through LDS, where a window is four bytes at an even offset).
// The kernel moves 2 + 1 (lifted 2 + 2(N-1)/N) bytes per value and is bound by memory: 8191 x
// 4096 lifted for 6:8 (118 MB) 18.2 us, 6.5 TB/s (part of it from the last-level cache); with a
// selection also by its network, 2048 x 14336 at 8:16 (88 MB) 21.9 us, 4.0 TB/s; one row 2.5 us.
// (In a replayed graph; under the profiler the selection takes 24.)
#include "i8_device.h"

namespace {

using namespace nmk;

// Codes of a row: see the header comment.  nonfinite rows have c = 0 and are written as zeros.
struct RowScale {
  float c, b, y;   // a = x c (c = 127 f), b = amax f, y = 1 / b; f a power of two
  float scale;
  bool zero;       // every code is 0
};

__device__ __forceinline__ RowScale row_scale(uint32_t mk) {
  RowScale r;
  const float amax = __uint_as_float(mk << 16);
  const bool bad = mk >= 0x7F80u;   // infinity or NaN: it is the row's scale
  r.zero = bad || mk == 0;
  r.scale = bad ? amax : mk == 0 ? 1.0f : amax / 127.0f;
  const float f = amax < 0x1p-40f ? 0x1p90f : amax >= 0x1p40f ? 0x1p-80f : 1.0f;
  r.b = r.zero ? 1.0f : amax * f;
  r.y = 1.0f / r.b;
  r.c = 127.0f * f;
  return r;
}

// bits whose low byte is the code of x (bf16 in the high half of a dword)
__device__ __forceinline__ uint32_t code_bits(uint32_t xhi, const RowScale& r) {
  const float a = __uint_as_float(xhi) * r.c;
  float q = a * r.y;
  const float e = __builtin_fmaf(-q, r.b, a);
  q = __builtin_fmaf(e, r.y, q);
  return __float_as_uint(q + 12582912.0f);   // 1.5 * 2^23
}

// four codes of two packed dwords
__device__ __forceinline__ uint32_t codes4(uint32_t d0, uint32_t d1, const RowScale& r) {
  const uint32_t c0 = code_bits(d0 << 16, r), c1 = code_bits(d0 & 0xFFFF0000u, r);
  const uint32_t c2 = code_bits(d1 << 16, r), c3 = code_bits(d1 & 0xFFFF0000u, r);
  return __builtin_amdgcn_perm(c1, c0, 0x0C0C0400u) | __builtin_amdgcn_perm(c3, c2, 0x04000C0Cu);
}

__device__ __forceinline__ uint32_t max2(uint32_t mk, uint32_t d) {
  const uint32_t lo = d & 0x7FFFu, hi = (d >> 16) & 0x7FFFu;
  mk = lo > mk ? lo : mk;
  return hi > mk ? hi : mk;
}

// A thread's unit: PU pieces of 8 values (16 bytes of input, 8 bytes of codes), the least that
// holds whole groups; UN units per thread, the workgroup as many waves as the row needs (an
// idle unit costs its loads' and its network's instructions: 8192 x 4096 at 5:16 took 41 us with
// half of them idle, 25 with none).  WAVE: a row per wave, four rows a workgroup.
// SEL: 0 none, M the group width (NK > 0: n known at compile time).  LIFT: 0 none, 4 the N = 4
// lift from registers, 1 any N through LDS.
template <bool WAVE, int UN, int SEL, int NK, int LIFT>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void k_quant_i8(
    const uint16_t* __restrict__ x, int64_t rows, int k, int64_t ldx, int n, int ns, int8_t* __restrict__ q, int64_t ldq,
    float* __restrict__ scale) {
  constexpr int PU = SEL > 8 ? SEL / 8 : 1;
  __shared__ uint32_t red[WAVE ? 1 : 16];
  extern __shared__ __align__(16) unsigned char codes[];   // LIFT == 1: the rows' codes
  const int NT = WAVE ? 64 : (int)blockDim.x;              // threads of a row
  const int tid = WAVE ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
  const int64_t row = WAVE ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (WAVE && row >= rows) return;   // whole waves; no barrier below for these
  unsigned char* const row_codes = codes + (WAVE ? (threadIdx.x >> 6) * ((k + 15) / 16 * 16) : 0);
  const uint16_t* xr = x + row * ldx;
  int8_t* qr = q + row * ldq;
  const int units = (k + 8 * PU - 1) / (8 * PU);

  uint4 v[UN][PU];
#pragma unroll
  for (int u = 0; u < UN; ++u) {
    const int c = u * NT + tid;
#pragma unroll
    for (int p = 0; p < PU; ++p) {
      const int k0 = (c * PU + p) * 8;
      v[u][p] = make_uint4(0u, 0u, 0u, 0u);
      if (c < units && k0 < k) v[u][p] = *reinterpret_cast<const uint4*>(xr + k0);   // ldx % 8 == 0: inside the row
    }
  }
  uint32_t mk = 0;
#pragma unroll
  for (int u = 0; u < UN; ++u) {
    const int c = u * NT + tid;
#pragma unroll
    for (int p = 0; p < PU; ++p) {
      const int left = k - (c * PU + p) * 8;   // values of this piece inside the row
      uint32_t d[4] = {v[u][p].x, v[u][p].y, v[u][p].z, v[u][p].w};
      if (left < 8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = left >= 2 * j + 2 ? d[j] : left == 2 * j + 1 ? (d[j] & 0xFFFFu) : 0u;
        v[u][p] = make_uint4(d[0], d[1], d[2], d[3]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) mk = max2(mk, d[j]);
    }
  }
  // the selection needs no scale: it runs while the other waves' maxima arrive
  if constexpr (SEL > 0) {
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      uint32_t d[4 * PU];
#pragma unroll
      for (int p = 0; p < PU; ++p) {
        d[4 * p] = v[u][p].x;
        d[4 * p + 1] = v[u][p].y;
        d[4 * p + 2] = v[u][p].z;
        d[4 * p + 3] = v[u][p].w;
      }
      constexpr int G = 4 * PU / (SEL / 2);   // groups per unit (2 for m = 4, else 1)
#pragma unroll
      for (int g = 0; g < G; ++g) {
        uint32_t w[SEL / 2];
#pragma unroll
        for (int j = 0; j < SEL / 2; ++j) w[j] = d[g * (SEL / 2) + j];
        uint32_t bits;
        if constexpr (NK > 0) bits = topn_bits_n<SEL, NK>(w);
        else bits = topn_bits<SEL>(w, n);
#pragma unroll
        for (int j = 0; j < SEL / 2; ++j) d[g * (SEL / 2) + j] = mask_pair(w[j], bits >> (2 * j));
      }
#pragma unroll
      for (int p = 0; p < PU; ++p) v[u][p] = make_uint4(d[4 * p], d[4 * p + 1], d[4 * p + 2], d[4 * p + 3]);
    }
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)mk, off, 64);
    mk = o > mk ? o : mk;
  }
  if constexpr (!WAVE) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = mk;
    __syncthreads();
    mk = red[0];
    for (int w = 1; w < (int)(blockDim.x >> 6); ++w) mk = red[w] > mk ? red[w] : mk;
  }
  const RowScale rs = row_scale(mk);
  if (tid == 0) scale[row] = rs.scale;

  const int kq16 = (k + 15) / 16 * 16;   // written length of an unlifted row
#pragma unroll
  for (int u = 0; u < UN; ++u) {
    const int c = u * NT + tid;
#pragma unroll
    for (int p = 0; p < PU; ++p) {
      const int k0 = (c * PU + p) * 8;
      const uint4 d = v[u][p];
      uint2 o = make_uint2(codes4(d.x, d.y, rs), codes4(d.z, d.w, rs));
      if (rs.zero) o = make_uint2(0u, 0u);
      if constexpr (LIFT == 0) {
        if (k0 < kq16) *reinterpret_cast<uint2*>(qr + k0) = o;   // past k: zeros
      } else if constexpr (LIFT == 4) {
        // 8 values (k % 8 == 0) -> windows [0, 4), [2, 6), [4, 8)
        if (k0 < k) {
          uint32_t* dst = reinterpret_cast<uint32_t*>(qr + k0 / 8 * 12);
          dst[0] = o.x;
          dst[1] = (o.x >> 16) | (o.y << 16);
          dst[2] = o.y;
        }
      } else {
        if (k0 < kq16) *reinterpret_cast<uint2*>(row_codes + k0) = o;
      }
    }
  }
  if constexpr (LIFT == 4) {
    // zeros from 12 k / 8 up to a multiple of 16
    const int kl = k / 8 * 12, kl16 = (kl + 15) / 16 * 16;
    if (tid < (kl16 - kl) / 4) reinterpret_cast<uint32_t*>(qr + kl)[tid] = 0u;
  }
  if constexpr (LIFT == 1) {
    if constexpr (WAVE) wave_lds_fence();
    else __syncthreads();
    const uint32_t wpg = (uint32_t)(ns - 1);
    const int dwords = k / (2 * ns) * (ns - 1);
    const int quads = (dwords + 3) / 4;
    for (int i = tid; i < quads; i += NT) {
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t j = 4 * i + e, g = j / wpg, w = j - g * wpg;
        o[e] = 0u;
        if ((int)j < dwords) {
          const uint16_t* s = reinterpret_cast<const uint16_t*>(row_codes + 2 * (ns * g + w));
          o[e] = s[0] | ((uint32_t)s[1] << 16);
        }
      }
      *reinterpret_cast<uint4*>(qr + 16 * (int64_t)i) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <bool WAVE, int UN, int SEL, int NK, int LIFT>
hipError_t launch_q(int threads, const uint16_t* x, int64_t rows, int64_t k, int64_t ldx, int n, int ns, int8_t* q,
                    int64_t ldq, float* scale, hipStream_t s) {
  const size_t lds = LIFT == 1 ? (size_t)((k + 15) / 16 * 16) * (WAVE ? 4 : 1) : 0;
  constexpr int64_t kRows = (1 << 22) - 4;   // of a launch: a grid holds under 2^32 threads
  for (int64_t r = 0; r < rows; r += kRows) {
    const int64_t part = rows - r < kRows ? rows - r : kRows;
    k_quant_i8<WAVE, UN, SEL, NK, LIFT><<<dim3((unsigned)(WAVE ? (part + 3) / 4 : part)), dim3(WAVE ? 256 : threads), lds, s>>>(
        x + r * ldx, part, (int)k, ldx, n, ns, q + r * ldq, ldq, scale + r);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// A row per wave up to 2048 values (4 pieces a lane); longer rows 2 pieces a thread up to 4096 values
// (4 for groups of 32, whose unit is 4), 4 up to 32768, 8 beyond.
template <int SEL, int NK, int LIFT>
hipError_t by_length(const uint16_t* x, int64_t rows, int64_t k, int64_t ldx, int n, int ns, int8_t* q, int64_t ldq,
                     float* scale, hipStream_t s) {
  constexpr int PU = SEL > 8 ? SEL / 8 : 1;
  if (k <= 2048) return launch_q<true, 4 / PU, SEL, NK, LIFT>(256, x, rows, k, ldx, n, ns, q, ldq, scale, s);
  const int pieces = PU <= 2 && k <= 4096 ? 2 : k <= 32768 ? 4 : 8;
  const int threads = (int)(((k + 15) / 16 * 16 + 512 * pieces - 1) / (512 * pieces) * 64);
  if constexpr (PU <= 2) {
    if (pieces == 2) return launch_q<false, 2 / PU, SEL, NK, LIFT>(threads, x, rows, k, ldx, n, ns, q, ldq, scale, s);
  }
  if (pieces == 4) return launch_q<false, 4 / PU, SEL, NK, LIFT>(threads, x, rows, k, ldx, n, ns, q, ldq, scale, s);
  return launch_q<false, 8 / PU, SEL, NK, LIFT>(threads, x, rows, k, ldx, n, ns, q, ldq, scale, s);
}

// A thread per 16 bytes of output (offline, once a weight: 14336 x 4096 17.7 us): block s of row r holds the positions of slots
// [64 s, 64 s + 64), bytes past the row filled with the slots 0, 1, 0, 1 (0x44).
__global__ __launch_bounds__(256) void k_meta_step_block(const uint8_t* __restrict__ meta, int64_t o, int64_t kc,
                                                         int64_t steps, uint8_t* __restrict__ out) {
  const int64_t stride = (kc + 7) / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < steps * o; i += (int64_t)gridDim.x * 256) {
    const int64_t st = i / o, r = i - st * o;
    const uint8_t* src = meta + r * stride;
    uint32_t d[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      d[e] = 0u;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int64_t at = 16 * st + 4 * e + b;
        uint32_t v = at < stride ? src[at] : 0x44u;
        if (at == stride - 1 && (kc & 7) != 0) v = (v & 0x0Fu) | 0x40u;   // half a byte of slots
        d[e] |= v << (8 * b);
      }
    }
    *reinterpret_cast<uint4*>(out + 16 * i) = make_uint4(d[0], d[1], d[2], d[3]);
  }
}

}  // namespace

namespace nml {

hipError_t launch_quant_i8(const uint16_t* x, int64_t rows, int64_t k, int64_t ldx, int n, int m, int ns, int8_t* q,
                           int64_t ldq, float* scale, hipStream_t s) {
  if (rows <= 0) return hipSuccess;
  if (rows > 0x7FFFFFFF || k > 65536) return hipErrorInvalidValue;
  if (ns == 4) return by_length<0, 0, 4>(x, rows, k, ldx, n, ns, q, ldq, scale, s);
  if (ns > 2) return by_length<0, 0, 1>(x, rows, k, ldx, n, ns, q, ldq, scale, s);
  switch (m) {
    case 0: return by_length<0, 0, 0>(x, rows, k, ldx, n, ns, q, ldq, scale, s);
#define NM_CASE(M)                                                                             \
  case M:                                                                                      \
    if (n == M / 2) return by_length<M, M / 2, 0>(x, rows, k, ldx, n, ns, q, ldq, scale, s);   \
    return by_length<M, 0, 0>(x, rows, k, ldx, n, ns, q, ldq, scale, s);
    NM_CASE(4) NM_CASE(8) NM_CASE(16) NM_CASE(32)
#undef NM_CASE
  }
  return hipErrorInvalidValue;
}

hipError_t launch_meta_step_block(const uint8_t* meta, int64_t o, int64_t kc, uint8_t* out, hipStream_t s) {
  const int64_t steps = (kc + 127) / 128, n = steps * o;
  if (n <= 0) return hipSuccess;
  const int64_t blocks = (n + 255) / 256, most = 1 << 20;
  k_meta_step_block<<<dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, s>>>(meta, o, kc, steps, out);
  return hipGetLastError();
}

}  // namespace nml
