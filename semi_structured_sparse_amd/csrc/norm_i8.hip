// RMS norm of rows with the residual's addition, written as int8 codes with one scale per row,
// after an n:m selection or lifted for (2N-2):2N weights (SlideSparse page, technical summary 2.B;
// Flexible (N:M) Activation Sparsity page, 2.A).
//
//   s = x + r, rounded to the stream's type     p = fp32(s w)
//   rstd = 1 / sqrt(sum s^2 / k + eps)          y = bf16(p fp32(rstd))
//   q = the integer nearest to 127 p / max|p|   scale = max|p| rstd / 127
//
// The row's factor rstd multiplies value and maximum alike, so the codes do not hang on it, nor
// on the order of the sum: they are those of p, and exact.  p has 24 bits, where one fp32
// quotient may fall on the wrong side of a half: t = p fp32(127 / max) is off by at most 127 *
// 2^-23 = 1.52e-5 (the quotient and the product round once each), so a code whose t lies more
// than 2e-5 from a half is right, and the others, one in 25000, are divided again in fp64.
// There 127 p is exact.  With p = P 2^a, max = M 2^b, P and M integers under 2^24, and a half (2 j + 1) / 2
// the difference is (254 P - (2 j + 1) M 2^(b - a)) / (2 M 2^(b - a)): no half, its numerator is 1 at
// least, 2 if b > a, and b - a is 8 at most where |p| passes max / 256, which every half does (1 / 254
// of max): over 2^-32 of a unit (127 (128 n - 1) / (256 (127 n - 1)) comes that near), and an fp64
// quotient of at most 127 is off by 2^-47.
// The sum of squares is carried in fp64, so that no row overflows it.
//
// One pass: a row's p stay in registers between the reductions (the largest |p| and the sum
// cross the workgroup together) and the outputs.  y is rounded to bf16 once; the codes come from the
// unrounded p.  Bound by memory: 4095 x 4096 bf16 with residual, sum, y and the 6:8 lift 34.5 us (5.6
// TB/s; a copy of 512 MB 5.35), 8192 x 8192 86 (5.5 TB/s), 8:16 94 (5.0); one row of 4096 3.7, a launch
// and two memory latencies.
#include "i8_device.h"
#include "layer_launch.h"

namespace {

using namespace nmk;
using namespace nml;

struct RowCode {
  float f, r;        // t = (p f) r: f a power of two that keeps r finite, r = 127 / (max f)
  float amax;
  bool zero;         // every code is 0
};

__device__ __forceinline__ RowCode row_code(uint32_t mk) {
  RowCode c;
  c.amax = __uint_as_float(mk);
  c.zero = mk == 0 || mk >= 0x7F800000u;
  c.f = c.amax < 0x1p-40f ? 0x1p90f : 1.0f;
  c.r = c.zero ? 0.0f : 127.0f / (c.amax * c.f);
  return c;
}

// bits whose low byte is the code of p
__device__ __forceinline__ uint32_t code_of(float p, const RowCode& c) {
  const float t = (p * c.f) * c.r;
  const float u = t + 12582912.0f;               // 1.5 * 2^23: the nearest integer, ties to even
  const float d = t - (u - 12582912.0f);
  uint32_t b = __float_as_uint(u);
  if (__builtin_expect(__builtin_fabsf(d) > 0.49998f, 0)) b = (uint32_t)(int)__builtin_rint(127.0 * (double)p / (double)c.amax);
  return b;
}

__device__ __forceinline__ uint32_t codes4(const float* p, const RowCode& c) {
  const uint32_t c0 = code_of(p[0], c), c1 = code_of(p[1], c), c2 = code_of(p[2], c), c3 = code_of(p[3], c);
  return __builtin_amdgcn_perm(c1, c0, 0x0C0C0400u) | __builtin_amdgcn_perm(c3, c2, 0x04000C0Cu);
}

// The value of the lane that PERM (two bits a lane) names in each quad.
template <int PERM>
__device__ __forceinline__ uint32_t quad(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, PERM, 0xF, 0xF, true);
}
constexpr int kSwap1 = 0xB1, kSwap2 = 0x4E, kTurn = 0x1B;   // lanes 1 0 3 2, 2 3 0 1, 3 2 1 0

// Eight keys that fall, then rise or the other way round, into falling order.
__device__ __forceinline__ void settle8(uint32_t (&s)[8]) {
#pragma unroll
  for (int d = 4; d >= 1; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((i & d) == 0) {
        const uint32_t x = s[i], y = s[i + d];
        s[i] = max(x, y);
        s[i + d] = min(x, y);
      }
}
// s against PERM's lane, its keys turned round: the larger ones where `up`, else the smaller ones.
// Of two falling runs these are their larger and their smaller half.
template <int PERM, bool TURN>
__device__ __forceinline__ void halve(uint32_t (&s)[8], bool up) {
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = quad<PERM>(s[TURN ? 7 - i : i]);
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = up ? max(s[i], o[i]) : min(s[i], o[i]);
}

// What a group keeps, its n largest magnitudes, ties to the lower index: every value whose key (the
// bits of |p|) is at least tau, the n-th largest, but not those of drop, the last of equal ones where
// the (n + 1)-th is tau too.  A lane holds 8 values: two groups of 4 (G = 0, 1), a group of 8, half
// of one of 16, a quarter of one of 32.  Wide groups are sorted within the lane and then across
// lanes by halving: where n = M / 2 (NK), the larger half's least key is tau.  (A whole group a lane
// takes the row in pieces with gaps between the lanes', for loads and stores alike: 8192 x 8192 8:16
// 107 us instead of 94, 16:32 145 instead of
// 98.)
struct Kept {
  uint32_t tau, drop;
};
template <int M, int NK>
__device__ __forceinline__ Kept kept(const float* p, int n) {
  constexpr int W = M < 8 ? M : 8;   // of the group in this lane
  const int lane = threadIdx.x & 63;
  if constexpr (NK > 0) n = NK;
  uint32_t k[W], s[W];
#pragma unroll
  for (int i = 0; i < W; ++i) s[i] = k[i] = __float_as_uint(p[i]) & 0x7FFFFFFFu;
  sort_desc_oem<W>(s);
  uint32_t tau, next;
  if constexpr (M > 8 && NK == M / 2) {
    if constexpr (M == 32) {
      halve<kSwap1, true>(s, (lane & 1) == 0);
      settle8(s);
    }
    constexpr int FAR = M == 32 ? kTurn : kSwap1;
    uint32_t lo[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) lo[i] = quad<FAR>(s[7 - i]);
    tau = max(s[0], lo[0]);
    next = min(s[0], lo[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      tau = min(tau, max(s[i], lo[i]));
      next = max(next, min(s[i], lo[i]));
    }
    if constexpr (M == 32) {
      tau = min(tau, quad<kSwap1>(tau));
      next = max(next, quad<kSwap1>(next));
    }
  } else {
    if constexpr (M > 8) {
      halve<kSwap1, true>(s, (lane & 1) == 0);
      settle8(s);
    }
    if constexpr (M == 32) {
      halve<kTurn, true>(s, (lane & 2) == 0);
      halve<kSwap1, false>(s, (lane & 1) == 0);
      settle8(s);
    }
    // rank n - 1 and n of the group: its lane q holds ranks [8 q, 8 q + 8)
    const int q = M == 32 ? lane & 3 : M == 16 ? lane & 1 : 0;
    tau = next = 0u;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      tau = 8 * q + j == n - 1 ? s[j] : tau;
      next = 8 * q + j == n ? s[j] : next;
    }
    if constexpr (M > 8) {
      tau |= quad<kSwap1>(tau);
      next |= quad<kSwap1>(next);
    }
    if constexpr (M == 32) {
      tau |= quad<kSwap2>(tau);
      next |= quad<kSwap2>(next);
    }
  }
  Kept o{tau, 0u};
  if (__any(next == tau && tau != 0u)) {   // zeros are zeros, kept or dropped
    int above = 0, equal = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      above += k[i] > tau ? 1 : 0;
      equal += k[i] == tau ? 1 : 0;
    }
    int before = 0;   // equal ones in the group's earlier lanes
    if constexpr (M > 8) {
      above += (int)quad<kSwap1>((uint32_t)above);
      const int other = (int)quad<kSwap1>((uint32_t)equal);
      before = lane & 1 ? other : 0;
      if constexpr (M == 32) {
        above += (int)quad<kSwap2>((uint32_t)above);
        const int far = (int)quad<kSwap2>((uint32_t)(equal + other));
        before += lane & 2 ? far : 0;
      }
    }
    int left = n - above - before;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const bool eq = k[i] == tau;
      o.drop |= (eq && left <= 0 ? 1u : 0u) << i;
      left -= eq ? 1 : 0;
    }
  }
  return o;
}

__device__ __forceinline__ void widen(const uint4& d, float* v) {
  const uint32_t e[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(e[j] << 16);
    v[2 * j + 1] = __uint_as_float(e[j] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void as_floats(const uint4& a, const uint4& b, float* v) {
  const uint32_t e[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(e[j]);
}

// two fp32 values as packed bf16, to nearest even
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

__device__ __forceinline__ uint4 narrow(const float* v) {
  uint32_t e[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) e[j] = bf16x2(v[2 * j], v[2 * j + 1]);
  return make_uint4(e[0], e[1], e[2], e[3]);
}

// P pieces of 8 values a thread, the workgroup as many waves as the row needs.
// WAVE: a row per wave, four rows a workgroup.  SEL: 0 none, M the group width (NK > 0: n known
// at compile time).  LIFT: 0 none, 4 the N = 4 lift from registers, 1 any N through LDS.
template <bool WAVE, int P, int SEL, int NK, int LIFT>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void k_rmsnorm_i8(NormArgs a) {
  __shared__ uint32_t red_max[WAVE ? 1 : 16];
  __shared__ double red_sum[WAVE ? 1 : 16];
  extern __shared__ __align__(16) unsigned char codes[];   // LIFT == 1: the rows' codes
  const int NT = WAVE ? 64 : (int)blockDim.x;              // threads of a row
  const int tid = WAVE ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
  const int64_t row = WAVE ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (WAVE && row >= a.rows) return;   // whole waves; no barrier below for these
  const int k = (int)a.k;
  auto at = [&](int i) { return (i * NT + tid) * 8; };   // first value of piece i

  // every load of the row first: rows are readable in whole pieces (leading dimensions % 8 == 0)
  uint4 xa[P], xb[P], ra[P], rb[P];
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < P; ++i) xa[i] = xb[i] = ra[i] = rb[i] = zero;
  if (a.x_bf16) {
    const uint16_t* xr = static_cast<const uint16_t*>(a.x) + row * a.ldx;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (at(i) < k) xa[i] = *reinterpret_cast<const uint4*>(xr + at(i));
  } else {
    const float* xr = static_cast<const float*>(a.x) + row * a.ldx;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (at(i) < k) {
        xa[i] = *reinterpret_cast<const uint4*>(xr + at(i));
        xb[i] = *reinterpret_cast<const uint4*>(xr + at(i) + 4);
      }
  }
  if (a.r != nullptr) {
    if (a.r_bf16) {
      const uint16_t* rr = static_cast<const uint16_t*>(a.r) + row * a.ldr;
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (at(i) < k) ra[i] = *reinterpret_cast<const uint4*>(rr + at(i));
    } else {
      const float* rr = static_cast<const float*>(a.r) + row * a.ldr;
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (at(i) < k) {
          ra[i] = *reinterpret_cast<const uint4*>(rr + at(i));
          rb[i] = *reinterpret_cast<const uint4*>(rr + at(i) + 4);
        }
    }
  }
  float p[P][8];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int left = k - at(i);
#pragma unroll
    for (int j = 0; j < 8; ++j) p[i][j] = 1.0f;
    if (a.weight == nullptr) continue;
    if (left >= 8) {
      as_floats(*reinterpret_cast<const uint4*>(a.weight + at(i)), *reinterpret_cast<const uint4*>(a.weight + at(i) + 4), p[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left) p[i][j] = a.weight[at(i) + j];
    }
  }

  uint32_t mk = 0;
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int left = k - at(i);   // values of this piece inside the row
    float s[8];
    if (a.x_bf16) widen(xa[i], s);
    else as_floats(xa[i], xb[i], s);
    if (a.r != nullptr) {
      float r[8];
      if (a.r_bf16) {
        widen(ra[i], r);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = s[j] + r[j];
        const uint4 d = narrow(s);   // the stream's type holds the sum: what is normed is what is stored
        widen(d, s);
        if (a.sum_out != nullptr) {
          uint16_t* o = static_cast<uint16_t*>(a.sum_out) + row * a.lds + at(i);
          if (left >= 8) {
            *reinterpret_cast<uint4*>(o) = d;
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (j < left) o[j] = (uint16_t)(__float_as_uint(s[j]) >> 16);
          }
        }
      } else {
        as_floats(ra[i], rb[i], r);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = s[j] + r[j];
        if (a.sum_out != nullptr) {
          float* o = static_cast<float*>(a.sum_out) + row * a.lds + at(i);
          if (left >= 8) {
            *reinterpret_cast<f32x4*>(o) = f32x4{s[0], s[1], s[2], s[3]};
            *reinterpret_cast<f32x4*>(o + 4) = f32x4{s[4], s[5], s[6], s[7]};
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (j < left) o[j] = s[j];
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s[j] = j < left ? s[j] : 0.0f;             // what lies past the row
      ss = __builtin_fma((double)s[j], (double)s[j], ss);
      p[i][j] = s[j] * p[i][j];
      const uint32_t m = __float_as_uint(p[i][j]) & 0x7FFFFFFFu;
      mk = m > mk ? m : mk;
    }
  }
  // the normed row's factor needs the reductions, the selection does not: it runs while the other
  // waves' arrive.  Dropped values are zeroed after the normed row is written.
  constexpr int GROUPS = SEL == 4 ? 2 : 1, GW = SEL == 4 ? 4 : 8;   // of a piece, and their values
  Kept keep[SEL > 0 ? P : 1][GROUPS];
  if constexpr (SEL > 0) {
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) keep[i][g] = kept<SEL, NK>(p[i] + g * GW, a.n);
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)mk, off, 64);
    mk = o > mk ? o : mk;
    ss += __shfl_xor(ss, off, 64);
  }
  if constexpr (!WAVE) {
    if ((threadIdx.x & 63) == 0) {
      red_max[threadIdx.x >> 6] = mk;
      red_sum[threadIdx.x >> 6] = ss;
    }
    __syncthreads();
    mk = red_max[0];
    ss = red_sum[0];
    for (int w = 1; w < (int)(blockDim.x >> 6); ++w) {
      mk = red_max[w] > mk ? red_max[w] : mk;
      ss += red_sum[w];
    }
  }
  const double rstd = 1.0 / __builtin_sqrt(ss / (double)(k > 0 ? k : 1) + (double)a.eps);
  const RowCode rc = row_code(mk);
  if (tid == 0) a.scale[row] = mk == 0 ? 1.0f : mk >= 0x7F800000u ? rc.amax : (float)((double)rc.amax * rstd / 127.0);
  if (a.y != nullptr) {
    const float f = (float)rstd;
    uint16_t* yr = a.y + row * a.ldy;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int left = k - at(i);
      if (left <= 0) continue;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = p[i][j] * f;
      const uint4 d = narrow(v);
      if (left >= 8) {
        *reinterpret_cast<uint4*>(yr + at(i)) = d;
      } else {
        const uint32_t e[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < left) yr[at(i) + j] = (uint16_t)(e[j >> 1] >> (16 * (j & 1)));
      }
    }
  }
  if constexpr (SEL > 0) {
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        const Kept w = keep[i][g];
#pragma unroll
        for (int e = 0; e < GW; ++e) {
          float& v = p[i][g * GW + e];
          v = (__float_as_uint(v) & 0x7FFFFFFFu) >= w.tau ? v : 0.0f;
        }
        if (__any(w.drop != 0u)) {
#pragma unroll
          for (int e = 0; e < GW; ++e)
            if ((w.drop >> e) & 1u) p[i][g * GW + e] = 0.0f;
        }
      }
  }

  int8_t* qr = a.q + row * a.ldq;
  unsigned char* const row_codes = codes + (WAVE ? (threadIdx.x >> 6) * ((k + 15) / 16 * 16) : 0);
  const int kq16 = (k + 15) / 16 * 16;   // written length of an unlifted row
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int k0 = at(i);
    uint2 o = make_uint2(codes4(p[i], rc), codes4(p[i] + 4, rc));
    if (rc.zero) o = make_uint2(0u, 0u);
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
  if constexpr (LIFT == 4) {
    // zeros from 12 k / 8 up to a multiple of 16
    const int kl = k / 8 * 12, kl16 = (kl + 15) / 16 * 16;
    if (tid < (kl16 - kl) / 4) reinterpret_cast<uint32_t*>(qr + kl)[tid] = 0u;
  }
  if constexpr (LIFT == 1) {
    if constexpr (WAVE) wave_lds_fence();
    else __syncthreads();
    const uint32_t wpg = (uint32_t)(a.ns - 1);
    const int dwords = k / (2 * a.ns) * (a.ns - 1);
    const int quads = (dwords + 3) / 4;
    for (int i = tid; i < quads; i += NT) {
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t j = 4 * i + e, g = j / wpg, w = j - g * wpg;
        o[e] = 0u;
        if ((int)j < dwords) {
          const uint16_t* s = reinterpret_cast<const uint16_t*>(row_codes + 2 * (a.ns * g + w));
          o[e] = s[0] | ((uint32_t)s[1] << 16);
        }
      }
      *reinterpret_cast<uint4*>(qr + 16 * (int64_t)i) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <bool WAVE, int P, int SEL, int NK, int LIFT>
hipError_t launch_n(int threads, const NormArgs& a, hipStream_t s) {
  const size_t lds = LIFT == 1 ? (size_t)((a.k + 15) / 16 * 16) * (WAVE ? 4 : 1) : 0;
  constexpr int64_t kRows = (1 << 22) - 4;   // of a launch: a grid holds under 2^32 threads
  for (int64_t r = 0; r < a.rows; r += kRows) {
    NormArgs b = a;
    b.rows = a.rows - r < kRows ? a.rows - r : kRows;
    b.x = static_cast<const char*>(a.x) + r * a.ldx * (a.x_bf16 ? 2 : 4);
    if (a.r != nullptr) b.r = static_cast<const char*>(a.r) + r * a.ldr * (a.r_bf16 ? 2 : 4);
    if (a.sum_out != nullptr) b.sum_out = static_cast<char*>(a.sum_out) + r * a.lds * (a.r_bf16 ? 2 : 4);
    if (a.y != nullptr) b.y = a.y + r * a.ldy;
    b.q = a.q + r * a.ldq;
    b.scale = a.scale + r;
    k_rmsnorm_i8<WAVE, P, SEL, NK, LIFT>
        <<<dim3((unsigned)(WAVE ? (b.rows + 3) / 4 : b.rows)), dim3(WAVE ? 256 : threads), lds, s>>>(b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// A row per wave up to 2048 values (4 pieces a lane), no barrier; longer rows 2 pieces a thread up to
// 12288 values, 4 beyond (us, 2 / 4 pieces: 8192 x 5120 58 / 62, 8192 x 8192 86 / 90, 8:16 94 / 93, 6000 x
// 10240 86 / 106, 4096 x 12288 69 / 85, 8:16 74 / 96, 6:8 lift 73 / 88, 4096 x 14336 6:8 lift 96 / 94, 4096 x
// 16384 8:16 127 / 99: 1024 threads of over 64 registers are alone on a CU).
template <int SEL, int NK, int LIFT>
hipError_t by_length(const NormArgs& a, hipStream_t s) {
  if (a.k <= 2048) return launch_n<true, 4, SEL, NK, LIFT>(256, a, s);
  const int pieces = a.k <= 12288 ? 2 : 4;
  const int threads = (int)(((a.k + 15) / 16 * 16 + 512 * pieces - 1) / (512 * pieces) * 64);
  return pieces == 2 ? launch_n<false, 2, SEL, NK, LIFT>(threads, a, s) : launch_n<false, 4, SEL, NK, LIFT>(threads, a, s);
}

}  // namespace

namespace nml {

hipError_t launch_rmsnorm_i8(const NormArgs& a, hipStream_t s) {
  if (a.rows <= 0) return hipSuccess;
  if (a.rows > 0x7FFFFFFF || a.k > 32768) return hipErrorInvalidValue;
  if (a.ns == 4) return by_length<0, 0, 4>(a, s);
  if (a.ns > 2) return by_length<0, 0, 1>(a, s);
  switch (a.m) {
    case 0: return by_length<0, 0, 0>(a, s);
#define NM_CASE(M)                                      \
  case M:                                               \
    if (a.n == M / 2) return by_length<M, M / 2, 0>(a, s); \
    return by_length<M, 0, 0>(a, s);
    NM_CASE(4) NM_CASE(8) NM_CASE(16) NM_CASE(32)
#undef NM_CASE
  }
  return hipErrorInvalidValue;
}

}  // namespace nml
