// bf16 products of few tokens (and of any shape) with an epilogue: the weights streamed from HBM
// straight into the operand registers of the matrix instructions.
//
//   y[t][o] = residual[t][o] + fn(sum_k x[t][k] w[o][k] + bias[o]),  W dense or 2:4
//
// With few tokens the weights' bytes bound the call: a workgroup owns 16 RW output rows, its waves
// share the reduction in contiguous parts, and each lane loads 16-byte weight pieces in operand
// layout, one batch of steps ahead of the one being multiplied; X, in L2, follows the same path.
// The waves' partial tiles are added in LDS, in their order, and leave through the epilogue.
// Where row blocks are too few to fill the chip the reduction is also cut across workgroups,
// whose partial sums a second kernel adds, again in order: a call's bits do not depend on timing.
// Sums are fp32 throughout; a bf16 output is rounded once, behind the epilogue.
//
// 1 x 4096 x 4096 from HBM 9.9 us (floor 5.9 at 5.7 TB/s, the rest launch, two memory latencies and the
// sum in LDS; 9.4 a call with weights from the cache), 2:4 9.0; 1 x 4096 x 14336 25.0 (floor 20.6).
//
// Operands: v_mfma_f32_16x16x32_bf16 takes from lane l eight values of row l % 16 at position
// 8 (l / 16) of a 32-position step, both sides alike.  v_smfmac_f32_16x16x64_bf16 takes the eight
// kept values of positions [16 (l / 16), + 16) of a 64-position step with their 16 bits of
// positions, and from X the values [8 (l / 16), + 8) and [32 + 8 (l / 16), + 8).
#include "lin_device.h"

namespace {

using namespace nmk;
using namespace nml;

constexpr int64_t kGridY = 65535;   // workgroups of tokens in the grid's y; more go on in z

// TB: blocks of 16 tokens; RW: blocks of 16 output rows; SP: 2:4 weights.
template <int TB, int RW, bool SP>
struct FewCfg {
  static constexpr int STEP = SP ? 64 : 32;                          // positions per matrix step
  static constexpr int REGS = RW * (SP ? 5 : 4) + TB * (SP ? 8 : 4);   // of one step's operands
  // registers of a wave: 128 (16 waves a workgroup) or 256 (8); two batches are live
  static constexpr bool BIG = TB >= 4;
  static constexpr int FIT = ((BIG ? 256 : 128) - 28 - 4 * RW * TB - 2 * (RW * (SP ? 2 : 1) + TB)) / (2 * REGS);
  static constexpr int UNROLL = FIT < 1 ? 1 : FIT > 8 ? 8 : FIT;
};

template <int TB, int RW, bool SP>
__global__ __launch_bounds__(TB >= 4 ? 512 : 1024) void k_lin_few(
    const uint16_t* __restrict__ x, int64_t ldx, const uint16_t* __restrict__ w, int64_t ldw,
    const uint8_t* __restrict__ meta, int64_t T, int64_t O, int k, LinEpi epi, float* __restrict__ part, int splits) {
  using C = FewCfg<TB, RW, SP>;
  constexpr int U = C::UNROLL;
  extern __shared__ __align__(16) float red[];   // [waves][RW][16 TB][16]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int fr = lane & 15, fq = lane >> 4;
  const int64_t nob = (O + 16 * RW - 1) / (16 * RW);
  const int64_t ob = blockIdx.x % nob, t0 = (blockIdx.y + (int64_t)blockIdx.z * kGridY) * 16 * TB;
  if (t0 >= T) return;   // the whole workgroup, in the last of z
  const int split = (int)(blockIdx.x / nob);
  const int steps = (k + C::STEP - 1) / C::STEP;
  const int P = splits * waves, p = split * waves + wave;
  const int s0 = (int)((int64_t)p * steps / P), s1 = (int)((int64_t)(p + 1) * steps / P);

  const uint16_t* xrow[TB];
#pragma unroll
  for (int j = 0; j < TB; ++j) {
    const int64_t t = t0 + 16 * j + fr;
    xrow[j] = x + (t < T ? t : T - 1) * ldx + 8 * fq;
  }
  const uint16_t* wrow[RW];
  const uint8_t* mrow[RW];
#pragma unroll
  for (int a = 0; a < RW; ++a) {
    int64_t o = (ob * RW + a) * 16 + fr;
    o = o < O ? o : O - 1;
    wrow[a] = w + o * ldw + 8 * fq;
    mrow[a] = SP ? meta + o * 16 + 2 * fq : nullptr;
  }
  f32x4 acc[RW][TB];
#pragma unroll
  for (int a = 0; a < RW; ++a)
#pragma unroll
    for (int j = 0; j < TB; ++j) acc[a][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  struct Batch {
    u32x4 w[U][RW];
    int m[U][SP ? RW : 1];
    u32x4 xl[U][TB], xh[U][SP ? TB : 1];
  };
  const int wlen = SP ? k / 2 : k;        // values of a weight row
  // whole: the step lies inside the part and the row on both sides; otherwise what lies past
  // either comes as zeros (whatever a row's padding holds)
  auto piece = [&](const uint16_t* row, int off, int left) {   // left: values of the piece inside
    const u32x4 v = *reinterpret_cast<const u32x4*>(left > 0 ? reinterpret_cast<const void*>(row + off) : &kZero16);
    return head_of(v, left);
  };
  auto fetch = [&](Batch& b, int s, bool whole) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = s + u, wo = q * 32, xo = q * C::STEP;
      if (whole) {
#pragma unroll
        for (int a = 0; a < RW; ++a) {
          b.w[u][a] = *reinterpret_cast<const u32x4*>(wrow[a] + wo);
          if constexpr (SP) b.m[u][a] = *reinterpret_cast<const uint16_t*>(mrow[a] + (q >> 1) * (O * 16) + 8 * (q & 1));
        }
#pragma unroll
        for (int j = 0; j < TB; ++j) {
          b.xl[u][j] = *reinterpret_cast<const u32x4*>(xrow[j] + xo);
          if constexpr (SP) b.xh[u][j] = *reinterpret_cast<const u32x4*>(xrow[j] + xo + 32);
        }
      } else {
        const bool in = q < s1;
        const int qm = in ? q : s1 - 1;
#pragma unroll
        for (int a = 0; a < RW; ++a) {
          b.w[u][a] = piece(wrow[a], wo, in ? wlen - wo - 8 * fq : 0);
          if constexpr (SP) b.m[u][a] = *reinterpret_cast<const uint16_t*>(mrow[a] + (qm >> 1) * (O * 16) + 8 * (qm & 1));
        }
#pragma unroll
        for (int j = 0; j < TB; ++j) {
          b.xl[u][j] = piece(xrow[j], xo, in ? k - xo - 8 * fq : 0);
          if constexpr (SP) b.xh[u][j] = piece(xrow[j], xo + 32, in ? k - xo - 32 - 8 * fq : 0);
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);   // the next batch's loads stay ahead of this one's products
  };
  auto consume = [&](const Batch& b) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < TB; ++j) {
        if constexpr (SP) {
          const u32x8 both = __builtin_shufflevector(b.xl[u][j], b.xh[u][j], 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
          for (int a = 0; a < RW; ++a)
            acc[a][j] = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(__builtin_bit_cast(bf16x8, b.w[u][a]),
                                                                  __builtin_bit_cast(bf16x16, both), acc[a][j], b.m[u][a], 0, 0);
        } else {
#pragma unroll
          for (int a = 0; a < RW; ++a)
            acc[a][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b.w[u][a]),
                                                                __builtin_bit_cast(bf16x8, b.xl[u][j]), acc[a][j], 0, 0, 0);
        }
      }
  };
  // batches of U steps, one in flight ahead of the one multiplied; the last one may pass the
  // part's or the row's end and is loaded with checks
  const int nb = (s1 - s0 + U - 1) / U;
  if (nb > 0) {
    Batch b0, b1;
    int b = 0;
    if (nb > 1) {
      fetch(b0, s0, true);
      for (; b + 3 < nb; b += 2) {
        fetch(b1, s0 + (b + 1) * U, true);
        consume(b0);
        fetch(b0, s0 + (b + 2) * U, true);
        consume(b1);
      }
      if (b + 3 == nb) {
        fetch(b1, s0 + (b + 1) * U, true);
        consume(b0);
        fetch(b0, s0 + (b + 2) * U, false);
        consume(b1);
        consume(b0);
      } else {
        fetch(b1, s0 + (b + 1) * U, false);
        consume(b0);
        consume(b1);
      }
    } else {
      fetch(b0, s0, false);
      consume(b0);
    }
  }

  // the waves' partial tiles: red[wave][a][token][row]
  constexpr int TILE = RW * TB * 256;
#pragma unroll
  for (int a = 0; a < RW; ++a)
#pragma unroll
    for (int j = 0; j < TB; ++j)
      *reinterpret_cast<f32x4*>(red + wave * TILE + ((a * TB + j) * 16 + fr) * 16 + 4 * fq) = acc[a][j];
  __syncthreads();
  const int64_t o4 = (O + 3) / 4 * 4;
  for (int e = threadIdx.x; e < TILE; e += blockDim.x) {
    const int r = e % (16 * RW), tl = e / (16 * RW);
    const int64_t o = ob * 16 * RW + r, t = t0 + tl;
    if (o >= O || t >= T) continue;
    const int at = ((r >> 4) * TB * 16 + tl) * 16 + (r & 15);
    float v = 0.0f;
    for (int wv = 0; wv < waves; ++wv) v += red[wv * TILE + at];
    if (part != nullptr) part[((int64_t)split * T + t) * o4 + o] = v;
    else lin_store(epi, v, t, o);
  }
}

// y from the splits' sums, part[split][t][o4]: one thread per 4 outputs, every load of up to 8
// splits in flight together.  whole: O and the rows of y and the residual keep their alignment.
__global__ __launch_bounds__(256) void k_lin_reduce(const float* __restrict__ part, int splits, uint32_t T, uint32_t O,
                                                    LinEpi epi, int whole) {
  const uint32_t q = (O + 3) / 4;
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= T * q) return;
  const uint32_t t = i / q, o = (i - t * q) * 4;
  const int64_t stride = (int64_t)T * (4 * q);
  const float* p = part + 4 * (int64_t)i;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  for (int b = 0; b < splits; b += 8) {
    f32x4 v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = *reinterpret_cast<const f32x4*>(p + (b + e < splits ? b + e : 0) * stride);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (b + e >= splits) break;
#pragma unroll
      for (int r = 0; r < 4; ++r) s[r] = s[r] + v[e][r];
    }
  }
  if (whole) {
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    if (epi.residual != nullptr) r = epi.bf16_out ? lin_load4<true>(epi, t, o) : lin_load4<false>(epi, t, o);
    float v[4] = {s[0], s[1], s[2], s[3]};
    if (epi.bias != nullptr) {
      const f32x4 b = *reinterpret_cast<const f32x4*>(epi.bias + o);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = v[e] + b[e];
    }
    lin_fns<4>(v, epi.fn);
    lin_store4(epi, v, r, t, o);
    return;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (o + r < O) lin_store(epi, s[r], t, o + r);
}

struct FewPlan {
  int tb, rw, waves;
  int64_t splits;
};

// Row blocks of a workgroup: every workgroup reads all of X again, so as many as leave 200
// workgroups.  Waves: four where there are 192 workgroups, whose two batches each keep enough loads
// in flight (1 x 4096 x 4096 with 4 / 8 / 16 waves: 10.2 / 10.1 / 10.6 us, 2:4 8.1 / 8.6 / 9.2, 4 x 4096
// x 14336 28.6 / 30.3 / 29.1).  Below, eight, and the reduction split up to one workgroup per CU,
// four steps a wave at least, if a wave has over eight unsplit (1 x 1024 x 4096: 16 waves unsplit
// 8.4 us, 16 in two ranges 8.2, 8 in four 7.7); sixteen where that leaves one range (1 x 256 x 2048:
// 5.2).
FewPlan few_plan(int64_t t, int64_t o, int64_t k, bool sparse) {
  FewPlan p;
  p.tb = t <= 16 ? 1 : t <= 32 ? 2 : 4;
  const int64_t steps = (k + (sparse ? 63 : 31)) / (sparse ? 64 : 32);
  const int64_t gy = (t + 16 * p.tb - 1) / (16 * p.tb);
  p.rw = p.tb > 2 ? 1 : p.tb == 2 ? 2 : 4;
  while (p.rw > 1 && ((o + 16 * p.rw - 1) / (16 * p.rw)) * gy < 200) p.rw /= 2;
  const int64_t blocks = ((o + 16 * p.rw - 1) / (16 * p.rw)) * gy;
  p.waves = blocks >= 192 ? 4 : 8;
  int64_t s = blocks > 0 ? 256 / blocks : 1;
  const int64_t room = steps / (4 * p.waves);
  if (s > room) s = room;
  if (steps <= 8 * p.waves) s = 1;
  p.splits = s < 2 ? 1 : s > 16 ? 16 : s;
  if (blocks <= 32 && p.splits == 1 && p.tb < 4 && steps >= 32) p.waves = 16;   // up to 32 KiB of partial tiles
  return p;
}

template <int TB, int RW, bool SP>
hipError_t few_launch(const LinArgs& a, const FewPlan& pl, float* part, hipStream_t s) {
  const int64_t nob = (a.o + 16 * RW - 1) / (16 * RW), gy = (a.t + 16 * TB - 1) / (16 * TB);
  const int64_t gz = (gy + kGridY - 1) / kGridY;
  if (nob * pl.splits * 64 * pl.waves > 0xFFFFFFFFll || gz > 65535) return hipErrorInvalidConfiguration;
  const size_t lds = (size_t)pl.waves * RW * TB * 256 * 4;
  k_lin_few<TB, RW, SP><<<dim3((unsigned)(nob * pl.splits), (unsigned)(gz > 1 ? kGridY : gy), (unsigned)gz), dim3(64 * pl.waves),
                          lds, s>>>(a.x, a.ldx, a.w, a.ldw, a.meta, a.t, a.o, (int)a.k, a.epi,
                                    pl.splits > 1 ? part : nullptr, (int)pl.splits);
  a.route.note(NM_TAKEN_FEW_STREAM | (SP ? NM_TAKEN_SPARSE_MMA : 0u));
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || pl.splits == 1) return e;
  return launch_lin_reduce(part, pl.splits, a.t, a.o, a.epi, a.route, s);
}

template <int TB, bool SP>
hipError_t few_rows(const LinArgs& a, const FewPlan& pl, float* part, hipStream_t s) {
  if constexpr (TB == 1) {
    if (pl.rw == 4) return few_launch<TB, 4, SP>(a, pl, part, s);
  }
  if constexpr (TB <= 2) {
    if (pl.rw == 2) return few_launch<TB, 2, SP>(a, pl, part, s);
  }
  return few_launch<TB, 1, SP>(a, pl, part, s);
}

}  // namespace

namespace nml {

hipError_t launch_lin_reduce(const float* part, int64_t splits, int64_t t, int64_t o, const LinEpi& e, const Route& r,
                             hipStream_t s) {
  const int64_t n = t * ((o + 3) / 4);
  if (n <= 0) return hipSuccess;
  if (n > 0x3FFFFFFF) return hipErrorInvalidConfiguration;   // plans split far smaller outputs only
  k_lin_reduce<<<dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s>>>(part, (int)splits, (uint32_t)t, (uint32_t)o, e,
                                                                         o % 4 == 0 && lin_whole(e));
  r.note(NM_TAKEN_REDUCE);
  return hipGetLastError();
}

int64_t lin_few_part_bytes(int64_t t, int64_t o, int64_t k, bool sparse) {
  const FewPlan p = few_plan(t, o, k, sparse);
  return p.splits > 1 ? p.splits * t * ((o + 3) / 4 * 4) * 4 : 0;
}

hipError_t launch_lin_few(const LinArgs& a, float* part, int64_t part_bytes, hipStream_t s) {
  const bool sp = a.meta != nullptr;
  FewPlan p = few_plan(a.t, a.o, a.k, sp);
  if (part == nullptr || part_bytes < lin_few_part_bytes(a.t, a.o, a.k, sp)) p.splits = 1;
  if (p.tb == 1) return sp ? few_rows<1, true>(a, p, part, s) : few_rows<1, false>(a, p, part, s);
  if (p.tb == 2) return sp ? few_rows<2, true>(a, p, part, s) : few_rows<2, false>(a, p, part, s);
  return sp ? few_rows<4, true>(a, p, part, s) : few_rows<4, false>(a, p, part, s);
}

}  // namespace nml
