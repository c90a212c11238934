// Few-token int8 products (and any shape): the weights streamed from HBM straight into the
// operand registers of the matrix instructions.
//
//   sum[t][o] = sum_k x[t][k] w[o][k]   (exact 32-bit integers)
//   y = (fp32(sum) * x_scale[t]) * w_scale[o] + beta_t c_o,  or act(gate) * up from two sums
//
// With few tokens the o k bytes of weights bound the call, so nothing else is allowed to
// wait: a workgroup owns 16 RW output rows, its waves share the reduction in contiguous
// parts, each lane loads 16-byte weight pieces directly in operand layout (no LDS) one batch
// ahead of the one being multiplied, and X (t k bytes, in L2) follows the same path.  The
// waves' integer partial tiles are added in LDS and leave through the epilogue; where too
// few row blocks exist to fill the chip the reduction is also cut across workgroups, whose
// partial sums a second kernel adds.  Sums are integers, so every split gives the same bits.
//
// Operands: v_mfma_i32_16x16x64_i8 takes from lane l sixteen bytes of row l % 16 at position
// 16 (l / 16) of a 64-position step, both sides alike.  v_smfmac_i32_16x16x128_i8 takes the
// sixteen kept codes of positions [32 (l / 16), + 32) of a 128-position step with their 32
// bits of positions, and from X the bytes [16 (l / 16), + 16) and [64 + 16 (l / 16), + 16).
// A step's last pieces may lie past the row: those loads go to sixteen zero bytes instead.
//
// Measured (us, in a replayed graph; weights in the 256 MB last-level cache / from HBM): 1 x 4096 x
// 4096 5.9 / 6.6 (2.5 TB/s), 8 x 4096 x 14336 13.5 / 15.6 (3.8 TB/s), 2:4 1 x 4096 x 14336 9.8 / 11.1
// (3.3 TB/s), GLU 1 x 14336 x 4096 25.7 / 26.1 (4.5 TB/s).  The bound is the weight stream; one-token
// calls of 17 MB are mostly a launch and two memory latencies, and from 16 tokens on X, read
// again by every row block, costs more than W.
#include "i8_device.h"

namespace {

using namespace nmk;
using namespace nml;

constexpr int64_t kGridY = 65535;   // workgroups of tokens in the grid's y; more go on in z

// TB: blocks of 16 tokens; RW: blocks of 16 output rows; SP: 2:4 weights; GLU: two weights.
template <int TB, int RW, bool SP, bool GLU>
struct FewCfg {
  static constexpr int NA = RW * (GLU ? 2 : 1);              // weight row blocks
  static constexpr int STEP = SP ? 128 : 64;                 // positions per matrix step
  static constexpr int REGS = NA * (SP ? 5 : 4) + TB * (SP ? 8 : 4);   // of one step's operands
  // registers of a wave: 128 (16 waves a workgroup) or 256 (8); two batches are live
  static constexpr bool BIG = TB >= 4;
  static constexpr int FIT = ((BIG ? 256 : 128) - 24 - 4 * NA * TB - 2 * (NA * (SP ? 2 : 1) + TB)) / (2 * REGS);
  static constexpr int UNROLL = FIT < 1 ? 1 : FIT > 4 ? 4 : FIT;
};

template <int TB, int RW, bool SP, bool GLU>
__global__ __launch_bounds__(TB >= 4 ? 512 : 1024) void k_few_i8(
    const int8_t* __restrict__ x, int64_t ldx, const int8_t* __restrict__ w0, const int8_t* __restrict__ w1, int64_t ldw,
    const uint8_t* __restrict__ m0, const uint8_t* __restrict__ m1, int64_t T, int64_t O, int k, I8Epi epi,
    int32_t* __restrict__ part, int splits) {
  using C = FewCfg<TB, RW, SP, GLU>;
  constexpr int NA = C::NA, U = C::UNROLL;
  extern __shared__ __align__(16) int red[];   // [waves][NA][16 TB][16]
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

  const int8_t* xrow[TB];
#pragma unroll
  for (int j = 0; j < TB; ++j) {
    const int64_t t = t0 + 16 * j + fr;
    xrow[j] = x + (t < T ? t : T - 1) * ldx + 16 * fq;
  }
  const int8_t* wrow[NA];
  const uint8_t* mrow[NA];
#pragma unroll
  for (int a = 0; a < NA; ++a) {
    int64_t o = (ob * RW + (GLU ? a >> 1 : a)) * 16 + fr;
    o = o < O ? o : O - 1;
    wrow[a] = (GLU && (a & 1) ? w1 : w0) + o * ldw + 16 * fq;
    mrow[a] = SP ? (GLU && (a & 1) ? m1 : m0) + o * 16 + 4 * fq : nullptr;
  }
  i32x4 acc[NA][TB];
#pragma unroll
  for (int a = 0; a < NA; ++a)
#pragma unroll
    for (int j = 0; j < TB; ++j) acc[a][j] = i32x4{0, 0, 0, 0};

  struct Batch {
    i32x4 w[U][NA];
    int m[U][NA];
    i32x4 xl[U][TB], xh[U][TB];
  };
  const int wlen = SP ? k / 2 : k;        // weight bytes of a row
  const int64_t mstep = O * 16;
  // whole: the step lies inside the part and the row on both sides; otherwise pieces past
  // either come as zeros
  auto piece = [&](const int8_t* row, int off, bool in) {
    return *reinterpret_cast<const i32x4*>(in ? row + off : reinterpret_cast<const int8_t*>(&kZero16));
  };
  auto load = [&](Batch& b, int u, int s, bool whole) {
    const int wo = s * 64, xo = s * C::STEP;
    const bool in = whole || s < s1;
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      b.w[u][a] = piece(wrow[a], wo, whole || (in && wo + 16 * fq < wlen));
      if constexpr (SP) b.m[u][a] = *reinterpret_cast<const int*>(mrow[a] + (in ? s : s1 - 1) * mstep);
    }
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      b.xl[u][j] = piece(xrow[j], xo, whole || (in && xo + 16 * fq < k));
      if constexpr (SP) b.xh[u][j] = piece(xrow[j], xo + 64, whole || (in && xo + 64 + 16 * fq < k));
    }
  };
  auto mma = [&](const Batch& b, int u) {
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      if constexpr (SP) {
        const i32x4 lo = b.xl[u][j], hi = b.xh[u][j];
        const i32x8 bv = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
        for (int a = 0; a < NA; ++a)
          acc[a][j] = __builtin_amdgcn_smfmac_i32_16x16x128_i8(b.w[u][a], bv, acc[a][j], b.m[u][a], 0, 0);
      } else {
#pragma unroll
        for (int a = 0; a < NA; ++a)
          acc[a][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b.w[u][a], b.xl[u][j], acc[a][j], 0, 0, 0);
      }
    }
  };
  auto fetch = [&](Batch& b, int s, bool whole) {
#pragma unroll
    for (int u = 0; u < U; ++u) load(b, u, s + u, whole);
    __builtin_amdgcn_sched_barrier(0);   // the next batch's loads stay ahead of this one's products
  };
  auto consume = [&](const Batch& b) {
#pragma unroll
    for (int u = 0; u < U; ++u) mma(b, u);
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
  constexpr int TILE = NA * TB * 256;
#pragma unroll
  for (int a = 0; a < NA; ++a)
#pragma unroll
    for (int j = 0; j < TB; ++j)
      *reinterpret_cast<i32x4*>(red + wave * TILE + ((a * TB + j) * 16 + fr) * 16 + 4 * fq) = acc[a][j];
  __syncthreads();
  constexpr int OUT = RW * TB * 256;       // outputs of the workgroup, row fastest
  const int64_t o4 = (O + 3) / 4 * 4;
  for (int e = threadIdx.x; e < OUT; e += blockDim.x) {
    const int r = e % (16 * RW), tl = e / (16 * RW);
    const int64_t o = ob * 16 * RW + r, t = t0 + tl;
    if (o >= O || t >= T) continue;
    const int blk = r >> 4, a = GLU ? 2 * blk : blk;
    const int at = (a * TB * 16 + tl) * 16 + (r & 15);
    int v0 = 0, v1 = 0;
    for (int wv = 0; wv < waves; ++wv) {
      v0 += red[wv * TILE + at];
      if constexpr (GLU) v1 += red[wv * TILE + at + TB * 256];
    }
    if (part != nullptr) {
      int32_t* pp = part + ((int64_t)split * (GLU ? 2 : 1) * T + t) * o4 + o;
      pp[0] = v0;
      if constexpr (GLU) pp[T * o4] = v1;
    } else {
      i8_store<GLU>(epi, v0, v1, t, o);
    }
  }
}

// y from the splits' sums, part[split][matrix][t][o4]: one thread per 4 outputs, every load of
// up to 8 splits in flight together.  whole: O and ldy are multiples of 4.
template <bool GLU>
__global__ __launch_bounds__(256) void k_i8_reduce(const int32_t* __restrict__ part, int splits, uint32_t T, uint32_t O,
                                                   I8Epi epi, int whole) {
  const uint32_t q = (O + 3) / 4;
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= T * q) return;
  const uint32_t t = i / q, o = (i - t * q) * 4;
  const int64_t mat = (int64_t)T * (4 * q), stride = (GLU ? 2 : 1) * mat;
  const int32_t* p = part + 4 * (int64_t)i;
  i32x4 s0 = {0, 0, 0, 0}, s1 = {0, 0, 0, 0};
  for (int s = 0; s < splits; s += 8) {
    i32x4 v0[8], v1[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool in = s + e < splits;   // past the last split: the first again, not added
      v0[e] = *reinterpret_cast<const i32x4*>(p + (in ? s + e : 0) * stride);
      if constexpr (GLU) v1[e] = *reinterpret_cast<const i32x4*>(p + mat + (in ? s + e : 0) * stride);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (s + e >= splits) break;
      s0 += v0[e];
      if constexpr (GLU) s1 += v1[e];
    }
  }
  if (!whole) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (o + r < O) i8_store<GLU>(epi, s0[r], s1[r], t, o + r);
    return;
  }
  const float xs = epi.x_scale[t];
  const f32x4 ws = *reinterpret_cast<const f32x4*>(epi.w_scale + o);
  const bool shifted = !GLU && epi.col_shift != nullptr;
  const float* ep = GLU ? epi.up_scale : epi.col_shift;
  const f32x4 es = GLU || shifted ? *reinterpret_cast<const f32x4*>(ep + o) : f32x4{0.f, 0.f, 0.f, 0.f};
  const float rb = shifted && epi.row_shift != nullptr ? epi.row_shift[t] : 1.f;
  f32x4 v;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if constexpr (GLU) v[r] = i8_gated(epi, s0[r], s1[r], xs, ws[r], es[r]);
    else v[r] = i8_scaled(s0[r], xs, ws[r]);
    if (shifted) v[r] = i8_shifted(v[r], rb, es[r]);
  }
  if (epi.bf16_out) {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(epi.y) + t * epi.ldy + o) =
        make_uint2(bf16_rne(v[0]) | (uint32_t)bf16_rne(v[1]) << 16, bf16_rne(v[2]) | (uint32_t)bf16_rne(v[3]) << 16);
  } else {
    f32x4* yp = reinterpret_cast<f32x4*>(static_cast<float*>(epi.y) + t * epi.ldy + o);
    if (epi.accumulate) v += *yp;
    *yp = v;
  }
}

struct FewPlan {
  int tb, rw, waves;
  int64_t splits;
};

// Row blocks of a workgroup: every workgroup reads all of X again, so as many as leave 200
// workgroups (four blocks against one at 8 x 14336 x 4096: 16.1 -> 11.4 us; a GLU has two
// weights in a block already).  Waves: few workgroups take more of them, to keep as many loads
// in flight per CU (16 up to 128 workgroups, 8 up to 512, 4 beyond), at least two steps each.
// Splits: where under 128 workgroups remain, up to one per CU, four steps a wave at least, and
// only where a wave has over eight weight pieces unsplit (1 x 512 x 8192, eight of them: 6.7 us
// either way, and outside a graph a launch more; x 11008 8.5 unsplit, 7.9 in two).
FewPlan few_plan(int64_t t, int64_t o, int64_t k, bool sparse, bool glu) {
  FewPlan p;
  p.tb = t <= 16 ? 1 : t <= 32 ? 2 : 4;
  const int64_t steps = (k + (sparse ? 127 : 63)) / (sparse ? 128 : 64);
  const int mats = glu ? 2 : 1;
  const int64_t gy = (t + 16 * p.tb - 1) / (16 * p.tb);
  p.rw = p.tb > 2 || glu ? 1 : p.tb == 2 ? 2 : 4;
  while (p.rw > 1 && ((o + 16 * p.rw - 1) / (16 * p.rw)) * gy < 200) p.rw /= 2;
  const int64_t blocks = ((o + 16 * p.rw - 1) / (16 * p.rw)) * gy;
  p.waves = blocks <= 128 ? 16 : blocks <= 512 ? 8 : 4;
  const int most = p.tb == 4 || p.rw * mats * p.tb > 4 ? 8 : 16;   // 64 KiB of partial tiles
  if (p.waves > most) p.waves = most;
  while (p.waves > 4 && steps < 2 * p.waves) p.waves /= 2;
  int64_t s = blocks > 0 ? 256 / blocks : 1;
  const int64_t room = steps / (4 * p.waves);
  if (s > room) s = room;
  if (steps * mats <= 8 * p.waves) s = 1;
  p.splits = s < 2 ? 1 : s > 16 ? 16 : s;
  return p;
}

template <int TB, int RW, bool SP, bool GLU>
hipError_t few_launch(const I8Args& a, const FewPlan& pl, int32_t* part, hipStream_t s) {
  using C = FewCfg<TB, RW, SP, GLU>;
  const int64_t nob = (a.o + 16 * RW - 1) / (16 * RW), gy = (a.t + 16 * TB - 1) / (16 * TB);
  const int64_t gz = (gy + kGridY - 1) / kGridY;
  if (nob * pl.splits * 64 * pl.waves > 0xFFFFFFFFll || gz > 65535) return hipErrorInvalidConfiguration;
  const size_t lds = (size_t)pl.waves * C::NA * TB * 256 * 4;
  k_few_i8<TB, RW, SP, GLU><<<dim3((unsigned)(nob * pl.splits), (unsigned)(gz > 1 ? kGridY : gy), (unsigned)gz), dim3(64 * pl.waves),
                                lds, s>>>(
      a.x, a.ldx, a.w, a.w_up, a.ldw, a.meta, a.up_meta, a.t, a.o, (int)a.k, a.epi, pl.splits > 1 ? part : nullptr,
      (int)pl.splits);
  a.route.note(NM_TAKEN_FEW_STREAM | (SP ? NM_TAKEN_SPARSE_MMA : 0u));
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || pl.splits == 1) return e;
  return launch_i8_reduce(part, pl.splits, GLU, a.t, a.o, a.epi, a.route, s);
}

template <int TB, bool SP, bool GLU>
hipError_t few_rows(const I8Args& a, const FewPlan& pl, int32_t* part, hipStream_t s) {
  if constexpr (TB == 1 && !GLU) {
    if (pl.rw == 4) return few_launch<TB, 4, SP, GLU>(a, pl, part, s);
  }
  if constexpr (TB <= 2 && !GLU) {
    if (pl.rw == 2) return few_launch<TB, 2, SP, GLU>(a, pl, part, s);
  }
  return few_launch<TB, 1, SP, GLU>(a, pl, part, s);
}

}  // namespace

namespace nml {

hipError_t launch_i8_reduce(const int32_t* part, int64_t splits, bool glu, int64_t t, int64_t o, const I8Epi& e,
                            const Route& r, hipStream_t s) {
  const int64_t n = t * ((o + 3) / 4);
  if (n <= 0) return hipSuccess;
  if (n > 0x3FFFFFFF) return hipErrorInvalidConfiguration;   // plans split far smaller outputs only
  const int whole = o % 4 == 0 && e.ldy % 4 == 0;
  const dim3 grid((unsigned)((n + 255) / 256)), block(256);
  if (glu) k_i8_reduce<true><<<grid, block, 0, s>>>(part, (int)splits, (uint32_t)t, (uint32_t)o, e, whole);
  else k_i8_reduce<false><<<grid, block, 0, s>>>(part, (int)splits, (uint32_t)t, (uint32_t)o, e, whole);
  r.note(NM_TAKEN_REDUCE);
  return hipGetLastError();
}

int64_t i8_few_part_bytes(int64_t t, int64_t o, int64_t k, bool sparse, bool glu) {
  const FewPlan p = few_plan(t, o, k, sparse, glu);
  return p.splits > 1 ? p.splits * (glu ? 2 : 1) * t * ((o + 3) / 4 * 4) * 4 : 0;
}

hipError_t launch_i8_few(const I8Args& a, int32_t* part, int64_t part_bytes, hipStream_t s) {
  const bool sp = a.meta != nullptr, glu = a.glu != 0;
  FewPlan p = few_plan(a.t, a.o, a.k, sp, glu);
  if (part == nullptr || part_bytes < i8_few_part_bytes(a.t, a.o, a.k, sp, glu)) p.splits = 1;
#define NM_FEW(TBV)                                                       \
  if (p.tb == TBV) {                                                      \
    if (sp && glu) return few_rows<TBV, true, true>(a, p, part, s);     \
    if (sp) return few_rows<TBV, true, false>(a, p, part, s);           \
    if (glu) return few_rows<TBV, false, true>(a, p, part, s);          \
    return few_rows<TBV, false, false>(a, p, part, s);                  \
  }
  NM_FEW(1) NM_FEW(2) NM_FEW(4)
#undef NM_FEW
  return hipErrorInvalidValue;
}

}  // namespace nml
