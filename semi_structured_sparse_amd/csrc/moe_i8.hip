// A mixture-of-experts layer of a few tokens in 8-bit integers:
//
//   h[t][e] = bf16(act(gate_e x_t) * up_e x_t)        for the experts e of token t
//   y[t]    = residual[t] + sum_e g[t][e] down_e Q(h[t][e])
//
// with the products of nm_glu_i8 and nm_spmm_i8 (exact 32-bit integer sums, fp32 scales) and the
// codes Q of nm_quant_i8.  The weights of the experts that are asked for bound the call, so they
// are streamed once, straight into the operand registers of the matrix instructions, as the
// few-token products do; the tokens of an expert are the columns of its products.
//
// Who asks for what: up to 64 tokens are one pass, so an expert's tokens are a 64-bit mask, set by
// LDS atomics whose order does not matter; a token that names an expert twice has it once, with
// both weights.  Experts with tokens are cut into items of at most 16 TB tokens, in ascending order,
// and a token's place in its item is its rank in the mask.  Each workgroup of the first kernel
// works that out for itself (a kernel of its own for it would cost a launch); one of them writes
// it down for the kernels behind it.
//
// Three kernels: the hidden rows' codes need a row's largest value, which only all of the gate and up
// products of an expert give, and the down products read codes.  The row's codes and scale are
// rounded as nm_quant_i8 rounds them, from bf16 hidden values; everything behind is fp32.
//
// Bound by the weights' bytes.  Measured (us, weights from HBM; gate and up + codes + down): 1 token 2/8
// 4096 x 14336 71, 43 + 4.8 + 23 (5.0 TB/s; floor 62 at 5.7); 64 tokens 6/64 4096 x 1408 215, 136 + 4.7 +
// 74 (5.2 TB/s; floor 194); 8 tokens 8/64 2:4 2048 x 1024 48, 25 + 3.9 + 15 and 2.1 for the parts' sum
// (floor 29: each kernel is only a few memory latencies long).
#include "i8_device.h"
#include "layer_launch.h"

namespace {

using namespace nmk;
using namespace nml;

constexpr int kPass = 64;      // tokens of a pass: bits of a mask
constexpr int kMaxParts = 8;   // of the down products' item sequence

struct Item {
  int expert, base, count;  // slots [base, base + count): the item's tokens in ascending order
  int pad;
};

// What a pass hands from kernel to kernel, in the workspace.
struct Plan {
  int* items;               // number of items
  Item* item;               // [slots]
  int* tok;                 // [slots] token of a slot
  float* g;                 // [slots] its weight
  uint16_t* h;              // bf16 [slots][ldh]
  int8_t* hq;               // [slots][ldh]
  float* hs;                // [slots]
  float* part;              // [parts][t][hidden], if the down products are cut
  int64_t ldh;
};

__device__ __forceinline__ i32x4 piece16(const int8_t* row, int off, bool in) {
  return *reinterpret_cast<const i32x4*>(in ? row + off : reinterpret_cast<const int8_t*>(&kZero16));
}

// Operands of U steps: v_mfma_i32_16x16x64_i8 and v_smfmac_i32_16x16x128_i8 as in few_i8.hip.
template <int U, int NA, int TB, bool SP>
struct Batch {
  i32x4 w[U][NA];
  int m[U][SP ? NA : 1];
  i32x4 xl[U][TB], xh[U][SP ? TB : 1];
};

template <int U, int NA, int TB, bool SP>
__device__ __forceinline__ void multiply(i32x4 (&acc)[NA][TB], const Batch<U, NA, TB, SP>& b) {
#pragma unroll
  for (int u = 0; u < U; ++u)
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
}

// Masks of the experts in LDS, from the pass's ids.  Every thread of the workgroup.
__device__ __forceinline__ void expert_masks(unsigned long long* mask, const int32_t* ids, int t, int top, int experts) {
  for (int e = threadIdx.x; e < experts; e += blockDim.x) mask[e] = 0ull;
  __syncthreads();
  for (int s = threadIdx.x; s < t * top; s += blockDim.x) {
    const int e = ids[s];
    if (e >= 0 && e < experts) atomicOr(&mask[e], 1ull << (s / top));
  }
  __syncthreads();
}

// Tokens and items of 16 TB before each expert: a lane's experts are [lane per, lane per + per).
// Returns the lane's own first numbers, tokens << 16 | items; whole: the same over all experts.
template <int TB>
__device__ __forceinline__ uint32_t before_lane(const unsigned long long* mask, int experts, int per, uint32_t& whole) {
  const int lane = threadIdx.x & 63;
  uint32_t own = 0;
  for (int v = 0; v < per; ++v) {
    const int e = lane * per + v;
    const int c = e < experts ? __popcll(mask[e]) : 0;
    own += (uint32_t)c << 16 | (uint32_t)((c + 16 * TB - 1) / (16 * TB));
  }
  uint32_t sum = own;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t o = (uint32_t)__shfl_up((int)sum, off, 64);
    sum += lane >= off ? o : 0u;
  }
  whole = (uint32_t)__builtin_amdgcn_readlane((int)sum, 63);
  return sum - own;
}

// Gate and up of an item's tokens (blockIdx.y the item) for 16 hidden units.  The waves share the
// reduction in contiguous parts, so that a workgroup reads whole rows.  Many short workgroups: what
// one waits for, its plan, its first weights, its sum, lies behind the others' weights.  (Two or
// four blocks of units a workgroup, their batches one sequence: 64 tokens 6/64 4096 x 1408 235 and 244
// us a layer instead of 221; a block a wave instead of a workgroup 237, and 1 token 2/8 4096 x
// 14336 80 instead of 73.)  Batches of four steps, two of 2:4 weights, whose registers leave room for
// twice the workgroups (8 tokens 8/64 2048 x 1024 50 us, with four 57).
template <int TB, bool SP>
__global__ __launch_bounds__(256) void k_moe_glu(MoeArgs a, Plan p, int t) {
  constexpr int NA = 2, STEP = SP ? 128 : 64, NW = 4;
  constexpr int U = TB == 1 ? (SP ? 2 : 4) : 2;
  constexpr int TILE = NA * TB * 256;
  __shared__ __align__(16) int red[NW * TILE];           // [waves][NA][16 TB][16] sums
  extern __shared__ __align__(16) unsigned char lds[];   // masks
  unsigned long long* const mask = reinterpret_cast<unsigned long long*>(lds);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fq = lane >> 4;
  expert_masks(mask, a.ids, t, a.top, a.experts);
  const int per = (a.experts + 63) / 64;
  uint32_t whole;
  const uint32_t first = before_lane<TB>(mask, a.experts, per, whole);
  const int items = (int)(whole & 0xFFFFu);

  if (blockIdx.x == 0 && blockIdx.y == 0 && wave == 0) {   // written down once
    if (lane == 0) *p.items = items;
    uint32_t at = first;
    for (int v = 0; v < per; ++v) {
      const int e = lane * per + v;
      if (e >= a.experts) break;
      const unsigned long long m = mask[e];
      const int c = __popcll(m), base = (int)(at >> 16);
      for (int b = 0; 16 * TB * b < c; ++b)
        p.item[(at & 0xFFFFu) + b] = Item{e, base + 16 * TB * b, min(16 * TB, c - 16 * TB * b), 0};
      int r = base;
      for (unsigned long long left = m; left != 0; left &= left - 1, ++r) {
        const int tok = __ffsll(left) - 1;
        float g = 0.0f;
        for (int j = 0; j < a.top; ++j) g += a.ids[tok * a.top + j] == e ? a.weights[tok * a.top + j] : 0.0f;
        p.tok[r] = tok;
        p.g[r] = g;
      }
      at += (uint32_t)c << 16 | (uint32_t)((c + 16 * TB - 1) / (16 * TB));
    }
  }
  const int it = (int)blockIdx.y;
  if (it >= items) return;   // the whole workgroup

  // the item's expert: the last lane whose first item is not behind it, then among its own
  const unsigned long long upto = __ballot((int)(first & 0xFFFFu) <= it);
  const int owner = 63 - __clzll((long long)upto);
  uint32_t at = (uint32_t)__builtin_amdgcn_readlane((int)first, owner);
  int e = owner * per;
  unsigned long long m = 0;
  for (int v = 0; v < per && e < a.experts; ++v, ++e) {
    m = mask[e];
    const int c = __popcll(m), n = (c + 16 * TB - 1) / (16 * TB);
    if (it < (int)(at & 0xFFFFu) + n) break;
    at += (uint32_t)c << 16 | (uint32_t)n;
  }
  e = __builtin_amdgcn_readfirstlane(e);
  const int blk = it - (int)(at & 0xFFFFu), total = __popcll(m);
  const int base = (int)(at >> 16) + 16 * TB * blk, count = min(16 * TB, total - 16 * TB * blk);
  // lane r receives the token of rank r
  const bool mine = (m >> lane) & 1ull;
  const int rank = __popcll(m & ((1ull << lane) - 1ull));
  const int token = __builtin_amdgcn_ds_permute(4 * (mine ? rank : total + lane - rank), lane);

  const int64_t O = a.inter;
  const int k = (int)a.hidden, wlen = SP ? k / 2 : k;
  const int8_t* xrow[TB];
  float xs[TB];   // of the thread's outputs: token 16 j + tid / 16, hidden unit tid % 16
#pragma unroll
  for (int j = 0; j < TB; ++j) {
    xrow[j] = a.x + (int64_t)__shfl(token, 16 * TB * blk + min(16 * j + fr, count - 1), 64) * a.ldx + 16 * fq;
    xs[j] = a.x_scale[__shfl(token, 16 * TB * blk + min(16 * j + (int)(threadIdx.x >> 4), count - 1), 64)];
  }
  const int64_t msteps = (k + 127) / 128;
  const int64_t ob = (int64_t)blockIdx.x * 16;
  const int64_t o_l = min(ob + fr, O - 1), o_t = min(ob + (threadIdx.x & 15), O - 1);
  const float gs = a.gate_scale[e * O + o_t], us = a.up_scale[e * O + o_t];   // of the thread's outputs
  const int8_t* wrow[NA] = {a.w_gate + (e * O + o_l) * a.ldw + 16 * fq, a.w_up + (e * O + o_l) * a.ldw + 16 * fq};
  const int64_t mat = (e * msteps * O + o_l) * 16 + 4 * fq;
  const uint8_t* mrow[NA] = {SP ? a.gate_meta + mat : nullptr, SP ? a.up_meta + mat : nullptr};

  const int steps = (k + STEP - 1) / STEP;
  const int s0 = wave * steps / NW, s1 = (wave + 1) * steps / NW;
  i32x4 acc[NA][TB];
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  // wholly inside the part and the row, or pieces past either as zeros
  auto fetch = [&](Batch<U, NA, TB, SP>& b, int s, bool all) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int wo = (s + u) * 64, xo = (s + u) * STEP;
      const bool in = all || s + u < s1;
#pragma unroll
      for (int i = 0; i < NA; ++i) {
        b.w[u][i] = piece16(wrow[i], wo, all || (in && wo + 16 * fq < wlen));
        if constexpr (SP) b.m[u][i] = *reinterpret_cast<const int*>(mrow[i] + (in ? s + u : s1 - 1) * O * 16);
      }
#pragma unroll
      for (int j = 0; j < TB; ++j) {
        b.xl[u][j] = piece16(xrow[j], xo, all || (in && xo + 16 * fq < k));
        if constexpr (SP) b.xh[u][j] = piece16(xrow[j], xo + 64, all || (in && xo + 64 + 16 * fq < k));
      }
    }
    __builtin_amdgcn_sched_barrier(0);   // the next batch's loads stay ahead of this one's products
  };
  const int nb = (s1 - s0 + U - 1) / U;
  if (nb > 0) {
    Batch<U, NA, TB, SP> b0, b1;
    fetch(b0, s0, nb > 1);
    for (int b = 0; b < nb; b += 2) {
      if (b + 1 < nb) fetch(b1, s0 + (b + 1) * U, b + 2 < nb);
      multiply<U, NA, TB, SP>(acc, b0);
      if (b + 1 >= nb) break;
      if (b + 2 < nb) fetch(b0, s0 + (b + 2) * U, b + 3 < nb);
      multiply<U, NA, TB, SP>(acc, b1);
    }
  }
  // the waves' partial tiles: red[wave][matrix][token][unit]
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j)
      *reinterpret_cast<i32x4*>(red + wave * TILE + ((i * TB + j) * 16 + fr) * 16 + 4 * fq) = acc[i][j];
  __syncthreads();
  const int64_t o = ob + (threadIdx.x & 15);
#pragma unroll
  for (int j = 0; j < TB; ++j) {
    const int tl = 16 * j + (int)(threadIdx.x >> 4);
    if (tl >= count || o >= O) continue;
    int v0 = 0, v1 = 0;
#pragma unroll
    for (int wv = 0; wv < NW; ++wv) {
      v0 += red[wv * TILE + tl * 16 + (threadIdx.x & 15)];
      v1 += red[wv * TILE + TB * 256 + tl * 16 + (threadIdx.x & 15)];
    }
    const float h = glu_gate(i8_scaled(v0, xs[j], gs), a.act) * i8_scaled(v1, xs[j], us);
    p.h[(int64_t)(base + tl) * p.ldh + o] = bf16_rne(h);
  }
}

__device__ __forceinline__ void moe_store(const MoeArgs& a, float v, int64_t tok, int64_t o) {
  if (a.bf16_out) {
    if (a.residual != nullptr)
      v += __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.residual)[tok * a.ldr + o] << 16);
    static_cast<uint16_t*>(a.y)[tok * a.ldy + o] = bf16_rne(v);
  } else {
    if (a.residual != nullptr) v += static_cast<const float*>(a.residual)[tok * a.ldr + o];
    static_cast<float*>(a.y)[tok * a.ldy + o] = v;
  }
}

// Down products of every item for 16 outputs, each token's summed with its weights.  The items'
// steps are one sequence of batches that the waves (of all blockIdx.y, where there are too few
// blocks of outputs to fill the chip) share in contiguous parts; a wave adds what it has of an
// item to its own sums in LDS, and the waves' sums are added in their order.  Batches of two steps
// (64 tokens 6/64 4096 x 1408 215 us a layer, with six 220), four for 2:4 items of 16, whose steps are
// half as many.
template <int TB, bool SP>
__global__ __launch_bounds__(512) void k_moe_down(MoeArgs a, Plan p, int t) {
  constexpr int STEP = SP ? 128 : 64;
  constexpr int U = SP && TB == 1 ? 4 : 2;
  extern __shared__ __align__(16) unsigned char lds[];   // [waves][t][16] sums
  float* const sums = reinterpret_cast<float*>(lds);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int fr = lane & 15, fq = lane >> 4;
  const int items = __builtin_amdgcn_readfirstlane(*p.items);
  float* const own = sums + wave * t * 16;
  for (int i = lane; i < t * 16; i += 64) own[i] = 0.0f;

  const int64_t O = a.hidden;
  const int k = (int)a.inter, wlen = SP ? k / 2 : k;
  const int64_t ob = (int64_t)blockIdx.x * 16;
  const int64_t o_l = ob + fr < O ? ob + fr : O - 1;
  const int64_t msteps = (k + 127) / 128;
  const int steps = (k + STEP - 1) / STEP, nbat = (steps + U - 1) / U;
  const int parts = waves * (int)gridDim.y, part = (int)blockIdx.y * waves + wave;
  const int g0 = (int)((int64_t)part * items * nbat / parts), g1 = (int)((int64_t)(part + 1) * items * nbat / parts);

  struct Work {                // a batch, and what its item's sums are scaled with
    Batch<U, 1, TB, SP> b;
    float hs[TB], g[TB];
    int tok[TB], count;
    f32x4 ws;
    bool last;                 // of the item, or of the wave's part
  };
  int li = -1;                 // item of the last fetch
  const int8_t *wrow = nullptr, *hrow[TB];
  const uint8_t* mrow = nullptr;
  Item item{};
  auto fetch = [&](Work& w, int g) {
    const int i = g / nbat, s = (g - i * nbat) * U;
    if (i != li) {
      li = i;
      item = p.item[i];
      item.expert = __builtin_amdgcn_readfirstlane(item.expert);
      item.base = __builtin_amdgcn_readfirstlane(item.base);
      item.count = __builtin_amdgcn_readfirstlane(item.count);
      wrow = a.w_down + (item.expert * O + o_l) * a.ldd + 16 * fq;
      if constexpr (SP) mrow = a.down_meta + (item.expert * msteps * O + o_l) * 16 + 4 * fq;
#pragma unroll
      for (int j = 0; j < TB; ++j) hrow[j] = p.hq + (item.base + min(16 * j + fr, item.count - 1)) * p.ldh + 16 * fq;
    }
    const bool all = s + U < steps;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int wo = (s + u) * 64, xo = (s + u) * STEP;
      w.b.w[u][0] = piece16(wrow, wo, all || wo + 16 * fq < wlen);
      if constexpr (SP) w.b.m[u][0] = *reinterpret_cast<const int*>(mrow + (s + u < steps ? s + u : steps - 1) * O * 16);
#pragma unroll
      for (int j = 0; j < TB; ++j) {
        w.b.xl[u][j] = piece16(hrow[j], xo, all || xo + 16 * fq < k);
        if constexpr (SP) w.b.xh[u][j] = piece16(hrow[j], xo + 64, all || xo + 64 + 16 * fq < k);
      }
    }
    w.last = s + U >= steps || g + 1 == g1;
    if (w.last) {
      w.count = item.count;
#pragma unroll
      for (int j = 0; j < TB; ++j) {
        const int r = item.base + min(16 * j + fr, item.count - 1);
        w.hs[j] = p.hs[r];
        w.g[j] = p.g[r];
        w.tok[j] = p.tok[r];
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t o = ob + 4 * fq + r;
        w.ws[r] = a.down_scale[item.expert * O + (o < O ? o : O - 1)];
      }
    }
    __builtin_amdgcn_sched_barrier(0);   // the next batch's loads stay ahead of this one's products
  };
  i32x4 acc[1][TB];
#pragma unroll
  for (int j = 0; j < TB; ++j) acc[0][j] = i32x4{0, 0, 0, 0};
  auto consume = [&](const Work& w) {
    multiply<U, 1, TB, SP>(acc, w.b);
    if (!w.last) return;
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      if (16 * j + fr < w.count) {   // an item's tokens are distinct: no two lanes meet
        f32x4* at = reinterpret_cast<f32x4*>(own + w.tok[j] * 16 + 4 * fq);
        f32x4 v = *at;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = __builtin_fmaf(w.g[j], i8_scaled(acc[0][j][r], w.hs[j], w.ws[r]), v[r]);
        *at = v;
      }
      acc[0][j] = i32x4{0, 0, 0, 0};
    }
  };
  wave_lds_fence();
  if (g0 < g1) {
    Work w0, w1;
    fetch(w0, g0);
    for (int g = g0; g < g1; g += 2) {
      if (g + 1 < g1) fetch(w1, g + 1);
      consume(w0);
      if (g + 1 >= g1) break;
      if (g + 2 < g1) fetch(w0, g + 2);
      consume(w1);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < t * 16; i += blockDim.x) {
    const int64_t o = ob + (i & 15), tok = i >> 4;
    if (o >= O) continue;
    float v = 0.0f;
    for (int wv = 0; wv < waves; ++wv) v += sums[wv * t * 16 + i];
    if (gridDim.y > 1) p.part[((int64_t)blockIdx.y * t + tok) * O + o] = v;
    else moe_store(a, v, tok, o);
  }
}

// y from the parts of blockIdx.y, part[part][t][hidden], in their order.
__global__ __launch_bounds__(256) void k_moe_sum(MoeArgs a, const float* __restrict__ part, int parts, int t) {
  const int64_t n = (int64_t)t * a.hidden;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float v[kMaxParts];
#pragma unroll
  for (int e = 0; e < kMaxParts; ++e) v[e] = part[(e < parts ? e : 0) * n + i];
  float s = 0.0f;
#pragma unroll
  for (int e = 0; e < kMaxParts; ++e) s += e < parts ? v[e] : 0.0f;
  const int64_t tok = i / a.hidden;
  moe_store(a, s, tok, i - tok * a.hidden);
}

int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }

// Parts that the down products' item sequence is cut in: up to a workgroup a CU, eight steps a wave at
// least (8 tokens 8/64 2:4 2048 x 1024, 128 blocks of outputs: 1 / 2 / 4 parts 57.5 / 49.3 / 51.5 us a
// layer).
int down_parts(int64_t t, int64_t experts, int64_t top, int64_t hidden, int64_t inter) {
  const int64_t blocks = (hidden + 15) / 16, slots = t * top, asked = slots < experts ? slots : experts;
  int64_t parts = blocks > 0 ? 256 / blocks : 1;
  const int64_t room = asked * ((inter + 63) / 64) / 64;   // steps: eight waves, eight each
  if (parts > room) parts = room;
  return parts < 2 ? 1 : parts > kMaxParts ? kMaxParts : (int)parts;
}

// Places in the workspace, and its size, for passes of up to kPass tokens.
int64_t lay_out(Plan& p, unsigned char* ws, int64_t t, int64_t experts, int64_t top, int64_t hidden, int64_t inter) {
  if (t > kPass) t = kPass;
  const int64_t slots = t * top;
  p.ldh = up16(inter);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    unsigned char* q = ws + at;
    at += up16(bytes);
    return q;
  };
  p.items = reinterpret_cast<int*>(take(16));
  p.item = reinterpret_cast<Item*>(take(slots * (int64_t)sizeof(Item)));
  p.tok = reinterpret_cast<int*>(take(slots * 4));
  p.g = reinterpret_cast<float*>(take(slots * 4));
  p.hs = reinterpret_cast<float*>(take(slots * 4));
  p.hq = reinterpret_cast<int8_t*>(take(slots * p.ldh));
  p.h = reinterpret_cast<uint16_t*>(take(slots * p.ldh * 2));
  const int parts = down_parts(t, experts, top, hidden, inter);
  p.part = reinterpret_cast<float*>(take(parts > 1 ? parts * t * hidden * 4 : 0));
  return at;
}

template <int TB, bool SP>
hipError_t launch_pass(const MoeArgs& a, const Plan& p, int t, hipStream_t s) {
  const int slots = t * a.top;
  const int asked = slots < a.experts ? slots : a.experts;
  const int items = slots < asked + slots / (16 * TB) ? slots : asked + slots / (16 * TB);
  const int64_t nob = (a.inter + 15) / 16, nod = (a.hidden + 15) / 16;
  if (nob > 0x7FFFFF || nod > 0x7FFFFF) return hipErrorInvalidConfiguration;
  if (a.inter > 0) {   // otherwise no batch of the down products exists, whatever the plan holds
    k_moe_glu<TB, SP><<<dim3((unsigned)nob, (unsigned)items), dim3(256), (size_t)(a.experts * 8 + 15) / 16 * 16, s>>>(a, p, t);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    e = launch_quant_i8(p.h, slots, a.inter, p.ldh, 0, 0, 2, p.hq, p.ldh, p.hs, s);
    if (e != hipSuccess) return e;
  }
  const int parts = down_parts(t, a.experts, a.top, a.hidden, a.inter);
  k_moe_down<TB, SP><<<dim3((unsigned)nod, (unsigned)parts), dim3(512), (size_t)8 * t * 64, s>>>(a, p, t);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || parts == 1) return e;
  k_moe_sum<<<dim3((unsigned)(((int64_t)t * a.hidden + 255) / 256)), dim3(256), 0, s>>>(a, p.part, parts, t);
  return hipGetLastError();
}

}  // namespace

namespace nml {

int64_t moe_workspace_bytes(int64_t t, int64_t experts, int64_t top, int64_t hidden, int64_t inter) {
  Plan p;
  int64_t most = lay_out(p, nullptr, t, experts, top, hidden, inter);
  const int64_t rest = t > kPass ? t % kPass : 0;
  const int64_t last = rest > 0 ? lay_out(p, nullptr, rest, experts, top, hidden, inter) : 0;
  return most > last ? most : last;
}

hipError_t launch_moe_i8(const MoeArgs& a, void* ws, hipStream_t s) {
  for (int64_t t0 = 0; t0 < a.t; t0 += kPass) {
    MoeArgs b = a;
    const int t = (int)(a.t - t0 < kPass ? a.t - t0 : kPass);
    const int64_t size = a.bf16_out ? 2 : 4;
    Plan p;
    lay_out(p, static_cast<unsigned char*>(ws), t, a.experts, a.top, a.hidden, a.inter);
    b.t = t;
    b.x = a.x + t0 * a.ldx;
    b.x_scale = a.x_scale + t0;
    b.ids = a.ids + t0 * a.top;
    b.weights = a.weights + t0 * a.top;
    if (a.residual != nullptr) b.residual = static_cast<const char*>(a.residual) + t0 * a.ldr * size;
    b.y = static_cast<char*>(a.y) + t0 * a.ldy * size;
    // Tokens of an item: those of an expert in one item if one may expect so (a second one reads the
    // expert's weights again), else the fewest, whose registers leave more loads in flight.  Measured
    // (us a layer, items of 16 / 32 / 64): 2/8 4096 x 14336 24 tokens 272 / 282 / 349, 32 291 / 301 /
    // 356, 64 440 / 384 / 414; 64 tokens 6/64 4096 x 1408 217 / 227 / 285, 6/32 2048 x 1024 75 / 79 / 83,
    // 8/16 2048 x 1024 104 / 97 / 99, 2/4 4096 x 8192 205 / 177 / 165, 4/4 345 / 277 / 236; 48 tokens 8/32
    // 2048 x 1024 79 / 82 / 86; 2:4 64 tokens 2/8 4096 x 14336 323 / 281 / 403, 8/16 2048 x 1024 94 / 89 /
    // 79, 4/4 4096 x 8192 286 / 232 / 209, 2/4 162 / 139 / 154 (where the one rule for dense and 2:4 takes
    // items of 64).
    const int tb = t <= 16 || t * a.top <= 12 * a.experts ? 1 : t <= 32 || t * a.top <= 20 * a.experts ? 2 : 4;
    hipError_t e;
    if (a.gate_meta != nullptr) {
      e = tb == 1 ? launch_pass<1, true>(b, p, t, s) : tb == 2 ? launch_pass<2, true>(b, p, t, s) : launch_pass<4, true>(b, p, t, s);
    } else {
      e = tb == 1 ? launch_pass<1, false>(b, p, t, s) : tb == 2 ? launch_pass<2, false>(b, p, t, s) : launch_pass<4, false>(b, p, t, s);
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace nml
