// bf16 tile products with an epilogue, staged direct to LDS:
//   y[t][o] = residual[t][o] + fn(sum_k x[t][k] w[o][k] + bias[o])
// W dense or 2:4 (kept values and step-blocked positions).
//
// gfx950 design:
//  * A K-step is KM chunks of 64 reduction positions: of each 128 bytes of every X row and of every
//    dense weight row (64 bytes of kept values and 8 of positions for 2:4), moved from global memory
//    into LDS by buffer loads of 16 bytes a lane.  A lane's row and piece are fixed for the whole call, so a step's
//    loads differ only in one scalar offset; a last step that passes the row's end sends its
//    lanes' offsets past the descriptor's range, which reads zeros.  A row that ends inside a
//    piece: what the last step staged past the end is zeroed in LDS, both sides, before it is
//    multiplied (a row's padding may hold a NaN).
//  * LDS rows are unpadded; piece c of row r lies at c ^ ((r >> 1) & 7) (64-byte rows:
//    c ^ ((r >> 2) & 3)), so a fragment read's 16 lanes fall on distinct banks.
//  * Output tiles are turned in LDS, a wave's 16 tokens at a time, so that bias, residual and y are
//    met in whole row pieces by the lanes that add and store them.
//  * Workgroups are remapped so that each XCD (own L2) runs a near-square block of tiles.
#include <type_traits>

#include "lin_device.h"

namespace {

using namespace nmk;
using namespace nml;

typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ int swz8(int r, int c) { return c ^ ((r >> 1) & 7); }   // 8 pieces per row
__device__ __forceinline__ int swz4(int r, int c) { return c ^ ((r >> 2) & 3); }   // 4 pieces per row

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00020000);
}
__device__ __forceinline__ void b2lds16(__amdgpu_buffer_rsrc_t r, void* lds, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, voff, soff, 0, 0);
}
constexpr uint32_t kPast = 0x80000000u;   // past every descriptor's range (< 2^31 bytes)

// A stage: the weight rows (and positions) and the X rows of a step, arrays of their own.
struct Stage {
  unsigned char *a, *b;
};

// The place of this workgroup in the order of all: workgroups go to the 8 XCDs in turn, and each XCD
// runs a contiguous range.
__device__ __forceinline__ int by_xcd() {
  const int n = (int)gridDim.x, x = blockIdx.x & 7;
  return x * (n >> 3) + min(x, n & 7) + (int)(blockIdx.x >> 3);
}

__device__ __forceinline__ void bar() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// K-loop over n >= 1 steps through NST stages (distinct static arrays, named by constant indices,
// so that the compiler tracks the requests into each one).  issue(st, s) requests step s into
// st; mend(st, s) makes up a landed step that the row's end falls into.  Ends with every request
// landed and every stage free.
//
// Step q requests step q + NST - 1 into the stage that step q - 1 used, reads its
// operands, all at once, and multiplies; then one wait (step q + 1 has landed, the operands have
// arrived) and one barrier.  Exactly L requests a wave and step; past the last step the last one
// is requested again, no one reads it.
template <int NST, int L, typename Frag, typename Issue, typename Mend, typename Read, typename Mma>
__device__ __forceinline__ void k_ring(int n, const Stage (&S)[4], Issue&& issue, Mend&& mend, Read&& read, Mma&& mma) {
  static_assert(NST >= 3 && NST <= 4 && L * (NST - 2) <= 63, "stages and requests per step");
#pragma unroll
  for (int j = 0; j + 1 < NST; ++j) issue(S[j], j < n ? j : n - 1);
  __builtin_amdgcn_s_waitcnt(vm_wait(L * (NST - 2)));
  bar();
  auto step = [&](int j, int q) {   // j = q % NST, a constant after unrolling
    mend(S[j], q);
    const int ahead = q + NST - 1;
    issue(S[(j + NST - 1) % NST], ahead < n ? ahead : n - 1);
    Frag f;
    read(f, S[j]);
    __builtin_amdgcn_sched_barrier(0);
    mma(f);
    // the reads too: the compiler may move products, and with them the waits for their operands,
    // past the barrier, behind which this stage is requested into
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0 & vm_wait(L * (NST - 2)));
    bar();
  };
  int s = 0;
  for (; s + NST <= n; s += NST) {
#pragma unroll
    for (int j = 0; j < NST; ++j) step(j, s + j);
  }
#pragma unroll
  for (int j = 0; j + 1 < NST; ++j) {
    if (s + j >= n) break;
    step(j, s + j);
  }
  __builtin_amdgcn_s_waitcnt(0);
  bar();
}

// f(0), f(step), ... below end, each with its number as a constant (sums that the compiler indexed by
// a variable would lie in memory)
template <int I, int END, int STEP, typename F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (I < END) {
    f(std::integral_constant<int, I>{});
    each<I + STEP, END, STEP>(f);
  }
}

// The parts that a wave's FI x FJ blocks of 16 x 16 sums leave in: BI x JB blocks each.
template <int FI, int FJ>
struct Turn {
  static constexpr int BI = FI < 4 ? FI : 4, W = 16 * BI;   // blocks and outputs of a row
  static constexpr int JB = FJ < 2 ? FJ : 2, ROWS = 16 * JB;
  static constexpr int BYTES = ROWS * W * 4;
  static_assert(FI % BI == 0 && FJ % JB == 0, "whole turns");
};

// A wave's finished outputs in parts ("turns") of W outputs by ROWS tokens, turned through its own LDS
// at `mine`: part (h, j) of NH x NJ starts at output o_of(h) and token t_of(j), and put(h, j) writes
// it, rows of W outputs, 16-byte piece c of row r at place(r, c).  Neighbouring lanes then hold
// neighbouring outputs of a row and meet bias, residual and y in whole row pieces: four outputs
// each where rows of y and of the residual keep that alignment, one each otherwise.  One wave may
// have its SIMD for itself, so what costs instructions is done once (types, addresses), and the
// next part's residual is loaded ahead of the use of this one's.  The parts run in a loop, each with
// its own put (unrolled, their code is eight times as long: 8192 x 14336 x 4096, gelu and bias, 736
// against 723 us).  bf16 outputs are rounded once, from the fp32 sum with bias, activation and residual.
template <int W, int ROWS>
struct Emit {
  static constexpr int PC = W / 4, RP = 64 / PC, NP = ROWS / RP;   // pieces of a row; rows of a pass; passes
  static constexpr int RS = 64 / W, N1 = ROWS / RS, NG = N1 < 16 ? N1 : 16;   // one output a lane: NG passes at a time
  static_assert(PC == 8 || PC == 16, "rows of 32 or 64 outputs");

  static __device__ __forceinline__ unsigned char* place(unsigned char* mine, int r, int c) {
    return mine + r * (4 * W) + 16 * (c ^ (r & (PC - 1)));
  }

  template <bool BF>
  struct Raw {   // four values of a residual row each
    using Four = typename std::conditional<BF, uint2, uint4>::type;
    Four d[NP];
  };
  // rows: of the part inside T (<= 0: none); o: the lane's first output
  template <bool BF>
  static __device__ __forceinline__ void residual4(Raw<BF>& r, const LinEpi& e, int rows, int64_t O, int64_t o, int64_t t_t,
                                                   int lane) {
    using E = typename std::conditional<BF, uint16_t, float>::type;
    if (rows <= 0 || o + 4 > O) return;
    const E* p = static_cast<const E*>(e.residual) + t_t * e.ldr + o;
    const int l = lane / PC;
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      const int row = RP * q + l < rows ? RP * q + l : rows - 1;   // past the last one its own, not used
      r.d[q] = *reinterpret_cast<const typename Raw<BF>::Four*>(p + row * e.ldr);
    }
  }
  template <bool BF>
  static __device__ __forceinline__ void out4(const Raw<BF>& r, const LinEpi& e, const f32x4& bias, int rows, int64_t O,
                                              int64_t o, int64_t t_t, int lane, unsigned char* mine) {
    using E = typename std::conditional<BF, uint16_t, float>::type;
    const int l = lane / PC;
    float v[4 * NP];
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      const f32x4 s = *reinterpret_cast<const f32x4*>(place(mine, RP * q + l, lane % PC));
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * q + i] = s[i];
    }
    wave_lds_fence();
    if (o + 4 > O) {
#pragma unroll
      for (int i = 0; i < 4 * NP; ++i)
        if (o + (i & 3) < O && RP * (i >> 2) + l < rows) lin_store(e, v[i], t_t + RP * (i >> 2) + l, o + (i & 3));
      return;
    }
    if (e.bias != nullptr) {
#pragma unroll
      for (int i = 0; i < 4 * NP; ++i) v[i] = v[i] + bias[i & 3];
    }
    lin_fns<4 * NP>(v, e.fn);
    if (e.residual != nullptr) {
#pragma unroll
      for (int q = 0; q < NP; ++q) {
        if constexpr (BF) {
          v[4 * q] = v[4 * q] + __uint_as_float(r.d[q].x << 16);
          v[4 * q + 1] = v[4 * q + 1] + __uint_as_float(r.d[q].x & 0xFFFF0000u);
          v[4 * q + 2] = v[4 * q + 2] + __uint_as_float(r.d[q].y << 16);
          v[4 * q + 3] = v[4 * q + 3] + __uint_as_float(r.d[q].y & 0xFFFF0000u);
        } else {
          v[4 * q] = v[4 * q] + __uint_as_float(r.d[q].x);
          v[4 * q + 1] = v[4 * q + 1] + __uint_as_float(r.d[q].y);
          v[4 * q + 2] = v[4 * q + 2] + __uint_as_float(r.d[q].z);
          v[4 * q + 3] = v[4 * q + 3] + __uint_as_float(r.d[q].w);
        }
      }
    }
    E* p = static_cast<E*>(e.y) + (t_t + l) * e.ldy + o;
    const int64_t next = RP * e.ldy;
    auto store = [&](int q) {
      if constexpr (BF)
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[4 * q], v[4 * q + 1]), pack_bf16(v[4 * q + 2], v[4 * q + 3]));
      else
        *reinterpret_cast<f32x4*>(p) = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      p += next;
    };
    if (rows >= ROWS) {
#pragma unroll
      for (int q = 0; q < NP; ++q) store(q);
    } else {
#pragma unroll
      for (int q = 0; q < NP; ++q)
        if (RP * q + l < rows) store(q);
    }
  }
  // one output a lane
  static __device__ __forceinline__ void out1(const LinEpi& epi, int64_t T, int64_t O, int64_t o_t, int64_t t_t, int lane,
                                              unsigned char* mine) {
    const int64_t o = o_t + lane % W, oc = o < O ? o : O - 1, tb = t_t + lane / W;
    const float bias = epi.bias != nullptr ? epi.bias[oc] : 0.0f;
#pragma unroll 1
    for (int g = 0; g < N1; g += NG) {
      float v[NG];
      uint32_t r[NG];   // past the last row or output: a neighbour's value, not used
      if (epi.residual != nullptr) {
        if (epi.bf16_out) {
#pragma unroll
          for (int p = 0; p < NG; ++p) {
            const int64_t t = tb + RS * (g + p) < T ? tb + RS * (g + p) : T - 1;
            r[p] = (uint32_t) static_cast<const uint16_t*>(epi.residual)[t * epi.ldr + oc] << 16;
          }
        } else {
#pragma unroll
          for (int p = 0; p < NG; ++p) {
            const int64_t t = tb + RS * (g + p) < T ? tb + RS * (g + p) : T - 1;
            r[p] = static_cast<const uint32_t*>(epi.residual)[t * epi.ldr + oc];
          }
        }
      }
#pragma unroll
      for (int p = 0; p < NG; ++p) {
        v[p] = *reinterpret_cast<const float*>(place(mine, RS * (g + p) + lane / W, lane % W / 4) + 4 * (lane & 3));
        if (epi.bias != nullptr) v[p] = v[p] + bias;
      }
      lin_fns<NG>(v, epi.fn);
#pragma unroll
      for (int p = 0; p < NG; ++p) {
        const int64_t t = tb + RS * (g + p);
        if (o >= O || t >= T) continue;
        if (epi.residual != nullptr) v[p] = v[p] + __uint_as_float(r[p]);
        if (epi.bf16_out) static_cast<uint16_t*>(epi.y)[t * epi.ldy + o] = (uint16_t)pack_bf16(v[p], 0.0f);
        else static_cast<float*>(epi.y)[t * epi.ldy + o] = v[p];
      }
    }
    wave_lds_fence();
  }
};

// put(n / NJ, n % NJ), numbers that it has as constants
template <int NH, int NJ, typename Put>
__device__ __forceinline__ void one_of(int n, Put&& put) {
  each<0, NH * NJ, 1>([&](auto m) __attribute__((always_inline)) {
    if (n == m) {
      // unlike any other part's: alike, the parts would become one whose sums are indexed by n
      asm volatile("; part %0" ::"n"(decltype(m)::value));
      put(std::integral_constant<int, m / NJ>{}, std::integral_constant<int, m % NJ>{});
      asm volatile("; part %0 written" ::"n"(decltype(m)::value));
    }
  });
}

template <int NH, int NJ, int W, int ROWS, bool BF, typename Put, typename OOf, typename TOf>
__device__ __forceinline__ void lin_emit4(const LinEpi& epi, int64_t T, int64_t O, int lane, unsigned char* mine, Put&& put,
                                          OOf&& o_of, TOf&& t_of) {
  using E = Emit<W, ROWS>;
  typename E::template Raw<BF> now, then;
  auto rows_of = [&](int j) {
    const int64_t left = T - t_of(j);
    return left < ROWS ? (int)left : ROWS;
  };
  const int lo = 4 * (lane % E::PC);
  f32x4 bias = {0.f, 0.f, 0.f, 0.f};
  if (epi.residual != nullptr) E::template residual4<BF>(then, epi, rows_of(0), O, o_of(0) + lo, t_of(0), lane);
#pragma unroll 1
  for (int n = 0; n < NH * NJ; ++n) {
    const int h = n / NJ, j = n % NJ;
    const int64_t o = o_of(h) + lo;
    if (j == 0 && epi.bias != nullptr && o + 4 <= O) bias = *reinterpret_cast<const f32x4*>(epi.bias + o);
    one_of<NH, NJ>(n, put);
    if (epi.residual != nullptr) {
      now = then;
      if (n + 1 < NH * NJ) {
        const int hn = (n + 1) / NJ, jn = (n + 1) % NJ;
        E::template residual4<BF>(then, epi, rows_of(jn), O, o_of(hn) + lo, t_of(jn), lane);
      }
    }
    wave_lds_fence();
    E::template out4<BF>(now, epi, bias, rows_of(j), O, o, t_of(j), lane, mine);
  }
}

template <int NH, int NJ, int W, int ROWS, typename Put, typename OOf, typename TOf>
__device__ __forceinline__ void lin_emit(const LinEpi& epi, int64_t T, int64_t O, int lane, unsigned char* mine, Put&& put,
                                         OOf&& o_of, TOf&& t_of) {
  if (lin_whole(epi)) {
    if (epi.bf16_out) lin_emit4<NH, NJ, W, ROWS, true>(epi, T, O, lane, mine, put, o_of, t_of);
    else lin_emit4<NH, NJ, W, ROWS, false>(epi, T, O, lane, mine, put, o_of, t_of);
    return;
  }
#pragma unroll 1
  for (int n = 0; n < NH * NJ; ++n) {
    one_of<NH, NJ>(n, put);
    wave_lds_fence();
    Emit<W, ROWS>::out1(epi, T, O, o_of(n / NJ), t_of(n % NJ), lane, mine);
  }
}

template <int FI, int FJ>
__device__ __forceinline__ void lin_finish(const f32x4 (&acc)[FI][FJ], const LinEpi& epi, float* __restrict__ part,
                                           int kpart, int64_t T, int64_t O, int64_t ob_w, int64_t tb_w, int lane,
                                           unsigned char* mine) {
  using C = Turn<FI, FJ>;
  const int fr = lane & 15, fq = lane >> 4;
  if (part != nullptr) {
    const int64_t o4 = (O + 3) / 4 * 4;
#pragma unroll
    for (int i = 0; i < FI; ++i) {
      const int64_t ob = ob_w + 16 * i + 4 * fq;
      if (ob >= O) continue;
#pragma unroll
      for (int j = 0; j < FJ; ++j) {
        const int64_t t = tb_w + 16 * j + fr;
        if (t < T) *reinterpret_cast<f32x4*>(part + ((int64_t)kpart * T + t) * o4 + ob) = acc[i][j];
      }
    }
    return;
  }
  lin_emit<FI / C::BI, FJ / C::JB, C::W, C::ROWS>(
      epi, T, O, lane, mine,
      [&](auto hc, auto jc) __attribute__((always_inline)) {
        constexpr int h = decltype(hc)::value, j = decltype(jc)::value * C::JB;
#pragma unroll
        for (int jj = 0; jj < C::JB; ++jj)
#pragma unroll
          for (int i = 0; i < C::BI; ++i)
            *reinterpret_cast<f32x4*>(Emit<C::W, C::ROWS>::place(mine, 16 * jj + fr, 4 * i + fq)) = acc[C::BI * h + i][j + jj];
      },
      [&](int h) { return ob_w + C::W * h; }, [&](int j) { return tb_w + C::ROWS * j; });
}

// BM x BN: weight rows by tokens of a tile; WM x WN waves; NST stages of KM chunks.
//
// Between the streaming kernel and the 256 x 256 tiles: too few tiles to fill the chip, so a step costs
// what its loads' latency leaves behind the ring, whatever it holds, and tiles and reduction ranges
// are chosen by estimated time (mid_plan).  Two chunks a step where the stages fit two workgroups a CU
// or the tile is short of work (40 x 4096 x 14336 2:4: 44 us with one chunk a step and the
// largest tile that gives 192 workgroups, 26 so).  Measured from HBM: 40 x 4096 x 14336 2:4 26.3 us (19 with its weights in the cache: 15.2 and the
// ranges' sum 4.0), floor 11.9 at 5.7 TB/s; 777 x 1025 x 1999 14.3, of it a step's load, launch and
// epilogue about 5, the rest 32 steps of 0.3.
template <int BM, int BN, int WM, int WN, bool SP, int NST, int KM>
__global__ __launch_bounds__(64 * WM * WN) void k_lin_tile(
    const uint16_t* __restrict__ x, int64_t ldx, const uint16_t* __restrict__ w, int64_t ldw,
    const uint8_t* __restrict__ meta, int64_t T, int64_t O, int k, LinEpi epi, float* __restrict__ part, int tiles_m,
    int tiles_n, int steps_per_split, int group) {
  constexpr int NW = WM * WN;
  constexpr int SM = BM / WM, SN = BN / WN, FI = SM / 16, FJ = SN / 16;
  constexpr int AROW = SP ? 64 : 128;          // weight bytes per row per step
  constexpr int RPG = SP ? 16 : 8;             // weight rows of one wave load (1 KiB)
  constexpr int A_CHUNK = BM * AROW, B_CHUNK = BN * 128;
  constexpr int V_BYTES = KM * A_CHUNK;
  constexpr int A_BYTES = V_BYTES + (SP ? BM * 8 * KM : 0), B_BYTES = KM * B_CHUNK;
  constexpr int NA = BM / RPG / NW, NB = BN / 8 / NW;
  static_assert(NA >= 1 && NB >= 1 && BM % (RPG * NW) == 0 && BN % (8 * NW) == 0, "load groups per wave");
  static_assert(!SP || (KM == 2 && BM == 16 * NW), "positions: of 16 rows a wave, 16 bytes a row and step, 4 a lane");
  constexpr int A3 = NST > 3 ? A_BYTES : 16, B3 = NST > 3 ? B_BYTES : 16;
  __shared__ __align__(16) unsigned char sA0[A_BYTES], sB0[B_BYTES], sA1[A_BYTES], sB1[B_BYTES], sA2[A_BYTES], sB2[B_BYTES],
      sA3[A3], sB3[B3];
  const Stage S[4] = {{sA0, sB0}, {sA1, sB1}, {sA2, sB2}, {sA3, sB3}};
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wmi = wave % WM, wni = wave / WM;
  const int fr = lane & 15, fq = lane >> 4;

  const int ntiles = tiles_m * tiles_n;
  const int place = by_xcd();
  const int kpart = __builtin_amdgcn_readfirstlane(place / ntiles);
  const int lin = place - kpart * ntiles;
  const int band = lin / (group * tiles_n);
  const int band_w = min(group, tiles_m - band * group);
  const int inband = lin - band * group * tiles_n;
  // wave-uniform (the division leaves them in vector registers; descriptors need scalars)
  const int tile_m = __builtin_amdgcn_readfirstlane(band * group + inband % band_w);
  const int tile_n = __builtin_amdgcn_readfirstlane(inband / band_w);
  const int64_t o0 = (int64_t)tile_m * BM, t0 = (int64_t)tile_n * BN;
  const int orows = (int)(O - o0 < BM ? O - o0 : BM), trows = (int)(T - t0 < BN ? T - t0 : BN);

  const int chunks = (k + 63) / 64, steps_all = (chunks + KM - 1) / KM;
  const int sb = kpart * steps_per_split;
  const int n = min(steps_all - sb, steps_per_split);
  const int wlen = SP ? k / 2 : k;             // values of a weight row

  // descriptors of the tile's rows, and the lane's offset of each of its loads
  const __amdgpu_buffer_rsrc_t rx = rsrc_of(x + t0 * ldx, (uint32_t)(trows * ldx * 2));
  const __amdgpu_buffer_rsrc_t rw = rsrc_of(w + o0 * ldw, (uint32_t)(orows * ldw * 2));
  uint32_t aoff[NA], boff[NB];
  uint32_t atail, btail;   // added in the last chunk: kPast where the piece starts past the row
  {
    const int last = chunks - 1;
#pragma unroll
    for (int q = 0; q < NA; ++q) {
      const int r = (wave + q * NW) * RPG + lane / (AROW / 16);
      const int c = SP ? swz4(r, lane & 3) : swz8(r, lane & 7);
      const int o = r < orows ? r : orows - 1;
      aoff[q] = (uint32_t)(o * (int)ldw * 2 + 16 * c);
      // one piece for every q: the rows of two loads differ by a multiple of 16, the swizzles' period
      if (q == 0) atail = last * (AROW / 2) + 8 * c >= wlen ? kPast : 0u;
    }
#pragma unroll
    for (int q = 0; q < NB; ++q) {
      const int r = (wave + q * NW) * 8 + (lane >> 3);
      const int c = swz8(r, lane & 7);
      const int t = r < trows ? r : trows - 1;
      boff[q] = (uint32_t)(t * (int)ldx * 2 + 16 * c);
      if (q == 0) btail = last * 64 + 8 * c >= k ? kPast : 0u;
    }
  }
  const uint8_t* mlane = nullptr;   // the lane's four bytes of positions in step 0
  if constexpr (SP) {
    const int r = wave * 16 + (lane >> 2);
    const int o = r < orows ? r : orows - 1;
    mlane = meta + (o0 + o) * 16 + 4 * (lane & 3);
  }

  f32x4 acc[FI][FJ];
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int j = 0; j < FJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto issue = [&](Stage st, int si) {
    unsigned char *const a = st.a, *const b = st.b;
    const int s = sb + si;
#pragma unroll
    for (int c = 0; c < KM; ++c) {
      const int ch = s * KM + c;   // past the last chunk: zeros
      const uint32_t at = ch == chunks - 1 ? atail : KM > 1 && ch >= chunks ? kPast : 0u;
#pragma unroll
      for (int q = 0; q < NA; ++q)
        b2lds16(rw, a + c * A_CHUNK + (wave + q * NW) * 1024, aoff[q] | at, (uint32_t)(ch * AROW));
    }
    if constexpr (SP) {
      __builtin_amdgcn_global_load_lds(mlane + s * (O * 16), (lds_void*)(a + V_BYTES + wave * 256), 4, 0, 0);
    }
#pragma unroll
    for (int c = 0; c < KM; ++c) {
      const int ch = s * KM + c;
      const uint32_t bt = ch == chunks - 1 ? btail : KM > 1 && ch >= chunks ? kPast : 0u;
#pragma unroll
      for (int q = 0; q < NB; ++q)
        b2lds16(rx, b + c * B_CHUNK + (wave + q * NW) * 1024, boff[q] | bt, (uint32_t)(ch * 128));
    }
  };
  // a row that ends inside a piece: values past it zeroed, one row a thread
  const bool ragged = (k & 7) != 0 || (SP && (wlen & 7) != 0);
  auto mend = [&](Stage st, int si) {
    if (!ragged || sb + si != steps_all - 1) return;
    const int xe = k & 63, we = wlen & (AROW / 2 - 1);   // values of the last chunk inside the row
    const int c = (chunks - 1) % KM;
    for (int r = tid; r < BN; r += 64 * NW) {
      unsigned char* const row = st.b + c * B_CHUNK + r * 128 + 16 * swz8(r, xe >> 3);
      for (int e = xe & 7; (k & 7) != 0 && e < 8; ++e) *reinterpret_cast<uint16_t*>(row + 2 * e) = 0;
    }
    for (int r = tid; r < BM; r += 64 * NW) {
      unsigned char* const row = st.a + c * A_CHUNK + r * AROW + 16 * (SP ? swz4(r, we >> 3) : swz8(r, we >> 3));
      for (int e = we & 7; (wlen & 7) != 0 && e < 8; ++e) *reinterpret_cast<uint16_t*>(row + 2 * e) = 0;
    }
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
    bar();
  };

  auto read_a = [&](const unsigned char* a, int ks, int i) {
    const int r = wmi * SM + i * 16 + fr;
    return *reinterpret_cast<const bf16x8*>(a + r * AROW + 16 * (SP ? swz4(r, fq) : swz8(r, 4 * ks + fq)));
  };
  auto read_b = [&](const unsigned char* b, int ks, int j) {
    const int r = wni * SN + j * 16 + fr;
    return *reinterpret_cast<const u32x4*>(b + r * 128 + 16 * swz8(r, 4 * ks + fq));
  };
  auto read_idx = [&](const unsigned char* a, int c, int i) {
    return (int)*reinterpret_cast<const uint16_t*>(a + V_BYTES + (wmi * SM + i * 16 + fr) * (8 * KM) + 8 * c + 2 * fq);
  };
  auto both = [](u32x4 lo, u32x4 hi) {
    return __builtin_bit_cast(bf16x16, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  // the operands of a whole step at once
  constexpr int KS = SP ? 1 : 2;
  struct Frag {
    bf16x8 a[KM][KS][FI];
    u32x4 b0[KM][FJ], b1[KM][FJ];
    int idx[KM][SP ? FI : 1];
  };
  auto read = [&](Frag& f, Stage st) {
#pragma unroll
    for (int c = 0; c < KM; ++c) {
#pragma unroll
      for (int i = 0; i < FI; ++i) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) f.a[c][ks][i] = read_a(st.a + c * A_CHUNK, ks, i);
        if constexpr (SP) f.idx[c][i] = read_idx(st.a, c, i);
      }
#pragma unroll
      for (int j = 0; j < FJ; ++j) {
        f.b0[c][j] = read_b(st.b + c * B_CHUNK, 0, j);
        f.b1[c][j] = read_b(st.b + c * B_CHUNK, 1, j);
      }
    }
  };
  auto mma = [&](const Frag& f) {
#pragma unroll
    for (int c = 0; c < KM; ++c) {
      if constexpr (SP) {
#pragma unroll
        for (int j = 0; j < FJ; ++j)
#pragma unroll
          for (int i = 0; i < FI; ++i)
            acc[i][j] = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(f.a[c][0][i], both(f.b0[c][j], f.b1[c][j]), acc[i][j],
                                                                  f.idx[c][i], 0, 0);
      } else {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int j = 0; j < FJ; ++j)
#pragma unroll
            for (int i = 0; i < FI; ++i)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  f.a[c][ks][i], __builtin_bit_cast(bf16x8, ks ? f.b1[c][j] : f.b0[c][j]), acc[i][j], 0, 0, 0);
      }
    }
  };
  if (n > 0) k_ring<NST, KM * (NA + NB) + (SP ? 1 : 0), Frag>(n, S, issue, mend, read, mma);

  // LDS of a wave to turn in: a quarter of the waves in each of four arrays
  constexpr int TURN = Turn<FI, FJ>::BYTES, QW = NW / 4;
  static_assert(A_BYTES >= QW * TURN && B_BYTES >= QW * TURN, "LDS of a wave to turn in");
  unsigned char* const mine =
      (wave < QW ? sA0 : wave < 2 * QW ? sB0 : wave < 3 * QW ? sA1 : sB1) + wave % QW * TURN;
  lin_finish<FI, FJ>(acc, epi, part, kpart, T, O, o0 + wmi * SM, t0 + wni * SN, lane, mine);
}

// ------------------------------------------------------------------------- the large products ---

// acc += a b on the accumulator half of the register file.  Written out so that the 256 sums stay
// where they are.  The compiler does not see this as a matrix instruction, so the waits it would
// insert are here: s_nop 1 ahead (an operand just written by a vector instruction), mma_done()
// before the sums are read.
__device__ __forceinline__ void mma_acc(f32x16& c, bf16x8 a, bf16x8 b) {
  asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
__device__ __forceinline__ void smma_acc(f32x16& c, bf16x8 a, u32x8 b, int idx) {
  asm volatile("s_nop 1\n\tv_smfmac_f32_32x32x32_bf16 %0, %1, %2, %3" : "+a"(c) : "v"(a), "v"(b), "v"(idx));
}
__device__ __forceinline__ void mma_done(f32x16 (&acc)[4][4]) {
  asm volatile("s_nop 15\n\ts_nop 15");
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) asm volatile("" : "+a"(acc[i][j]));
}
// one sum, read when it is used (read together they would need 256 more registers)
__device__ __forceinline__ float acc_read(float a) {
  float v;
  asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a));
  return v;
}

// 256 x 256 tiles by 4 waves of 128 x 128, one per SIMD.  A wave reads 256 rows of LDS for 128 x 128
// outputs (the 8-wave form, 192 for 64 x 128: there LDS' reads and the stages' writes together
// take as long as the products).  A wave's rows and tokens lie half in the tile's first and half in
// its last 128, so that a step's stage is four regions, AT and AB (weight rows), BL and BR (tokens),
// and the step four phases, a quadrant of 64 x 64 each: AT BL, AT BR, AB BR, AB BL.  Each phase reads
// one region, the one the next phase needs, into the registers of the one it will no longer need:
//   phase     multiplies   reads             requests (into what was read a phase before)
//   0 of s    AT BL        BR of s           BL of s + 2
//   1         AT BR        AB of s           BR of s + 2
//   2         AB BR        AT of s + 1       AB of s + 2
//   3         AB BL        BL of s + 1       AT of s + 3
// (BL of the next step takes BR's registers: the two swap roles every step.)  A region is needed six
// phases, one and a half steps, after its request, and each phase ends with one wait (at most the
// six phases' requests since are outstanding, never none) and one barrier, so up to 96 KiB are in
// flight per CU and no phase waits for a request's latency.  Reads and requests are placed between
// the matrix instructions, which a phase has 16 of.
// v_mfma_f32_32x32x16_bf16: lane (c, h) = (lane & 31, lane >> 5) holds values 8 h + [0, 8) of a
// 16-position part of row c, of either side; its sums are rows 8 (v / 4) + 4 h + v % 4 of token c.
//
// Bound by power: the matrix pipe is busy in 82% of cycles without an epilogue, 73% with bias and
// gelu, and the card runs them at 1.45 GHz; the same loop with nothing but its matrix instructions
// takes 506-528 us at 8192 x 4096 x 14336, with nothing but its loads 518-534.  Measured (cards differ
// by 5%): 8192 x 4096 x 14336 684 us (8 waves of 64 x 128 on two stages 722), 8192 x 14336 x 4096 with
// bias and gelu 741-780 (without 707-735), 4096 x 4096 x 4096 104 (110).  On a card where they take 692,
// 755 (with a bias) and 110 the library's bf16 products of these sizes, which have no epilogue, take
// 616, 667 and 95.
__global__ __launch_bounds__(256) void k_lin_big(
    const uint16_t* __restrict__ x, int64_t ldx, const uint16_t* __restrict__ w, int64_t ldw, int64_t T, int64_t O, int k,
    LinEpi epi, int tiles_m, int tiles_n, int group) {
  constexpr int REGION = 128 * 128;   // rows of 128 bytes
  __shared__ __align__(16) unsigned char at0[REGION], at1[REGION], ab0[REGION], ab1[REGION], bl0[REGION], bl1[REGION],
      br0[REGION], br1[REGION];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wmi = wave & 1, wni = wave >> 1;
  const int c = lane & 31, h = lane >> 5;

  const int lin = by_xcd();
  const int band = lin / (group * tiles_n);
  const int band_w = min(group, tiles_m - band * group);
  const int inband = lin - band * group * tiles_n;
  // wave-uniform (the division leaves them in vector registers; descriptors need scalars)
  const int tile_m = __builtin_amdgcn_readfirstlane(band * group + inband % band_w);
  const int tile_n = __builtin_amdgcn_readfirstlane(inband / band_w);
  const int64_t o0 = (int64_t)tile_m * 256, t0 = (int64_t)tile_n * 256;
  const int orows = (int)(O - o0 < 256 ? O - o0 : 256), trows = (int)(T - t0 < 256 ? T - t0 : 256);
  const int n = (k + 63) / 64;   // steps, >= 1

  // descriptors of the tile's rows, and the lane's offset of each load: four of a region
  const __amdgpu_buffer_rsrc_t rx = rsrc_of(x + t0 * ldx, (uint32_t)(trows * ldx * 2));
  const __amdgpu_buffer_rsrc_t rw = rsrc_of(w + o0 * ldw, (uint32_t)(orows * ldw * 2));
  uint32_t woff[2][4], xoff[2][4];
  uint32_t tail;   // in the last step: kPast where the lane's piece starts past the row
  {
    const int p = swz8(wave * 8 + (lane >> 3), lane & 7);   // one piece for every load: rows differ by multiples of 32
    tail = (n - 1) * 64 + 8 * p >= k ? kPast : 0u;
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = 128 * half + (wave + 4 * q) * 8 + (lane >> 3);
        woff[half][q] = (uint32_t)((r < orows ? r : orows - 1) * (int)ldw * 2 + 16 * p);
        xoff[half][q] = (uint32_t)((r < trows ? r : trows - 1) * (int)ldx * 2 + 16 * p);
      }
  }
  // request q of a region of step s; past the last step the last again (no one reads it)
  auto request = [&](__amdgpu_buffer_rsrc_t rsrc, unsigned char* region, uint32_t off, int q, int s) {
    const int sc = s < n ? s : n - 1;
    b2lds16(rsrc, region + (wave + 4 * q) * 1024, off | (sc == n - 1 ? tail : 0u), (uint32_t)(sc * 128));
  };
  // fragments: block b (of 2) and part ks (of 4) of a region's 64 rows of this wave
  int apos[4], bpos[4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    apos[ks] = (wmi * 64 + c) * 128 + 16 * swz8(c, 2 * ks + h);
    bpos[ks] = (wni * 64 + c) * 128 + 16 * swz8(c, 2 * ks + h);
  }
  struct Frag {
    bf16x8 v[4][2];   // [part][block]
  };
  auto read = [&](Frag& f, const unsigned char* region, const int (&pos)[4], int e) {   // read e of 8
    f.v[e >> 1][e & 1] = *reinterpret_cast<const bf16x8*>(region + pos[e >> 1] + (e & 1) * 4096);
  };

  f32x16 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  // a row that ends inside a piece: the last step's values past it zeroed, one row a thread
  auto mend = [&](unsigned char* at, unsigned char* ab, unsigned char* bl, unsigned char* br) {
    const int e0 = k & 7, p = (k & 63) >> 3, r = tid & 127;
    unsigned char* const ra = (tid < 128 ? at : ab) + r * 128 + 16 * swz8(r, p);
    unsigned char* const rb = (tid < 128 ? bl : br) + r * 128 + 16 * swz8(r, p);
    for (int e = e0; e < 8; ++e) {
      *reinterpret_cast<uint16_t*>(ra + 2 * e) = 0;
      *reinterpret_cast<uint16_t*>(rb + 2 * e) = 0;
    }
  };
  const bool ragged = (k & 7) != 0;

  Frag fat, fab, f0, f1;   // f0, f1: BL and BR of an even step, BR and BL of an odd one
  // a phase: quadrant (I, J) from fa, fb; next region into fn; requests of region rq
  auto phase = [&](auto I, auto J, const Frag& fa, const Frag& fb, Frag& fn, const unsigned char* rd, const int (&pos)[4],
                   __amdgpu_buffer_rsrc_t rsrc, unsigned char* rq, const uint32_t (&off)[4], int s) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int ks = e >> 2, i = (e >> 1) & 1, j = e & 1;
      mma_acc(acc[2 * I + i][2 * J + j], fa.v[ks][i], fb.v[ks][j]);
      if (e < 8) read(fn, rd, pos, e);
      else if (e < 12) request(rsrc, rq, off[e - 8], e - 8, s);
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0 & vm_wait(24));
    bar();
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  // step s in stage cur, the next in nxt; fl, fr: BL (held) and BR of this step
  auto step = [&](Frag& fl, Frag& fr, unsigned char* atn, unsigned char* abc, unsigned char* blc, unsigned char* bln,
                  unsigned char* brc, unsigned char* abn, unsigned char* brn, int s) __attribute__((always_inline)) {
    phase(I0{}, I0{}, fat, fl, fr, brc, bpos, rx, blc, xoff[0], s + 2);
    phase(I0{}, I1{}, fat, fr, fab, abc, apos, rx, brc, xoff[1], s + 2);
    if (ragged && s == n - 2) {   // the last step, before any of it is read
      __builtin_amdgcn_s_waitcnt(vm_wait(0));
      bar();
      mend(atn, abn, bln, brn);
      __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
      bar();
    }
    phase(I1{}, I1{}, fab, fr, fat, atn, apos, rw, abc, woff[1], s + 2);
    phase(I1{}, I0{}, fab, fl, fr, bln, bpos, rw, atn, woff[0], s + 3);
  };
  auto request_all = [&](unsigned char* at, unsigned char* bl, unsigned char* br, unsigned char* ab, int s) {
#pragma unroll
    for (int q = 0; q < 4; ++q) request(rw, at, woff[0][q], q, s);
#pragma unroll
    for (int q = 0; q < 4; ++q) request(rx, bl, xoff[0][q], q, s);
#pragma unroll
    for (int q = 0; q < 4; ++q) request(rx, br, xoff[1][q], q, s);
#pragma unroll
    for (int q = 0; q < 4; ++q) request(rw, ab, woff[1][q], q, s);
  };
  request_all(at0, bl0, br0, ab0, 0);
  request_all(at1, bl1, br1, ab1, 1);
  if (ragged && n == 1) {
    __builtin_amdgcn_s_waitcnt(vm_wait(0));
    bar();
    mend(at0, ab0, bl0, br0);
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
  }
  __builtin_amdgcn_s_waitcnt(vm_wait(24));
  bar();
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    read(fat, at0, apos, e);
    read(f0, bl0, bpos, e);
  }
  __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
  bar();
#pragma unroll
  for (int q = 0; q < 4; ++q) request(rw, at0, woff[0][q], q, 2);
  __builtin_amdgcn_s_waitcnt(vm_wait(24));
  bar();
  int s = 0;
  for (; s + 2 <= n; s += 2) {
    step(f0, f1, at1, ab0, bl0, bl1, br0, ab1, br1, s);
    step(f1, f0, at0, ab1, bl1, bl0, br1, ab0, br0, s + 1);
  }
  if (s < n) step(f0, f1, at1, ab0, bl0, bl1, br0, ab1, br1, s);
  __builtin_amdgcn_s_waitcnt(0);
  bar();
  mma_done(acc);

  // turns of 64 outputs (two blocks) by 32 tokens, 8 KiB a wave
  unsigned char* const mine = wave == 0 ? at0 : wave == 1 ? at1 : wave == 2 ? ab0 : ab1;
  using E = Emit<64, 32>;
  lin_emit<2, 4, 64, 32>(
      epi, T, O, lane, mine,
      [&](auto hc, auto jc) __attribute__((always_inline)) {
        constexpr int hh = decltype(hc)::value, j = decltype(jc)::value;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const f32x16& a = acc[2 * hh + i][j];
            *reinterpret_cast<f32x4*>(E::place(mine, c, 8 * i + 2 * g + h)) =
                f32x4{acc_read(a[4 * g]), acc_read(a[4 * g + 1]), acc_read(a[4 * g + 2]), acc_read(a[4 * g + 3])};
          }
      },
      [&](int hh) { return o0 + 128 * hh + 64 * wmi; },
      [&](int j) { return t0 + 128 * (j >> 1) + 64 * wni + 32 * (j & 1); });
}

// 256 x 256 tiles of 2:4 products by 4 waves of 128 x 128.  The sparse instruction takes X twice as fast
// as the dense one, so a step's stage is 50 KiB for half the products and three stages fit: nothing
// but the wave itself hides a latency, so operands are read two phases of 16 matrix instructions
// ahead, a read or a request between two of them.
//  * v_smfmac_f32_32x32x32_bf16: lane (c, h) = (lane & 31, lane >> 5) holds the 8 kept values of row c at
//    positions [16 h, + 16) of a 32-position phase with their 16 bits of positions, and of X the
//    values [8 h, + 8) and [16 + 8 h, + 8).
//  * A step of 64 positions is two phases.  When a step begins, its operands are in registers and the
//    next step's have landed: one wait, one barrier, and the stage takes the requests of the step
//    after the next two.
// The matrix pipe is busy in 44% of cycles, LDS in 24% (11% of these conflicts, in the positions), at
// 1.78 GHz (bias and gelu, 8192 x 14336 x 4096): less than the dense product's share, since a
// step's barrier comes after half its matrix cycles.  Measured: 8192 x 14336 x 4096 528 us (8
// waves of 64 x 128 on two stages 656), 8192 x 4096 x 14336 504 (713), 4096 x 4096 x 4096 78 (94); on
// another card 542, 519 and 87 with a bias.
__global__ __launch_bounds__(256) void k_lin_big24(
    const uint16_t* __restrict__ x, int64_t ldx, const uint16_t* __restrict__ w, int64_t ldw,
    const uint8_t* __restrict__ meta, int64_t T, int64_t O, int k, LinEpi epi, int tiles_m, int tiles_n, int group) {
  constexpr int NW = 4;
  constexpr int V_BYTES = 256 * 64, A_BYTES = V_BYTES + 256 * 8, B_BYTES = 256 * 128;   // values, positions; X
  constexpr int NA = 4, NB = 8, NM = 2, NL = NA + NB + NM;   // loads of a wave per step
  __shared__ __align__(16) unsigned char s0[A_BYTES + B_BYTES], s1[A_BYTES + B_BYTES], s2[A_BYTES + B_BYTES];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wmi = wave & 1, wni = wave >> 1;
  const int c = lane & 31, h = lane >> 5;

  const int lin = by_xcd();
  const int band = lin / (group * tiles_n);
  const int band_w = min(group, tiles_m - band * group);
  const int inband = lin - band * group * tiles_n;
  // wave-uniform (the division leaves them in vector registers; descriptors need scalars)
  const int tile_m = __builtin_amdgcn_readfirstlane(band * group + inband % band_w);
  const int tile_n = __builtin_amdgcn_readfirstlane(inband / band_w);
  const int64_t o0 = (int64_t)tile_m * 256, t0 = (int64_t)tile_n * 256;
  const int orows = (int)(O - o0 < 256 ? O - o0 : 256), trows = (int)(T - t0 < 256 ? T - t0 : 256);
  const int n = (k + 63) / 64;   // steps, >= 1

  const __amdgpu_buffer_rsrc_t rx = rsrc_of(x + t0 * ldx, (uint32_t)(trows * ldx * 2));
  const __amdgpu_buffer_rsrc_t rw = rsrc_of(w + o0 * ldw, (uint32_t)(orows * ldw * 2));
  uint32_t aoff[NA], boff[NB];
  uint32_t atail, btail;   // in the last step: kPast where the lane's piece starts past the row
#pragma unroll
  for (int q = 0; q < NA; ++q) {
    const int r = (wave + q * NW) * 16 + (lane >> 2);
    const int p = swz4(r, lane & 3);
    aoff[q] = (uint32_t)((r < orows ? r : orows - 1) * (int)ldw * 2 + 16 * p);
    if (q == 0) atail = (n - 1) * 32 + 8 * p >= k / 2 ? kPast : 0u;
  }
#pragma unroll
  for (int q = 0; q < NB; ++q) {
    const int r = (wave + q * NW) * 8 + (lane >> 3);
    const int p = swz8(r, lane & 7);
    boff[q] = (uint32_t)((r < trows ? r : trows - 1) * (int)ldx * 2 + 16 * p);
    if (q == 0) btail = (n - 1) * 64 + 8 * p >= k ? kPast : 0u;
  }
  const uint8_t* mlane[NM];   // the lane's positions in step 0: 32 rows of two lanes a load
#pragma unroll
  for (int q = 0; q < NM; ++q) {
    const int r = wave * 64 + q * 32 + (lane >> 1);
    mlane[q] = meta + (o0 + (r < orows ? r : orows - 1)) * 16 + 4 * (lane & 1);
  }
  int ls = 0;   // the step being requested; past the last one the last again (no one reads it)
  uint32_t at = 0, bt = 0;
  int64_t ms = 0;
  auto begin_loads = [&](int s) {
    ls = s < n ? s : n - 1;
    at = ls == n - 1 ? atail : 0u;
    bt = ls == n - 1 ? btail : 0u;
    ms = (ls >> 1) * (O * 16) + 8 * (ls & 1);
  };
  auto load = [&](unsigned char* st, int q) {   // load q of step ls into stage st
    if (q < NA) {
      b2lds16(rw, st + (wave + q * NW) * 1024, aoff[q] | at, (uint32_t)(ls * 64));
    } else if (q < NA + NB) {
      const int p = q - NA;
      b2lds16(rx, st + A_BYTES + (wave + p * NW) * 1024, boff[p] | bt, (uint32_t)(ls * 128));
    } else {
      const int p = q - NA - NB;
      __builtin_amdgcn_global_load_lds(mlane[p] + ms, (lds_void*)(st + V_BYTES + wave * 512 + p * 256), 4, 0, 0);
    }
  };
  auto lds4 = [](const unsigned char* p) { return *reinterpret_cast<const u32x4*>(p); };
  // fragment addresses: rows 32 i + c of the wave's 128, whose swizzle does not depend on i
  const int ab = (wmi * 128 + c) * 64, bb = A_BYTES + (wni * 128 + c) * 128;
  const int mb = V_BYTES + (wmi * 128 + c) * 8 + 2 * h;
  int apos[2], bpos[4];   // pieces 2 e + h of a weight row, of a token row
#pragma unroll
  for (int e = 0; e < 2; ++e) apos[e] = ab + 16 * swz4(c, 2 * e + h);
#pragma unroll
  for (int e = 0; e < 4; ++e) bpos[e] = bb + 16 * swz8(c, 2 * e + h);

  f32x16 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  struct Frag {
    bf16x8 a[4];
    u32x8 b[4];
    int idx[4];
  };
  auto read = [&](Frag& f, const unsigned char* st, int ks, int e) {   // read e of 12 (two for X)
    if (e < 4) f.a[e] = __builtin_bit_cast(bf16x8, lds4(st + apos[ks] + e * 2048));
    else if (e < 8) f.idx[e - 4] = *reinterpret_cast<const uint16_t*>(st + mb + 4 * ks + (e - 4) * 256);
    else f.b[e - 8] = __builtin_shufflevector(lds4(st + bpos[2 * ks] + (e - 8) * 4096),
                                              lds4(st + bpos[2 * ks + 1] + (e - 8) * 4096), 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto phase = [&](const Frag& f, Frag& fn, const unsigned char* rd, int ks, bool LOAD, unsigned char* wr)
      __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int j = e >> 2, i = e & 3;
      smma_acc(acc[i][j], f.a[i], f.b[j], f.idx[i]);
      if (e < 12) read(fn, rd, ks, e < 8 ? ((e & 1) ? 4 + e / 2 : e / 2) : e);
      if (LOAD && e < NL) load(wr, e);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  static_assert(NL <= 16, "a load per product");
  // a row that ends inside a piece: the last step's values past it zeroed, a row of each side a thread
  const int wlen = k / 2;
  const bool ragged = (k & 7) != 0 || (wlen & 7) != 0;
  auto mend = [&](unsigned char* st) {
    unsigned char* const ra = st + tid * 64 + 16 * swz4(tid, (wlen & 31) >> 3);
    unsigned char* const rb = st + A_BYTES + tid * 128 + 16 * swz8(tid, (k & 63) >> 3);
    for (int e = wlen & 7; (wlen & 7) != 0 && e < 8; ++e) *reinterpret_cast<uint16_t*>(ra + 2 * e) = 0;
    for (int e = k & 7; (k & 7) != 0 && e < 8; ++e) *reinterpret_cast<uint16_t*>(rb + 2 * e) = 0;
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
    bar();
  };
  Frag f0, f1, f2;   // part p of step s is the (2 s + p) % 3rd
  begin_loads(0);
#pragma unroll
  for (int q = 0; q < NL; ++q) load(s0, q);
  begin_loads(1);
#pragma unroll
  for (int q = 0; q < NL; ++q) load(s1, q);
  begin_loads(2);
#pragma unroll
  for (int q = 0; q < NL; ++q) load(s2, q);
  __builtin_amdgcn_s_waitcnt(vm_wait(2 * NL));
  bar();
  if (ragged && n == 1) mend(s0);
#pragma unroll
  for (int e = 0; e < 12; ++e) read(f0, s0, 0, e);
#pragma unroll
  for (int e = 0; e < 12; ++e) read(f1, s0, 1, e);
  // step s of (fa, fb): its operands are all read by now, so its stage takes the loads of
  // step s + 3 while those of step s + 1 come from nxt: (fc, fa)
  auto step = [&](Frag& fa, Frag& fb, Frag& fc, unsigned char* cur, unsigned char* nxt, int s) __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0 & vm_wait(NL));   // step s + 1 landed; reads of step s arrived
    bar();
    if (ragged && s == n - 2) mend(nxt);   // the last step, before any of it is read
    begin_loads(s + 3);
    phase(fa, fc, nxt, 0, true, cur);
    phase(fb, fa, nxt, 1, false, nullptr);
  };
  int s = 0;
  for (; s + 3 <= n; s += 3) {
    step(f0, f1, f2, s0, s1, s);
    step(f2, f0, f1, s1, s2, s + 1);
    step(f1, f2, f0, s2, s0, s + 2);
  }
  if (s < n) step(f0, f1, f2, s0, s1, s);
  if (s + 1 < n) step(f2, f0, f1, s1, s2, s + 1);
  __builtin_amdgcn_s_waitcnt(0);   // loads and reads past the last step
  bar();
  mma_done(acc);

  unsigned char* const mine = s0 + wave * 8192;
  using E = Emit<64, 32>;
  lin_emit<2, 4, 64, 32>(
      epi, T, O, lane, mine,
      [&](auto hc, auto jc) __attribute__((always_inline)) {
        constexpr int hh = decltype(hc)::value, j = decltype(jc)::value;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const f32x16& a = acc[2 * hh + i][j];
            *reinterpret_cast<f32x4*>(E::place(mine, c, 8 * i + 2 * g + h)) =
                f32x4{acc_read(a[4 * g]), acc_read(a[4 * g + 1]), acc_read(a[4 * g + 2]), acc_read(a[4 * g + 3])};
          }
      },
      [&](int hh) { return o0 + 128 * wmi + 64 * hh; }, [&](int j) { return t0 + 128 * wni + 32 * j; });
}

template <int BM, int BN, int WM, int WN, bool SP, int NST, int KM>
hipError_t launch_cfg(const LinArgs& a, int64_t splits, float* part, hipStream_t s) {
  const int64_t tm = (a.o + BM - 1) / BM, tn = (a.t + BN - 1) / BN, ntiles = tm * tn;
  if (tm > 0x7FFFFFFF || tn > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  const int64_t steps = ((a.k + 63) / 64 + KM - 1) / KM;
  if (splits < 1 || part == nullptr) splits = 1;
  const int64_t per = steps > 0 ? (steps + splits - 1) / splits : 1;
  splits = steps > 0 ? (steps + per - 1) / per : 1;
  if (ntiles * splits > 0x7FFFFFFF / (WM * WN * 32)) return hipErrorInvalidConfiguration;   // a grid holds under 2^32 threads
  // o-tiles per band of the tile order: an XCD runs 32 tiles at a time
  const int64_t group = tm < 8 ? tm : 8;
  k_lin_tile<BM, BN, WM, WN, SP, NST, KM><<<dim3((unsigned)(ntiles * splits)), dim3(64 * WM * WN), 0, s>>>(
      a.x, a.ldx, a.w, a.ldw, a.meta, a.t, a.o, (int)a.k, a.epi, splits > 1 ? part : nullptr, (int)tm, (int)tn, (int)per,
      (int)group);
  a.route.note(NM_TAKEN_TILE_LDS | (SP ? NM_TAKEN_SPARSE_MMA : 0u) | (splits > 1 ? NM_TAKEN_TILE_SPLIT : 0u));
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  return launch_lin_reduce(part, splits, a.t, a.o, a.epi, a.route, s);
}

template <bool SP>
hipError_t launch_kind(const LinArgs& a, int shape, int64_t splits, float* part, hipStream_t s) {
  switch (shape) {
    case 0: return launch_cfg<128, 128, 4, 2, SP, 3, SP ? 2 : 1>(a, splits, part, s);
    case 1: return launch_cfg<128, 64, 4, 2, SP, SP ? 3 : 4, SP ? 2 : 1>(a, splits, part, s);
    case 2: return launch_cfg<64, 64, 2, 2, SP, 4, SP ? 2 : 1>(a, splits, part, s);
    case 3: return launch_cfg<64, 32, 2, 2, SP, 4, 2>(a, splits, part, s);
  }
  const int64_t tm = (a.o + 255) / 256, tn = (a.t + 255) / 256;
  if (tm > 0x7FFFFFFF || tn > 0x7FFFFFFF || tm * tn > 0xFFFFFF) return hipErrorInvalidConfiguration;   // under 2^32 threads
  const dim3 grid((unsigned)(tm * tn)), block(256);
  const int group = (int)(tm < 8 ? tm : 8);
  if constexpr (SP)
    k_lin_big24<<<grid, block, 0, s>>>(a.x, a.ldx, a.w, a.ldw, a.meta, a.t, a.o, (int)a.k, a.epi, (int)tm, (int)tn, group);
  else
    k_lin_big<<<grid, block, 0, s>>>(a.x, a.ldx, a.w, a.ldw, a.t, a.o, (int)a.k, a.epi, (int)tm, (int)tn, group);
  a.route.note(NM_TAKEN_TILE_LDS | (SP ? NM_TAKEN_SPARSE_MMA : 0u));
  return hipGetLastError();
}

struct MidPlan {
  int shape;        // 128 x 128, 128 x 64, 64 x 64, 64 x 32 (weight rows x tokens)
  int64_t splits;
};

// The tile and the number of reduction ranges of least estimated time:
//   chunks of a range * time of one * rounds of 256 workgroups (whole ones where the stages leave a
//   CU one workgroup; the weights' stream at 5 TB/s where that is longer), and where the reduction
//   is split 2.8 us for the second kernel and its partial sums, written and read, at 3.2 TB/s.
// A chunk's time is that of its loads' latency behind the barrier, whatever it holds, up to 256
// workgroups: measured (with weights from HBM) and fitted with the other constants over 28 sizes of
// 16 to 777 tokens.  Over 48 others of 40 to 3000 tokens the plan chosen is 1.4% slower than the best
// of 16 on average (with parts of a round throughout 4.5%: 600 x 4096 x 4096 128 x 64 54, 128 x 128 40 us).
// Some of them (us, tile x ranges): 40 x 4096 x 14336 64 x 32 x 2 40.6, 64 x 64 x 4 30.7, 128 x 64 x 8
// 31.1, unsplit 59-120; 128 x 4096 x 14336 64 x 32 58.5, 64 x 64 x 2 44.6, 128 x 64 x 4 42.6, 128 x 128 x
// 8 40.3; 64 x 14336 x 4096 64 x 64 31.9, x 2 36.6, 64 x 32 38.0; 600 x 2048 x 2048 128 x 64 13.9, 64 x
// 64 15.1, 64 x 32 16.5; 2:4 40 x 4096 x 14336 128 x 64 x 8 24.5, 64 x 64 x 4 24.5, 64 x 32 x 4 31.5;
// 64 x 4096 x 4096 64 x 32 x 2 11.7, 64 x 64 x 4 12.5; 128 x 4096 x 14336 128 x 64 x 4 32.0, 128 x 128 x
// 8 32.5, 64 x 64 x 4 40.3.
MidPlan mid_plan(int64_t t, int64_t o, int64_t k, bool sparse) {
  constexpr int kBM[4] = {128, 128, 64, 64}, kBN[4] = {128, 64, 64, 32};
  constexpr int kRanges[8] = {1, 2, 3, 4, 6, 8, 12, 16};
  constexpr double kChunk[2][4] = {{0.60, 0.45, 0.31, 0.255}, {0.50, 0.34, 0.286, 0.168}};   // us
  constexpr bool kAlone[2][4] = {{true, true, false, true}, {true, true, true, false}};   // on a CU
  const int64_t chunks = (k + 63) / 64;
  const double stream = (double)o * (double)k * (sparse ? 1.125 : 2.0) / 5.0e6;
  MidPlan best{3, 1};
  double least = 0;
  for (int sh = 3; sh >= 0; --sh) {
    const double tiles = (double)((o + kBM[sh] - 1) / kBM[sh]) * (double)((t + kBN[sh] - 1) / kBN[sh]);
    for (int r : kRanges) {
      if (r > 1 && (chunks < 8 * r || tiles * r > 1024)) break;
      const double full = tiles * r / 256, rounds = full <= 1.0 ? 1.0 : kAlone[sparse][sh] ? __builtin_ceil(full) : full;
      double us = (double)((chunks + r - 1) / r) * kChunk[sparse][sh] * rounds;
      if (us < stream) us = stream;
      if (r > 1) us += 2.8 + (double)r * (double)t * (double)o * 8 / 3.2e6;
      if ((sh == 3 && r == 1) || us < least) {
        least = us;
        best = {sh, r};
      }
    }
  }
  return best;
}

}  // namespace

namespace nml {

bool lin_tile_eligible(const LinArgs& a) {
  // descriptors hold 256 rows in under 2^31 bytes
  return a.k > 0 && a.ldx < (1 << 22) && a.ldw < (1 << 22);
}

int64_t lin_mid_part_bytes(int64_t t, int64_t o, int64_t k, bool sparse) {
  const int64_t s = mid_plan(t, o, k, sparse).splits;
  return s > 1 ? s * t * ((o + 3) / 4 * 4) * 4 : 0;
}

hipError_t launch_lin_tile(const LinArgs& a, bool large, float* part, int64_t part_bytes, hipStream_t s) {
  MidPlan p{-1, 1};   // 256 x 256 tiles
  if (!large) {
    const bool sp = a.meta != nullptr;
    p = mid_plan(a.t, a.o, a.k, sp);
    // the tile stays the split plan's (40 x 4096 x 14336 67 us, 2:4 73, with a workspace 37 and 26)
    if (part == nullptr || part_bytes < lin_mid_part_bytes(a.t, a.o, a.k, sp)) p.splits = 1;
  }
  return a.meta != nullptr ? launch_kind<true>(a, p.shape, p.splits, part, s)
                           : launch_kind<false>(a, p.shape, p.splits, part, s);
}

}  // namespace nml
