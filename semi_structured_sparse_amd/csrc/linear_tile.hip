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

__device__ __forceinline__ void bar() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// K-loops over n >= 1 steps through NST stages (distinct static arrays, named by constant indices,
// so that the compiler tracks the requests into each one).  issue(st, s) requests step s into
// st; mend(st, s) makes up a landed step that the row's end falls into.  Both end with every
// request landed and every stage free.

// Two stages of large steps: a step's requests go out before the step ahead of it is multiplied
// and are waited for after it.
template <typename Issue, typename Mend, typename Compute>
__device__ __forceinline__ void k_loop2(int n, Stage a, Stage b, Issue&& issue, Mend&& mend, Compute&& compute) {
  issue(a, 0);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  for (int s = 0; s < n; s += 2) {
    mend(a, s);
    if (s + 1 < n) issue(b, s + 1);
    compute(a);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (s + 1 < n) {
      mend(b, s + 1);
      if (s + 2 < n) issue(a, s + 2);
      compute(b);
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
    }
  }
}

// Small steps: step q requests step q + NST - 1 into the stage that step q - 1 used, reads its
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

// What a wave does with its finished sums: FI x FJ blocks of 16 x 16, lane (fr, fq) = (lane & 15,
// lane >> 4) holding outputs 4 fq + [0, 4) of each block's range for token fr.  ob_w, tb_w: the wave's
// first output and token.  With a split reduction the sums go to part.  Otherwise 16 JB tokens at
// a time are turned through the wave's own LDS at `mine` (rows of W outputs, 16-byte piece c of row
// r at c ^ (r & (W / 4 - 1))): neighbouring lanes hold neighbouring outputs of a row, four each
// where rows of y and the residual keep that alignment, one each otherwise.  The residual's
// loads go out together, ahead of the turn.
template <int FI, int FJ>
struct Turn {
  static constexpr int BI = FI < 4 ? FI : 4, W = 16 * BI, PC = W / 4;   // blocks, outputs and pieces of a row
  static constexpr int JB = FJ < 2 ? FJ : 2, ROWS = 16 * JB;
  static constexpr int BYTES = ROWS * W * 4;
  static_assert(FI % BI == 0 && FJ % JB == 0 && (PC == 8 || PC == 16), "rows of 32 or 64 outputs");
};

// f(0), f(step), ... below end, each with its number as a constant (sums that the compiler indexed by
// a variable would lie in memory)
template <int I, int END, int STEP, typename F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (I < END) {
    f(std::integral_constant<int, I>{});
    each<I + STEP, END, STEP>(f);
  }
}

template <int FI, int FJ>
__device__ __forceinline__ void lin_finish(const f32x4 (&acc)[FI][FJ], const LinEpi& epi, float* __restrict__ part,
                                           int kpart, int64_t T, int64_t O, int64_t ob_w, int64_t tb_w, int lane,
                                           unsigned char* mine) {
  using C = Turn<FI, FJ>;
  constexpr int W = C::W, PC = C::PC, ROWS = C::ROWS;
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
  auto place = [&](int r, int c) { return mine + r * (4 * W) + 16 * (c ^ (r & (PC - 1))); };
  auto put = [&](auto hc, auto jc) __attribute__((always_inline)) {
    constexpr int h = decltype(hc)::value, j = decltype(jc)::value;
#pragma unroll
    for (int jj = 0; jj < C::JB; ++jj)
#pragma unroll
      for (int i = 0; i < C::BI; ++i)
        *reinterpret_cast<f32x4*>(place(16 * jj + fr, 4 * i + fq)) = acc[C::BI * h + i][j + jj];
    wave_lds_fence();
  };
  if (lin_whole(epi)) {
    constexpr int RP = 64 / PC, NP = ROWS / RP;   // rows of a pass, passes
    each<0, FI / C::BI, 1>([&](auto h) __attribute__((always_inline)) {
      const int64_t o = ob_w + W * h + 4 * (lane % PC);
      const bool whole = o + 4 <= O;
      f32x4 bias = {0.f, 0.f, 0.f, 0.f};
      if (epi.bias != nullptr && whole) bias = *reinterpret_cast<const f32x4*>(epi.bias + o);
      each<0, FJ, C::JB>([&](auto j) __attribute__((always_inline)) {
        const int64_t tb = tb_w + 16 * j + lane / PC;
        uint4 r[NP];   // past the last row: its values, not used
        if (epi.residual != nullptr && whole) {
          if (epi.bf16_out) {
#pragma unroll
            for (int p = 0; p < NP; ++p) r[p] = lin_load4<true>(epi, tb + RP * p < T ? tb + RP * p : T - 1, o);
          } else {
#pragma unroll
            for (int p = 0; p < NP; ++p) r[p] = lin_load4<false>(epi, tb + RP * p < T ? tb + RP * p : T - 1, o);
          }
        }
        put(h, j);
        float v[4 * NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const f32x4 s = *reinterpret_cast<const f32x4*>(place(RP * p + lane / PC, lane % PC));
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * p + e] = s[e];
        }
        wave_lds_fence();
        if (whole) {
          if (epi.bias != nullptr) {
#pragma unroll
            for (int e = 0; e < 4 * NP; ++e) v[e] = v[e] + bias[e & 3];
          }
          lin_fns<4 * NP>(v, epi.fn);
#pragma unroll
          for (int p = 0; p < NP; ++p)
            if (tb + RP * p < T) lin_store4(epi, v + 4 * p, r[p], tb + RP * p, o);
        } else {
#pragma unroll
          for (int e = 0; e < 4 * NP; ++e)
            if (o + (e & 3) < O && tb + RP * (e >> 2) < T) lin_store(epi, v[e], tb + RP * (e >> 2), o + (e & 3));
        }
      });
    });
    return;
  }
  constexpr int RS = 64 / W, NP = ROWS / RS, NG = NP < 16 ? NP : 16;   // rows of a pass, passes, passes at a time
  each<0, FI / C::BI, 1>([&](auto h) __attribute__((always_inline)) {
    const int64_t o = ob_w + W * h + lane % W, oc = o < O ? o : O - 1;
    const float bias = epi.bias != nullptr ? epi.bias[oc] : 0.0f;
    each<0, FJ, C::JB>([&](auto j) __attribute__((always_inline)) {
      put(h, j);
      const int64_t tb = tb_w + 16 * j + lane / W;
#pragma unroll 1
      for (int g = 0; g < NP; g += NG) {
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
          v[p] = *reinterpret_cast<const float*>(place(RS * (g + p) + lane / W, lane % W / 4) + 4 * (lane & 3));
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
    });
  });
}

// BM x BN: weight rows by tokens of a tile; WM x WN waves; NST stages of KM chunks.
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
  constexpr int MROWS = BM / NW;               // rows whose positions a wave loads: 2 KM lanes each
  static_assert(NA >= 1 && NB >= 1 && BM % (RPG * NW) == 0 && BN % (8 * NW) == 0, "load groups per wave");
  static_assert(!SP || MROWS * KM == 16 || MROWS * KM == 32, "positions: 8 KM bytes a row, 4 a lane");
  constexpr int A2 = NST > 2 ? A_BYTES : 16, B2 = NST > 2 ? B_BYTES : 16, A3 = NST > 3 ? A_BYTES : 16, B3 = NST > 3 ? B_BYTES : 16;
  __shared__ __align__(16) unsigned char sA0[A_BYTES], sB0[B_BYTES], sA1[A_BYTES], sB1[B_BYTES], sA2[A2], sB2[B2], sA3[A3],
      sB3[B3];
  const Stage S[4] = {{sA0, sB0}, {sA1, sB1}, {sA2, sB2}, {sA3, sB3}};
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wmi = wave % WM, wni = wave / WM;
  const int fr = lane & 15, fq = lane >> 4;

  const int ntiles = tiles_m * tiles_n;
  const int kpart = __builtin_amdgcn_readfirstlane(blockIdx.x / ntiles);
  int lin = blockIdx.x - kpart * ntiles;
  if ((ntiles & 7) == 0 && gridDim.x == (unsigned)ntiles) lin = (blockIdx.x & 7) * (ntiles >> 3) + (blockIdx.x >> 3);
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
    const int r = wave * MROWS + lane / (2 * KM) % MROWS;
    const int o = r < orows ? r : orows - 1;
    mlane = meta + (o0 + o) * 16 + 4 * (lane % (2 * KM));
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
      const uint32_t at = ch < chunks - 1 ? 0u : ch == chunks - 1 ? atail : kPast;
#pragma unroll
      for (int q = 0; q < NA; ++q)
        b2lds16(rw, a + c * A_CHUNK + (wave + q * NW) * 1024, aoff[q] | at, (uint32_t)(ch * AROW));
    }
    if constexpr (SP) {
      if (MROWS * KM == 32 || lane < 32)
        __builtin_amdgcn_global_load_lds(KM == 2 ? mlane + s * (O * 16) : mlane + (s >> 1) * (O * 16) + 8 * (s & 1),
                                         (lds_void*)(a + V_BYTES + wave * MROWS * 8 * KM), 4, 0, 0);
    }
#pragma unroll
    for (int c = 0; c < KM; ++c) {
      const int ch = s * KM + c;
      const uint32_t bt = ch < chunks - 1 ? 0u : ch == chunks - 1 ? btail : kPast;
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
  // 256-row tiles: fragments a block ahead; the wait for them sits before the next reads (while a
  // direct-to-LDS load is in flight the compiler can only wait for all LDS reads)
  auto compute = [&](Stage st) {
    const unsigned char *const a = st.a, *const b = st.b;
    if constexpr (SP) {
      bf16x8 af[FI];
      int idx[FI];
#pragma unroll
      for (int i = 0; i < FI; ++i) {
        af[i] = read_a(a, 0, i);
        idx[i] = read_idx(a, 0, i);
      }
      bf16x16 bcur = both(read_b(b, 0, 0), read_b(b, 1, 0)), bnxt;
#pragma unroll
      for (int j = 0; j < FJ; ++j) {
        __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
        __builtin_amdgcn_sched_barrier(0);
        if (j + 1 < FJ) bnxt = both(read_b(b, 0, j + 1), read_b(b, 1, j + 1));
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < FI; ++i)
          acc[i][j] = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(af[i], bcur, acc[i][j], idx[i], 0, 0);
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
        bcur = bnxt;
      }
    } else {
      u32x4 b0[FJ], b1[FJ];
#pragma unroll
      for (int j = 0; j < FJ; ++j) b0[j] = read_b(b, 0, j);
      bf16x8 acur = read_a(a, 0, 0), anxt;
      constexpr int BPS = (FJ + FI - 1) / FI;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
        for (int i = 0; i < FI; ++i) {
          __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
          __builtin_amdgcn_sched_barrier(0);
          if (i + 1 < FI) anxt = read_a(a, ks, i + 1);
          else if (ks == 0) anxt = read_a(a, 1, 0);
          if (ks == 0) {
#pragma unroll
            for (int q = 0; q < BPS; ++q)
              if (i * BPS + q < FJ) b1[i * BPS + q] = read_b(b, 1, i * BPS + q);
          }
          __builtin_amdgcn_sched_barrier(0);
          __builtin_amdgcn_s_setprio(1);
#pragma unroll
          for (int j = 0; j < FJ; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(acur, __builtin_bit_cast(bf16x8, ks ? b1[j] : b0[j]),
                                                                acc[i][j], 0, 0, 0);
          __builtin_amdgcn_s_setprio(0);
          __builtin_amdgcn_sched_barrier(0);
          acur = anxt;
        }
      }
    }
  };
  // smaller tiles: the operands of a whole step at once (k_ring)
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
  if (n > 0) {
    if constexpr (NST == 2) k_loop2(n, S[0], S[1], issue, mend, compute);
    else k_ring<NST, KM * (NA + NB) + (SP ? 1 : 0), Frag>(n, S, issue, mend, read, mma);
  }

  // LDS of a wave to turn in: a quarter of the waves in each of four arrays
  constexpr int TURN = Turn<FI, FJ>::BYTES, QW = NW / 4;
  static_assert(A_BYTES >= QW * TURN && B_BYTES >= QW * TURN, "LDS of a wave to turn in");
  unsigned char* const mine =
      (wave < QW ? sA0 : wave < 2 * QW ? sB0 : wave < 3 * QW ? sA1 : sB1) + wave % QW * TURN;
  lin_finish<FI, FJ>(acc, epi, part, kpart, T, O, o0 + wmi * SM, t0 + wni * SN, lane, mine);
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
  return launch_cfg<256, 256, SP ? 2 : 4, SP ? 4 : 2, SP, 2, 1>(a, 1, nullptr, s);
}

struct MidPlan {
  int shape;        // 128 x 128, 128 x 64, 64 x 64, 64 x 32 (weight rows x tokens)
  int64_t splits;
};

// The tile and the number of reduction ranges of least estimated time:
//   chunks of a range * time of one * rounds of 256 workgroups (one per CU; the weights' stream at 5
//   TB/s where that is longer), and where the reduction is split 2.8 us for the second kernel and
//   its partial sums, written and read, at 3.2 TB/s.
// A chunk's time is that of its loads' latency behind the barrier, whatever it holds, up to 256
// workgroups: measured (with weights from HBM) and fitted with the other constants over 28 sizes of
// 16 to 777 tokens, 16 plans each: the plan chosen is 2% slower than the best of the 16 on average.
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
  const int64_t chunks = (k + 63) / 64;
  const double stream = (double)o * (double)k * (sparse ? 1.125 : 2.0) / 5.0e6;
  MidPlan best{3, 1};
  double least = 0;
  for (int sh = 3; sh >= 0; --sh) {
    const double tiles = (double)((o + kBM[sh] - 1) / kBM[sh]) * (double)((t + kBN[sh] - 1) / kBN[sh]);
    for (int r : kRanges) {
      if (r > 1 && (chunks < 8 * r || tiles * r > 1024)) break;
      const double rounds = tiles * r <= 256 ? 1.0 : tiles * r / 256;
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
    if (part == nullptr || part_bytes < lin_mid_part_bytes(a.t, a.o, a.k, sp)) p.splits = 1;
  }
  return a.meta != nullptr ? launch_kind<true>(a, p.shape, p.splits, part, s)
                           : launch_kind<false>(a, p.shape, p.splits, part, s);
}

}  // namespace nml
