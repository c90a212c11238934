// Int8 tile products, staged direct to LDS:
//   sum[t][o] = sum_k x[t][k] w[o][k]  in 32-bit integers, W dense or 2:4 (values and step-blocked
//   positions), y = (fp32(sum) x_scale[t]) w_scale[o] + beta_t c_o, or act(gate) * up (GLU).
//
// gfx950 design:
//  * A K-step is 128 reduction positions: 128 bytes of every X row and of every dense weight row
//    (64 bytes of kept codes and 16 of positions for 2:4), moved from global memory into LDS by
//    buffer loads of 16 bytes a lane.  A lane's row and piece are fixed for the whole call, so
//    a step's loads differ only in one scalar offset; a last step that passes the row's end
//    sends its lanes' offsets past the descriptor's range, which reads zeros.
//  * LDS rows are unpadded; piece c of row r lies at c ^ ((r >> 1) & 7) (64-byte rows:
//    c ^ ((r >> 2) & 3)), so a fragment read's 16 lanes fall on distinct banks.
//  * GLU: the weight rows of a tile alternate in blocks of 16 between gate and up, so a lane
//    holds both sums of its outputs and the tile writes only their combination.
//  * Output tiles are turned in LDS so that whole 128- or 256-byte row pieces are stored.
//  * Workgroups are remapped so that each XCD (own L2) runs a near-square block of tiles.
#include "i8_device.h"

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

// A stage: the weight rows (and positions) and the X rows of a step, arrays of their own (as one
// array, 8192 x 14336 x 4096 took 433 us instead of 389).
struct Stage {
  unsigned char *a, *b;
};

// K-loops over n >= 1 steps through NST stages (distinct static arrays, named by constant indices,
// so that the compiler tracks the requests into each one).  issue(st, s) requests step s into
// st, exactly L requests a wave.  Both end with every request landed and every stage free.

// Two stages of large steps: a step's requests go out before the step ahead of it is multiplied
// and are waited for after it.
template <typename Issue, typename Compute>
__device__ __forceinline__ void k_loop2(int n, Stage a, Stage b, Issue&& issue, Compute&& compute) {
  issue(a, 0);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  for (int s = 0; s < n; s += 2) {
    if (s + 1 < n) issue(b, s + 1);
    compute(a);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (s + 1 < n) {
      if (s + 2 < n) issue(a, s + 2);
      compute(b);
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
    }
  }
}

// Small steps: step q requests step q + NST - 1 into the stage that step q - 1 used, reads its
// operands, all at once, and multiplies; then one wait (step q + 1 has landed, the operands have
// arrived) and one barrier.
// Past the last step the last one is requested again; no one reads it.  (Reading operands a
// step ahead, during the products, measured 2-6% slower; six stages, which leave a CU one
// workgroup instead of two, 1-20% slower than four.)
template <int NST, int L, typename Frag, typename Issue, typename Read, typename Mma>
__device__ __forceinline__ void k_ring(int n, const Stage (&S)[4], Issue&& issue, Read&& read, Mma&& mma) {
  static_assert(NST >= 3 && NST <= 4 && L * (NST - 2) <= 63, "stages and requests per step");
  auto bar = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
#pragma unroll
  for (int j = 0; j + 1 < NST; ++j) issue(S[j], j < n ? j : n - 1);
  __builtin_amdgcn_s_waitcnt(vm_wait(L * (NST - 2)));
  bar();
  auto step = [&](int j, int q) {   // j = q % NST, a constant after unrolling
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

// Two fp32 values as packed bf16, to nearest even.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

// The output factors of a tile in LDS (requested before the K-loop: loaded after it they cost
// 4 us a tile): w_scale, then up_scale (GLU) or col_shift of BO outputs, past O the last one.
// Waves 0 .. 2 BO / 64 - 1 load 64 each (GLU tiles of 32 outputs: both halves of one load).
template <int BO, bool GLU, int NW>
__device__ __forceinline__ void load_factors(const I8Epi& epi, int64_t o0, int64_t O, int wave, int lane, float* sw) {
  static_assert(BO % 64 == 0 || (GLU && BO == 32), "a load of 64 factors is of one kind, or of two whole ones");
  const float* const second = GLU ? epi.up_scale : epi.col_shift;
#pragma unroll
  for (int q = 0; q < (2 * BO / 64 + NW - 1) / NW; ++q) {
    const int g = wave + q * NW, e = g * 64 + lane;   // factor e: kind e / BO of output e % BO
    if (g >= 2 * BO / 64 || (g * 64 >= BO && second == nullptr)) break;
    int64_t o = o0 + e % BO;
    o = o < O ? o : O - 1;
    __builtin_amdgcn_global_load_lds((e < BO ? epi.w_scale : second) + o, (lds_void*)(sw + g * 64), 4, 0, 0);
  }
}

// What a wave does with its finished sums: FI x FJ blocks of 16 x 16, lane (fr, fq) = (lane & 15,
// lane >> 4) holding rows 4 fq + [0, 4) of each block's row range for token fr.  ob_w, tb_w: the
// wave's first output and token; ow: that output in the tile.  With a split reduction the sums
// go to part, otherwise they are scaled.  TURN (256 x 256 tiles): each block column is turned
// through the wave's own 4 KiB of LDS at `mine` (a row of 64 outputs per token, 16-byte piece c
// of row r at c ^ r) and stored as whole row pieces, 128 bytes of bf16 or 256 of fp32.  Smaller
// tiles store a lane's four outputs at once.  Where rows of y do not keep that alignment, both
// turn (smaller tiles in 2 KiB) and neighbouring lanes store neighbouring outputs: stored one by
// one from where the sums lie, 4096 x 4095 x 2048 took 53 us instead of 34, 777 x 1025 x 2048 8.4
// instead of 7.8.
template <int FI, int FJ, bool GLU, bool TURN>
__device__ __forceinline__ void i8_finish(const i32x4 (&acc)[FI][FJ], const I8Epi& epi, int32_t* __restrict__ part,
                                          int kpart, int64_t T, int64_t O, int64_t ob_w, int64_t tb_w, int lane,
                                          unsigned char* mine, const float* sw, int BO, int ow) {
  const int fr = lane & 15, fq = lane >> 4;
  constexpr int NO = GLU ? FI / 2 : FI;         // output blocks of 16
  const int64_t ob0 = ob_w + 4 * fq, tb0 = tb_w + fr;
  if (part != nullptr) {
    const int64_t o4 = (O + 3) / 4 * 4;
#pragma unroll
    for (int i = 0; i < NO; ++i) {
      const int64_t ob = ob0 + 16 * i;
      if (ob >= O) continue;
#pragma unroll
      for (int j = 0; j < FJ; ++j) {
        const int64_t t = tb0 + 16 * j;
        if (t >= T) continue;
        int32_t* pp = part + ((int64_t)kpart * (GLU ? 2 : 1) * T + t) * o4 + ob;
        *reinterpret_cast<i32x4*>(pp) = acc[GLU ? 2 * i : i][j];
        if constexpr (GLU) *reinterpret_cast<i32x4*>(pp + T * o4) = acc[2 * i + 1][j];
      }
    }
    return;
  }
  // the tokens' factors first: a load per block column would stall each of them
  float xs[FJ], rb[FJ];
#pragma unroll
  for (int j = 0; j < FJ; ++j) {
    const int64_t t = tb0 + 16 * j < T ? tb0 + 16 * j : T - 1;
    xs[j] = epi.x_scale[t];
    rb[j] = !GLU && epi.row_shift != nullptr ? epi.row_shift[t] : 1.f;
  }
  const bool shifted = !GLU && epi.col_shift != nullptr;
  struct Scales {
    f32x4 w, e;   // w_scale, and up_scale (GLU) or col_shift
  };
  auto scales = [&](int i) {   // of the lane's four outputs in block i
    const float* at = sw + ow + 16 * i + 4 * fq;   // in the tile
    return Scales{*reinterpret_cast<const f32x4*>(at),
                  GLU || shifted ? *reinterpret_cast<const f32x4*>(at + BO) : f32x4{0.f, 0.f, 0.f, 0.f}};
  };
  auto values = [&](const Scales& sc, int i, int j) {
    f32x4 v;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int s0 = acc[GLU ? 2 * i : i][j][r], s1 = GLU ? acc[GLU ? 2 * i + 1 : i][j][r] : 0;
      if constexpr (GLU) v[r] = i8_gated(epi, s0, s1, xs[j], sc.w[r], sc.e[r]);
      else v[r] = i8_scaled(s0, xs[j], sc.w[r]);
    }
    if (shifted) {
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = i8_shifted(v[r], rb[j], sc.e[r]);
    }
    return v;
  };
  if constexpr (TURN) {
    static_assert(NO % 4 == 0, "rows of 64 outputs");
    if (epi.bf16_out) {
      const bool whole = epi.ldy % 8 == 0;
#pragma unroll
      for (int h = 0; h < NO / 4; ++h) {
        const int64_t oh = ob_w + 64 * h;
        Scales sc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[i] = scales(4 * h + i);
#pragma unroll
        for (int j = 0; j < FJ; ++j) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f32x4 v = values(sc[i], 4 * h + i, j);
            *reinterpret_cast<uint2*>(mine + fr * 128 + 16 * ((2 * i + (fq >> 1)) ^ (fr & 7)) + 8 * (fq & 1)) =
                make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
          }
          wave_lds_fence();
          if (!whole) {
            if (oh + lane < O) {
              uint16_t* yp = static_cast<uint16_t*>(epi.y) + (tb_w + 16 * j) * epi.ldy + oh + lane;
              const int rows = (int)(T - tb_w - 16 * j < 16 ? T - tb_w - 16 * j : 16);
#pragma unroll 8
              for (int r = 0; r < rows; ++r, yp += epi.ldy)
                *yp = *reinterpret_cast<const uint16_t*>(mine + r * 128 + 16 * ((lane >> 3) ^ (r & 7)) + 2 * (lane & 7));
            }
            wave_lds_fence();
            continue;
          }
          uint4 d[2];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const int row = 8 * p + (lane >> 3);
            d[p] = *reinterpret_cast<const uint4*>(mine + row * 128 + 16 * ((lane & 7) ^ (row & 7)));
          }
          wave_lds_fence();
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const int64_t t = tb_w + 16 * j + 8 * p + (lane >> 3), o = oh + 8 * (lane & 7);
            if (t >= T || o >= O) continue;
            uint16_t* yp = static_cast<uint16_t*>(epi.y) + t * epi.ldy + o;
            if (o + 8 <= O) {
              *reinterpret_cast<uint4*>(yp) = d[p];
            } else {
              const uint32_t e[4] = {d[p].x, d[p].y, d[p].z, d[p].w};
#pragma unroll
              for (int r = 0; r < 8; ++r)
                if (o + r < O) yp[r] = (uint16_t)(e[r >> 1] >> (16 * (r & 1)));
            }
          }
        }
      }
      return;
    }
    if (!epi.bf16_out) {
      const bool whole = epi.ldy % 4 == 0;
#pragma unroll
      for (int h = 0; h < NO / 4; ++h) {
        const int64_t oh = ob_w + 64 * h;
        Scales sc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[i] = scales(4 * h + i);
#pragma unroll
        for (int j = 0; j < FJ; ++j) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<f32x4*>(mine + fr * 256 + 16 * ((4 * i + fq) ^ fr)) = values(sc[i], 4 * h + i, j);
          wave_lds_fence();
          if (!whole) {
            if (oh + lane < O) {
              float* yp = static_cast<float*>(epi.y) + (tb_w + 16 * j) * epi.ldy + oh + lane;
              const int rows = (int)(T - tb_w - 16 * j < 16 ? T - tb_w - 16 * j : 16);
#pragma unroll 8
              for (int r = 0; r < rows; ++r, yp += epi.ldy) {
                const float e = *reinterpret_cast<const float*>(mine + r * 256 + 16 * ((lane >> 2) ^ r) + 4 * (lane & 3));
                *yp = epi.accumulate ? *yp + e : e;
              }
            }
            wave_lds_fence();
            continue;
          }
          f32x4 d[4];
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const int row = 4 * p + (lane >> 4);
            d[p] = *reinterpret_cast<const f32x4*>(mine + row * 256 + 16 * ((lane & 15) ^ (row & 15)));
          }
          wave_lds_fence();
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const int64_t t = tb_w + 16 * j + 4 * p + (lane >> 4), o = oh + 4 * (lane & 15);
            if (t >= T || o >= O) continue;
            float* yp = static_cast<float*>(epi.y) + t * epi.ldy + o;
            if (o + 4 <= O) {
              if (epi.accumulate) d[p] += *reinterpret_cast<const f32x4*>(yp);
              *reinterpret_cast<f32x4*>(yp) = d[p];
            } else {
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (o + r < O) yp[r] = epi.accumulate ? yp[r] + d[p][r] : d[p][r];
            }
          }
        }
      }
      return;
    }
  }
  if constexpr (!TURN) {
    if (epi.ldy % 4 == 0) {   // four outputs start on a multiple of their size
#pragma unroll
      for (int i = 0; i < NO; ++i) {
        const Scales sc = scales(i);
        const int64_t ob = ob0 + 16 * i;
        if (ob >= O) continue;
#pragma unroll
        for (int j = 0; j < FJ; ++j) {
          const int64_t t = tb0 + 16 * j;
          if (t >= T) continue;
          f32x4 v = values(sc, i, j);
          if (epi.bf16_out) {
            uint16_t* yp = static_cast<uint16_t*>(epi.y) + t * epi.ldy + ob;
            const uint2 d = make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
            if (ob + 4 <= O) {
              *reinterpret_cast<uint2*>(yp) = d;
            } else {
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (ob + r < O) yp[r] = (uint16_t)((r < 2 ? d.x : d.y) >> (16 * (r & 1)));
            }
          } else {
            float* yp = static_cast<float*>(epi.y) + t * epi.ldy + ob;
            if (ob + 4 <= O) {
              if (epi.accumulate) v += *reinterpret_cast<const f32x4*>(yp);
              *reinterpret_cast<f32x4*>(yp) = v;
            } else {
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (ob + r < O) yp[r] = epi.accumulate ? yp[r] + v[r] : v[r];
            }
          }
        }
      }
      return;
    }
    static_assert(NO <= 2, "2 KiB hold 16 tokens of 32 outputs");
    constexpr int W = 16 * NO;   // outputs of a row
    auto piece = [](int r, int c) { return r * (4 * W) + 16 * (NO == 2 ? swz8(r, c) : swz4(r, c)); };
    const int64_t o = ob_w + lane % W;
#pragma unroll
    for (int j = 0; j < FJ; ++j) {
#pragma unroll
      for (int i = 0; i < NO; ++i) *reinterpret_cast<f32x4*>(mine + piece(fr, 4 * i + fq)) = values(scales(i), i, j);
      wave_lds_fence();
      float e[W / 4];
#pragma unroll
      for (int p = 0; p < W / 4; ++p)
        e[p] = *reinterpret_cast<const float*>(mine + piece(64 / W * p + lane / W, lane % W / 4) + 4 * (lane & 3));
      wave_lds_fence();
#pragma unroll
      for (int p = 0; p < W / 4; ++p) {
        const int64_t t = tb_w + 16 * j + 64 / W * p + lane / W;
        if (t >= T || o >= O) continue;
        if (epi.bf16_out) {
          static_cast<uint16_t*>(epi.y)[t * epi.ldy + o] = (uint16_t)bf16x2(e[p], 0.f);
        } else {
          float* yp = static_cast<float*>(epi.y) + t * epi.ldy + o;
          *yp = epi.accumulate ? *yp + e[p] : e[p];
        }
      }
    }
  }
}

// BM x BN: weight rows by tokens of a tile (GLU: BM / 2 outputs); WM x WN waves; NST stages.
// Two stages of 256 x 256 (dense): bound by the matrix pipe under the card's power limit.  8192 x
// 14336 x 4096 379-405 us on different cards, 2.4-2.5 POPS; the products alone on the same codes
// take 281 us (on constant ones 238: the clock falls with the bits that change).  GLU 4096 x
// 14336 x 4096 383-395 us.
// Rings of smaller tiles (us; weights in the last-level cache / from HBM): with few tokens bound
// by the weights' stream (61 x 4096 x 14336 15.4 / 21.9 with its reduction, 2:4 16 x 14336 x 4096
// 8.9 / 11.6, 3.2 TB/s, GLU 8 x 14336 x 4096 24.4 / 27.1, 4.3 TB/s); in
// between by the latency of a step's requests (2:4 333 x 4096 over 128 positions 4.9, over 6144
// 17.2 / 23.5: 47 further steps of 0.26 / 0.40; dense 777 x 1025 over 16 4.7, over 1024 6.7, 2048
// 8.1, 1999 9.4: rows 2000 bytes apart share cache lines with their neighbours).
template <int BM, int BN, int WM, int WN, bool SP, bool GLU, int NST>
__global__ __launch_bounds__(64 * WM * WN) void k_i8_tile(
    const int8_t* __restrict__ x, int64_t ldx, const int8_t* __restrict__ w0, const int8_t* __restrict__ w1, int64_t ldw,
    const uint8_t* __restrict__ m0, const uint8_t* __restrict__ m1, int64_t T, int64_t O, int k, I8Epi epi,
    int32_t* __restrict__ part, int tiles_m, int tiles_n, int steps_per_split, int group) {
  constexpr int NW = WM * WN;
  constexpr int SM = BM / WM, SN = BN / WN, FI = SM / 16, FJ = SN / 16;
  constexpr int BO = GLU ? BM / 2 : BM;        // outputs of a tile
  constexpr int AROW = SP ? 64 : 128;          // weight bytes per row per step
  constexpr int RPG = SP ? 16 : 8;             // weight rows of one wave load (1 KiB)
  constexpr int V_BYTES = BM * AROW;
  constexpr int A_BYTES = V_BYTES + (SP ? BM * 16 : 0), B_BYTES = BN * 128;
  constexpr int NA = BM / RPG / NW, NB = BN / 8 / NW;
  static_assert(NA >= 1 && NB >= 1 && BM % (RPG * NW) == 0 && BN % (8 * NW) == 0, "load groups per wave");
  static_assert(!SP || BM == 16 * NW, "positions: 16 rows a wave, 4 bytes a lane");
  static_assert(!GLU || FI % 2 == 0, "GLU: gate and up blocks in one wave");
  constexpr int A2 = NST > 2 ? A_BYTES : 16, B2 = NST > 2 ? B_BYTES : 16, A3 = NST > 3 ? A_BYTES : 16, B3 = NST > 3 ? B_BYTES : 16;
  __shared__ __align__(16) unsigned char sA0[A_BYTES], sB0[B_BYTES], sA1[A_BYTES], sB1[B_BYTES], sA2[A2], sB2[B2], sA3[A3],
      sB3[B3];
  const Stage S[4] = {{sA0, sB0}, {sA1, sB1}, {sA2, sB2}, {sA3, sB3}};
  __shared__ __align__(16) float sw[2 * BO];
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
  const int64_t o0 = (int64_t)tile_m * BO, t0 = (int64_t)tile_n * BN;
  const int orows = (int)(O - o0 < BO ? O - o0 : BO), trows = (int)(T - t0 < BN ? T - t0 : BN);

  const int steps_all = (k + 127) / 128;
  const int sb = kpart * steps_per_split;
  const int n = min(steps_all - sb, steps_per_split);

  // descriptors of the tile's rows, and the lane's offset of each of its loads
  const __amdgpu_buffer_rsrc_t rx = rsrc_of(x + t0 * ldx, (uint32_t)(trows * ldx));
  const __amdgpu_buffer_rsrc_t rw0 = rsrc_of(w0 + o0 * ldw, (uint32_t)(orows * ldw));
  const __amdgpu_buffer_rsrc_t rw1 = GLU ? rsrc_of(w1 + o0 * ldw, (uint32_t)(orows * ldw)) : rw0;
  uint32_t aoff[NA], boff[NB];
  uint32_t atail, btail;   // added in the last step: kPast where the piece starts past the row
  {
    const int last = (steps_all - 1) * 128;
#pragma unroll
    for (int q = 0; q < NA; ++q) {
      const int r = (wave + q * NW) * RPG + lane / (AROW / 16);
      const int c = SP ? swz4(r, lane & 3) : swz8(r, lane & 7);
      int o = GLU ? (r >> 5) * 16 + (r & 15) : r;
      o = o < orows ? o : orows - 1;
      aoff[q] = (uint32_t)(o * (int)ldw + 16 * c);
      // one piece for every q: the rows of two loads differ by a multiple of 16, the swizzles' period
      if (q == 0) atail = (SP ? last / 2 + 16 * c >= k / 2 : last + 16 * c >= k) ? kPast : 0u;
    }
#pragma unroll
    for (int q = 0; q < NB; ++q) {
      const int r = (wave + q * NW) * 8 + (lane >> 3);
      const int c = swz8(r, lane & 7);
      const int t = r < trows ? r : trows - 1;
      boff[q] = (uint32_t)(t * (int)ldx + 16 * c);
      if (q == 0) btail = last + 16 * c >= k ? kPast : 0u;
    }
  }
  const uint8_t* mlane = nullptr;   // the lane's four bytes of positions in step block 0
  if constexpr (SP) {
    const int r = wave * 16 + (lane >> 2);
    int o = GLU ? (r >> 5) * 16 + (r & 15) : r;
    o = o < orows ? o : orows - 1;
    mlane = (GLU && (wave & 1) ? m1 : m0) + (o0 + o) * 16 + 4 * (lane & 3);
  }

  if (part == nullptr) load_factors<BO, GLU, NW>(epi, o0, O, wave, lane, sw);

  i32x4 acc[FI][FJ];
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int j = 0; j < FJ; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

  auto issue = [&](Stage st, int si) {
    unsigned char *const a = st.a, *const b = st.b;
    const int s = sb + si;
    const uint32_t at = s == steps_all - 1 ? atail : 0u, bt = s == steps_all - 1 ? btail : 0u;
#pragma unroll
    for (int q = 0; q < NA; ++q) {
      const int grp = wave + q * NW;
      const bool second = GLU && ((SP ? grp : grp >> 1) & 1);
      b2lds16(second ? rw1 : rw0, a + grp * 1024, aoff[q] + at, (uint32_t)(s * AROW));
    }
    if constexpr (SP)
      __builtin_amdgcn_global_load_lds(mlane + (int64_t)s * O * 16, (lds_void*)(a + V_BYTES + wave * 256), 4, 0, 0);
#pragma unroll
    for (int q = 0; q < NB; ++q) b2lds16(rx, b + (wave + q * NW) * 1024, boff[q] + bt, (uint32_t)(s * 128));
  };

  auto read_b = [&](const unsigned char* b, int ks, int j) {
    const int r = wni * SN + j * 16 + fr;
    return *reinterpret_cast<const i32x4*>(b + r * 128 + 16 * swz8(r, 4 * ks + fq));
  };
  // 256-row tiles (dense): an A fragment a row block ahead, the second half's B fragments during
  // the first
  auto compute = [&](Stage st) {
    const unsigned char *const a = st.a, *const b = st.b;
    auto read_a = [&](int ks, int i) {
      const int r = wmi * SM + i * 16 + fr;
      return *reinterpret_cast<const i32x4*>(a + r * 128 + 16 * swz8(r, 4 * ks + fq));
    };
    i32x4 b0[FJ], b1[FJ];
#pragma unroll
    for (int j = 0; j < FJ; ++j) b0[j] = read_b(b, 0, j);
    i32x4 acur = read_a(0, 0), anxt;
    constexpr int BPS = (FJ + FI - 1) / FI;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
      for (int i = 0; i < FI; ++i) {
        __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
        __builtin_amdgcn_sched_barrier(0);
        if (i + 1 < FI) anxt = read_a(ks, i + 1);
        else if (ks == 0) anxt = read_a(1, 0);
        if (ks == 0) {
#pragma unroll
          for (int q = 0; q < BPS; ++q)
            if (i * BPS + q < FJ) b1[i * BPS + q] = read_b(b, 1, i * BPS + q);
        }
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int j = 0; j < FJ; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(acur, ks ? b1[j] : b0[j], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
        acur = anxt;
      }
    }
  };
  // smaller tiles: the operands of a whole step at once (k_ring)
  constexpr int KS = SP ? 1 : 2;
  struct Frag {
    i32x4 a[KS][FI], b0[FJ], b1[FJ];
    int idx[SP ? FI : 1];
  };
  auto read = [&](Frag& f, Stage st) {
    const unsigned char *const a = st.a, *const b = st.b;
#pragma unroll
    for (int i = 0; i < FI; ++i) {
      const int r = wmi * SM + i * 16 + fr;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
        f.a[ks][i] = *reinterpret_cast<const i32x4*>(a + r * AROW + 16 * (SP ? swz4(r, fq) : swz8(r, 4 * ks + fq)));
      if constexpr (SP) f.idx[i] = *reinterpret_cast<const int*>(a + V_BYTES + r * 16 + 4 * fq);
    }
#pragma unroll
    for (int j = 0; j < FJ; ++j) {
      f.b0[j] = read_b(b, 0, j);
      f.b1[j] = read_b(b, 1, j);
    }
  };
  auto mma = [&](const Frag& f) {
#pragma unroll
    for (int j = 0; j < FJ; ++j)
#pragma unroll
      for (int i = 0; i < FI; ++i) {
        if constexpr (SP) {
          const i32x8 bv = __builtin_shufflevector(f.b0[j], f.b1[j], 0, 1, 2, 3, 4, 5, 6, 7);
          acc[i][j] = __builtin_amdgcn_smfmac_i32_16x16x128_i8(f.a[0][i], bv, acc[i][j], f.idx[i], 0, 0);
        } else {
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.a[0][i], f.b0[j], acc[i][j], 0, 0, 0);
        }
      }
    if constexpr (!SP) {
#pragma unroll
      for (int j = 0; j < FJ; ++j)
#pragma unroll
        for (int i = 0; i < FI; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.a[KS - 1][i], f.b1[j], acc[i][j], 0, 0, 0);
    }
  };
  if (n > 0) {
    if constexpr (NST == 2) {
      static_assert(!SP, "2:4 products of this size: k_i8_big");
      k_loop2(n, S[0], S[1], issue, compute);
    } else {
      k_ring<NST, NA + NB + (SP ? 1 : 0), Frag>(n, S, issue, read, mma);
    }
  }

  constexpr bool TURN = NST == 2;
  static_assert(TURN ? B_BYTES >= NW * 4096 : A_BYTES >= NW / 2 * 2048, "LDS of a wave to turn in");
  unsigned char* const mine = TURN ? sB0 + wave * 4096 : (wave < NW / 2 ? sA0 : sA1) + wave % (NW / 2) * 2048;
  const int ow = GLU ? wmi * SM / 2 : wmi * SM;
  i8_finish<FI, FJ, GLU, TURN>(acc, epi, part, kpart, T, O, o0 + ow, t0 + wni * SN, lane, mine, sw, BO, ow);
}

// ----------------------------------------------------------- the large 2:4 products ---

// acc += a b on the accumulator half of the register file.  Written out because the compiler,
// with all 256 registers of that half taken by sums, moved or spilled a hundred of them per
// step (658 us against 277 at 8192 x 4096 x 14336).  It does not see this as a matrix
// instruction, so the waits it would insert are here: s_nop 1 ahead (an operand just written
// by a vector instruction), mma_done() before the sums are read.
__device__ __forceinline__ void smma_acc(i32x16& c, i32x4 a, i32x8 b, int idx) {
  asm volatile("s_nop 1\n\tv_smfmac_i32_32x32x64_i8 %0, %1, %2, %3" : "+a"(c) : "v"(a), "v"(b), "v"(idx));
}
template <int N>
__device__ __forceinline__ void mma_done(i32x16 (&acc)[N][N]) {
  asm volatile("s_nop 15\n\ts_nop 15");
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) asm volatile("" : "+a"(acc[i][j]));
}
// one sum, read when it is used (read together they would need 256 more registers)
__device__ __forceinline__ int acc_read(int a) {
  int v;
  asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a));
  return v;
}

// The finished sums of a wave's 4 x 4 blocks of 32 x 32: lane (c, h) = (lane & 31, lane >> 5)
// holds, in register v, row 8 (v / 4) + 4 h + v % 4 of token c.  GLU: the rows of a block are 16
// gate rows and the 16 up rows of the same outputs, registers v and v + 8.  As i8_finish: rows
// of 64 outputs and 32 tokens are turned in the wave's own 8 KiB of LDS and stored whole.
// WHOLE: rows of y keep the alignment (a form of its own: as one, the registers of the other cost
// aligned outputs 2 us of 28 at 4096 x 4096 x 2048); otherwise neighbouring lanes store
// neighbouring outputs.
template <bool GLU, bool WHOLE>
__device__ __forceinline__ void i8_finish_big(const i32x16 (&acc)[4][4], const I8Epi& epi, int64_t T, int64_t O,
                                              int64_t ob_w, int64_t tb_w, int lane, unsigned char* mine,
                                              const float* sw, int ow) {
  const int c = lane & 31, h = lane >> 5;
  constexpr int BO = GLU ? 128 : 256;
  constexpr int NB = GLU ? 4 : 2;      // blocks of 64 outputs
  constexpr int NG = GLU ? 2 : 4;      // groups of 4 outputs of a lane per block: outputs 8 g + 4 h + [0, 4)
  constexpr int NH = GLU ? 1 : 2;      // 64-output parts of the wave
  const bool shifted = !GLU && epi.col_shift != nullptr;
  float xs[4], rb[4];                  // the tokens' factors first: a load per block would stall each
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t t = tb_w + 32 * j + c < T ? tb_w + 32 * j + c : T - 1;
    xs[j] = epi.x_scale[t];
    rb[j] = !GLU && epi.row_shift != nullptr ? epi.row_shift[t] : 1.f;
  }
#pragma unroll
  for (int hh = 0; hh < NH; ++hh) {
    const int64_t oh = ob_w + 64 * hh;
    f32x4 ws[NB][NG], es[NB][NG];   // w_scale, and up_scale (GLU) or col_shift
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float* at = sw + ow + 64 * hh + (GLU ? 16 : 32) * b + 8 * g + 4 * h;
        ws[b][g] = *reinterpret_cast<const f32x4*>(at);
        es[b][g] = GLU || shifted ? *reinterpret_cast<const f32x4*>(at + BO) : f32x4{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[NB][NG][4];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const i32x16& blk = acc[GLU ? b : 2 * hh + b][j];
            const int s0 = acc_read(blk[4 * g + r]);
            if constexpr (GLU) {
              const int s1 = acc_read(blk[8 + 4 * g + r]);
              v[b][g][r] = i8_gated(epi, s0, s1, xs[j], ws[b][g][r], es[b][g][r]);
            } else {
              v[b][g][r] = i8_scaled(s0, xs[j], ws[b][g][r]);
            }
          }
      if (shifted) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int r = 0; r < 4; ++r) v[b][g][r] = i8_shifted(v[b][g][r], rb[j], es[b][g][r]);
      }
      const int64_t tj = tb_w + 32 * j;
      if (epi.bf16_out) {
        // rows of 128 bytes: 8-byte halves of piece p of token c at p ^ ((c >> 1) & 7)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const int p = (GLU ? 2 : 4) * b + g;
            *reinterpret_cast<uint2*>(mine + c * 128 + 16 * (p ^ ((c >> 1) & 7)) + 8 * h) =
                make_uint2(bf16x2(v[b][g][0], v[b][g][1]), bf16x2(v[b][g][2], v[b][g][3]));
          }
        wave_lds_fence();
        if constexpr (!WHOLE) {
          if (oh + lane < O) {
            uint16_t* yp = static_cast<uint16_t*>(epi.y) + tj * epi.ldy + oh + lane;
            const int rows = (int)(T - tj < 32 ? T - tj : 32);
#pragma unroll 8
            for (int r = 0; r < rows; ++r, yp += epi.ldy)
              *yp = *reinterpret_cast<const uint16_t*>(mine + r * 128 + 16 * ((lane >> 3) ^ ((r >> 1) & 7)) + 2 * (lane & 7));
          }
          wave_lds_fence();
          continue;
        }
        uint4 d[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int row = 8 * p + (lane >> 3);
          d[p] = *reinterpret_cast<const uint4*>(mine + row * 128 + 16 * ((lane & 7) ^ ((row >> 1) & 7)));
        }
        wave_lds_fence();
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int64_t t = tj + 8 * p + (lane >> 3), o = oh + 8 * (lane & 7);
          if (t >= T || o >= O) continue;
          uint16_t* yp = static_cast<uint16_t*>(epi.y) + t * epi.ldy + o;
          if (o + 8 <= O) {
            *reinterpret_cast<uint4*>(yp) = d[p];
          } else {
            const uint32_t e[4] = {d[p].x, d[p].y, d[p].z, d[p].w};
#pragma unroll
            for (int r = 0; r < 8; ++r)
              if (o + r < O) yp[r] = (uint16_t)(e[r >> 1] >> (16 * (r & 1)));
          }
        }
      } else {
        // rows of 256 bytes: piece p of token c at p ^ (c & 15)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const int p = (GLU ? 4 : 8) * b + 2 * g + h;
            *reinterpret_cast<f32x4*>(mine + c * 256 + 16 * (p ^ (c & 15))) =
                f32x4{v[b][g][0], v[b][g][1], v[b][g][2], v[b][g][3]};
          }
        wave_lds_fence();
        if constexpr (!WHOLE) {
          if (oh + lane < O) {
            float* yp = static_cast<float*>(epi.y) + tj * epi.ldy + oh + lane;
            const int rows = (int)(T - tj < 32 ? T - tj : 32);
#pragma unroll 8
            for (int r = 0; r < rows; ++r, yp += epi.ldy) {
              const float e = *reinterpret_cast<const float*>(mine + r * 256 + 16 * ((lane >> 2) ^ (r & 15)) + 4 * (lane & 3));
              *yp = epi.accumulate ? *yp + e : e;
            }
          }
          wave_lds_fence();
          continue;
        }
        f32x4 d[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const int row = 4 * p + (lane >> 4);
          d[p] = *reinterpret_cast<const f32x4*>(mine + row * 256 + 16 * ((lane & 15) ^ (row & 15)));
        }
        wave_lds_fence();
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const int64_t t = tj + 4 * p + (lane >> 4), o = oh + 4 * (lane & 15);
          if (t >= T || o >= O) continue;
          float* yp = static_cast<float*>(epi.y) + t * epi.ldy + o;
          if (o + 4 <= O) {
            if (epi.accumulate) d[p] += *reinterpret_cast<const f32x4*>(yp);
            *reinterpret_cast<f32x4*>(yp) = d[p];
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (o + r < O) yp[r] = epi.accumulate ? yp[r] + d[p][r] : d[p][r];
          }
        }
      }
    }
  }
}

// 256 x 256 tiles of 2:4 products by 4 waves of 128 x 128 (one per SIMD, 256 sums a lane).  A wave
// reads 256 rows of LDS for 128 x 128 outputs, so LDS, which bounds the 8-wave form (twice the
// matrix rate of dense products on the same X bytes), moves three quarters as much: 8192 x
// 4096 x 14336 311 -> 271 us, GLU 4096 x 14336 x 4096 313 -> 303 us.  (Dense products gain
// nothing: 384 us with 8 waves, 394-417 with 4.)  Nothing but the wave itself hides a latency,
// so operands are read two phases of 16 matrix instructions ahead, a read or a request
// between two of them:
//  * v_smfmac_i32_32x32x64_i8: lane (c, h) = (lane & 31, lane >> 5) holds the 16 kept codes of
//    row c at positions [32 h, + 32) of a 64-position phase with their 32 bits of positions,
//    and of X the bytes [16 h, + 16) and [32 + 16 h, + 16).
//  * A step of 128 positions is two phases; 3 stages of 52 KiB.  When a step begins, its operands
//    are in registers and the next step's have landed: one wait, one barrier, and the stage
//    takes the requests of the step after the next two.
// What bounds it: with no requests and real data 211 us (the matrix pipe alone 165 us: power
// holds its clock down, the same loop on constant operands takes 132), the requests' LDS
// writes and L2 latency 60 us, epilogue 30 us.  LDS itself is not full: reading the positions
// without their two-way bank conflicts (29% of its active cycles) changes nothing.
template <bool GLU>
__global__ __launch_bounds__(256) void k_i8_big(
    const int8_t* __restrict__ x, int64_t ldx, const int8_t* __restrict__ w0, const int8_t* __restrict__ w1, int64_t ldw,
    const uint8_t* __restrict__ m0, const uint8_t* __restrict__ m1, int64_t T, int64_t O, int k, I8Epi epi, int tiles_m,
    int tiles_n, int group) {
  constexpr int BM = 256, BN = 256, NW = 4;
  constexpr int BO = GLU ? BM / 2 : BM;
  constexpr int V_BYTES = BM * 64, A_BYTES = V_BYTES + BM * 16, B_BYTES = BN * 128;   // codes, positions; X
  constexpr int NA = BM / 16 / NW, NB = BN / 8 / NW, NL = NA + NB + 1;   // loads of a wave per step
  __shared__ __align__(16) unsigned char s0[A_BYTES + B_BYTES], s1[A_BYTES + B_BYTES], s2[A_BYTES + B_BYTES];
  __shared__ __align__(16) float sw[2 * BO];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wmi = wave & 1, wni = wave >> 1;
  const int c = lane & 31, h = lane >> 5;

  const int ntiles = tiles_m * tiles_n;
  int lin = blockIdx.x;
  if ((ntiles & 7) == 0) lin = (blockIdx.x & 7) * (ntiles >> 3) + (blockIdx.x >> 3);
  const int band = lin / (group * tiles_n);
  const int band_w = min(group, tiles_m - band * group);
  const int inband = lin - band * group * tiles_n;
  // wave-uniform (the division leaves them in vector registers; descriptors need scalars)
  const int tile_m = __builtin_amdgcn_readfirstlane(band * group + inband % band_w);
  const int tile_n = __builtin_amdgcn_readfirstlane(inband / band_w);
  const int64_t o0 = (int64_t)tile_m * BO, t0 = (int64_t)tile_n * BN;
  const int orows = (int)(O - o0 < BO ? O - o0 : BO), trows = (int)(T - t0 < BN ? T - t0 : BN);
  const int n = (k + 127) / 128;   // steps, >= 1

  // descriptors and offsets as in k_i8_tile; a wave's weight loads are all of one matrix
  const bool up = GLU && (wave & 1);
  const __amdgpu_buffer_rsrc_t rx = rsrc_of(x + t0 * ldx, (uint32_t)(trows * ldx));
  const __amdgpu_buffer_rsrc_t rw = rsrc_of((up ? w1 : w0) + o0 * ldw, (uint32_t)(orows * ldw));
  uint32_t aoff[NA], boff[NB];
  uint32_t amask = 0, bmask = 0;   // kPast where the lane's piece of the last step starts past the row
  const int last = (n - 1) * 128;
#pragma unroll
  for (int q = 0; q < NA; ++q) {
    const int r = (wave + q * NW) * 16 + (lane >> 2);
    const int p = swz4(r, lane & 3);
    int o = GLU ? (r >> 5) * 16 + (r & 15) : r;
    o = o < orows ? o : orows - 1;
    aoff[q] = (uint32_t)(o * (int)ldw + 16 * p);
    if (q == 0) amask = last / 2 + 16 * p >= k / 2 ? kPast : 0u;
  }
#pragma unroll
  for (int q = 0; q < NB; ++q) {
    const int r = (wave + q * NW) * 8 + (lane >> 3);
    const int p = swz8(r, lane & 7);
    const int t = r < trows ? r : trows - 1;
    boff[q] = (uint32_t)(t * (int)ldx + 16 * p);
    if (q == 0) bmask = last + 16 * p >= k ? kPast : 0u;
  }
  const uint8_t* mlane;   // the lane's positions in step block 0
  const int64_t mstep = O * 16;
  {
    const int r = wave * 64 + lane;
    int o = GLU ? (r >> 5) * 16 + (r & 15) : r;
    o = o < orows ? o : orows - 1;
    mlane = (GLU && ((lane >> 4) & 1) ? m1 : m0) + (o0 + o) * 16;
  }
  int ls = 0;   // the step being requested; past the last one the last again (no one reads it)
  auto begin_loads = [&](int s) {
    ls = s < n ? s : n - 1;
    const uint32_t am = ls == n - 1 ? amask : 0u, bm = ls == n - 1 ? bmask : 0u;
#pragma unroll
    for (int q = 0; q < NA; ++q) aoff[q] |= am;
#pragma unroll
    for (int q = 0; q < NB; ++q) boff[q] |= bm;
  };
  auto load = [&](unsigned char* st, int q) {   // load q of step ls into stage st
    if (q < NA) {
      b2lds16(rw, st + (wave + q * NW) * 1024, aoff[q], (uint32_t)(ls * 64));
    } else if (q < NA + NB) {
      const int p = q - NA;
      b2lds16(rx, st + A_BYTES + (wave + p * NW) * 1024, boff[p], (uint32_t)(ls * 128));
    } else {
      __builtin_amdgcn_global_load_lds(mlane + ls * mstep, (lds_void*)(st + V_BYTES + wave * 1024), 16, 0, 0);
    }
  };
  auto bar = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  auto lds4 = [](const unsigned char* p) { return *reinterpret_cast<const i32x4*>(p); };
  // fragment addresses: rows 32 i + c of the wave's 128, whose swizzle does not depend on i
  const int ab = (wmi * 128 + c) * 64, bb = A_BYTES + (wni * 128 + c) * 128;
  const int ms = V_BYTES + (wmi * 128 + c) * 16 + 4 * h;
  int apos[2], bpos[4];   // pieces 2 e + h of a weight row, of a token row
#pragma unroll
  for (int e = 0; e < 2; ++e) apos[e] = ab + 16 * swz4(c, 2 * e + h);
#pragma unroll
  for (int e = 0; e < 4; ++e) bpos[e] = bb + 16 * swz8(c, 2 * e + h);

  load_factors<BO, GLU, NW>(epi, o0, O, wave, lane, sw);

  i32x16 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = i32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};

  struct Frag {
    i32x4 a[4];
    i32x8 b[4];
    int idx[4];
  };
  auto read = [&](Frag& f, const unsigned char* st, int ks, int e) {   // read e of 12 (two for X)
    if (e < 4) f.a[e] = lds4(st + apos[ks] + e * 2048);
    else if (e < 8) f.idx[e - 4] = *reinterpret_cast<const int*>(st + ms + 8 * ks + (e - 4) * 512);
    else f.b[e - 8] = __builtin_shufflevector(lds4(st + bpos[2 * ks] + (e - 8) * 4096),
                                              lds4(st + bpos[2 * ks + 1] + (e - 8) * 4096), 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto phase = [&](const Frag& f, Frag& fn, const unsigned char* rd, int ks, bool LOAD, unsigned char* wr) {
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
#pragma unroll
  for (int e = 0; e < 12; ++e) read(f0, s0, 0, e);
#pragma unroll
  for (int e = 0; e < 12; ++e) read(f1, s0, 1, e);
  // step s of (fa, fb): its operands are all read by now, so its stage takes the loads of
  // step s + 3 while those of step s + 1 come from nxt: (fc, fa)
  auto step = [&](Frag& fa, Frag& fb, Frag& fc, unsigned char* cur, unsigned char* nxt, int s) {
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0 & vm_wait(NL));   // step s + 1 landed; reads of step s arrived
    bar();
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
  const int ow = GLU ? wmi * 64 : wmi * 128;
  if (epi.bf16_out ? epi.ldy % 8 == 0 : epi.ldy % 4 == 0)
    i8_finish_big<GLU, true>(acc, epi, T, O, o0 + ow, t0 + wni * 128, lane, s0 + wave * 8192, sw, ow);
  else
    i8_finish_big<GLU, false>(acc, epi, T, O, o0 + ow, t0 + wni * 128, lane, s0 + wave * 8192, sw, ow);
}

template <int BM, int BN, int WM, int WN, bool SP, bool GLU, int NST>
hipError_t launch_cfg(const I8Args& a, int64_t splits, int32_t* part, hipStream_t s) {
  constexpr int BO = GLU ? BM / 2 : BM;
  const int64_t tm = (a.o + BO - 1) / BO, tn = (a.t + BN - 1) / BN, ntiles = tm * tn;
  if (tm > 0x7FFFFFFF || tn > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  const int64_t steps = (a.k + 127) / 128;
  if (splits < 1 || part == nullptr) splits = 1;
  const int64_t per = steps > 0 ? (steps + splits - 1) / splits : 1;
  splits = steps > 0 ? (steps + per - 1) / per : 1;
  if (ntiles * splits > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  // o-tiles per band of the tile order: an XCD runs 32 tiles at a time
  const int64_t group = tm < 8 ? tm : 8;
  k_i8_tile<BM, BN, WM, WN, SP, GLU, NST><<<dim3((unsigned)(ntiles * splits)), dim3(64 * WM * WN), 0, s>>>(
      a.x, a.ldx, a.w, a.w_up, a.ldw, a.meta, a.up_meta, a.t, a.o, (int)a.k, a.epi, splits > 1 ? part : nullptr, (int)tm,
      (int)tn, (int)per, (int)group);
  a.route.note(NM_TAKEN_TILE_LDS | (SP ? NM_TAKEN_SPARSE_MMA : 0u) | (splits > 1 ? NM_TAKEN_TILE_SPLIT : 0u));
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  return launch_i8_reduce(part, splits, GLU, a.t, a.o, a.epi, a.route, s);
}

template <bool SP, bool GLU>
hipError_t launch_kind(const I8Args& a, int shape, int64_t splits, int32_t* part, hipStream_t s) {
  if (shape < 0) {
    if constexpr (SP) {
      constexpr int BO = GLU ? 128 : 256;
      const int64_t tm = (a.o + BO - 1) / BO, tn = (a.t + 255) / 256;
      if (tm > 0x7FFFFFFF || tn > 0x7FFFFFFF || tm * tn > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
      k_i8_big<GLU><<<dim3((unsigned)(tm * tn)), dim3(256), 0, s>>>(
          a.x, a.ldx, a.w, a.w_up, a.ldw, a.meta, a.up_meta, a.t, a.o, (int)a.k, a.epi, (int)tm, (int)tn,
          (int)(tm < 8 ? tm : 8));
      a.route.note(NM_TAKEN_TILE_LDS | NM_TAKEN_SPARSE_MMA);
      return hipGetLastError();
    } else if constexpr (GLU) {
      return launch_cfg<256, 256, 2, 4, false, true, 2>(a, 1, nullptr, s);
    } else {
      return launch_cfg<256, 256, 4, 2, false, false, 2>(a, 1, nullptr, s);
    }
  }
  switch (shape) {
    case 0: return launch_cfg<128, 128, 4, 2, SP, GLU, 3>(a, splits, part, s);
    case 1: return launch_cfg<128, 64, 4, 2, SP, GLU, 4>(a, splits, part, s);
    case 2: return launch_cfg<64, 64, 2, 2, SP, GLU, 4>(a, splits, part, s);
  }
  return launch_cfg<64, 32, 2, 2, SP, GLU, 4>(a, splits, part, s);
}

struct MidPlan {
  int shape;        // 128 x 128, 128 x 64, 64 x 64, 64 x 32 (weight rows x tokens)
  int64_t splits;
};

// The largest tile that gives 192 workgroups (of 128 tokens only above 64); with none, the
// smallest, a reduction of over 32 steps cut in ranges of at least 16 up to one workgroup per
// CU.  A split costs the partial sums and a second kernel, 3-5 us against 0.13-0.15 us for each step
// of a short list of tiles (100 x 500 x 2048 unsplit 5.0, in 8 ranges 7.7; x 8192 12.3 unsplit, 7.8 in
// 4, 8.4 in 8; 40 x 256 x 14336 17.4 unsplit, 8.4 in 7, 9.3 in 14, 12.5 in 32), so it is the last
// choice, except that 64 x 32 tiles pay for each step however little it holds: over 64 steps, 64 x
// 64 tiles in two ranges (weights from HBM, us, in two ranges / 64 x 32 unsplit: 128 x 4096 x 8320
// 17.7 / 19.1, x 10240 21.1 / 23.8, x 14336 25.3 / 31.2, 100 x 4100 x 8320 19.9 / 19.8, x 14336 28.4 /
// 31.6, 64 x 6400 x 8320 18.9 / 20.4, 2:4 128 x 4096 x 8320 16.7 / 17.6, x 14336 23.3 / 27.5, GLU 40 x
// 4096 x 8320 18.8 / 20.0, x 14336 27.7 / 32.5).  Measured with weights in the last-level cache (us;
// 128 x 128 / 128 x 64 / 64 x 64 / 64 x 32, split to fill the chip): dense 61 x 4096 x 14336 18.6 /
// 17.8 / 15.9 / 15.3, 777 x 1025 x 1999 16.8 / 13.9 / 9.5 / 10.3, 128 x 4096 x 4096 17.8 / 13.5 / 11.0 /
// 8.5, 512 x 4096 x 4096 19.1 / 13.4 / 15.6 / 20.1, 2048^3 13.1 / 15.9 / 17.4 / 21.4; 2:4 333 x 4096 x
// 6144 19.4 / 16.8 / 19.6 / 20.6, 128 x 4096 x 14336 20.2 / 16.7 / 16.9 / 19.4, 1024 x 4096 x 4096
// 18.2 / 21.8 / 25.9 / 33.2; GLU 64 x 14336 x 4096 26.4 / 25.5 / 29.1 / 33.7, 2:4 17.2 / 15.8 / 16.2 /
// 20.1.
MidPlan mid_plan(int64_t t, int64_t o, int64_t k, bool glu) {
  const int64_t steps = (k + 127) / 128;
  const int bm[4] = {128, 128, 64, 64}, bn[4] = {128, 64, 64, 32};
  auto tiles = [&](int sh) {
    const int64_t bo = glu ? bm[sh] / 2 : bm[sh];
    return ((o + bo - 1) / bo) * ((t + bn[sh] - 1) / bn[sh]);
  };
  MidPlan p{3, 1};
  if (t > 32) {
    for (int sh = t > 64 ? 0 : 1; sh < 4; ++sh) {
      if (tiles(sh) < 192) continue;
      if (sh == 3 && steps > 64) return {2, 2};
      return {sh, 1};
    }
  }
  p.splits = tiles(3) > 0 ? 256 / tiles(3) : 1;
  if (p.splits > steps / 16) p.splits = steps / 16;
  if (steps <= 32 || p.splits < 1) p.splits = 1;
  return p;
}

}  // namespace

namespace nml {

bool i8_tile_eligible(const I8Args& a) {
  // descriptors hold 256 rows in under 2^31 bytes
  return a.k > 0 && a.ldx < (1 << 23) && a.ldw < (1 << 23);
}

int64_t i8_mid_part_bytes(int64_t t, int64_t o, int64_t k, bool glu) {
  const int64_t s = mid_plan(t, o, k, glu).splits;
  return s > 1 ? s * (glu ? 2 : 1) * t * ((o + 3) / 4 * 4) * 4 : 0;
}

hipError_t launch_i8_tile(const I8Args& a, bool large, int32_t* part, int64_t part_bytes, hipStream_t s) {
  const bool sp = a.meta != nullptr, glu = a.glu != 0;
  MidPlan p{-1, 1};   // 256 x 256 tiles
  if (!large) {
    p = mid_plan(a.t, a.o, a.k, glu);
    if (part == nullptr || part_bytes < i8_mid_part_bytes(a.t, a.o, a.k, glu)) p.splits = 1;
  }
  if (sp && glu) return launch_kind<true, true>(a, p.shape, p.splits, part, s);
  if (sp) return launch_kind<true, false>(a, p.shape, p.splits, part, s);
  if (glu) return launch_kind<false, true>(a, p.shape, p.splits, part, s);
  return launch_kind<false, false>(a, p.shape, p.splits, part, s);
}

}  // namespace nml
