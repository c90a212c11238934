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

// The two-stage K-loop: each step issues the next step's loads, multiplies, then waits for all
// loads and synchronises.
template <typename Issue, typename Compute>
__device__ __forceinline__ void k_loop2(int n, unsigned char* a0, unsigned char* b0, unsigned char* a1, unsigned char* b1,
                                        Issue&& issue, Compute&& compute) {
  issue(a0, b0, 0);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  for (int s = 0; s < n; s += 2) {
    if (s + 1 < n) issue(a1, b1, s + 1);
    compute(a0, b0);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (s + 1 < n) {
      if (s + 2 < n) issue(a0, b0, s + 2);
      compute(a1, b1);
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
    }
  }
}

// BM x BN: weight rows by tokens of a tile (GLU: BM / 2 outputs); WM x WN waves; NST stages.
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
  constexpr int NMW = SP ? BM / 64 : 0;        // waves that load positions (64 rows each)
  static_assert(NA >= 1 && NB >= 1 && BM % (RPG * NW) == 0 && BN % (8 * NW) == 0 && NMW <= NW, "load groups per wave");
  static_assert(!GLU || FI % 2 == 0, "GLU: gate and up blocks in one wave");
  constexpr int A2 = NST >= 3 ? A_BYTES : 16, B2 = NST >= 3 ? B_BYTES : 16;
  __shared__ __align__(16) unsigned char sA0[A_BYTES], sB0[B_BYTES];
  __shared__ __align__(16) unsigned char sA1[A_BYTES], sB1[B_BYTES];
  __shared__ __align__(16) unsigned char sA2[A2], sB2[B2];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wmi = wave % WM, wni = wave / WM;
  const int fr = lane & 15, fq = lane >> 4;

  const int ntiles = tiles_m * tiles_n;
  const int kpart = blockIdx.x / ntiles;
  int lin = blockIdx.x - kpart * ntiles;
  if ((ntiles & 7) == 0 && gridDim.x == (unsigned)ntiles) lin = (blockIdx.x & 7) * (ntiles >> 3) + (blockIdx.x >> 3);
  const int band = lin / (group * tiles_n);
  const int band_w = min(group, tiles_m - band * group);
  const int inband = lin - band * group * tiles_n;
  const int tile_m = band * group + inband % band_w, tile_n = inband / band_w;
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
      // the piece is the same for every q: the rows of two loads differ by a multiple of 16 (2:4)
      // or, at 8 waves, 64, and at 4 waves, 32 rows
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
  uint32_t moff = 0;
  const uint8_t* mbase = nullptr;   // positions of the tile's rows in step block 0
  if constexpr (SP) {
    const int r = (wave < NMW ? wave : 0) * 64 + lane;
    int o = GLU ? (r >> 5) * 16 + (r & 15) : r;
    o = o < orows ? o : orows - 1;
    moff = (uint32_t)(o * 16);
    mbase = m0 + o0 * 16;
  }

  i32x4 acc[FI][FJ];
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int j = 0; j < FJ; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

  auto issue = [&](unsigned char* a, unsigned char* b, int si) {
    const int s = sb + si;
    const uint32_t at = s == steps_all - 1 ? atail : 0u, bt = s == steps_all - 1 ? btail : 0u;
#pragma unroll
    for (int q = 0; q < NA; ++q) {
      const int grp = wave + q * NW;
      const bool second = GLU && ((SP ? grp : grp >> 1) & 1);
      b2lds16(second ? rw1 : rw0, a + grp * 1024, aoff[q] + at, (uint32_t)(s * AROW));
    }
    if constexpr (SP) {
      if (wave < NMW) {
        const uint8_t* mp = mbase + (int64_t)s * O * 16;
        if constexpr (GLU) {
          // rows alternate between the two weights in blocks of 16: a pointer per lane
          const uint8_t* up = m1 + o0 * 16 + (int64_t)s * O * 16;
          const uint8_t* src = ((lane >> 4) & 1 ? up : mp) + moff;
          __builtin_amdgcn_global_load_lds(src, (lds_void*)(a + V_BYTES + wave * 1024), 16, 0, 0);
        } else {
          __builtin_amdgcn_global_load_lds(mp + moff, (lds_void*)(a + V_BYTES + wave * 1024), 16, 0, 0);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < NB; ++q) b2lds16(rx, b + (wave + q * NW) * 1024, boff[q] + bt, (uint32_t)(s * 128));
  };

  auto read_b = [&](const unsigned char* b, int ks, int j) {
    const int r = wni * SN + j * 16 + fr;
    return *reinterpret_cast<const i32x4*>(b + r * 128 + 16 * swz8(r, 4 * ks + fq));
  };
  auto compute = [&](const unsigned char* a, const unsigned char* b) {
    if constexpr (SP) {
      i32x4 af[FI];
      int idx[FI];
#pragma unroll
      for (int i = 0; i < FI; ++i) {
        const int r = wmi * SM + i * 16 + fr;
        af[i] = *reinterpret_cast<const i32x4*>(a + r * 64 + 16 * swz4(r, fq));
        idx[i] = *reinterpret_cast<const int*>(a + V_BYTES + r * 16 + 4 * fq);
      }
      i32x4 lo = read_b(b, 0, 0), hi = read_b(b, 1, 0), nlo, nhi;
#pragma unroll
      for (int j = 0; j < FJ; ++j) {
        __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
        __builtin_amdgcn_sched_barrier(0);
        if (j + 1 < FJ) {
          nlo = read_b(b, 0, j + 1);
          nhi = read_b(b, 1, j + 1);
        }
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
        const i32x8 bv = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
        for (int i = 0; i < FI; ++i)
          acc[i][j] = __builtin_amdgcn_smfmac_i32_16x16x128_i8(af[i], bv, acc[i][j], idx[i], 0, 0);
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
        lo = nlo;
        hi = nhi;
      }
    } else {
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
    }
  };
  if (n > 0) {
    if constexpr (NST == 2) {
      k_loop2(n, sA0, sB0, sA1, sB1, issue, compute);
    } else {
      unsigned char* const SA[3] = {sA0, sA1, sA2};
      unsigned char* const SB[3] = {sB0, sB1, sB2};
      lds_ring<NST, NA + NB>(n, SA, SB, issue, compute);
    }
  }

  // lane: outputs ob + [0, 4) of each block row, token tb of each block column
  constexpr int NO = GLU ? FI / 2 : FI;         // output blocks of 16
  const int64_t ob0 = o0 + (GLU ? wmi * SM / 2 : wmi * SM) + 4 * fq;
  const int64_t tb0 = t0 + wni * SN + fr;
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
  const int esz = epi.bf16_out ? 2 : 4;
  struct Scales {
    float w[4], u[4], c[4];
  };
  auto scales = [&](int i) {   // of the lane's four outputs in block i
    Scales sc;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t o = ob0 + 16 * i + r < O ? ob0 + 16 * i + r : O - 1;
      sc.w[r] = epi.w_scale[o];
      sc.u[r] = GLU ? epi.up_scale[o] : 0.f;
      sc.c[r] = !GLU && epi.col_shift != nullptr ? epi.col_shift[o] : 0.f;
    }
    return sc;
  };
  auto value = [&](const Scales& sc, int i, int j, int r, float xs, float rb) {
    const int s0 = acc[GLU ? 2 * i : i][j][r], s1 = GLU ? acc[GLU ? 2 * i + 1 : i][j][r] : 0;
    if (!GLU && epi.col_shift == nullptr) return ((float)s0 * xs) * sc.w[r];
    return i8_value<GLU>(epi, s0, s1, xs, sc.w[r], sc.u[r], rb, sc.c[r]);
  };
  constexpr bool TURN = B_BYTES >= NW * 4096 && NO % 4 == 0;
  // pieces of 16 bytes of an output row: whole rows of 64 outputs, aligned
  const bool vec = TURN && (epi.ldy * esz) % 16 == 0;
  if (TURN && vec) {
    // 64 outputs x 16 tokens at a time: fp32 rows of 256 bytes in the wave's 4 KiB, piece c of
    // row r at c ^ r
    unsigned char* const mine = sB0 + wave * 4096;
#pragma unroll
    for (int h = 0; h < NO / 4; ++h) {
      const int64_t oh = o0 + (GLU ? wmi * SM / 2 : wmi * SM) + 64 * h;
      Scales sc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[i] = scales(4 * h + i);
#pragma unroll
      for (int j = 0; j < FJ; ++j) {
        const int64_t t = tb0 + 16 * j, tc = t < T ? t : T - 1;
        const float xs = epi.x_scale[tc];
        const float rb = !GLU && epi.row_shift != nullptr ? epi.row_shift[tc] : 1.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f32x4 v;
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = value(sc[i], 4 * h + i, j, r, xs, rb);
          *reinterpret_cast<f32x4*>(mine + fr * 256 + 16 * ((4 * i + fq) ^ fr)) = v;
        }
        __builtin_amdgcn_wave_barrier();
        if (epi.bf16_out) {
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const int row = 8 * p + (lane >> 3), c = 2 * (lane & 7);
            const f32x4 u = *reinterpret_cast<const f32x4*>(mine + row * 256 + 16 * (c ^ row));
            const f32x4 v = *reinterpret_cast<const f32x4*>(mine + row * 256 + 16 * ((c + 1) ^ row));
            const int64_t tt = t0 + wni * SN + 16 * j + row, o = oh + 4 * c;
            if (tt >= T || o >= O) continue;
            uint16_t* yp = static_cast<uint16_t*>(epi.y) + tt * epi.ldy + o;
            uint16_t h8[8];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              h8[r] = bf16_rne(u[r]);
              h8[4 + r] = bf16_rne(v[r]);
            }
            if (o + 8 <= O) {
              *reinterpret_cast<uint4*>(yp) =
                  make_uint4(h8[0] | (uint32_t)h8[1] << 16, h8[2] | (uint32_t)h8[3] << 16, h8[4] | (uint32_t)h8[5] << 16,
                             h8[6] | (uint32_t)h8[7] << 16);
            } else {
#pragma unroll
              for (int r = 0; r < 8; ++r)
                if (o + r < O) yp[r] = h8[r];
            }
          }
        } else {
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const int row = 4 * p + (lane >> 4), c = lane & 15;
            f32x4 v = *reinterpret_cast<const f32x4*>(mine + row * 256 + 16 * (c ^ row));
            const int64_t tt = t0 + wni * SN + 16 * j + row, o = oh + 4 * c;
            if (tt >= T || o >= O) continue;
            float* yp = static_cast<float*>(epi.y) + tt * epi.ldy + o;
            if (o + 4 <= O) {
              if (epi.accumulate) v += *reinterpret_cast<const f32x4*>(yp);
              *reinterpret_cast<f32x4*>(yp) = v;
            } else {
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (o + r < O) yp[r] = epi.accumulate ? yp[r] + v[r] : v[r];
            }
          }
        }
        __builtin_amdgcn_wave_barrier();
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < NO; ++i) {
    const Scales sc = scales(i);
#pragma unroll
    for (int j = 0; j < FJ; ++j) {
      const int64_t t = tb0 + 16 * j;
      if (t >= T) continue;
      const float xs = epi.x_scale[t];
      const float rb = !GLU && epi.row_shift != nullptr ? epi.row_shift[t] : 1.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t o = ob0 + 16 * i + r;
        if (o >= O) continue;
        const float v = value(sc, i, j, r, xs, rb);
        if (epi.bf16_out) {
          static_cast<uint16_t*>(epi.y)[t * epi.ldy + o] = bf16_rne(v);
        } else {
          float* p = static_cast<float*>(epi.y) + t * epi.ldy + o;
          *p = epi.accumulate ? *p + v : v;
        }
      }
    }
  }
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
hipError_t launch_kind(const I8Args& a, bool large, int64_t splits, int32_t* part, hipStream_t s) {
  if (large) {
    if constexpr (GLU || SP) return launch_cfg<256, 256, 2, 4, SP, GLU, 2>(a, splits, part, s);
    else return launch_cfg<256, 256, 4, 2, SP, GLU, 2>(a, splits, part, s);
  }
  if (a.t <= 64) return launch_cfg<128, 64, 4, 2, SP, GLU, 3>(a, splits, part, s);
  return launch_cfg<128, 128, 4, 2, SP, GLU, 3>(a, splits, part, s);
}

// splits of the 128-row tiles: one workgroup per CU, at least two steps each
int64_t mid_splits(int64_t t, int64_t o, int64_t k, bool glu) {
  const int64_t bn = t <= 64 ? 64 : 128, bo = glu ? 64 : 128;
  const int64_t tiles = ((o + bo - 1) / bo) * ((t + bn - 1) / bn), steps = (k + 127) / 128;
  int64_t s = tiles > 0 ? 256 / tiles : 1;
  if (s > steps / 2) s = steps / 2;
  return s < 1 ? 1 : s;
}

}  // namespace

namespace nml {

bool i8_tile_eligible(const I8Args& a) {
  // descriptors hold 256 rows in under 2^31 bytes
  return a.k > 0 && a.ldx < (1 << 23) && a.ldw < (1 << 23);
}

int64_t i8_mid_part_bytes(int64_t t, int64_t o, int64_t k, bool glu) {
  const int64_t s = mid_splits(t, o, k, glu);
  return s > 1 ? s * (glu ? 2 : 1) * t * ((o + 3) / 4 * 4) * 4 : 0;
}

hipError_t launch_i8_tile(const I8Args& a, bool large, int32_t* part, int64_t part_bytes, hipStream_t s) {
  const bool sp = a.meta != nullptr, glu = a.glu != 0;
  int64_t splits = 1;
  if (!large && part != nullptr && part_bytes >= i8_mid_part_bytes(a.t, a.o, a.k, glu)) splits = mid_splits(a.t, a.o, a.k, glu);
  if (sp && glu) return launch_kind<true, true>(a, large, splits, part, s);
  if (sp) return launch_kind<true, false>(a, large, splits, part, s);
  if (glu) return launch_kind<false, true>(a, large, splits, part, s);
  return launch_kind<false, false>(a, large, splits, part, s);
}

}  // namespace nml
