// C ABI of the int8 layers: host-side validation and dispatch (nm_quant_i8, nm_meta_block,
// nm_spmm_i8, nm_glu_i8).  Arguments are checked completely before the first HIP call.
#include "i8_launch.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// rows x ld elements of up to 8 bytes addressable in 64 bits
bool span_ok(int64_t rows, int64_t ld) {
  int64_t e, b;
  return rows >= 0 && ld >= 0 && !__builtin_mul_overflow(rows, ld, &e) && !__builtin_mul_overflow(e, (int64_t)8, &b);
}

nm_status hip_status(hipError_t e) { return e == hipSuccess ? NM_OK : NM_EHIP; }

int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }

// a product's arguments (nm_spmm_i8 and nm_glu_i8 alike)
nm_status check_i8(const nml::I8Args& a, const void* ws, int64_t ws_bytes) {
  if (a.t < 0 || a.o < 0 || a.k < 0 || ws_bytes < 0) return NM_ESHAPE;
  if (a.epi.bf16_out != NM_Y_F32 && a.epi.bf16_out != NM_Y_BF16) return NM_EINVAL;
  if (a.epi.accumulate != 0 && a.epi.accumulate != 1) return NM_EINVAL;
  if (a.epi.row_shift != nullptr && a.epi.col_shift == nullptr) return NM_EINVAL;
  const bool glu = a.glu != 0;
  if (glu && (a.meta != nullptr) != (a.up_meta != nullptr)) return NM_EINVAL;
  if (a.t > 0 && a.o > 0) {
    if (a.epi.y == nullptr || a.epi.x_scale == nullptr || a.epi.w_scale == nullptr) return NM_EINVAL;
    if (glu && a.epi.up_scale == nullptr) return NM_EINVAL;
    if (a.k > 0 && (a.x == nullptr || a.w == nullptr || (glu && a.w_up == nullptr))) return NM_EINVAL;
  }
  const bool sp = a.meta != nullptr;
  if (sp && a.k % 4 != 0) return NM_ESHAPE;
  const int64_t wlen = sp ? a.k / 2 : a.k;
  if (a.ldx < a.k || a.ldw < wlen || a.epi.ldy < a.o) return NM_ESHAPE;
  if (!span_ok(a.t, a.ldx) || !span_ok(a.o, a.ldw) || !span_ok(a.t, a.epi.ldy) || !span_ok(a.t, a.o)) return NM_ESHAPE;
  if (sp && !span_ok(a.o, a.k)) return NM_ESHAPE;
  if (a.ldx % 16 != 0 || a.ldw % 16 != 0) return NM_EALIGN;
  const void* ptrs[] = {a.x, a.w, a.w_up, a.meta, a.up_meta, a.epi.x_scale, a.epi.w_scale, a.epi.up_scale,
                        a.epi.row_shift, a.epi.col_shift, a.epi.y, ws};
  for (const void* p : ptrs)
    if (!aligned16(p)) return NM_EALIGN;
  if (a.k > NM_I8_MAX_K) return NM_EUNSUPPORTED;
  if (a.epi.accumulate && a.epi.bf16_out) return NM_EUNSUPPORTED;
  if (a.t > NM_I8_MAX_ROWS || a.o > NM_I8_MAX_ROWS) return NM_EUNSUPPORTED;   // a grid holds under 2^32 threads
  return NM_OK;
}

enum class Kind { kFew, kMid, kLarge };

// Up to 32 tokens the streaming kernel, whose row blocks need no partial sums, unless 64 x 32
// tiles fill the chip unsplit (192 of them) or X, which every row block of the streaming kernel
// reads again, is long.  Measured (us, streaming / tiles, weights in the 256 MB last-level cache;
// then the same with weights from HBM): dense 1 x 4096 x 4096 5.9 / 7.9; 6.6 / 10.9, 16 x 4096 x
// 4096 7.0 / 8.1; 7.8 / 11.2, 32 x 4096 x 4096 8.9 / 8.3; 9.9 / 11.5, 8 x 4096 x 14336 13.5 / 14.2;
// 15.6 / 16.2, 16 x 4096 x 14336 15.7 / 14.6; 18.6 / 16.4, 32 x 4096 x 14336 22.1 / 15.0; 27.3 /
// 16.8, 1 x 14336 x 4096 12.5 / 10.8; 17.7 / 15.6, 16 x 14336 x 4096 14.3 / 11.4; 19.4 / 15.3, 16 x
// 14336 x 256 4.5 / 3.3; 5.3 / 4.0; 2:4 1 x 4096 x 14336 9.8 / 11.5; 11.1 / 14.1, 16 x 4096 x 14336
// 14.5 / 12.4; 15.7 / 14.4, 16 x 14336 x 4096 11.7 / 8.9; 13.1 / 11.6.
//
// Above, 256 x 256 tiles from 160 of them, smaller tiles below, whatever the reduction's length.
// Measured (us, smaller / 256 x 256; tiles): dense 2048 x 4096 x 4096 40 / 48 (128; weights from HBM
// 46 / 54), 2048 x 4096 x 14336 112 / 145 (128; 138 / 168), 2100 x 4096 x 14336 173 / 158 (144), 700 x
// 14336 x 1024 24 / 19 (168), 3000 x 4096 x 2048 35 / 29 (192), 4096 x 4096 x 4096 90 / 60 (256); GLU
// 1536 x 4096 x 14336 196 / 162 (192), 512 x 14336 x 4096 71 / 54 (224); 2:4 512 x 14336 x 4096 31 /
// 35 (112), 2048 x 4096 x 4096 32 / 34 (128; 39 / 42), 2048 x 4096 x 14336 94 / 91 (128; 115 / 120),
// 2100 x 4096 x 14336 143 / 112 (144), 700 x 14336 x 1024 20 / 18 (168), 4096 x 4096 x 4096 75 / 47
// (256); GLU 256 x 14336 x 4096 30 / 35 (112), 512 x 14336 x 4096 56 / 42 (224).  So the two meet
// between 128 and 144 tiles, dense and 2:4.
// Just over a round of 256 tiles the second round is mostly idle and the two are level: 2560 x
// 7168 x 4096 (280) 99 / 97, 3000 x 6144 x 4096 (288) 98 / 97, 1200 x 14336 x 4096 (280) 98 / 97, 2:4
// 78 / 76, 78 / 75, 76 / 75; only GLU 600 x 14336 x 4096 (336) loses, 94 / 98, 2:4 71 / 75.
// Short reductions, 8192 x 4096 over 64, 128, 256, 512, 1024 (512 tiles, fp32 out): dense 41 / 27,
// 42 / 27, 45 / 31, 50 / 39, 67 / 49, 2:4 31 / 30, 32 / 30, 39 / 33, 49 / 38, 66 / 48; bf16 38 / 18,
// 38 / 18, 41 / 21, 46 / 28, 63 / 40, 2:4 26 / 22, 27 / 23, 29 / 25, 35 / 31, 47 / 41.  GLU 4096 x
// 4096 over 128 and 512 35 / 21 and 44 / 31, but 2:4 22 / 26 and 31 / 34: the one kind that smaller
// tiles would serve better there.
Kind plan_i8(int64_t t, int64_t o, int64_t k, bool glu, uint32_t route) {
  if (route & NM_ROUTE_FEW_STREAM) return Kind::kFew;
  if (route & NM_ROUTE_FEW_TILE) return Kind::kMid;
  if (route & NM_ROUTE_TILE_LDS) return Kind::kLarge;
  if (t <= 32) {
    const int64_t bo = glu ? 32 : 64;
    return (o + bo - 1) / bo >= 192 || (t > 8 && t * k > 16 * 8192) ? Kind::kMid : Kind::kFew;
  }
  const int64_t bo = glu ? 128 : 256;
  return ((o + bo - 1) / bo) * ((t + 255) / 256) >= 160 ? Kind::kLarge : Kind::kMid;
}

nm_status run_i8(const nml::I8Args& a, void* ws, int64_t ws_bytes, hipStream_t s) {
  if (a.t == 0 || a.o == 0) return NM_OK;
  const Kind kind = plan_i8(a.t, a.o, a.k, a.glu != 0, a.route.flags);
  int32_t* part = static_cast<int32_t*>(ws);
  if (kind == Kind::kFew || !nml::i8_tile_eligible(a)) return hip_status(nml::launch_i8_few(a, part, ws_bytes, s));
  return hip_status(nml::launch_i8_tile(a, kind == Kind::kLarge, part, ws_bytes, s));
}

}  // namespace

extern "C" {

nm_status nm_quant_i8(const void* x, int64_t rows, int64_t k, int64_t ldx, int n, int m, int ns, int8_t* q,
                      int64_t ldq, float* scale, void* stream) {
  if (m != 0 && m != 4 && m != 8 && m != 16 && m != 32) return m < 0 ? NM_EINVAL : NM_EUNSUPPORTED;
  if (m != 0 && (n < 1 || n > m)) return NM_EINVAL;
  if (ns < 2 || ns > 8) return NM_EINVAL;
  if (m != 0 && ns != 2) return NM_EUNSUPPORTED;
  if (rows < 0 || k < 0) return NM_ESHAPE;
  if (m != 0 && k % m != 0) return NM_ESHAPE;
  if (ns > 2 && k % (2 * ns) != 0) return NM_ESHAPE;
  if (rows > 0 && (scale == nullptr || (k > 0 && (x == nullptr || q == nullptr)))) return NM_EINVAL;
  const int64_t kq = ns > 2 ? k / (2 * ns) * 4 * (ns - 1) : k;
  if (ldx < k || ldq < up16(kq)) return NM_ESHAPE;
  if (!span_ok(rows, ldx) || !span_ok(rows, ldq)) return NM_ESHAPE;
  if (!aligned16(x) || !aligned16(q) || !aligned16(scale) || ldx % 8 != 0 || ldq % 16 != 0) return NM_EALIGN;
  if (k > 65536 || rows > 0x7FFFFFFF) return NM_EUNSUPPORTED;
  return hip_status(nml::launch_quant_i8(static_cast<const uint16_t*>(x), rows, k, ldx, n, m, ns, q, ldq, scale,
                                         reinterpret_cast<hipStream_t>(stream)));
}

int64_t nm_meta_block_bytes(int64_t o, int64_t kc) {
  if (o <= 0 || kc <= 0 || !span_ok(o, kc)) return 0;
  return (kc + 127) / 128 * o * 16;
}

nm_status nm_meta_block(const void* meta, int64_t o, int64_t kc, void* out, void* stream) {
  if (o < 0 || kc < 0 || kc % 4 != 0 || !span_ok(o, kc)) return NM_ESHAPE;
  if (o > 0 && kc > 0 && (meta == nullptr || out == nullptr)) return NM_EINVAL;
  if (!aligned16(meta) || !aligned16(out)) return NM_EALIGN;
  return hip_status(nml::launch_meta_step_block(static_cast<const uint8_t*>(meta), o, kc, static_cast<uint8_t*>(out),
                                                reinterpret_cast<hipStream_t>(stream)));
}

nm_status nm_spmm_i8(const int8_t* x, int64_t t, int64_t k, int64_t ldx, const float* x_scale, const int8_t* w,
                     int64_t o, int64_t ldw, const float* w_scale, const void* w_meta, const float* row_shift,
                     const float* col_shift, void* y, int64_t ldy, nm_ydtype y_dtype, int accumulate,
                     void* workspace, int64_t workspace_bytes, uint32_t route, uint32_t* route_taken,
                     void* stream) {
  nml::I8Args a{};
  a.x = x; a.ldx = ldx; a.w = w; a.ldw = ldw; a.meta = static_cast<const uint8_t*>(w_meta);
  a.t = t; a.o = o; a.k = k;
  a.epi = nml::I8Epi{x_scale, w_scale, nullptr, row_shift, col_shift, y, ldy, (int)y_dtype, accumulate, 0};
  a.route.flags = route;
  a.route.taken = route_taken;
  const nm_status st = check_i8(a, workspace, workspace_bytes);
  return st != NM_OK ? st : run_i8(a, workspace, workspace_bytes, reinterpret_cast<hipStream_t>(stream));
}

nm_status nm_glu_i8(const int8_t* x, int64_t t, int64_t k, int64_t ldx, const float* x_scale, const int8_t* w_gate,
                    const float* gate_scale, const void* gate_meta, const int8_t* w_up, const float* up_scale,
                    const void* up_meta, int64_t inter, int64_t ldw, nm_glu_act act, void* y, int64_t ldy,
                    nm_ydtype y_dtype, void* workspace, int64_t workspace_bytes, uint32_t route,
                    uint32_t* route_taken, void* stream) {
  if (act != NM_GLU_SILU && act != NM_GLU_GELU_TANH) return NM_EINVAL;
  nml::I8Args a{};
  a.x = x; a.ldx = ldx; a.w = w_gate; a.w_up = w_up; a.ldw = ldw;
  a.meta = static_cast<const uint8_t*>(gate_meta); a.up_meta = static_cast<const uint8_t*>(up_meta);
  a.t = t; a.o = inter; a.k = k;
  a.glu = 1;
  a.epi = nml::I8Epi{x_scale, gate_scale, up_scale, nullptr, nullptr, y, ldy, (int)y_dtype, 0, (int)act};
  a.route.flags = route;
  a.route.taken = route_taken;
  const nm_status st = check_i8(a, workspace, workspace_bytes);
  return st != NM_OK ? st : run_i8(a, workspace, workspace_bytes, reinterpret_cast<hipStream_t>(stream));
}

int64_t nm_i8_workspace_size(int64_t t, int64_t o, int64_t k, int sparse, int glu, uint32_t route) {
  if (t <= 0 || o <= 0 || k <= 0 || k > NM_I8_MAX_K || !span_ok(t, o)) return 0;
  const Kind kind = plan_i8(t, o, k, glu != 0, route);
  if (kind == Kind::kLarge) return 0;
  return kind == Kind::kFew ? nml::i8_few_part_bytes(t, o, k, sparse != 0, glu != 0)
                            : nml::i8_mid_part_bytes(t, o, k, glu != 0);
}

}  // extern "C"
