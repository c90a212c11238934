// C ABI of the operators around the products: host-side validation and dispatch
// (nm_linear, nm_rmsnorm_i8, nm_moe_route, nm_moe_i8).  Arguments are checked completely before the first HIP call.
#include "layer_launch.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename... P>
bool all_aligned(P... p) { return (aligned16(p) && ...); }

// rows x ld elements of up to 8 bytes addressable in 64 bits
bool span_ok(int64_t rows, int64_t ld) {
  int64_t e, b;
  return rows >= 0 && ld >= 0 && !__builtin_mul_overflow(rows, ld, &e) && !__builtin_mul_overflow(e, (int64_t)8, &b);
}

bool is_dtype(int d) { return d == NM_Y_F32 || d == NM_Y_BF16; }

bool finite(float v) { return v - v == 0.0f; }

nm_status hip_status(hipError_t e) { return e == hipSuccess ? NM_OK : NM_EHIP; }

int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }

enum class Kind { kFew, kMid, kLarge };

// Few tokens over short reductions: the streaming kernel, whose row blocks need no partial sums but
// read X again each.  Otherwise 256 x 256 tiles where there are enough of them to fill the chip,
// smaller tiles below.  Measured (us, streaming / smaller tiles, weights from HBM): 1 x 4096 x 4096
// 10.5 / 11.8, 4 11.2 / 12.2, 8 11.9 / 12.2, 16 13.5 / 12.4, 32 17.5 / 13.4; 1 x 4096 x 14336 25.0 / 27.3, 4
// 29.0 / 28.0, 16 37.9 / 29.1; 1 x 14336 x 4096 31.9 / 26.8; 8 x 256 x 2048 5.9 / 6.7, 32 9.0 / 7.0; 16 x
// 4096 x 1024 6.5 / 6.4; 2:4 1 x 4096 x 4096 9.0 / 9.3, 4 9.7 / 9.6, 8 10.3 / 9.7; 1 x 4096 x 14336 22.0 /
// 21.9; 1 x 14336 x 4096 22.1 / 18.9; 8 x 256 x 2048 5.7 / 6.6.
// From 160 tiles of 256 x 256 these (us, smaller / 256 x 256 tiles; their number, bias, bf16 out, weights
// from HBM): dense 2048 x 4096 x 4096 83 / 87 (128), 2304 x 4096 x 4096 114 / 82 (144), 2560 x 4096 x
// 4096 116 / 84 (160), 700 x 14336 x 1024 39 / 33 (168), 3000 x 4096 x 2048 68 / 52 (192), 4096 x 4096 x
// 4096 164 / 109 (256), 4352 x 4096 x 4096 198 / 175 (272), 1200 x 14336 x 4096 189 / 179 (280), 3000 x
// 6144 x 4096 184 / 177 (288), 1500 x 14336 x 4096 223 / 186 (336), 2304 x 4096 x 14336 385 / 264 (144),
// 4352 x 4096 x 14336 655 / 567 (272); 2:4 2048 x 4096 x 4096 69 / 78 (128), 2304 x 4096 x 4096 97 / 77
// (144), 2560 x 4096 x 4096 98 / 78 (160), 700 x 14336 x 1024 36 / 31 (168), 4096 x 4096 x 4096 136 / 85
// (256), 2560 x 7168 x 4096 154 / 137 (280), 5120 x 4096 x 4096 165 / 149 (320).  So they stay ahead where
// a second round is mostly idle, and would be from 144 on.
Kind plan_linear(int64_t t, int64_t o, int64_t k, bool sparse, uint32_t route) {
  if (route & NM_ROUTE_FEW_STREAM) return Kind::kFew;
  if (route & NM_ROUTE_FEW_TILE) return Kind::kMid;
  if (route & NM_ROUTE_TILE_LDS) return Kind::kLarge;
  if (t <= 16 && o < 8192 && t * k <= (sparse ? 16384 : 32768)) return Kind::kFew;
  return ((o + 255) / 256) * ((t + 255) / 256) >= 160 ? Kind::kLarge : Kind::kMid;
}

}  // namespace

extern "C" {

nm_status nm_linear(const void* x, int64_t t, int64_t k, int64_t ldx, const void* w, int64_t o, int64_t ldw,
                    const void* w_meta, const float* bias, nm_fn fn, const void* residual, int64_t ldr, void* y,
                    int64_t ldy, nm_ydtype y_dtype, void* workspace, int64_t workspace_bytes, uint32_t route,
                    uint32_t* route_taken, void* stream) {
  if (!is_dtype(y_dtype) || fn < NM_FN_NONE || fn > NM_FN_GELU_TANH) return NM_EINVAL;
  if (t < 0 || o < 0 || k < 0 || workspace_bytes < 0) return NM_ESHAPE;
  const bool sp = w_meta != nullptr, some = t > 0 && o > 0;
  if (sp && k % 4 != 0) return NM_ESHAPE;
  if (some && (y == nullptr || (k > 0 && (x == nullptr || w == nullptr)))) return NM_EINVAL;
  if (ldx < k || ldw < (sp ? k / 2 : k) || ldy < o || (residual != nullptr && ldr < o)) return NM_ESHAPE;
  if (!span_ok(t, ldx) || !span_ok(o, ldw) || !span_ok(t, ldy) || !span_ok(t, o) || (sp && !span_ok(o, k)) ||
      (residual != nullptr && !span_ok(t, ldr)))
    return NM_ESHAPE;
  if (ldx % 8 != 0 || ldw % 8 != 0 || !all_aligned(x, w, w_meta, bias, residual, y, workspace)) return NM_EALIGN;
  if (k > NM_LINEAR_MAX_K || t > NM_LINEAR_MAX_ROWS || o > NM_LINEAR_MAX_ROWS) return NM_EUNSUPPORTED;
  if (!some) return NM_OK;
  nml::LinArgs a{};
  a.x = static_cast<const uint16_t*>(x); a.w = static_cast<const uint16_t*>(w);
  a.meta = static_cast<const uint8_t*>(w_meta);
  a.ldx = ldx; a.ldw = ldw; a.t = t; a.o = o; a.k = k;
  a.epi = nml::LinEpi{bias, residual, y, ldr, ldy, (int)fn, y_dtype == NM_Y_BF16};
  a.route.flags = route;
  a.route.taken = route_taken;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  float* part = static_cast<float*>(workspace);
  const Kind kind = plan_linear(t, o, k, sp, route);
  if (kind == Kind::kFew || !nml::lin_tile_eligible(a)) return hip_status(nml::launch_lin_few(a, part, workspace_bytes, s));
  return hip_status(nml::launch_lin_tile(a, kind == Kind::kLarge, part, workspace_bytes, s));
}

int64_t nm_linear_workspace_size(int64_t t, int64_t o, int64_t k, int sparse, uint32_t route) {
  if (t <= 0 || o <= 0 || k <= 0 || k > NM_LINEAR_MAX_K || t > NM_LINEAR_MAX_ROWS || o > NM_LINEAR_MAX_ROWS) return 0;
  const Kind kind = plan_linear(t, o, k, sparse != 0, route);
  if (kind == Kind::kLarge) return 0;
  return kind == Kind::kFew ? nml::lin_few_part_bytes(t, o, k, sparse != 0) : nml::lin_mid_part_bytes(t, o, k, sparse != 0);
}

nm_status nm_rmsnorm_i8(const void* x, nm_ydtype x_dtype, int64_t rows, int64_t k, int64_t ldx, const void* residual,
                        int64_t ldr, void* sum_out, int64_t lds, nm_ydtype stream_dtype, const float* weight, float eps,
                        int n, int m, int ns, void* y, int64_t ldy, int8_t* q, int64_t ldq, float* scale, void* stream) {
  if (m != 0 && m != 4 && m != 8 && m != 16 && m != 32) return m < 0 ? NM_EINVAL : NM_EUNSUPPORTED;
  if (m != 0 && (n < 1 || n > m)) return NM_EINVAL;
  if (ns < 2 || ns > 8) return NM_EINVAL;
  if (!is_dtype(x_dtype) || !is_dtype(stream_dtype)) return NM_EINVAL;
  if (!(eps > 0.0f) || !finite(eps)) return NM_EINVAL;
  if (sum_out != nullptr && residual == nullptr) return NM_EINVAL;
  if (m != 0 && ns != 2) return NM_EUNSUPPORTED;
  if (rows < 0 || k < 0) return NM_ESHAPE;
  if (m != 0 && k % m != 0) return NM_ESHAPE;
  if (ns > 2 && k % (2 * ns) != 0) return NM_ESHAPE;
  if (rows > 0 && (scale == nullptr || (k > 0 && (x == nullptr || q == nullptr)))) return NM_EINVAL;
  const int64_t kq = ns > 2 ? k / (2 * ns) * 4 * (ns - 1) : k;
  const bool has_r = residual != nullptr, has_s = sum_out != nullptr, has_y = y != nullptr;
  if (ldx < k || ldq < up16(kq) || (has_r && ldr < k) || (has_s && lds < k) || (has_y && ldy < k)) return NM_ESHAPE;
  if (!span_ok(rows, ldx) || !span_ok(rows, ldq) || (has_r && !span_ok(rows, ldr)) || (has_s && !span_ok(rows, lds)) ||
      (has_y && !span_ok(rows, ldy)))
    return NM_ESHAPE;
  if (!all_aligned(x, residual, sum_out, weight, y, q, scale)) return NM_EALIGN;
  if (ldx % 8 != 0 || ldq % 16 != 0 || (has_r && ldr % 8 != 0) || (has_s && lds % 8 != 0) || (has_y && ldy % 8 != 0))
    return NM_EALIGN;
  if (k > 32768 || rows > 0x7FFFFFFF) return NM_EUNSUPPORTED;
  const nml::NormArgs a{x, residual, sum_out, weight, static_cast<uint16_t*>(y), q, scale, rows, k, ldx, ldr, lds, ldy,
                        ldq, x_dtype == NM_Y_BF16, stream_dtype == NM_Y_BF16, eps, n, m, ns};
  return hip_status(nml::launch_rmsnorm_i8(a, reinterpret_cast<hipStream_t>(stream)));
}

nm_status nm_moe_route(const float* logits, int64_t t, int64_t experts, int64_t ldl, const float* bias, nm_router kind,
                       int top, int renormalize, float scale, int32_t* ids, float* weights, void* stream) {
  if (kind != NM_ROUTER_SOFTMAX && kind != NM_ROUTER_SIGMOID) return NM_EINVAL;
  if (renormalize != 0 && renormalize != 1) return NM_EINVAL;
  if (!finite(scale) || top < 1) return NM_EINVAL;
  if (t < 0 || experts < top || ldl < experts || !span_ok(t, ldl)) return NM_ESHAPE;
  if (t > 0 && (logits == nullptr || ids == nullptr || weights == nullptr)) return NM_EINVAL;
  if (!all_aligned(logits, bias, ids, weights)) return NM_EALIGN;
  if (bias != nullptr && kind != NM_ROUTER_SIGMOID) return NM_EUNSUPPORTED;
  if (experts > NM_MOE_MAX_EXPERTS || top > NM_MOE_MAX_TOP || t > (1 << 25)) return NM_EUNSUPPORTED;
  const nml::RouteArgs a{logits, bias, ids, weights, t, experts, ldl, top, kind == NM_ROUTER_SIGMOID, renormalize, scale};
  return hip_status(nml::launch_moe_route(a, reinterpret_cast<hipStream_t>(stream)));
}

nm_status nm_moe_i8(const nm_moe_args* args, void* stream) {
  if (args == nullptr) return NM_EINVAL;
  const nm_moe_args& g = *args;
  if (g.act != NM_GLU_SILU && g.act != NM_GLU_GELU_TANH) return NM_EINVAL;
  if (!is_dtype(g.y_dtype) || g.top < 1 || g.experts < 1) return NM_EINVAL;
  const bool sp = g.gate_meta != nullptr;
  if ((g.up_meta != nullptr) != sp || (g.down_meta != nullptr) != sp) return NM_EINVAL;
  if (g.t < 0 || g.hidden < 0 || g.inter < 0 || g.workspace_bytes < 0) return NM_ESHAPE;
  if (sp && (g.hidden % 4 != 0 || g.inter % 4 != 0)) return NM_ESHAPE;
  const int64_t wk = sp ? g.hidden / 2 : g.hidden, dk = sp ? g.inter / 2 : g.inter;
  if (g.ldx < g.hidden || g.ldw < wk || g.ldd < dk || g.ldy < g.hidden || (g.residual != nullptr && g.ldr < g.hidden))
    return NM_ESHAPE;
  int64_t rows_i, rows_h;
  if (__builtin_mul_overflow((int64_t)g.experts, g.inter, &rows_i) ||
      __builtin_mul_overflow((int64_t)g.experts, g.hidden, &rows_h) || !span_ok(rows_i, g.ldw) || !span_ok(rows_h, g.ldd) ||
      !span_ok(rows_i, g.hidden) || !span_ok(rows_h, g.inter) || !span_ok(g.t, g.ldx) || !span_ok(g.t, g.ldy) ||
      !span_ok(g.t, g.top) || (g.residual != nullptr && !span_ok(g.t, g.ldr)))
    return NM_ESHAPE;
  const bool some = g.t > 0 && g.hidden > 0;
  if (some && (g.y == nullptr || g.ids == nullptr || g.weights == nullptr)) return NM_EINVAL;
  if (some && g.inter > 0 &&
      (g.x == nullptr || g.x_scale == nullptr || g.w_gate == nullptr || g.w_up == nullptr || g.w_down == nullptr ||
       g.gate_scale == nullptr || g.up_scale == nullptr || g.down_scale == nullptr))
    return NM_EINVAL;
  if (g.ldx % 16 != 0 || g.ldw % 16 != 0 || g.ldd % 16 != 0) return NM_EALIGN;
  if (!all_aligned(g.x, g.x_scale, g.ids, g.weights, g.w_gate, g.w_up, g.gate_scale, g.up_scale, g.gate_meta, g.up_meta,
                   g.w_down, g.down_scale, g.down_meta, g.residual, g.y, g.workspace))
    return NM_EALIGN;
  if (g.hidden > NM_I8_MAX_K || g.inter > 65536 || g.experts > NM_MOE_MAX_EXPERTS || g.top > NM_MOE_MAX_TOP)
    return NM_EUNSUPPORTED;
  if (!some) return NM_OK;
  if (g.workspace == nullptr || g.workspace_bytes < nml::moe_workspace_bytes(g.t, g.experts, g.top, g.hidden, g.inter)) return NM_EINVAL;
  nml::MoeArgs a{};
  a.x = g.x; a.x_scale = g.x_scale; a.ids = g.ids; a.weights = g.weights;
  a.w_gate = g.w_gate; a.w_up = g.w_up; a.w_down = g.w_down;
  a.gate_scale = g.gate_scale; a.up_scale = g.up_scale; a.down_scale = g.down_scale;
  a.gate_meta = static_cast<const uint8_t*>(g.gate_meta);
  a.up_meta = static_cast<const uint8_t*>(g.up_meta);
  a.down_meta = static_cast<const uint8_t*>(g.down_meta);
  a.residual = g.residual; a.y = g.y;
  a.ldx = g.ldx; a.ldw = g.ldw; a.ldd = g.ldd; a.ldr = g.ldr; a.ldy = g.ldy;
  a.t = g.t; a.hidden = g.hidden; a.inter = g.inter;
  a.experts = g.experts; a.top = g.top; a.act = (int)g.act; a.bf16_out = g.y_dtype == NM_Y_BF16;
  return hip_status(nml::launch_moe_i8(a, g.workspace, reinterpret_cast<hipStream_t>(stream)));
}

int64_t nm_moe_i8_workspace_size(int64_t t, int64_t experts, int64_t top, int64_t hidden, int64_t inter, int sparse) {
  (void)sparse;
  if (t <= 0 || experts <= 0 || top <= 0 || hidden <= 0 || inter < 0) return 0;
  if (hidden > NM_I8_MAX_K || inter > 65536 || experts > NM_MOE_MAX_EXPERTS || top > NM_MOE_MAX_TOP) return 0;
  return nml::moe_workspace_bytes(t, experts, top, hidden, inter);
}

}  // extern "C"
