// C-ABI entry points of microscaled activations and of routing by scores: host-side checks and enqueue.
#include <cmath>

#include "mx_checks.hpp"

using namespace mx;

namespace {

bool format_ok(int f) { return f == MX_FORMAT_MXFP8 || f == MX_FORMAT_MXFP4; }
// Whole 16 bytes of scales go to the LDS at once where rows begin at multiples of them.
bool q_scales_aligned(const uint8_t* s, int64_t K) { return K % 512 != 0 || aligned(s, 16); }

// For either format: sizes alone say how large a workspace is.
size_t linear_bytes(int64_t T, int64_t K, int64_t N) {
  return std::max(quantized_plan(T, K, N, false, false, MX_FORMAT_MXFP8).bytes,
                  quantized_plan(T, K, N, false, false, MX_FORMAT_MXFP4).bytes);
}

// What both routing calls share.
int route_args(const void* logits, int logits_type, int score, float scale, int64_t T, int64_t E, int64_t k) {
  if (T < 1 || T > MAX_T || E < 1 || E > MX_MAX_EXPERTS || k < 1 || k > MX_MAX_TOPK || k > E) return MX_ERR_SHAPE;
  if ((logits_type != MX_TYPE_BF16 && logits_type != MX_TYPE_F32) ||
      (score != MX_SCORE_SOFTMAX && score != MX_SCORE_SIGMOID) || !std::isfinite(scale))
    return MX_ERR_ARG;
  return aligned(logits, logits_type == MX_TYPE_F32 ? 4 : 2) ? MX_OK : MX_ERR_ALIGN;
}

}  // namespace

extern "C" {

int mx_quantize(const void* x, int x_type, int format, uint8_t* codes, uint8_t* scales, uint16_t* values, int64_t rows,
                int64_t K, void* stream) {
  if (!x || !codes || !scales) return MX_ERR_NULL;
  if (rows < 1 || K < 32 || K % 32 != 0 || rows > MAX_VALUES / K) return MX_ERR_SHAPE;
  if (!format_ok(format) || (x_type != MX_TYPE_BF16 && x_type != MX_TYPE_F32)) return MX_ERR_ARG;
  if (!aligned(x, 16) || !aligned(codes, 16) || !opt_aligned(values, 16)) return MX_ERR_ALIGN;
  return launch_quantize(x, x_type == MX_TYPE_F32, format, rows, K, codes, scales, values,
                         static_cast<hipStream_t>(stream));
}

int mx_norm_residual_quantize(const uint16_t* x, const uint16_t* b, const uint16_t* w_post, const uint16_t* gate,
                              int gate_mode, float scale, const uint16_t* w_pre, float eps, uint16_t* y, uint16_t* xn,
                              int format, uint8_t* codes, uint8_t* scales, int64_t T, int64_t H, void* stream) {
  if (!x || !w_pre || !codes || !scales || (b && !y)) return MX_ERR_NULL;
  if (!norm_sizes_ok(T, H) || H % 32 != 0) return MX_ERR_SHAPE;
  if (gate_mode < MX_GATE_NONE || gate_mode > MX_GATE_FULL || (gate_mode != MX_GATE_NONE) != (gate != nullptr) ||
      (!b && (w_post || gate || y)) || !format_ok(format) || !std::isfinite(scale) || !std::isfinite(eps) || eps <= 0.f)
    return MX_ERR_ARG;
  if (!aligned(x, 16) || !opt_aligned(b, 16) || !opt_aligned(w_post, 16) || !aligned(w_pre, 16) ||
      !opt_aligned(gate, gate_mode == MX_GATE_TOKEN ? 2 : 16) || !opt_aligned(y, 16) || !opt_aligned(xn, 16) ||
      !aligned(codes, 16))
    return MX_ERR_ALIGN;
  return launch_norm_residual_quantize(x, b, w_post, gate, gate_mode, scale, w_pre, eps, y, xn, format, codes, scales,
                                       (int)T, (int)H, static_cast<hipStream_t>(stream));
}

size_t mx_linear_quantized_workspace_size(int64_t T, int64_t K, int64_t N) {
  return sizes_ok(T, K, N) ? linear_bytes(T, K, N) : 0;
}

int mx_linear_quantized(const uint8_t* a_codes, const uint8_t* a_scales, int format, const uint8_t* w_codes,
                        const uint8_t* w_scales, const uint16_t* bias, const uint16_t* residual, float scale, int act,
                        uint16_t* y, uint16_t* z, int64_t T, int64_t K, int64_t N, void* workspace,
                        size_t workspace_bytes, void* stream) {
  if (!a_codes || !a_scales || !w_codes || !w_scales || !y) return MX_ERR_NULL;
  if (!sizes_ok(T, K, N)) return MX_ERR_SHAPE;
  if (!format_ok(format) || !act_ok(act) || !std::isfinite(scale)) return MX_ERR_ARG;
  if (!aligned(a_codes, 16) || !aligned(w_codes, 16) || !aligned(y, 16) || !opt_aligned(bias, 16) ||
      !opt_aligned(residual, 16) || !opt_aligned(z, 16) || !q_scales_aligned(a_scales, K) ||
      !q_scales_aligned(w_scales, K))
    return MX_ERR_ALIGN;
  const int st = workspace_ok(workspace, workspace_bytes, linear_bytes(T, K, N));
  if (st != MX_OK) return st;
  return launch_linear_quantized(a_codes, a_scales, format, w_codes, w_scales, bias, residual, scale, act, y, z, (int)T,
                                 (int)K, (int)N, workspace, static_cast<hipStream_t>(stream));
}

size_t mx_gate_up_quantized_workspace_size(int64_t T, int64_t H, int64_t I) {
  if (!gated_ok(T, H, I)) return 0;
  size_t most = 0;
  for (int f : {MX_FORMAT_MXFP8, MX_FORMAT_MXFP4})
    for (bool quantized : {false, true}) most = std::max(most, quantized_plan(T, H, I, true, quantized, f).bytes);
  return most;
}

int mx_gate_up_quantized(const uint8_t* a_codes, const uint8_t* a_scales, int format, const uint8_t* w_gate_up,
                         const uint8_t* s_gate_up, const uint16_t* bias, int act, uint16_t* h, int h_format,
                         uint8_t* h_codes, uint8_t* h_scales, uint16_t* z, int64_t T, int64_t H, int64_t I,
                         void* workspace, size_t workspace_bytes, void* stream) {
  if (!a_codes || !a_scales || !w_gate_up || !s_gate_up || (!h && (!h_codes || !h_scales))) return MX_ERR_NULL;
  if (!gated_ok(T, H, I) || (!h && I % 32 != 0)) return MX_ERR_SHAPE;
  if (!format_ok(format) || !act_ok(act) || (h ? h_codes || h_scales : !format_ok(h_format))) return MX_ERR_ARG;
  if (!aligned(a_codes, 16) || !aligned(w_gate_up, 16) || !opt_aligned(h, 16) || !opt_aligned(h_codes, 16) ||
      !opt_aligned(bias, 16) || !opt_aligned(z, 16) || !q_scales_aligned(a_scales, H) || !q_scales_aligned(s_gate_up, H))
    return MX_ERR_ALIGN;
  const int st = workspace_ok(workspace, workspace_bytes, mx_gate_up_quantized_workspace_size(T, H, I));
  if (st != MX_OK) return st;
  return launch_gate_up_quantized(a_codes, a_scales, format, w_gate_up, s_gate_up, bias, act, h, h_format, h_codes,
                                  h_scales, z, (int)T, (int)H, (int)I, workspace, static_cast<hipStream_t>(stream));
}

int moe_route_scored(const void* logits, int logits_type, const float* bias, int score, int64_t n_group,
                     int64_t topk_group, int group_score, int renormalize, float scale, int32_t* ids, float* gates,
                     int64_t T, int64_t E, int64_t top_k, void* stream) {
  if (!logits || !ids || !gates) return MX_ERR_NULL;
  const int st = route_args(logits, logits_type, score, scale, T, E, top_k);
  if (st != MX_OK && st != MX_ERR_ALIGN) return st;
  if (n_group < 1 || n_group > MX_MAX_GROUPS || E % n_group != 0 || topk_group < 1 || topk_group > n_group ||
      top_k > topk_group * (E / n_group))
    return MX_ERR_SHAPE;
  if (group_score != MX_GROUP_TOP2 && group_score != MX_GROUP_MAX) return MX_ERR_ARG;
  if (st != MX_OK || !opt_aligned(bias, 4) || !aligned(ids, 4) || !aligned(gates, 4)) return MX_ERR_ALIGN;
  RouteScored a{};
  a.logits = logits, a.bias = bias, a.bf16 = logits_type == MX_TYPE_BF16, a.sigmoid = score == MX_SCORE_SIGMOID;
  a.top2 = group_score == MX_GROUP_TOP2, a.renormalize = renormalize != 0, a.scale = scale;
  a.T = T, a.E = (int)E, a.k = (int)top_k;
  a.groups = topk_group == n_group ? 1 : (int)n_group, a.kept = (int)topk_group;  // all groups kept: as none
  return launch_route_scored(a, ids, gates, static_cast<hipStream_t>(stream));
}

int moe_route_scored_backward(const float* dgates, const void* logits, int logits_type, const int32_t* ids, int score,
                              int renormalize, float scale, void* dlogits, int64_t T, int64_t E, int64_t top_k,
                              void* stream) {
  if (!dgates || !logits || !ids || !dlogits) return MX_ERR_NULL;
  const int st = route_args(logits, logits_type, score, scale, T, E, top_k);
  if (st != MX_OK) return st;
  if (!aligned(dgates, 4) || !aligned(ids, 4) || !aligned(dlogits, logits_type == MX_TYPE_F32 ? 4 : 2)) return MX_ERR_ALIGN;
  RouteScored a{};
  a.logits = logits, a.bf16 = logits_type == MX_TYPE_BF16, a.sigmoid = score == MX_SCORE_SIGMOID;
  a.renormalize = renormalize != 0, a.scale = scale, a.T = T, a.E = (int)E, a.k = (int)top_k;
  return launch_route_scored_backward(a, dgates, ids, dlogits, static_cast<hipStream_t>(stream));
}

}  // extern "C"
