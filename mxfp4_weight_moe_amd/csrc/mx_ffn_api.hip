// C-ABI entry points of the dense feed-forward operators: host-side checks and enqueue.
#include <cmath>

#include "mx_checks.hpp"

using namespace mx;

namespace {

size_t norm_backward_bytes(int64_t T, int64_t H, int arrays) {
  return (size_t)norm_backward_groups(T, H) * (size_t)H * arrays * 4;
}
size_t round256(size_t v) { return (v + 255) / 256 * 256; }

struct BlockPlan {
  bool post;  // a norm, gate or neither after the down projection
  size_t xn, h, b, ws, ws_bytes, bytes;
};
BlockPlan block_plan(int64_t T, int64_t H, int64_t I, bool pre, bool post) {
  BlockPlan p{};
  size_t off = 0;
  auto take = [&](size_t n) {
    const size_t at = off;
    off += round256(n);
    return at;
  };
  p.post = post;
  p.h = take((size_t)T * I * 2);
  if (pre) p.xn = take((size_t)T * H * 2);
  if (post) p.b = take((size_t)T * H * 2);
  p.ws_bytes = std::max(forward_plan(T, H, I, true).bytes, forward_plan(T, I, H, false).bytes);
  p.ws = take(p.ws_bytes);
  p.bytes = off;
  return p;
}

}  // namespace

extern "C" {

size_t mx_linear_fused_workspace_size(int64_t T, int64_t K, int64_t N) {
  return sizes_ok(T, K, N) ? forward_plan(T, K, N, false).bytes : 0;
}

int mx_linear_fused(const uint16_t* x, const uint8_t* w_codes, const uint8_t* w_scales, const uint16_t* bias,
                    const uint16_t* residual, float scale, int act, uint16_t* y, uint16_t* z, int64_t T, int64_t K,
                    int64_t N, void* workspace, size_t workspace_bytes, void* stream) {
  if (!x || !w_codes || !w_scales || !y) return MX_ERR_NULL;
  if (!sizes_ok(T, K, N)) return MX_ERR_SHAPE;
  if (!act_ok(act) || !std::isfinite(scale)) return MX_ERR_ARG;
  if (!aligned(x, 16) || !aligned(w_codes, 16) || !aligned(y, 16) || !opt_aligned(bias, 16) ||
      !opt_aligned(residual, 16) || !opt_aligned(z, 16) || !scales_aligned(w_scales, K))
    return MX_ERR_ALIGN;
  const int st = workspace_ok(workspace, workspace_bytes, forward_plan(T, K, N, false).bytes);
  if (st != MX_OK) return st;
  return launch_linear_fused(x, w_codes, w_scales, bias, residual, scale, act, y, z, (int)T, (int)K, (int)N, workspace,
                             static_cast<hipStream_t>(stream));
}

size_t mx_linear_fused_backward_workspace_size(int64_t T, int64_t K, int64_t N) {
  return sizes_ok(T, K, N) ? backward_workspace(T, K, N, N, true, true, true).bytes : 0;
}

int mx_linear_fused_backward(const uint16_t* dy, const uint16_t* z, const uint8_t* w_codes, const uint8_t* w_scales,
                             float scale, int act, uint16_t* dx, float* dbias, int64_t T, int64_t K, int64_t N,
                             void* workspace, size_t workspace_bytes, void* stream) {
  if (!dy || (!dx && !dbias) || (dx && (!w_codes || !w_scales)) || (act != MX_ACT_NONE && !z)) return MX_ERR_NULL;
  if (!sizes_ok(T, K, N)) return MX_ERR_SHAPE;
  if (!act_ok(act) || !std::isfinite(scale)) return MX_ERR_ARG;
  if (act == MX_ACT_NONE) z = nullptr;
  if (!aligned(dy, 16) || !opt_aligned(z, 16) || !opt_aligned(w_codes, 16) || !opt_aligned(dx, 16) ||
      !opt_aligned(dbias, 4))
    return MX_ERR_ALIGN;
  const int st = workspace_ok(workspace, workspace_bytes, mx_linear_fused_backward_workspace_size(T, K, N));
  if (st != MX_OK) return st;
  return launch_linear_fused_backward(dy, z, w_codes, w_scales, scale, act, dx, dbias, (int)T, (int)K, (int)N, workspace,
                                      static_cast<hipStream_t>(stream));
}

size_t mx_gate_up_workspace_size(int64_t T, int64_t H, int64_t I) {
  return gated_ok(T, H, I) ? forward_plan(T, H, I, true).bytes : 0;
}

int mx_gate_up(const uint16_t* x, const uint8_t* w_gate_up, const uint8_t* s_gate_up, const uint16_t* bias, int act,
               uint16_t* h, uint16_t* z, int64_t T, int64_t H, int64_t I, void* workspace, size_t workspace_bytes,
               void* stream) {
  if (!x || !w_gate_up || !s_gate_up || !h) return MX_ERR_NULL;
  if (!gated_ok(T, H, I)) return MX_ERR_SHAPE;
  if (!act_ok(act)) return MX_ERR_ARG;
  if (!aligned(x, 16) || !aligned(w_gate_up, 16) || !aligned(h, 16) || !opt_aligned(bias, 16) || !opt_aligned(z, 16) ||
      !scales_aligned(s_gate_up, H))
    return MX_ERR_ALIGN;
  const int st = workspace_ok(workspace, workspace_bytes, forward_plan(T, H, I, true).bytes);
  if (st != MX_OK) return st;
  return launch_gate_up_dense(x, w_gate_up, s_gate_up, bias, act, h, z, (int)T, (int)H, (int)I, workspace,
                              static_cast<hipStream_t>(stream));
}

size_t mx_gate_up_backward_workspace_size(int64_t T, int64_t H, int64_t I) {
  return gated_ok(T, H, I) ? backward_workspace(T, H, 2 * I, I, true, true, true).bytes : 0;
}

int mx_gate_up_backward(const uint16_t* dh, const uint16_t* z, const uint8_t* w_gate_up, const uint8_t* s_gate_up,
                        int act, uint16_t* dx, float* dbias, int64_t T, int64_t H, int64_t I, void* workspace,
                        size_t workspace_bytes, void* stream) {
  if (!dh || !z || (!dx && !dbias) || (dx && (!w_gate_up || !s_gate_up))) return MX_ERR_NULL;
  if (!gated_ok(T, H, I)) return MX_ERR_SHAPE;
  if (!act_ok(act)) return MX_ERR_ARG;
  if (!aligned(dh, 16) || !aligned(z, 16) || !opt_aligned(w_gate_up, 16) || !opt_aligned(dx, 16) ||
      !opt_aligned(dbias, 4))
    return MX_ERR_ALIGN;
  const int st = workspace_ok(workspace, workspace_bytes, mx_gate_up_backward_workspace_size(T, H, I));
  if (st != MX_OK) return st;
  return launch_gate_up_backward(dh, z, w_gate_up, s_gate_up, act, dx, dbias, (int)T, (int)H, (int)I, workspace,
                                 static_cast<hipStream_t>(stream));
}

int mx_norm_residual(const uint16_t* x, const uint16_t* b, const uint16_t* w_post, const uint16_t* gate, int gate_mode,
                     float scale, const uint16_t* w_pre, float eps, uint16_t* y, uint16_t* xn, int64_t T, int64_t H,
                     void* stream) {
  if (!x || (!b && !w_pre) || (b && !y) || (w_pre && !xn)) return MX_ERR_NULL;
  if (!norm_sizes_ok(T, H)) return MX_ERR_SHAPE;
  if (gate_mode < MX_GATE_NONE || gate_mode > MX_GATE_FULL || (gate_mode != MX_GATE_NONE) != (gate != nullptr) ||
      (!b && (w_post || gate || y)) || (!w_pre && xn) || !std::isfinite(scale) || !std::isfinite(eps) || eps <= 0.f)
    return MX_ERR_ARG;
  if (!aligned(x, 16) || !opt_aligned(b, 16) || !opt_aligned(w_post, 16) || !opt_aligned(w_pre, 16) ||
      !opt_aligned(gate, gate_mode == MX_GATE_TOKEN ? 2 : 16) || !opt_aligned(y, 16) || !opt_aligned(xn, 16))
    return MX_ERR_ALIGN;
  return launch_norm_residual(x, b, w_post, gate, gate_mode, scale, w_pre, eps, y, xn, (int)T, (int)H,
                              static_cast<hipStream_t>(stream));
}

size_t mx_norm_residual_backward_workspace_size(int64_t T, int64_t H) {
  return norm_sizes_ok(T, H) ? norm_backward_bytes(T, H, 3) : 0;
}

int mx_norm_residual_backward(const uint16_t* dy, const uint16_t* dxn, const uint16_t* y, const uint16_t* b,
                              const uint16_t* w_post, const uint16_t* gate, int gate_mode, float scale,
                              const uint16_t* w_pre, float eps, uint16_t* dx, uint16_t* db, void* dgate,
                              float* dw_post, float* dw_pre, int64_t T, int64_t H, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (!dx || (!b && !w_pre) || (w_pre && (!dxn || !y)) || (!w_pre && !dy)) return MX_ERR_NULL;
  if (!norm_sizes_ok(T, H)) return MX_ERR_SHAPE;
  if (gate_mode < MX_GATE_NONE || gate_mode > MX_GATE_FULL || (gate_mode != MX_GATE_NONE) != (gate != nullptr) ||
      (!b && (w_post || gate || db)) || (!w_post && dw_post) || (!gate && dgate) || (!w_pre && (dw_pre || dxn)) ||
      !std::isfinite(scale) || !std::isfinite(eps) || eps <= 0.f)
    return MX_ERR_ARG;
  if (!opt_aligned(dy, 16) || !opt_aligned(dxn, 16) || !opt_aligned(y, 16) || !opt_aligned(b, 16) ||
      !opt_aligned(w_post, 16) || !opt_aligned(w_pre, 16) || !opt_aligned(gate, gate_mode == MX_GATE_TOKEN ? 2 : 16) ||
      !aligned(dx, 16) || !opt_aligned(db, 16) || !opt_aligned(dgate, gate_mode == MX_GATE_FULL ? 16 : 4) ||
      !opt_aligned(dw_post, 4) || !opt_aligned(dw_pre, 4))
    return MX_ERR_ALIGN;
  const int st = workspace_ok(workspace, workspace_bytes, norm_backward_bytes(T, H, 3));
  if (st != MX_OK) return st;
  return launch_norm_residual_backward(dy, dxn, y, b, w_post, gate, gate_mode, scale, w_pre, eps, dx, db, dgate, dw_post,
                                       dw_pre, (int)T, (int)H, static_cast<float*>(workspace),
                                       static_cast<hipStream_t>(stream));
}

size_t mx_ffn_block_workspace_size(int64_t T, int64_t H, int64_t I) {
  return block_ok(T, H, I) ? block_plan(T, H, I, true, true).bytes : 0;
}

int mx_ffn_block(const uint16_t* x, const uint16_t* w_pre, const uint8_t* w_gate_up, const uint8_t* s_gate_up,
                 const uint16_t* bias_gate_up, int act, const uint8_t* w_down, const uint8_t* s_down,
                 const uint16_t* bias_down, const uint16_t* w_post, const uint16_t* gate, int gate_mode, float scale,
                 float eps, uint16_t* y, int64_t T, int64_t H, int64_t I, void* workspace, size_t workspace_bytes,
                 void* stream) {
  if (!x || !w_gate_up || !s_gate_up || !w_down || !s_down || !y) return MX_ERR_NULL;
  if (!block_ok(T, H, I)) return MX_ERR_SHAPE;
  if ((w_pre || w_post || gate) && !norm_sizes_ok(T, H)) return MX_ERR_SHAPE;
  if (gate_mode < MX_GATE_NONE || gate_mode > MX_GATE_FULL || (gate_mode != MX_GATE_NONE) != (gate != nullptr) ||
      !act_ok(act) || !std::isfinite(scale) || !std::isfinite(eps) || eps <= 0.f)
    return MX_ERR_ARG;
  if (!aligned(x, 16) || !opt_aligned(w_pre, 16) || !aligned(w_gate_up, 16) || !scales_aligned(s_gate_up, H) ||
      !opt_aligned(bias_gate_up, 16) || !aligned(w_down, 16) || !scales_aligned(s_down, I) ||
      !opt_aligned(bias_down, 16) || !opt_aligned(w_post, 16) || !opt_aligned(gate, gate_mode == MX_GATE_TOKEN ? 2 : 16) ||
      !aligned(y, 16))
    return MX_ERR_ALIGN;
  int st = workspace_ok(workspace, workspace_bytes, mx_ffn_block_workspace_size(T, H, I));
  if (st != MX_OK) return st;
  const BlockPlan p = block_plan(T, H, I, w_pre != nullptr, w_post || gate);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint16_t* h = reinterpret_cast<uint16_t*>(ws + p.h);
  const uint16_t* in = x;
  if (w_pre) {
    uint16_t* xn = reinterpret_cast<uint16_t*>(ws + p.xn);
    st = launch_norm_residual(x, nullptr, nullptr, nullptr, MX_GATE_NONE, 1.f, w_pre, eps, nullptr, xn, (int)T, (int)H, s);
    if (st != MX_OK) return st;
    in = xn;
  }
  st = launch_gate_up_dense(in, w_gate_up, s_gate_up, bias_gate_up, act, h, nullptr, (int)T, (int)H, (int)I, ws + p.ws, s);
  if (st != MX_OK) return st;
  if (!p.post)
    return launch_linear_fused(h, w_down, s_down, bias_down, x, scale, MX_ACT_NONE, y, nullptr, (int)T, (int)I, (int)H,
                               ws + p.ws, s);
  uint16_t* b = reinterpret_cast<uint16_t*>(ws + p.b);
  st = launch_linear_fused(h, w_down, s_down, bias_down, nullptr, 1.f, MX_ACT_NONE, b, nullptr, (int)T, (int)I, (int)H,
                           ws + p.ws, s);
  if (st != MX_OK) return st;
  return launch_norm_residual(x, b, w_post, gate, gate_mode, scale, nullptr, eps, y, nullptr, (int)T, (int)H, s);
}

}  // extern "C"
