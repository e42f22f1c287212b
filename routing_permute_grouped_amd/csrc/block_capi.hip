// C ABI entry points of moe_block.h: host-side validation, then the kernel launchers.
// Every check runs before any HIP call, so a rejected call never touches the GPU.
#include <hip/hip_runtime.h>
#include <math.h>

#include "moe_block.h"
#include "border.hpp"
#include "checks.hpp"
#include "few.hpp"
#include "route_bwd.hpp"

using namespace moe;

namespace {

bool few_sizes_ok(int T, int k, int F, int Fs) {
  return T >= 1 && T <= kFewTokens && k >= 1 && k <= kMaxK && dim_ok(F) && (Fs == 0 || dim_ok(Fs));
}

moe_status_t few_layer(int fmt, const FewCall& c, size_t ws_bytes, void* stream) {
  if (!aligned16(c.x) || !aligned16(c.out) || !aligned4(c.topk_idx) || !aligned4(c.topk_w) ||
      !aligned16(c.workspace) || (c.wg && !aligned16(c.wg)) || (c.bias && !aligned4(c.bias)))
    return MOE_EINVAL;
  for (int i = 0; i < 3; ++i) {
    if (!aligned16(c.w[i])) return MOE_EINVAL;
    if (fmt == kFewMx4 && !aligned4(c.s[i])) return MOE_EINVAL;
    if (c.Fs > 0 && !aligned16(c.ws[i])) return MOE_EINVAL;
  }
  if (!few_sizes_ok(c.T, c.k, c.F, c.Fs) || !dim_ok(c.D) || c.E < 1 || c.E > kMaxExperts ||
      c.k > c.E)
    return MOE_ESHAPE;
  if (fmt == kFewMx4 && (c.D % 128 != 0 || c.F % 128 != 0)) return MOE_ESHAPE;
  if (ws_bytes < few_workspace_bytes(fmt, c.T, c.k, c.F, c.Fs)) return MOE_EWORKSPACE;
  return hip_status(launch_few(fmt, c, static_cast<hipStream_t>(stream)));
}

bool opt16(const void* p) { return !p || aligned16(p); }
bool opt4(const void* p) { return !p || aligned4(p); }
bool norm_sizes_ok(int T, int D) {
  return T >= 1 && T <= (1 << 30) && dim_ok(D) && D <= kBorderMaxD;
}
bool route_bwd_sizes_ok(int T, int D, int E) {
  return T >= 1 && T <= (1 << 30) && dim_ok(D) && E >= 1 && E <= kMaxExperts;
}

}  // namespace

extern "C" {

size_t moe_layer_few_workspace_bytes(moe_dtype_t dt, int T, int k, int F, int Fs) {
  if (!dtype_ok(dt) || !few_sizes_ok(T, k, F, Fs)) return 0;
  return few_workspace_bytes(dt == MOE_F32 ? kFewF32 : kFewBf16, T, k, F, Fs);
}

moe_status_t moe_layer_few(moe_dtype_t dt, const void* x, const void* wg, const float* bias,
                           int T, int D, int F, int E, int k, int renorm, const void* w1,
                           const void* w3, const void* w2, int Fs, const void* ws1,
                           const void* ws3, const void* ws2, int32_t* topk_idx, float* topk_w,
                           void* out, void* workspace, size_t ws_bytes, void* stream) {
  if (!dtype_ok(dt)) return MOE_EINVAL;
  const FewCall c = {x,  wg, bias, T, D, F, E, k, renorm, Fs, {w1, w3, w2}, {nullptr, nullptr, nullptr},
                     {ws1, ws3, ws2}, topk_idx, topk_w, out, workspace};
  return few_layer(dt == MOE_F32 ? kFewF32 : kFewBf16, c, ws_bytes, stream);
}

moe_status_t moe_layer_few_mxfp4(const void* x, const void* wg, const float* bias, int T, int D,
                                 int F, int E, int k, int renorm, const void* w1q,
                                 const void* w1s, const void* w3q, const void* w3s,
                                 const void* w2q, const void* w2s, int Fs, const void* ws1,
                                 const void* ws3, const void* ws2, int32_t* topk_idx,
                                 float* topk_w, void* out, void* workspace, size_t ws_bytes,
                                 void* stream) {
  const FewCall c = {x,  wg, bias, T, D, F, E, k, renorm, Fs, {w1q, w3q, w2q}, {w1s, w3s, w2s},
                     {ws1, ws3, ws2}, topk_idx, topk_w, out, workspace};
  return few_layer(kFewMx4, c, ws_bytes, stream);
}

moe_status_t moe_norm(moe_dtype_t dt, const void* r, const void* gamma, float eps, int T, int D,
                      void* x, float* rstd, void* stream) {
  if (!dtype_ok(dt) || !aligned16(r) || !aligned16(gamma) || !aligned16(x) || !opt4(rstd) ||
      !(eps > 0.0f) || !isfinite(eps))
    return MOE_EINVAL;
  if (!norm_sizes_ok(T, D)) return MOE_ESHAPE;
  BorderCall c = {};
  c.resid = r;
  c.gamma_next = gamma;
  c.eps = eps;
  c.T = T;
  c.D = D;
  c.x_next = x;
  c.rstd_next = rstd;
  return hip_status(launch_border(dt, c, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_combine_norm(moe_dtype_t dt, const void* resid, const void* y_perm,
                              const int32_t* dst_row, const float* topk_w, const void* shared,
                              const float* gate, const void* gamma_post, const void* gamma_next,
                              float scale, float eps, int T, int D, int k, int64_t m_cap,
                              void* out, void* x_next, void* u, float* rstd_post,
                              float* rstd_next, void* stream) {
  if (!dtype_ok(dt) || !aligned16(resid) || !aligned16(out) || !opt16(shared) || !opt4(gate) ||
      !opt16(gamma_post) || !opt16(gamma_next) || !opt16(u) || !opt4(rstd_post) ||
      !opt4(rstd_next) || !isfinite(scale) || !(eps > 0.0f) || !isfinite(eps))
    return MOE_EINVAL;
  if (y_perm ? !aligned16(y_perm) || !aligned4(dst_row) || !opt4(topk_w) : !shared)
    return MOE_EINVAL;
  // a result that no norm writes is refused, not left as it was
  if (gamma_next ? !aligned16(x_next) : x_next || rstd_next) return MOE_EINVAL;
  if (!gamma_post && rstd_post) return MOE_EINVAL;
  if (!norm_sizes_ok(T, D)) return MOE_ESHAPE;
  if (y_perm) {
    if (!tk_ok(T, k) || k < 1 || k > kMaxK) return MOE_ESHAPE;
    if (m_cap < 1 || m_cap > INT32_MAX) return MOE_ECAPACITY;
  }
  BorderCall c = {};
  c.resid = resid;
  c.y = y_perm;
  c.dst = dst_row;
  c.w = topk_w;
  c.shared = shared;
  c.gate = gate;
  c.gamma_post = gamma_post;
  c.gamma_next = gamma_next;
  c.scale = scale;
  c.eps = eps;
  c.T = T;
  c.D = D;
  c.k = k;
  c.m_cap = m_cap;
  c.block = true;
  c.out = out;
  c.x_next = x_next;
  c.u = u;
  c.rstd_post = rstd_post;
  c.rstd_next = rstd_next;
  return hip_status(launch_border(dt, c, static_cast<hipStream_t>(stream)));
}

size_t moe_norm_workspace_bytes(int T, int D) {
  return norm_sizes_ok(T, D) ? border_workspace_bytes(T, D) : 0;
}

moe_status_t moe_norm_backward(moe_dtype_t dt, const void* dx, const void* r, const void* gamma,
                               const float* rstd, const void* dresid, int T, int D, void* dr,
                               float* dgamma, void* workspace, size_t ws_bytes, void* stream) {
  if (!dtype_ok(dt) || !aligned16(dx) || !aligned16(r) || !aligned16(gamma) || !aligned4(rstd) ||
      !opt16(dresid) || !aligned16(dr) || !opt4(dgamma) || !aligned16(workspace))
    return MOE_EINVAL;
  if (!norm_sizes_ok(T, D)) return MOE_ESHAPE;
  if (ws_bytes < border_workspace_bytes(T, D)) return MOE_EWORKSPACE;
  BorderBwdCall c = {};
  c.dout = dresid;
  c.dx_next = dx;
  c.out = r;
  c.gamma_next = gamma;
  c.rstd_next = rstd;
  c.T = T;
  c.D = D;
  c.dresid = dr;
  c.dgamma_next = dgamma;
  c.partial = static_cast<float*>(workspace);
  return hip_status(launch_border_backward(dt, c, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_combine_norm_backward(moe_dtype_t dt, const void* dout, const void* dx_next,
                                       const void* u, const void* out, const float* gate,
                                       const void* gamma_post, const void* gamma_next,
                                       const float* rstd_post, const float* rstd_next,
                                       float scale, int T, int D, void* du, void* dresid,
                                       float* dgate, float* dgamma_post, float* dgamma_next,
                                       void* workspace, size_t ws_bytes, void* stream) {
  if (!dtype_ok(dt) || !opt16(dout) || !opt16(dx_next) || (!dout && !dx_next) || !opt4(gate) ||
      !opt16(gamma_post) || !aligned16(du) || !aligned16(dresid) || !opt4(dgate) ||
      !opt4(dgamma_post) || !opt4(dgamma_next) || !aligned16(workspace) || !isfinite(scale))
    return MOE_EINVAL;
  if (dx_next && (!aligned16(out) || !aligned16(gamma_next) || !aligned4(rstd_next)))
    return MOE_EINVAL;
  if (gamma_post ? !aligned4(rstd_post) : dgamma_post != nullptr) return MOE_EINVAL;
  if (!dx_next && dgamma_next) return MOE_EINVAL;
  // u is read for the norm after the block and for the gate's gradient
  if (!opt16(u) || ((gamma_post || dgate) && !u)) return MOE_EINVAL;
  if (!norm_sizes_ok(T, D)) return MOE_ESHAPE;
  if (ws_bytes < border_workspace_bytes(T, D)) return MOE_EWORKSPACE;
  BorderBwdCall c = {};
  c.dout = dout;
  c.dx_next = dx_next;
  c.u = u;
  c.out = out;
  c.gate = gate;
  c.gamma_post = gamma_post;
  c.gamma_next = gamma_next;
  c.rstd_post = rstd_post;
  c.rstd_next = rstd_next;
  c.scale = scale;
  c.T = T;
  c.D = D;
  c.block = true;
  c.du = du;
  c.dresid = dresid;
  c.dgate = dgate;
  c.dgamma_post = dgamma_post;
  c.dgamma_next = dgamma_next;
  c.partial = static_cast<float*>(workspace);
  return hip_status(launch_border_backward(dt, c, static_cast<hipStream_t>(stream)));
}

size_t moe_route_backward_workspace_bytes(moe_dtype_t dt, int T, int D, int E) {
  if (!dtype_ok(dt) || !route_bwd_sizes_ok(T, D, E)) return 0;
  return route_bwd_workspace_bytes(dt, T, D, E);
}

moe_status_t moe_route_backward(moe_dtype_t dt, const float* dtopk_w, const int32_t* topk_idx,
                                const float* logits, const void* x, const void* wg,
                                const float* dlogits_add, const void* dx_add, int T, int D,
                                int E, int k, int renorm, float* dlogits, void* dx, float* dwg,
                                float* dbias, void* workspace, size_t ws_bytes, void* stream) {
  if (!dtype_ok(dt) || !aligned4(dtopk_w) || !aligned4(topk_idx) || !aligned4(logits) ||
      !opt16(x) || !opt16(wg) || !opt4(dlogits_add) || !opt16(dx_add) || !aligned4(dlogits) ||
      !opt16(dx) || !opt16(dwg) || !opt4(dbias) || !aligned16(workspace))
    return MOE_EINVAL;
  if ((dx && !wg) || (dwg && !x)) return MOE_EINVAL;
  if (!route_bwd_sizes_ok(T, D, E) || k < 1 || k > E || k > kMaxK || !tk_ok(T, k))
    return MOE_ESHAPE;
  if (ws_bytes < route_bwd_workspace_bytes(dt, T, D, E)) return MOE_EWORKSPACE;
  const RouteBwdCall c = {dtopk_w, topk_idx, logits, x,  wg,  dlogits_add, dx_add, T, D, E, k,
                          renorm,  dlogits,  dx,     dwg, dbias, workspace};
  return hip_status(launch_route_backward(dt, c, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
