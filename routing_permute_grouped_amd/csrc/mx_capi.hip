// C ABI entry points of moe_mx.h: host-side validation, then the kernel launchers.
// Every check runs before any HIP call, so a rejected call never touches the GPU.
#include <hip/hip_runtime.h>

#include "moe_mx.h"
#include "checks.hpp"

using namespace moe;

namespace {

// sizes of [R, C] block-scaled rows under a scale layout
moe_status_t mx_rows_ok(int64_t R, int C, moe_mx_layout_t layout, const void* scales) {
  if (layout != MOE_MX_ROWS && layout != MOE_MX_KSTEPS) return MOE_EINVAL;
  if (!scales || (layout == MOE_MX_KSTEPS && !aligned4(scales))) return MOE_EINVAL;
  if (R < 1 || C < 32 || C % 32 != 0 || C > kMaxDim || R > ((int64_t)1 << 31)) return MOE_ESHAPE;
  if (layout == MOE_MX_KSTEPS && C % 128 != 0) return MOE_ESHAPE;
  return MOE_OK;
}

// what the grouped calls share: segment metadata, workspace, sizes
moe_status_t segments_ok(const int32_t* offsets, const int32_t* counts,
                         const int32_t* tile_expert, int E, int D, int F, int m_tile,
                         int64_t m_cap, const void* workspace) {
  if (!aligned4(offsets) || !aligned4(tile_expert) || (counts && !aligned4(counts)))
    return MOE_EINVAL;
  if (workspace && !aligned16(workspace)) return MOE_EINVAL;
  if (E < 1 || E > kMaxExperts || !dim_ok(D) || !dim_ok(F) || !mtile_ok(m_tile)) return MOE_ESHAPE;
  if ((int64_t)D * F >= ((int64_t)1 << 31)) return MOE_ESHAPE;
  if (m_cap < 1 || m_cap % m_tile != 0 || m_cap > INT32_MAX) return MOE_ECAPACITY;
  return MOE_OK;
}

moe_status_t dequantize(bool fp4, moe_dtype_t dt, const void* q, const void* scales, int64_t R,
                        int C, moe_mx_layout_t layout, void* out, void* stream) {
  if (!dtype_ok(dt) || !aligned16(q) || !aligned16(out)) return MOE_EINVAL;
  const moe_status_t st = mx_rows_ok(R, C, layout, scales);
  if (st != MOE_OK) return st;
  return hip_status(launch_dequantize_mx(dt, fp4, q, scales, R, C, layout == MOE_MX_KSTEPS, out,
                                         static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

moe_status_t moe_quantize_mxfp4(moe_dtype_t dt, const void* x, int64_t R, int C, void* q,
                                void* scales, moe_mx_layout_t layout, void* stream) {
  if (!dtype_ok(dt) || !aligned16(x) || !aligned16(q)) return MOE_EINVAL;
  const moe_status_t st = mx_rows_ok(R, C, layout, scales);
  if (st != MOE_OK) return st;
  return hip_status(launch_quantize_mx4(dt, x, R, C, q, scales, layout == MOE_MX_KSTEPS,
                                        static_cast<hipStream_t>(stream)));
}

moe_status_t moe_dequantize_mxfp4(moe_dtype_t dt, const void* q, const void* scales, int64_t R,
                                  int C, moe_mx_layout_t layout, void* out, void* stream) {
  return dequantize(true, dt, q, scales, R, C, layout, out, stream);
}

moe_status_t moe_dequantize_mxfp8(moe_dtype_t dt, const void* q, const void* scales, int64_t R,
                                  int C, moe_mx_layout_t layout, void* out, void* stream) {
  return dequantize(false, dt, q, scales, R, C, layout, out, stream);
}

moe_status_t moe_permute_mxfp4(const void* xq, const void* xs, const int32_t* topk_idx, int T,
                               int D, int E, int k, int m_tile, int64_t m_cap, void* xq_perm,
                               void* xs_perm, int32_t* counts, int32_t* offsets,
                               int32_t* dst_row, int32_t* src_row, int32_t* tile_expert,
                               void* workspace, size_t ws_bytes, int32_t* dev_err,
                               void* stream) {
  if (!aligned16(xq) || !aligned4(xs) || !aligned16(xq_perm) || !aligned4(xs_perm) ||
      !aligned4(topk_idx) || !aligned4(counts) || !aligned4(offsets) || !aligned4(dst_row) ||
      !aligned4(src_row) || !aligned4(tile_expert) || !aligned4(workspace) || !aligned4(dev_err))
    return MOE_EINVAL;
  if (!tk_ok(T, k) || !dim_ok(D) || D % 128 != 0 || E < 1 || E > kMaxExperts || k < 1 || k > E ||
      k > kMaxK || !mtile_ok(m_tile))
    return MOE_ESHAPE;
  const int64_t need = moe_capacity(T, k, E, m_tile);
  if (m_cap < need || m_cap % m_tile != 0 || m_cap > INT32_MAX) return MOE_ECAPACITY;
  if (ws_bytes < permute_workspace_bytes(T, k, E)) return MOE_EWORKSPACE;
  return hip_status(launch_permute_mx(4, xq, xs, topk_idx, T, D, E, k, m_tile, m_cap, xq_perm,
                                      xs_perm, counts, offsets, dst_row, src_row, tile_expert,
                                      workspace, dev_err, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_grouped_fc1_swiglu_mxfp4(const void* xq_perm, const void* xs_perm,
                                          const int32_t* offsets, const int32_t* counts,
                                          const int32_t* tile_expert, int E, int D, int F,
                                          int m_tile, int64_t m_cap, const void* w1q,
                                          const void* w1s, const void* w3q, const void* w3s,
                                          void* h, void* workspace, size_t ws_bytes,
                                          void* stream) {
  if (!aligned16(xq_perm) || !aligned16(xs_perm) || !aligned16(w1q) || !aligned16(w1s) ||
      !aligned16(w3q) || !aligned16(w3s) || !aligned16(h))
    return MOE_EINVAL;
  const moe_status_t st =
      segments_ok(offsets, counts, tile_expert, E, D, F, m_tile, m_cap, workspace);
  if (st != MOE_OK) return st;
  if (D % 128 != 0) return MOE_ESHAPE;
  if (!workspace) ws_bytes = 0;
  return hip_status(launch_grouped_mx4(true, xq_perm, xs_perm, offsets, counts, E, D, F, m_cap,
                                       w1q, w1s, w3q, w3s, h, ws_bytes ? workspace : nullptr,
                                       ws_bytes, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_grouped_fc2_mxfp4(const void* hq, const void* hs, const int32_t* offsets,
                                   const int32_t* counts, const int32_t* tile_expert, int E,
                                   int D, int F, int m_tile, int64_t m_cap, const void* w2q,
                                   const void* w2s, void* y_perm, void* workspace,
                                   size_t ws_bytes, void* stream) {
  if (!aligned16(hq) || !aligned16(hs) || !aligned16(w2q) || !aligned16(w2s) || !aligned16(y_perm))
    return MOE_EINVAL;
  const moe_status_t st =
      segments_ok(offsets, counts, tile_expert, E, D, F, m_tile, m_cap, workspace);
  if (st != MOE_OK) return st;
  if (F % 128 != 0) return MOE_ESHAPE;
  if (!workspace) ws_bytes = 0;
  return hip_status(launch_grouped_mx4(false, hq, hs, offsets, counts, E, F, D, m_cap, w2q, w2s,
                                       w2q, w2s, y_perm, ws_bytes ? workspace : nullptr, ws_bytes,
                                       static_cast<hipStream_t>(stream)));
}

moe_status_t moe_grouped_swiglu_masked_mxfp4(const void* x_masked, const int32_t* counts, int E,
                                             int D, int F, int cap, const void* w1q,
                                             const void* w1s, const void* w3q, const void* w3s,
                                             const void* w2q, const void* w2s, void* h, void* y,
                                             void* stream) {
  if (!aligned16(x_masked) || !aligned4(counts) || !aligned16(w1q) || !aligned4(w1s) ||
      !aligned16(w3q) || !aligned4(w3s) || !aligned16(w2q) || !aligned4(w2s) || !aligned16(h) ||
      !aligned16(y))
    return MOE_EINVAL;
  if (E < 1 || E > kMaxExperts || !dim_ok(D) || D % 128 != 0 || !dim_ok(F) || F % 128 != 0)
    return MOE_ESHAPE;
  if ((int64_t)D * F >= ((int64_t)1 << 31)) return MOE_ESHAPE;
  if (!cap_ok(E, cap) || cap > 65536) return MOE_ECAPACITY;
  return hip_status(launch_decode_mx4(x_masked, counts, E, D, F, cap, w1q, w1s, w3q, w3s, w2q,
                                      w2s, h, y, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_grouped_fc1_swiglu_ckpt8(const void* x_perm, const int32_t* offsets,
                                          const int32_t* counts, const int32_t* tile_expert,
                                          int E, int D, int F, int m_tile, int64_t m_cap,
                                          const void* w1, const void* w3, void* h,
                                          void* ab_codes, void* ab_scales, void* workspace,
                                          size_t ws_bytes, void* stream) {
  if (!aligned16(x_perm) || !aligned16(w1) || !aligned16(w3) || !aligned16(h) ||
      !aligned16(ab_codes) || !aligned4(ab_scales))
    return MOE_EINVAL;
  const moe_status_t st =
      segments_ok(offsets, counts, tile_expert, E, D, F, m_tile, m_cap, workspace);
  if (st != MOE_OK) return st;
  if (!workspace) ws_bytes = 0;
  return hip_status(launch_grouped_fc1_ckpt8(x_perm, offsets, counts, E, D, F, m_cap, w1, w3, h,
                                             ab_codes, ab_scales, ws_bytes ? workspace : nullptr,
                                             ws_bytes, static_cast<hipStream_t>(stream)));
}

size_t moe_ckpt8_scratch_bytes(int F, int64_t m_cap) {
  if (!dim_ok(F) || m_cap < 1 || m_cap > INT32_MAX) return 0;
  return ckpt8_scratch_bytes(F, m_cap);
}

moe_status_t moe_grouped_dgrad_swiglu_ckpt8(const void* dout_perm, const int32_t* offsets,
                                            const int32_t* counts, const int32_t* tile_expert,
                                            int E, int D, int F, int m_tile, int64_t m_cap,
                                            const void* w2, const void* ab_codes,
                                            const void* ab_scales, const int32_t* src_row,
                                            const int32_t* dst_row, const float* topk_w, int T,
                                            int k, void* dab, void* hw, float* dtopk_w,
                                            void* scratch, size_t scratch_bytes,
                                            void* workspace, size_t ws_bytes, void* stream) {
  if (!aligned16(dout_perm) || !aligned16(w2) || !aligned16(ab_codes) ||
      !aligned4(ab_scales) || !aligned16(dab) || !aligned16(hw))
    return MOE_EINVAL;
  if (topk_w && (!aligned4(topk_w) || !aligned4(src_row))) return MOE_EINVAL;
  if (dtopk_w &&
      (!topk_w || !aligned4(dtopk_w) || !aligned4(dst_row) || !aligned16(scratch)))
    return MOE_EINVAL;
  const moe_status_t st =
      segments_ok(offsets, counts, tile_expert, E, D, F, m_tile, m_cap, workspace);
  if (st != MOE_OK) return st;
  if (topk_w && (!tk_ok(T, k) || k < 1 || k > kMaxK)) return MOE_ESHAPE;
  if (dtopk_w && scratch_bytes < ckpt8_scratch_bytes(F, m_cap)) return MOE_EWORKSPACE;
  if (!workspace) ws_bytes = 0;
  return hip_status(launch_grouped_dgrad_ckpt8(
      dout_perm, offsets, counts, E, D, F, m_cap, w2, ab_codes, ab_scales, src_row, dst_row,
      topk_w, topk_w ? T * k : 0, dab, hw, dtopk_w, scratch, ws_bytes ? workspace : nullptr,
      ws_bytes, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
