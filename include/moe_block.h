/*
 * moe_block.h - operators inside and around a whole expert block (moe.h): the layer for a few
 * tokens in three kernels, the norms, gate and residual at a block's border, the router's
 * backward. The conventions, status codes and types of moe.h hold for every call here.
 *
 *   decode     moe_norm -> moe_layer_few -> moe_combine_norm (its out as `shared`)
 *   training   forward   moe_norm -> moe_route -> moe_permute -> moe_grouped_fc1_swiglu
 *                          -> moe_grouped_fc2 -> moe_combine_norm (also the next block's norm)
 *              backward  moe_combine_norm_backward -> moe_combine_backward
 *                          -> moe_grouped_dgrad_swiglu, moe_grouped_dgrad_fc1, moe_grouped_wgrad
 *                          -> moe_combine (no weights) -> moe_route_backward (adds to its dx)
 *                          -> moe_norm_backward
 */
#ifndef MOE_MI355X_BLOCK_H
#define MOE_MI355X_BLOCK_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * moe_layer_few - the whole layer for T <= 32 tokens:
 *   h[t,j] = silu(x[t] w1[e]^T) * (x[t] w3[e]^T) for e = topk_idx[t,j], rounded to dt,
 *   out[t] = sum_j topk_w[t,j] * (h[t,j] w2[e]^T) + shared(x[t]),
 * float32 sums, one rounding of out (the rows y of moe_grouped_swiglu are not rounded on the
 * way, so out is a little closer to the formula than the chain of calls). Three kernels, or two with
 * the routing given.
 *   x [T,D]; w1, w3 [E,F,D]; w2 [E,D,F] (dt)
 *   wg [E,D] (dt) and bias [E] float32 or NULL: the routing is moe_route's, bit for bit, and
 *     topk_idx [T,k], topk_w [T,k] are outputs. wg NULL: they are inputs (renorm and bias are
 *     not looked at); a slot whose index lies outside [0, E) is skipped, and two slots of a
 *     token may hold one expert (their weights add).
 *   Fs > 0: shared experts as one, ws1, ws3 [Fs,D], ws2 [D,Fs] (dt), added unweighted. Fs = 0:
 *     none (the pointers are not looked at).
 *   -> out [T,D] (dt)
 * workspace: device scratch of at least moe_layer_few_workspace_bytes(dt, T, k, F, Fs) bytes,
 * 16-byte aligned, clobbered; calls that share it must not overlap. The inactive experts'
 * weights are not read. Equal calls give equal bits; a token's last bits may depend on which
 * others are in the call and on whether the call routes (the order of sums follows both).
 * T in [1, 32]; D, F, Fs multiples of 64 up to 65536; E and k as moe_route.
 * Errors: MOE_EINVAL, MOE_ESHAPE, MOE_EWORKSPACE, MOE_EHIP.
 *
 * moe_layer_few_mxfp4 - the same in bf16 with the routed experts' weights in MXFP4 (moe_mx.h):
 *   codes w1q, w3q [E,F,D/2], w2q [E,D,F/2], scales in MOE_MX_KSTEPS over the weights' rows; the
 *   weights' values enter the products exactly. D and F multiples of 128. The workspace is
 *   moe_layer_few_workspace_bytes(MOE_BF16, ...). Where many rows of h are wide (T*k*F*2 bytes past
 *   the 160 KiB of LDS) the calls of the masked layout (moe_grouped_swiglu_masked_mxfp4) are the
 *   faster ones from about 8 tokens: 8 experts of D = 4096, F = 14336, top-2, whole layers in us, this
 *   call and the masked chain, 4 tokens 109 and 119, 8 143 and 142, 16 187 and 162, 32 251 and 167.
 */
moe_status_t moe_layer_few(moe_dtype_t dt, const void* x, const void* wg, const float* bias,
                           int T, int D, int F, int E, int k, int renorm, const void* w1,
                           const void* w3, const void* w2, int Fs, const void* ws1,
                           const void* ws3, const void* ws2, int32_t* topk_idx, float* topk_w,
                           void* out, void* workspace, size_t ws_bytes, void* stream);
moe_status_t moe_layer_few_mxfp4(const void* x, const void* wg, const float* bias, int T, int D,
                                 int F, int E, int k, int renorm, const void* w1q,
                                 const void* w1s, const void* w3q, const void* w3s,
                                 const void* w2q, const void* w2s, int Fs, const void* ws1,
                                 const void* ws3, const void* ws2, int32_t* topk_idx,
                                 float* topk_w, void* out, void* workspace, size_t ws_bytes,
                                 void* stream);

/* Workspace bytes of the two calls above. Returns 0 on bad sizes. */
size_t moe_layer_few_workspace_bytes(moe_dtype_t dt, int T, int k, int F, int Fs);

/*
 * moe_norm - the norm before a block:
 *   r [T,D], gamma [D] (dt) -> x [T,D] (dt) = r * rstd * gamma,
 *   rstd [T] float32 (or NULL) = 1 / sqrt(mean_d r^2 + eps)
 * in float32 with one rounding of x. Only the mean of squares is taken (no mean is subtracted).
 *
 * moe_norm_backward - with rh = r * rstd:
 *   dr [T,D] (dt) = dresid + rstd * (dx gamma - rh * mean_d(dx gamma rh)),
 *   dgamma [D] float32 = sum_t dx rh, or NULL
 *   dresid [T,D] (dt) or NULL: the gradient that reaches r beside the norm, as on a residual
 *   stream.
 *
 * moe_combine_norm - the border of a block: combine, the norm after the block, its gate and
 * scale, the residual sum and the norm before the next block in one pass over the rows:
 *   u = sum_j topk_w[t,j] * y_perm[dst_row[t,j]] (+ shared[t])     as moe_combine
 *   z = u * rstd_post * gamma_post                                 (u without gamma_post)
 *   out = resid + scale * gate[t] * z                              (gate NULL: 1)
 *   x_next = out * rstd_next * gamma_next
 *   resid [T,D]; y_perm [m_cap,D], dst_row [T,k], topk_w [T,k] float32 or NULL (weights 1), or
 *   y_perm NULL: u = shared (T rows a caller has already, then needed); shared [T,D] or NULL;
 *   gate [T] float32 or NULL; gamma_post, gamma_next [D] (dt) or NULL
 *   -> out [T,D], x_next [T,D] (needed with gamma_next), and, each where not NULL, u [T,D] (dt),
 *      rstd_post [T], rstd_next [T] float32: what the backward reads. rstd_post is only taken with
 *      gamma_post, x_next and rstd_next only with gamma_next (else MOE_EINVAL).
 * Float32 between the reads and one rounding of each result (x_next is of out before its
 * rounding, z of u before its). Slots whose dst_row is outside [0, m_cap) are skipped. out may
 * be resid's buffer (in place); no other buffers may overlap.
 *
 * moe_combine_norm_backward - its backward, to u (the output gradient that moe_combine_backward
 * and moe_grouped_dgrad_swiglu_ckpt8's permute take, and the shared experts') and to resid:
 *   uh = u * rstd_post, oh = out * rstd_next,
 *   G = dout + rstd_next * (dx_next gamma_next - oh * mean_d(dx_next gamma_next oh)) -> dresid
 *   du = scale * gate * rstd_post * (gamma_post G - uh * mean_d(gamma_post G uh))
 *        (scale * gate * G without gamma_post)
 *   dgate [T] float32 = scale * sum_d G z; dgamma_post [D], dgamma_next [D] float32
 *   dout or dx_next may be NULL (not both): that gradient is zero. With dx_next: out, gamma_next,
 *   rstd_next. With gamma_post: rstd_post. dgate, dgamma_post and dgamma_next may be NULL.
 *
 * workspace of the backward calls: device scratch of at least moe_norm_workspace_bytes(T, D),
 * 16-byte aligned, clobbered; calls that share it must not overlap. The sums over tokens run in
 * a fixed order. eps > 0. D a multiple of 64 up to 16384; T in
 * [1, 2^30].
 * Errors: MOE_EINVAL (also eps or scale that is not finite), MOE_ESHAPE, MOE_ECAPACITY (m_cap),
 * MOE_EWORKSPACE, MOE_EHIP.
 */
moe_status_t moe_norm(moe_dtype_t dt, const void* r, const void* gamma, float eps, int T, int D,
                      void* x, float* rstd, void* stream);
moe_status_t moe_norm_backward(moe_dtype_t dt, const void* dx, const void* r, const void* gamma,
                               const float* rstd, const void* dresid, int T, int D, void* dr,
                               float* dgamma, void* workspace, size_t ws_bytes, void* stream);
moe_status_t moe_combine_norm(moe_dtype_t dt, const void* resid, const void* y_perm,
                              const int32_t* dst_row, const float* topk_w, const void* shared,
                              const float* gate, const void* gamma_post, const void* gamma_next,
                              float scale, float eps, int T, int D, int k, int64_t m_cap,
                              void* out, void* x_next, void* u, float* rstd_post,
                              float* rstd_next, void* stream);
moe_status_t moe_combine_norm_backward(moe_dtype_t dt, const void* dout, const void* dx_next,
                                       const void* u, const void* out, const float* gate,
                                       const void* gamma_post, const void* gamma_next,
                                       const float* rstd_post, const float* rstd_next,
                                       float scale, int T, int D, void* du, void* dresid,
                                       float* dgate, float* dgamma_post, float* dgamma_next,
                                       void* workspace, size_t ws_bytes, void* stream);

/* Workspace bytes of the two backward calls. Returns 0 on bad sizes. */
size_t moe_norm_workspace_bytes(int T, int D);

/*
 * moe_route_backward - the router's backward from the gradient of the top-k weights
 * (moe_combine_backward's dtopk_w). With p = softmax(logits) of moe_route's logits:
 *   renorm = 0: dl_e = p_e * (dp_e - sum_i p_i dp_i), dp_e = sum of dtopk_w over the token's
 *               slots that hold e
 *   renorm = 1: dl_e = sum over those slots of w_j * (dtopk_w_j - sum_i w_i dtopk_w_i), w the
 *               selected probabilities divided by their sum
 *   dlogits [T,E] float32 = dl + dlogits_add (the gradient of a loss on the logits; NULL: none)
 *   dx [T,D] (dt) = dlogits wg + dx_add (rounded once; dx_add [T,D] (dt) or NULL),
 *   dwg [E,D] float32 = dlogits^T x, dbias [E] float32 = sum_t dlogits
 * dx, dwg and dbias may be NULL: not computed. Slots whose index lies outside [0, E) are
 * skipped (of a token with no other dl is zero, whatever its logits are; its x must still be finite
 * for dwg); two slots of a token may hold one expert. Float32 sums in a fixed order; in bf16
 * dlogits enters dx as the sum of two bf16 values (2^-17 of its size is dropped, against dx's
 * own rounding of 2^-9) and dwg as that of three (nothing is dropped).
 *   dtopk_w [T,k] float32, topk_idx [T,k], logits [T,E] float32, x [T,D], wg [E,D] (dt)
 * workspace: device scratch of at least moe_route_backward_workspace_bytes(dt, T, D, E),
 * 16-byte aligned, clobbered; calls that share it must not overlap.
 * T*k in [1, 2^30]; D a multiple of 64 up to 65536; E in [1, 1024], k in [1, min(E, 32)].
 * Errors: MOE_EINVAL, MOE_ESHAPE, MOE_EWORKSPACE, MOE_EHIP.
 */
moe_status_t moe_route_backward(moe_dtype_t dt, const float* dtopk_w, const int32_t* topk_idx,
                                const float* logits, const void* x, const void* wg,
                                const float* dlogits_add, const void* dx_add, int T, int D,
                                int E, int k, int renorm, float* dlogits, void* dx, float* dwg,
                                float* dbias, void* workspace, size_t ws_bytes, void* stream);

/* Workspace bytes of moe_route_backward. Returns 0 on bad sizes. */
size_t moe_route_backward_workspace_bytes(moe_dtype_t dt, int T, int D, int E);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MI355X_BLOCK_H */
