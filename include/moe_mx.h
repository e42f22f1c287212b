/*
 * moe_mx.h - block-scaled operators of the MoE expert layer (moe.h): 4-bit weights and
 * payload, and 8-bit checkpoints of fc1's pre-activations. The conventions, status codes
 * and types of moe.h hold for every call here.
 *
 *   prefill with 4-bit weights:
 *     moe_route -> moe_quantize_mxfp4 (x) -> moe_permute_mxfp4
 *       -> moe_grouped_fc1_swiglu_mxfp4 -> moe_quantize_mxfp4 (h) -> moe_grouped_fc2_mxfp4
 *       -> moe_combine
 *   decode with 4-bit weights:
 *     moe_route -> moe_permute_masked -> moe_grouped_swiglu_masked_mxfp4 -> moe_combine
 *   training with an 8-bit checkpoint:
 *     forward   moe_route -> moe_permute -> moe_grouped_fc1_swiglu_ckpt8
 *                 -> moe_grouped_fc2 -> moe_combine
 *     backward  moe_permute (dout) -> moe_grouped_dgrad_swiglu_ckpt8
 *                 -> moe_grouped_dgrad_fc1 -> moe_permute (x)
 *                 -> moe_grouped_wgrad twice -> moe_combine
 *
 * Formats. Both share one power of two 2^X per 32 consecutive values of a row, stored as
 * the byte X + 127 (E8M0). X is the smallest integer >= -127 with max|v| <= L * 2^X over the
 * block, L the format's largest value, so nothing saturates; X = -127 for a block of zeros.
 *   MXFP4  codes in E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives, L = 6), two a
 *          byte, the element of even index in the low half: rows of C/2 bytes
 *   MXFP8  codes in OCP E4M3 (L = 448), one a byte: rows of C bytes
 * A code is v / 2^X rounded to nearest, ties to the even code; the sign is kept, -0 included.
 * A block that holds an infinity or a NaN gets the byte 255 (E8M0's NaN) and zero codes, and
 * whatever reads it gives NaN. Scales lie in rows or in k-step words (moe_mx_layout_t).
 */
#ifndef MOE_MI355X_MX_H
#define MOE_MI355X_MX_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * moe_quantize_mxfp4 - rows to MXFP4.
 *   x [R,C] (dt) -> q [R,C/2] codes, scales in `layout`
 *   (MOE_MX_ROWS: C a multiple of 32; MOE_MX_KSTEPS: C a multiple of 128, scales 4-byte
 *   aligned; C <= 65536, R <= 2^31). Used with MOE_MX_ROWS for token rows before the
 *   permute, with MOE_MX_KSTEPS for h and, once, for weights (R = E*F rows of D values, or
 *   E*D rows of F).
 * moe_dequantize_mxfp4 / moe_dequantize_mxfp8 - the values of MXFP4 / MXFP8 rows, the same
 *   sizes: q, scales -> out [R,C] (dt), rounded once to dt (only bf16 values below 2^-126
 *   are rounded at all; a value past the largest finite one is an infinity).
 * Errors: MOE_EINVAL (also an unknown layout), MOE_ESHAPE, MOE_EHIP.
 */
moe_status_t moe_quantize_mxfp4(moe_dtype_t dt, const void* x, int64_t R, int C, void* q,
                                void* scales, moe_mx_layout_t layout, void* stream);
moe_status_t moe_dequantize_mxfp4(moe_dtype_t dt, const void* q, const void* scales, int64_t R,
                                  int C, moe_mx_layout_t layout, void* out, void* stream);
moe_status_t moe_dequantize_mxfp8(moe_dtype_t dt, const void* q, const void* scales, int64_t R,
                                  int C, moe_mx_layout_t layout, void* out, void* stream);

/*
 * moe_permute_mxfp4 - moe_permute_mxfp8 for 4-bit rows: moe_permute's metadata, the code rows
 * of xq [T,D/2] copied to xq_perm [m_cap,D/2], the scales xs [T,D/32] (MOE_MX_ROWS) gathered
 * into xs_perm in MOE_MX_KSTEPS over m_cap rows; zero bytes in pad rows; rows at or past
 * offsets[E] are not written. D a multiple of 128.
 * Errors: MOE_EINVAL, MOE_ESHAPE, MOE_ECAPACITY, MOE_EWORKSPACE, MOE_EHIP.
 */
moe_status_t moe_permute_mxfp4(const void* xq, const void* xs, const int32_t* topk_idx, int T,
                               int D, int E, int k, int m_tile, int64_t m_cap, void* xq_perm,
                               void* xs_perm, int32_t* counts, int32_t* offsets,
                               int32_t* dst_row, int32_t* src_row, int32_t* tile_expert,
                               void* workspace, size_t ws_bytes, int32_t* dev_err,
                               void* stream);

/*
 * moe_grouped_fc1_swiglu_mxfp4 / moe_grouped_fc2_mxfp4 - the two grouped products on MXFP4
 * rows and weights (the scaled FP4 MFMA, float32 sums, bf16 results):
 *   fc1: xq_perm [m_cap,D/2], w1q, w3q [E,F,D/2]
 *        -> h [m_cap,F] = silu(x w1[e]^T) * (x w3[e]^T) per segment row
 *   fc2: hq [m_cap,F/2], w2q [E,D,F/2] -> y_perm [m_cap,D] = h w2[e]^T per segment row
 * Scales in MOE_MX_KSTEPS, 16-byte aligned: the rows' over m_cap rows, the weights' over their
 * E*F (fc2: E*D) rows. Segments, counts, tile_expert, m_tile and the optional workspace as
 * moe_grouped_swiglu: with counts, pad rows are not read and give exact zeros; rows at or
 * past offsets[E] are neither read nor written. fc1: D a multiple of 128, F of 64; fc2: F a
 * multiple of 128, D of 64; D*F < 2^31. Every m_tile.
 * Errors: MOE_EINVAL, MOE_ESHAPE, MOE_ECAPACITY, MOE_EHIP.
 */
moe_status_t moe_grouped_fc1_swiglu_mxfp4(const void* xq_perm, const void* xs_perm,
                                          const int32_t* offsets, const int32_t* counts,
                                          const int32_t* tile_expert, int E, int D, int F,
                                          int m_tile, int64_t m_cap, const void* w1q,
                                          const void* w1s, const void* w3q, const void* w3s,
                                          void* h, void* workspace, size_t ws_bytes,
                                          void* stream);
moe_status_t moe_grouped_fc2_mxfp4(const void* hq, const void* hs, const int32_t* offsets,
                                   const int32_t* counts, const int32_t* tile_expert, int E,
                                   int D, int F, int m_tile, int64_t m_cap, const void* w2q,
                                   const void* w2s, void* y_perm, void* workspace,
                                   size_t ws_bytes, void* stream);

/*
 * moe_grouped_swiglu_masked_mxfp4 - moe_grouped_swiglu_masked with MXFP4 weights and bf16
 * rows: for rows [e*cap, e*cap + min(counts[e], cap)) of every expert e
 *   h = silu(x w1[e]^T) * (x w3[e]^T) rounded to bf16, y = h w2[e]^T rounded to bf16,
 * float32 sums; the other rows of x_masked, h and y are neither read nor written, and an
 * expert without rows has none of its weights read. The weights' values enter the products
 * exactly (a 4-bit code times a power of two is a bf16 value). Each 64 rows of a slab read
 * the weights once. Calls with few rows in all sum over k in two halves, so a row's last bits
 * may depend on how many other rows there are; equal calls give equal bits.
 *   x_masked [E*cap,D], w1q, w3q [E,F,D/2], w2q [E,D,F/2], scales in MOE_MX_KSTEPS over the
 *   weights' rows -> h [E*cap,F], y [E*cap,D].
 * D and F multiples of 128, D*F < 2^31; cap a multiple of 16, at most 65536, E*cap < 2^31.
 * Errors: MOE_EINVAL, MOE_ESHAPE, MOE_ECAPACITY (cap), MOE_EHIP.
 */
moe_status_t moe_grouped_swiglu_masked_mxfp4(const void* x_masked, const int32_t* counts, int E,
                                             int D, int F, int cap, const void* w1q,
                                             const void* w1s, const void* w3q, const void* w3s,
                                             const void* w2q, const void* w2s, void* h, void* y,
                                             void* stream);

/*
 * moe_grouped_fc1_swiglu_ckpt8 - moe_grouped_fc1_swiglu (bf16) that keeps the
 * pre-activations for the backward as MXFP8 in place of bf16:
 *   -> h [m_cap,F] bf16, bit for bit what moe_grouped_fc1_swiglu with ab gives, both without a
 *                    workspace (with one the two calls may cut different tiles over k:
 *                    another order of sums; without ab a decode-sized call sums otherwise too)
 *      ab_codes [m_cap,2F] e4m3 codes of [a | b], ab_scales [m_cap,2F/32] bytes
 *                    (4-byte aligned)
 * Blocks are 32 consecutive columns of a or of b, quantised from the float32 sums. Pad rows
 * give exact zeros. Per row 2F*33/32 bytes in place of 4F. Arguments otherwise, workspace
 * and errors as moe_grouped_fc1_swiglu.
 */
moe_status_t moe_grouped_fc1_swiglu_ckpt8(const void* x_perm, const int32_t* offsets,
                                          const int32_t* counts, const int32_t* tile_expert,
                                          int E, int D, int F, int m_tile, int64_t m_cap,
                                          const void* w1, const void* w3, void* h,
                                          void* ab_codes, void* ab_scales, void* workspace,
                                          size_t ws_bytes, void* stream);

/*
 * moe_grouped_dgrad_swiglu_ckpt8 - the backward of combine, fc2 and silu(a)*b from that
 * checkpoint, which needs neither h nor y_perm of the forward. With a, b the checkpoint's
 * values, w the row's top-k weight (topk_w[src_row[row]]; topk_w NULL: 1) and
 * u = dout_perm w2[e] (float32, not rounded):
 *   dout_perm [m_cap,D] bf16: the output gradient moved to the permuted rows, unweighted
 *                    (moe_permute of dout with the forward's routing)
 *   -> dab [m_cap,2F] = [w*u*b*silu'(a) | w*u*silu(a)], for moe_grouped_dgrad_fc1 and the
 *                    wgrad of w1 and w3
 *      hw [m_cap,F]  = w*silu(a)*b, for the wgrad of w2: dW2 = dout_perm^T hw
 *      dtopk_w [T,k] float32 = sum over F of u*silu(a)*b of the slot's row (dst_row), 0 for
 *                    slots without a row; NULL: not computed
 * each rounded once to its type. The sums over F run in a fixed order. Pad rows give exact
 * zeros; rows at or past offsets[E] are neither read nor written.
 * src_row [m_cap], dst_row [T,k] as moe_permute writes them; T and k give topk_w's and
 * dtopk_w's size. topk_w needs src_row; dtopk_w needs topk_w, dst_row and `scratch`; without
 * topk_w all of these may be NULL (T and k are then not looked at). scratch: device memory
 * of at least moe_ckpt8_scratch_bytes(F, m_cap), 16-byte aligned, clobbered; calls
 * that share it or the workspace must not overlap.
 * Sizes, m_tile and workspace as moe_grouped_swiglu.
 * Errors: MOE_EINVAL, MOE_ESHAPE, MOE_ECAPACITY, MOE_EWORKSPACE (scratch), MOE_EHIP.
 */
moe_status_t moe_grouped_dgrad_swiglu_ckpt8(const void* dout_perm, const int32_t* offsets,
                                            const int32_t* counts, const int32_t* tile_expert,
                                            int E, int D, int F, int m_tile, int64_t m_cap,
                                            const void* w2, const void* ab_codes,
                                            const void* ab_scales, const int32_t* src_row,
                                            const int32_t* dst_row, const float* topk_w, int T,
                                            int k, void* dab, void* hw, float* dtopk_w,
                                            void* scratch, size_t scratch_bytes,
                                            void* workspace, size_t ws_bytes, void* stream);

/* Scratch bytes of moe_grouped_dgrad_swiglu_ckpt8 with dtopk_w. Returns 0 on bad sizes. */
size_t moe_ckpt8_scratch_bytes(int F, int64_t m_cap);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MI355X_MX_H */
