/*
 * moe_layer.h -- C ABI of the operators around the expert block of
 * moe_lora.h, on B200 (sm_100a): the residual norm before and after a block,
 * the dense gated feed-forward block (a shared expert, or a layer without
 * routing) and dropout from a counter-based generator.
 *
 * The conventions are moe_lora.h's: device pointers, dense row-major tensors,
 * caller-owned buffers, no allocation, no synchronisation, all work enqueued
 * on `stream` of the current device, argument errors returned before anything
 * is launched, results the same from run to run.  An output may not overlap
 * an input except where a call says so.  Limits: 0 <= T <= 2^30 (T = 0
 * launches nothing but the zeros of weight gradients).
 *
 * Element types: MOE_DTYPE_*; all tensors of a call have the same one except
 * where a type is named.  Sums and statistics are fp32.
 */
#ifndef MOE_LAYER_H_
#define MOE_LAYER_H_

#include "moe_lora.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_DTYPE_BF16 0
#define MOE_DTYPE_FP16 1
#define MOE_DTYPE_FP32 2

/* ------------------------------------------------------------ residual norm
 * With x^ = x / sqrt(mean(x^2) + eps) over a row of H:
 *   b = y^ (w_offset + w_post)     b = y where w_post is NULL
 *   b = keep b / (1 - p)           dropout (below); none where p = 0
 *   r = res + scale gate b         res NULL: 0; gate NULL: 1
 *   n = r^ (w_offset + w_pre)      only with w_pre; from the unrounded r
 * y, res, r, n [T, H]; w_post, w_pre [H]; gate by gate_kind: [T], [H] or
 * [T, H]; stats fp32 [2, T]: 1 / sqrt(mean + eps) of y and of r, for the
 * backward (needed with w_post or w_pre).  r may be NULL when only n is
 * wanted; r may be y or res, n may be y or res.  1 <= H <= 16384, any
 * multiple of the element's size as the address (16-byte aligned tensors with H a multiple
 * of 8, of 4 for fp32, are read in 16-byte pieces).
 *
 * Backward, from dr (the gradient of r, NULL: 0) and dn (of n; given exactly
 * when w_pre is), the forward's y, r and stats, and its parameters:
 *   dres [T, H]  total gradient of r (= of res); may be NULL when dy is given
 *   dy   [T, H]  gradient of y; NULL for a call whose r is y itself (no
 *                w_post, gate, dropout or scale: dres is then y's gradient)
 *   dgate, dw_post, dw_pre: given exactly when gate, w_post, w_pre are, in
 *                their shapes; sums over rows are fp32, rounded once.
 *   ws           of moe_residual_norm_bwd_workspace_bytes, 4-byte aligned
 * dres and dy may be dr or dn. */
#define MOE_GATE_NONE 0
#define MOE_GATE_TOKEN 1
#define MOE_GATE_CHANNEL 2
#define MOE_GATE_ELEMENT 3
MOE_API moe_status_t moe_residual_norm_fwd(const void* y, const void* res, const void* w_post,
                                           const void* gate, int gate_kind, float scale,
                                           const void* w_pre, float w_offset, float eps, double p,
                                           const int64_t* rng, int T, int H, int dtype, void* r,
                                           void* n, float* stats, moe_stream_t stream);
MOE_API size_t moe_residual_norm_bwd_workspace_bytes(int T, int H, int dtype);
MOE_API moe_status_t moe_residual_norm_bwd(const void* dr, const void* dn, const void* y,
                                           const void* r, const float* stats, const void* w_post,
                                           const void* gate, int gate_kind, float scale,
                                           const void* w_pre, float w_offset, double p,
                                           const int64_t* rng, int T, int H, int dtype,
                                           void* dres, void* dy, void* dgate, void* dw_post,
                                           void* dw_pre, void* ws, size_t ws_bytes,
                                           moe_stream_t stream);

/* ---------------------------------------------------------------- dropout
 * out[t, c] = x[t, c] / (1 - p) where kept, else 0 (whatever x holds there);
 * the backward is the same call on the gradient with the same rng.
 *   rng  int64 [2] on the device: seed and offset.  The 32 random bits of
 *        (t, c) are word c % 4 of Philox4x32-10 at counter (c / 4, t, low and
 *        high word of offset) and key (low and high word of seed); kept where
 *        they are at least round(p 2^32).  The caller changes seed or offset
 *        between draws that must differ (in place, also between replays of a
 *        captured graph).
 * 0 <= p <= 1; x, out [T, H], out may be x; 1 <= H <= 2^30. */
MOE_API moe_status_t moe_dropout(const void* x, int T, int H, int dtype, double p,
                                 const int64_t* rng, void* out, moe_stream_t stream);

/* -------------------------------------------------------------- gated FFN
 *   [g | u] = X W1^T,  h = act(g) u,  Y = add + h W2^T      (add NULL: 0)
 * X, Y, add [T, H]; W1 [2I, H] (gate rows first, as one expert of gate_up);
 * W2 [H, I]; bf16 or fp16; H and I multiples of 16 and >= 64; all pointers
 * 16-byte aligned.  Y may be add.  act: silu, or gelu in its tanh form.
 * h and dZ (below) are rounded to the element type between the products, as
 * the tensor cores' operands; g, u and all sums are kept in fp32.  In fp16 a
 * value of h or dZ past 65504 becomes infinite, and what is summed from it
 * infinite or NaN: its row of Y or dX, its column of dW2 or row of dW1.  The
 * other rows are not affected.
 *   saved  of moe_ffn_saved_bytes: g, u and h for the backward; NULL for
 *          inference, which then needs ws of moe_ffn_workspace_bytes.
 * Backward: dX = add + dZ W1 with dZ = [dh u act'(g) | dh act(g)], dh = dY W2; dW1 [2I, H] = dZ^T X and dW2 [H, I] = dY^T h
 * both given, or both NULL for frozen weights; dX may be add; ws of
 * moe_ffn_workspace_bytes. */
#define MOE_ACT_SILU 0
#define MOE_ACT_GELU_TANH 1
MOE_API size_t moe_ffn_saved_bytes(int T, int H, int I);
MOE_API size_t moe_ffn_workspace_bytes(int T, int H, int I);
/* Which kernel a product of a call with these sizes runs on (host-side, no GPU
 * needed; need_dw: a backward with dW1 and dW2): MOE_FFN_TOKENS, _PAIRS or
 * _PAIRS_MERGED (dX, dW1 and dW2 in one launch), else 16 n + s for 128 x n
 * tiles with K split over a cluster of s CTAs; -1: no such product. */
#define MOE_FFN_GATE_UP 0
#define MOE_FFN_DOWN 1
#define MOE_FFN_DH 2
#define MOE_FFN_DX 3
#define MOE_FFN_DW1 4
#define MOE_FFN_DW2 5
#define MOE_FFN_TOKENS 0
#define MOE_FFN_PAIRS 1
#define MOE_FFN_PAIRS_MERGED 2
MOE_API int moe_ffn_kernel(int T, int H, int I, int product, int need_dw);
MOE_API moe_status_t moe_ffn_fwd(const void* X, const void* W1, const void* W2, int T, int H,
                                 int I, int dtype, int act, const void* add, void* Y, void* saved,
                                 size_t saved_bytes, void* ws, size_t ws_bytes,
                                 moe_stream_t stream);
MOE_API moe_status_t moe_ffn_bwd(const void* dY, const void* X, const void* W1, const void* W2,
                                 int T, int H, int I, int dtype, int act, const void* saved,
                                 size_t saved_bytes, const void* add, void* dX, void* dW1,
                                 void* dW2, void* ws, size_t ws_bytes, moe_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_LAYER_H_ */
