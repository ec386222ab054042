/*
 * wqmlp_blocks.h -- C ABI of libwqmlp, third part: blocks with 4-bit weights and what stands around them.  The
 * linear with AWQ int4 group-32 weights and the gradient through it, a whole mixture-of-experts layer for a few
 * tokens, and the norms before and after a block with its gate and residual, forward and backward.
 *
 * The conventions of wqmlp.h hold for every call here: device pointers of the current device, 16-byte
 * aligned, dense row-major; nothing is allocated or synchronised and every call can be captured into a
 * hipGraph; argument errors are found before anything is enqueued; the same return codes.  Calls that may
 * run at the same time (streams, threads, captured graphs) need workspaces of their own.  Sums are float32
 * (float64 where said) in an order fixed by the shape, so a call's results are reproducible bit for bit.
 */
#ifndef WQMLP_BLOCKS_H
#define WQMLP_BLOCKS_H

#include "wqmlp.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Linear with AWQ int4 group-32 weights:
 *   y[m,n] = sum_k x[m,k] dq[n,k],   dq = RN_f16(fma(q, scale, RN_f16(-zero * scale))) as in moe_awq_m1_run
 *   x     [M, K]  WQ_F32, WQ_BF16 or WQ_F16
 *   bank          one expert's [N, K] weights: awq_pack_bank / awq_bank_bytes with E = 1 (an expert of a larger
 *                 bank starts at a multiple of awq_bank_bytes(1, N, K, meta_layout)); meta_layout 3 or 4
 *   y     [M, N]  float32
 * K: a multiple of 32; N and M: any.  The products are exact in float32 and summed there: weights are float16
 * values, float16 x enters as it is, bfloat16 and float32 rows (or pieces of 512 and 1024 k of them) are scaled by a power
 * of two so that their largest finite magnitude lies in [2^14, 2^15) and enter as one (bfloat16) or two (float32) float16 terms: a
 * bfloat16 element is off by at most 2^-39 of its row's largest, a float32 one by 2^-22 of itself or 2^-39 of its
 * row's largest, whichever is more.  A row's result does not depend on the other rows' values; NaN and infinities
 * stay in their row.  Weights have to decode to finite values: an infinite one may make NaN of its results.  M == 0 is a valid
 * empty call.
 */
size_t awq_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int x_dtype);
int awq_linear_run(int64_t M, int64_t N, int64_t K, const void* x, int x_dtype, const void* bank, int meta_layout,
                   void* workspace, size_t workspace_bytes, float* y, void* stream);

/*
 * The gradient of awq_linear_run with respect to its input, through the frozen packed weights:
 *   dx[m,k] = sum_n dy[m,n] dq[n,k]
 * dy [M,N]: WQ_F32 or WQ_BF16; dx [M,K]: dx_dtype, WQ_F32 or WQ_BF16; bank and meta_layout as above.  K: a
 * multiple of 32; N and M: any.  Numerics as for qlinear_backward: each row of dy is scaled by a power of two so that
 * its largest finite magnitude lies in [2^14, 2^15) and enters float16 MFMAs.  bfloat16 dy: one float16 term, off
 * by at most 2^-39 of the row's largest.  float32 dy into a float32 dx: two terms, 2^-22 of the element or 2^-51 of the
 * row's largest; into a bfloat16 dx: rounded once to float16, 2^-11 of the element (dx's own rounding is 2^-8) or 2^-39
 * of the row's largest.  NaN and infinities of dy stay in their row.  M == 0 is a valid empty call.
 */
size_t awq_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K, int dy_dtype, int dx_dtype);
int awq_linear_backward(int64_t M, int64_t N, int64_t K, const void* dy, int dy_dtype, const void* bank, int meta_layout,
                        void* workspace, size_t workspace_bytes, void* dx, int dx_dtype, void* stream);

/*
 * A mixture-of-experts layer with AWQ int4 group-32 experts for M tokens at once (moe_awq_m1_run is its step for
 * one token and ready-made ids, in float16):
 *   logits[m,e] = RN_f32(sum_h x[m,h] router[e,h]), summed in float64
 *   ids[m,:]    the topk largest logits, largest first; equal ones by the lower index; NaN below all others
 *   weights     softmax of the chosen logits (flags with WQ_MOE_RENORM) or their share in the softmax of all E
 *   out[m,o]  = sum over k, in order, of weights[m,k] * sum_i act[m,k,i] dq2[e][o,i],  e = ids[m,k]
 *   act[m,k,i] = silu(g) * u,  g = sum_h x[m,h] dq13[e][i,h],  u = the same with row i + I
 *   x       [M, H]    WQ_F32, WQ_BF16 or WQ_F16
 *   router  [E, H]    router_dtype (any of the three); NULL: ids and weights are inputs (flags is then 0), where an
 *                     id outside [0, E) contributes nothing and repeated ids keep their weights
 *   ids, weights [M, topk]  int32, float32
 *   w13_bank, w2_bank as for moe_awq_m1_run; meta_layout 3 or 4
 *   out     [M, H]    out_dtype (any of the three), rounded once
 * 0 <= M <= WQ_MOE_MAX_TOKENS, 1 <= topk <= min(E, WQ_MOE_MAX_TOPK) (given ids: topk may exceed E), H and I
 * multiples of 32 up to WQ_MOE_MAX_WIDTH.  Numerics as for awq_linear_run: products and sums are float32, float32 x and
 * act enter as two float16 terms; no intermediate is rounded to 16 bits (moe_awq_m1_run rounds g, u, act and each route's
 * result to float16).  A token's result is the same bits whatever the other tokens are and however many.  Where x holds an
 * infinity or NaN its row's ids are those of the order above, and its out may be NaN.  An expert is read from HBM once for
 * all of its tokens; more tokens than a pass holds (at most 16) read it again through the caches.
 */
#define WQ_MOE_MAX_TOKENS 256
#define WQ_MOE_MAX_WIDTH 16384
enum { WQ_MOE_RENORM = 1 };
size_t moe_awq_workspace_bytes(int64_t M, int64_t E, int64_t topk, int64_t H, int64_t I);
int moe_awq_run(int64_t M, int64_t E, int64_t topk, int64_t H, int64_t I, const void* x, int x_dtype, const void* router,
                int router_dtype, int32_t* ids, float* weights, const void* w13_bank, const void* w2_bank, int meta_layout,
                void* workspace, size_t workspace_bytes, void* out, int out_dtype, int flags, void* stream);

/*
 * What stands between one block (an MLP, say) and the next: the norm of the block's result, its gate and
 * residual scale, the residual stream and the norm before the next block, row by row:
 *   norm(t; w)[m,i] = t[m,i] / sqrt(mean_i t[m,i]^2 + eps) * (offset + w[i])
 *   p = norm(y; post), or y where post is NULL
 *   h_out[m,i] = h[m,i] + alpha * gate[m / (M/G), i] * p[m,i]         (h itself where y is NULL)
 *   x[m,i] = norm(h_out; pre), of h_out as it is stored (rounded to h_dtype)
 *   h, h_out [M, H]  h_dtype: the residual stream; h_out may be h itself, and is NULL where y is
 *   y        [M, H]  y_dtype: the block's result, or NULL (only the norm before a block)
 *   post, pre [H]    w_dtype: the norms' weights (offset 1: weights stored as their distance from one); pre NULL:
 *                    no second norm (x is then NULL, too)
 *   gate     [G, H]  g_dtype, or NULL for one; G divides M, and gate row j serves the M/G rows from j M/G on:
 *                    G = 1 a gate per channel, G = M one for every element, between them one per sequence
 *   x        [M, H]  x_dtype: the next block's input
 * All types: WQ_F32, WQ_BF16 or WQ_F16 (the type of an absent tensor is ignored).  H: a multiple of 8.  eps >= 0.
 * Arithmetic is float32, rounded once to h_out and once to x: a row's squares, their sum and (backward) its products with the
 * gradients are formed as they stand and have to lie in float32's normal range, or below eps.  M == 0 is a valid empty call (with a
 * gate of any G, 0 among them).
 */
int block_norm_run(int64_t M, int64_t H, const void* h, int h_dtype, const void* y, int y_dtype, const void* post,
                   const void* pre, int w_dtype, const void* gate, int64_t G, int g_dtype, float alpha, float offset,
                   float eps, void* h_out, void* x, int x_dtype, void* stream);

/*
 * The gradients of block_norm_run.  h is the stream after the block (h_out as block_norm_run stored it), y as there;
 * dh = dL/dh_out from later uses of the stream [M, H] h_dtype (NULL: zeros), dx = dL/dx [M, H] x_dtype (NULL with
 * pre NULL).  With r(t) = 1 / sqrt(mean t^2 + eps), n(t) = t r(t), w+ = offset + w:
 *   du = dh + r(h) (dn - n(h) mean_i(dn n(h))),  dn = dx pre+            dh_in = du   (h_dtype)
 *   dpre = sum_m dx n(h)                                                (float32 [H])
 *   dgate[g] = sum over the gate row's rows of alpha du p               (float32 [G, H])
 *   dp = alpha gate du;  dpost = sum_m dp n(y)                          (float32 [H])
 *   dy = r(y) (dp post+ - n(y) mean_i(dp post+ n(y))), or dp where post is NULL     (y_dtype)
 * Each output may be NULL and is then not written; at least one is not.  dh_in may be dh itself.  An output whose
 * input is NULL (dy, dgate, dpost without y; dpost without post; dgate without gate; dpre without pre) is
 * WQ_EINVAL.  Sums over rows are float32, in an order fixed by M, H and G.
 * M == 0 writes the weights' gradients, where given, with zeros.
 */
size_t block_norm_backward_workspace_bytes(int64_t M, int64_t H, int64_t G);
int block_norm_backward(int64_t M, int64_t H, const void* h, int h_dtype, const void* y, int y_dtype, const void* dh,
                        const void* dx, int x_dtype, const void* post, const void* pre, int w_dtype, const void* gate,
                        int64_t G, int g_dtype, float alpha, float offset, float eps, void* workspace,
                        size_t workspace_bytes, void* dh_in, void* dy, float* dpost, float* dgate, float* dpre,
                        void* stream);

#ifdef __cplusplus
}
#endif

#endif /* WQMLP_BLOCKS_H */
