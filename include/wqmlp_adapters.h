/*
 * wqmlp_adapters.h -- C ABI of libwqmlp, second part: low-rank adapters beside the quantised projections
 * (serving and training), the gradient through a frozen quantised projection, and the AdamW step that
 * trains the adapters.
 *
 * The conventions of wqmlp.h hold for every call here: device pointers of the current device, 16-byte
 * aligned, dense row-major; nothing is allocated or synchronised and every call can be captured into a
 * hipGraph; argument errors are found before anything is enqueued; the same return codes.  Calls that may
 * run at the same time (streams, threads, captured graphs) need workspaces of their own.  All sums are
 * float32 in an order fixed by the shape, so a call's results are reproducible bit for bit.
 */
#ifndef WQMLP_ADAPTERS_H
#define WQMLP_ADAPTERS_H

#include "wqmlp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Adapter ranks: multiples of 8 up to this (an adapter of smaller rank is padded with zero rows of a). */
#define WQ_LORA_MAX_RANK 256
/* Elements per scale of the 8-bit optimizer states. */
#define WQ_ADAMW_BLOCK 256
/* With 8-bit optimizer states (in adamw_table_build's state_bits): a positive v keeps a positive code. */
#define WQ_ADAMW_KEEP_V 256
/* Tensors one AdamW table can hold. */
#define WQ_ADAMW_MAX_TENSORS (1 << 20)

/*
 * E low-rank adapters of rank R beside one shared projection of K inputs and N outputs, row by row:
 *   e = ids[m];  out[m,n] = y[m,n] + scale[e] * sum_r (sum_k x[m,k] a[e,r,k]) * b[e,n,r]
 * and out[m,:] = y[m,:] where ids[m] is outside [0, E) (a row without an adapter; its x is not used).
 *   x     [M, K]     WQ_F32, WQ_BF16 or WQ_F16
 *   a     [E, R, K]  and  b [E, N, R]: both of w_dtype (WQ_F32, WQ_BF16 or WQ_F16)
 *   scale [E]        float32 (alpha / rank, say)
 *   ids   [M]        int32, device; rows of one adapter need not be neighbours, though runs of rows with
 *                    one id (a request's tokens) are what the kernels are shaped for
 *   y     [M, N]     float32: the projection's result (qlinear_run); NULL stands for zeros
 *   out   [M, N]     float32; may be y itself
 * The result is that of float32 arithmetic: operands enter the matrix cores as sums of bfloat16 terms that
 * hold all their bits down to 2^-133, bfloat16's smallest step (a float32 operand is off by at most 2^-134), and
 * so does the rank-R intermediate, which is float32.  An adapter's values reach only the rows that
 * name it, whatever they are (NaN and infinities included); where a row's own operands hold an infinity,
 * or a float32 above 3.38e38, its result may be NaN.  K: a multiple of 16; N: any; R: a multiple of 8 up to WQ_LORA_MAX_RANK.
 * M == 0 is a valid empty call (x, ids, y, out and the workspace may then be NULL).
 * The fused MLP calls take no adapters: an MLP with adapters is qlinear_run and lora_run for each of its
 * projections, with the activation (and its gradient) between them the caller's.
 */
size_t lora_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t E, int64_t R, int backward);
int lora_run(int64_t M, int64_t K, int64_t N, int64_t E, int64_t R, const void* x, int x_dtype,
             const void* a, const void* b, int w_dtype, const float* scale, const int32_t* ids,
             const float* y, void* workspace, size_t workspace_bytes, float* out, void* stream);

/*
 * The gradients of lora_run for a given dy = dL/dout (whose own part passes to y unchanged):
 *   t[m,r]  = sum_k x[m,k] a[e,r,k]                  dt[m,r] = scale[e] sum_n dy[m,n] b[e,n,r]
 *   db[e,n,r] = scale[e] sum_{m: ids[m] = e} dy[m,n] t[m,r]
 *   da[e,r,k] = sum_{m: ids[m] = e} dt[m,r] x[m,k]
 *   dx[m,k] = dx0[m,k] + sum_r dt[m,r] a[e,r,k]      (dx0 where the row has no adapter)
 * t is computed again from x.  dy [M,N]: WQ_F32 or WQ_BF16; dx0 and dx [M,K]: dx_dtype, WQ_F32, WQ_BF16 or
 * WQ_F16 (dx rounded once from float32); dx0 NULL stands for zeros and may be dx itself (the gradient that
 * qlinear_backward left there); da [E,R,K] and db [E,N,R] float32, written whole (zeros for an adapter
 * that no row names).  Each of dx, da and db may be NULL and is then not computed, at least one is not.
 * The workspace is lora_workspace_bytes(..., backward = 1).  M == 0 writes da and db, where given, with
 * zeros (dy, x, ids, dx0 and dx may then be NULL).  Precision and infinities as for lora_run: where a row of dy
 * or x holds an infinity, its dx and its adapter's da and db may be NaN.
 */
int lora_backward(int64_t M, int64_t K, int64_t N, int64_t E, int64_t R, const void* dy, int dy_dtype,
                  const void* x, int x_dtype, const void* a, const void* b, int w_dtype, const float* scale,
                  const int32_t* ids, const void* dx0, int dx_dtype, void* workspace, size_t workspace_bytes,
                  void* dx, float* da, float* db, void* stream);

/*
 * The gradient of qlinear_run with respect to its input, through the frozen packed weights:
 *   dx[m,k] = sum_n dy[m,n] dq(W[n,k])
 * fmt, w, scale and global_scale as for qlinear_run.  dy [M,N]: WQ_F32 or WQ_BF16; dx [M,K]: dx_dtype,
 * WQ_F32 or WQ_BF16.  K: a multiple of 16 (FP8) or 64 (NVFP4); N: any.
 * Each row of dy (FP8: times scale[n], one float32 rounding) is scaled by a power of two so that its
 * largest finite magnitude lies in [2^14, 2^15) and enters float16 MFMAs (a row below 2^-112 as one of 2^-112).
 * dx bfloat16: rounded once to float16; an element is off by at most 2^-11 of itself (dx's own rounding is
 * 2^-8) or 2^-39 of its row's largest, whichever is more.  dx float32: as two float16 terms; 2^-22 of the
 * element or 2^-51 of the row's largest.  A caller who wants more than float16 holds of dy in a bfloat16 dx
 * asks for float32 and rounds it.  Weights decode exactly; sums are float32.  NaN and infinities of dy stay in
 * their row and act there as float32 products would.
 * M == 0 is a valid empty call.
 */
size_t qlinear_backward_workspace_bytes(int fmt, int64_t M, int64_t N, int64_t K, int dx_dtype);
int qlinear_backward(int fmt, int64_t M, int64_t N, int64_t K, const void* dy, int dy_dtype, const uint8_t* w,
                     const float* scale, float global_scale, void* workspace, size_t workspace_bytes, void* dx,
                     int dx_dtype, void* stream);

/*
 * One AdamW step over many tensors in one launch.  For every element, with g = grad_scale * grad, step t:
 *   m = beta1 m + (1 - beta1) g            v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay) - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 *   copy = p rounded to copy_dtype (the adapter weights that lora_run reads), where a copy is kept
 * eps: 0, or taken as at least 2^-126.
 * p is float32 (master weights), g float32 or bfloat16.  State forms (state_bits):
 *   32  m, v float32
 *    8  blocks of WQ_ADAMW_BLOCK consecutive elements (the last may be short) with one power-of-two float32
 *       scale each: m = m_scale * E4M3 code, v = v_scale * E5M2 code, sign bit unused.  The new block scale
 *       is the smallest 2^e (e in [-100, 100]) with max |m| <= 448 * 2^e (v: 57344 * 2^e), 1 for a zero
 *       block; what even 2^100 leaves above the largest code takes that code.  Codes are rounded stochastically: beta2 = 0.999 moves v by far less than half a code step,
 *       which rounding to nearest would drop in every step.  x' = |x| / scale keeps its 3 (v: 2) mantissa
 *       bits after 16 random bits r are added right below them, or below 2^-6 (v: 2^-14) becomes
 *       floor(x' 2^9 + r 2^-16) 2^-9 (v: 2^16, 2^-16).  r are the low (m) and high (v) 16 bits of
 *       mix(key + 0x9E3779B9 i) for element i of tensor j, key = mix(mix(seed + 0x9E3779B9 t) + j), with
 *       mix(h): h ^= h>>16; h *= 0x7FEB352D; h ^= h>>15; h *= 0x846CA68B; h ^= h>>16 on 32 bits (constants:
 *       C. Wellons, "Prospecting for Hash Functions", 2018).
 *       A code of m reaches down to 2^-18 of its block's largest m, one of v to 2^-32 of the largest v, which is
 *       2^-16 in gradient: below that v becomes 0 beside an m that does not, and the next step divides by
 *       sqrt((1 - beta2) g^2) alone, many times lr where g is small.  Blocks whose gradients lie that far apart
 *       want float32 states, or WQ_ADAMW_KEEP_V:
 *    8 | WQ_ADAMW_KEEP_V  the same, but a v that is positive before its rounding gets at least the smallest code,
 *       2^-16.  Elements below 2^-16 of their block's largest gradient then take shorter steps than float32 states
 *       give them, never longer ones than those ever do.  (To adamw_run such a table is one of 8-bit states.)
 * In both 8-bit forms p takes the step with m and v before their rounding, and a state that is not finite gets
 * a NaN code and does not count for its block's scale.
 *
 * The tensors' addresses live in a table in device memory that is built once:
 *   adamw_table_build fills `table` (adamw_table_bytes(count) bytes) from `tensors`, a HOST array of count
 *   descriptors that is not used after the call; its tensors must stay where they are while the table is
 *   in use, must not overlap, and n == 0 is allowed.  Rebuild it when a gradient buffer moves.
 *   adamw_run takes one step over the table's tensors.  step (int64, >= 1) and lr (float32) are read from
 *   device memory, so that a captured graph can be replayed over many steps.  elems: the sum of n, which
 *   sizes the launch (0: an empty call) and nothing else.  A table built for the other state_bits is left
 *   untouched.  Steps over the same tensors must not run at the same time, nor before the build that wrote
 *   the table.
 */
typedef struct {
  int64_t n;        /* elements */
  float* p;         /* [n] */
  const void* g;    /* [n] g_dtype */
  void* m;          /* [n] float32, or E4M3 codes */
  void* v;          /* [n] float32, or E5M2 codes */
  float* m_scale;   /* [ceil(n / WQ_ADAMW_BLOCK)] (8-bit states), else NULL */
  float* v_scale;
  void* copy;       /* [n] copy_dtype, or NULL */
  int32_t g_dtype;  /* WQ_F32 or WQ_BF16 */
  int32_t copy_dtype; /* WQ_BF16 or WQ_F16; ignored where copy is NULL */
} wq_adamw_tensor;
size_t adamw_table_bytes(int64_t count);
int adamw_table_build(int64_t count, const wq_adamw_tensor* tensors, int state_bits, void* table,
                      size_t table_bytes, void* stream);
int adamw_run(int64_t count, int64_t elems, int state_bits, const void* table, const int64_t* step,
              const float* lr, double beta1, double beta2, double eps, double weight_decay, float grad_scale,
              uint32_t seed, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* WQMLP_ADAPTERS_H */
