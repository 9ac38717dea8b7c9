/*
 * libmoe_block: the operators of the transformer block around one MoE layer
 * (include/moe.h) on one B200 (sm_100a), and the layer's experts in 8-bit
 * integers:
 *
 *   residual norm   the norm after a block's output, its gate and scale, the
 *                   residual add ("a token with no entry passes on the
 *                   residual, which the caller adds": moe_combine) and the
 *                   next block's pre-norm, in one pass; and its backward
 *   gradient clip   the global norm of many gradient tensors, and their
 *                   clipped copies
 *   8-bit experts   activations quantised per token, expert weights per
 *                   output channel, and the grouped products between them
 *
 * The conventions of moe.h hold: device pointers to contiguous row-major
 * memory owned by the caller, work enqueued on `stream` of the current
 * device (which must own the pointers), no allocation, no synchronisation,
 * host-side validation before the first launch, bounded device-side waits.
 * Statuses, dtypes, activations and streams are moe.h's. Errors of a bounded
 * wait go to the first 256 bytes of the workspace, as there:
 * moe_workspace_init zeroes them once, moe_read_error reads them.
 *
 * Every call may be captured into a CUDA graph. A workspace serves one call
 * at a time: calls that may overlap on the GPU (two streams, two graphs
 * replayed on two streams) need one each.
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- residual norms ----------------------------------------------------
 * A row's sum of squares is fp32: it has to fit (a root mean square below
 * 1.8e19 / d^1/2); squares below 2^-126 count in steps of 2^-149, beside eps.
 * Rows of any size in between, zeros among them, and any eps give the gradients
 * of their formulas, as far as those fit the outputs' type. */

#define MOE_NORM_MAX_D 16384

typedef struct {
  int n;           /* tokens, >= 0 (0: no token tensor is read; sums over tokens are zeroed) */
  int d;           /* model dim, 1..MOE_NORM_MAX_D; any value */
  moe_dtype dtype; /* of x, y, gate, out, h and their gradients */
  float eps;       /* > 0, added to the mean square */
  /* the weights multiply as (w + weight_offset): 0, or 1 for weights stored
   * around zero */
  float weight_offset;
  float res_scale;   /* a: scale of the residual */
  float block_scale; /* b: scale of the block's (normed, gated) output */
  /* gate rows: 0 = one row for all tokens; T > 0 = one row for each T
   * consecutive tokens (row t / T), the last one may cover fewer */
  int gate_tokens;
  long long gate_stride; /* elements between gate rows (and dgate rows), >= d */
} moe_norm_config;

/* Checks a config. */
MOE_API moe_status moe_norm_validate(const moe_norm_config* cfg);

/* Workspace bytes of the two backward calls (256-byte aligned; partial sums
 * only, nothing to initialise). */
MOE_API moe_status moe_norm_workspace_size(const moe_norm_config* cfg, size_t* bytes);

/* Pre-norm: rstd[t] = (mean_j x[t,j]^2 + eps)^-1/2,
 * h[t,j] = x[t,j] rstd[t] (w[j] + weight_offset). x, h [n,d]; w [d] fp32;
 * rstd [n] fp32 (NULL: not stored). h may be x. Sums, norms and products are
 * fp32, rounded once into h. */
MOE_API moe_status moe_norm_forward(const moe_norm_config* cfg, const void* x, const float* w,
                                    void* h, float* rstd, moe_stream_t stream);

/* Its gradient: dx = dres + d<dh, h>/dx and dw = d<dh, h>/dw, with dres [n,d]
 * the gradient that reaches x along the residual (NULL: none). x, w, rstd as
 * in the forward; dx [n,d] (may be dres or dh); dw [d] fp32. Row sums go
 * through the workspace in a fixed order: the result is the same each time. */
MOE_API moe_status moe_norm_backward(const moe_norm_config* cfg, const void* dres,
                                     const void* dh, const void* x, const float* w,
                                     const float* rstd, void* dx, float* dw, void* ws,
                                     size_t ws_bytes, moe_stream_t stream);

/* Post-norm, gate, scale, residual and the next pre-norm:
 *   v[t]   = y[t] rstd_post[t] (w_post + weight_offset)   (w_post NULL: v = y)
 *   out[t] = res_scale x[t] + block_scale gate[row(t)] v[t]  (gate NULL: 1)
 *   h[t]   = out[t] rstd_next[t] (w_next + weight_offset)  (w_next and h NULL: none)
 * with rstd the (mean square + eps)^-1/2 of y and of out. x, y, out, h [n,d];
 * gate [rows, d] with gate_stride; w_post, w_next [d] fp32; rstd_post,
 * rstd_next [n] fp32 (NULL: not stored; stored with w_post / w_next only). h is
 * taken from out before out is rounded. out may be x or y, h may be y or x (not
 * both the same); no other overlap. */
MOE_API moe_status moe_residual_norm_forward(const moe_norm_config* cfg, const void* x,
                                             const void* y, const float* w_post,
                                             const void* gate, const float* w_next, void* out,
                                             void* h, float* rstd_post, float* rstd_next,
                                             moe_stream_t stream);

/* Gradients of <dout, out> + <dh, h>. out is the forward's output, y its
 * input, rstd_post / rstd_next what it stored (needed with w_post / w_next).
 * dout NULL: out has no other use; dh and w_next NULL: there was no next
 * norm (one of dout, dh is needed; out, rstd_next and dw_next only with dh).
 *   D = dout + d<dh, h>/dout; dx = res_scale D; dz = block_scale D;
 *   dgate[r] = sum over its tokens of dz v; dy and dw_post through the norm
 * dx, dy [n,d], dgate [rows,d] (stride gate_stride; NULL without gate), dw_post
 * and dw_next [d] fp32. dx may be dout and dy may be dh; no other overlap.
 * Sums over tokens are fp32 in a fixed order through the workspace. */
MOE_API moe_status moe_residual_norm_backward(
    const moe_norm_config* cfg, const void* dout, const void* dh, const void* out, const void* y,
    const float* w_post, const void* gate, const float* w_next, const float* rstd_post,
    const float* rstd_next, void* dx, void* dy, float* dw_post, void* dgate, float* dw_next,
    void* ws, size_t ws_bytes, moe_stream_t stream);

/* ---- global gradient norm and clip ------------------------------------- */

typedef struct {
  const void* grad; /* device; element-aligned, any length */
  void* out;        /* device: the clipped copy; may be grad itself */
  long long numel;  /* >= 0 */
  moe_dtype dtype;  /* of grad and out */
} moe_grad_tensor;

/* Workspace bytes for `count` tensors (256-byte aligned; nothing to
 * initialise). */
MOE_API moe_status moe_grad_workspace_size(int count, size_t* bytes);

/* norm[0] = (sum over all elements of all tensors of g^2)^1/2. `tensors` is a
 * HOST array, read during the call; `out` members are ignored. Elements are
 * squared and summed so that values of any magnitude count (no overflow or
 * underflow before the root); partial sums are fp64 and joined in a fixed
 * order. An infinite element, or a norm above the largest fp32, gives +inf, a
 * NaN gives NaN. A tensor listed twice counts twice. norm: device, fp32. */
MOE_API moe_status moe_grad_norm(const moe_grad_tensor* tensors, int count, float* norm, void* ws,
                                 size_t ws_bytes, moe_stream_t stream);

/* The norm, and the tensors scaled so that it is at most max_norm:
 * norm[0] as above, norm[1] = min(1, max_norm / (norm[0] + 1e-6)) (NaN if the
 * norm is), out = grad * norm[1], rounded once. max_norm >= 0; +inf is no limit,
 * norm[1] is 1 then unless the norm is NaN. An out is its own grad (in place;
 * with norm[1] == 1 nothing is rewritten) or memory that no other listed tensor
 * touches. */
MOE_API moe_status moe_grad_clip(const moe_grad_tensor* tensors, int count, float max_norm,
                                 float* norm, void* ws, size_t ws_bytes, moe_stream_t stream);

/* ---- 8-bit experts ------------------------------------------------------ */

#define MOE_I8_MAX_GROUPS (MOE_MAX_EXPERTS + MOE_MAX_SHARED)
#define MOE_I8_MAX_K 65536 /* 127 * 127 * K stays inside the int32 accumulator */

/* Symmetric quantisation, row by row: scale[r] = max_j |x[r,j]| / 127 in fp32,
 * q[r,j] = x[r,j] / scale[r] rounded to the nearest integer, ties to even
 * (decided on the exact quotient), at most 127. A row of zeros, or one so small
 * that its scale rounds to 0 (max |x| up to 63 * 2^-149), gets scale 0 and
 * zeros; a row with an infinity or a NaN gets scale NaN and zeros, so that
 * every product with it is NaN. x [rows, cols] of `dtype` (cols >= 1), q [rows, cols] int8,
 * scale [rows] fp32. With starts / counts [groups] (both or neither), only
 * rows starts[g] .. starts[g] + counts[g] - 1 of each group are read and
 * written (groups in ascending order of their rows, inside [0, rows)); the
 * others are left as they were. The same call quantises weights [E*out, in]
 * per output channel. */
MOE_API moe_status moe_quantize_rows(long long rows, int cols, moe_dtype dtype, const void* x,
                                     int8_t* q, float* scale, const int32_t* starts,
                                     const int32_t* counts, int groups, moe_stream_t stream);

/* Activation of a product's epilogue: none, or moe_act's */
typedef enum {
  MOE_I8_RELU = MOE_ACT_RELU,
  MOE_I8_GELU = MOE_ACT_GELU,
  MOE_I8_SWIGLU = MOE_ACT_SWIGLU,
  MOE_I8_NONE = 3
} moe_i8_act;

typedef struct {
  int groups;      /* weight matrices, 1..MOE_I8_MAX_GROUPS */
  int rows;        /* rows of the activation and output buffers, >= 0 */
  int k;           /* reduction length, a multiple of 16, 16..MOE_I8_MAX_K */
  int n_out;       /* output channels, a multiple of 16 */
  moe_i8_act act;
  moe_dtype dtype; /* of the output */
} moe_gemm_i8_config;

MOE_API moe_status moe_gemm_i8_validate(const moe_gemm_i8_config* cfg);

/* Workspace bytes (256-byte aligned; moe_workspace_init once). */
MOE_API moe_status moe_gemm_i8_workspace_size(const moe_gemm_i8_config* cfg, size_t* bytes);

/* Grouped product in 8-bit integers: for each group g and its rows r =
 * starts[g] .. starts[g] + counts[g] - 1,
 *   u[r,o] = x_scale[r] w_scale[g,o] sum_j xq[r,j] w[g,o,j]
 *   out[r,o] = act(u[r,o]), or silu(u) v with v from w3 / w3_scale (SwiGLU)
 * x: xq [rows,k] int8, x_scale [rows] fp32; w, w3 [groups,n_out,k] int8,
 * w_scale, w3_scale [groups,n_out] fp32; out [rows,n_out]. The sum over j is
 * exact (int32); scales (the sum times w_scale, then times x_scale) and
 * activation are fp32, rounded once into out. Rows outside every group are left
 * as they were. starts and counts NULL: one group (groups == 1) of all `rows`
 * rows. Groups must lie in ascending order inside [0, rows) and not overlap; a
 * group that does not fit is cut to what does. Rows start anywhere (no
 * alignment). xq, w, w3 and out 16-byte aligned. */
MOE_API moe_status moe_gemm_i8(const moe_gemm_i8_config* cfg, const int8_t* xq,
                               const float* x_scale, const int32_t* starts,
                               const int32_t* counts, const int8_t* w, const float* w_scale,
                               const int8_t* w3, const float* w3_scale, void* out, void* ws,
                               size_t ws_bytes, moe_stream_t stream);

/* Dispatch of quantised rows: token t of X [n,d] is quantised once (as
 * moe_quantize_rows does) and its bytes and scale are written to every
 * dispatched row of its list tok_row[t, :] (moe_route_out; entries < 0 end
 * nothing and are skipped) and, for each shared expert s < n_shared, to row
 * shared_row_base + s * roundup(n, 128) + t, the rows moe_combine reads its
 * shared experts from. starts / counts [E + n_shared] receive the groups of
 * moe_gemm_i8 over these rows: routed expert e has offsets[e] and its counts[e],
 * shared expert s its n rows. `rows`, `slots` and `shared_row_base` are
 * moe_sizes' values. q [rows, d] int8, scale [rows] fp32. d any multiple of 16. */
typedef struct {
  int n, d, E, n_shared;
  int slots;           /* columns of tok_row */
  int rows;            /* rows of q */
  int shared_row_base; /* also the bound on routed rows */
  moe_dtype dtype;     /* of X */
} moe_dispatch_i8_config;

MOE_API moe_status moe_dispatch_i8(const moe_dispatch_i8_config* cfg, const void* X,
                                   const moe_route_out* route, int8_t* q, float* scale,
                                   int32_t* starts, int32_t* counts, moe_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_BLOCK_H */
