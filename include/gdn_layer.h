/*
 * gdn_layer.h - C ABI of the operators of a recurrent layer around and beside
 * the gated delta rule: the selective state space scan, the short causal
 * convolution, and the root-mean-square norm.  Same library, conventions and
 * status codes as gdn_qdq.h: every pointer is caller-owned device memory,
 * nothing is allocated, argument errors are returned before any launch, calls
 * are asynchronous on `cuda_stream`, a malformed cu_seqlens skips the
 * sequences concerned (those that are no range of the call's tokens, and those
 * that start before the one in front of them; their outputs are left as they
 * were; what the other sequences of that call receive is not defined) and is
 * reported by gdn_last_error().  All sums, states and statistics are fp32; a result is
 * rounded once, to its own type.  Results do not depend on timing: nothing is
 * added in an order that changes from run to run.
 *
 * Layouts: a "token" of a strided tensor is one contiguous row (all its heads,
 * or all its channels); consecutive tokens, across batch rows too, lie `stride`
 * elements apart, so that a slice of a projection's output is read in place.
 * Dense calls (cu_seqlens == NULL) have n_seq sequences of T tokens; packed
 * calls have T tokens in all and int32 cu_seqlens [n_seq + 1], as in
 * gdn_prefill.  Outputs are contiguous.  No output may overlap an input
 * except where it is said.
 */
#ifndef GDN_LAYER_H_
#define GDN_LAYER_H_

#include "gdn_qdq.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GDN_ACT_NONE = 0, GDN_ACT_SILU = 1 } gdn_activation;

/*
 * gdn_conv_prefill - causal convolution of every channel over the tokens of
 * its sequence:  pre_t = bias + sum_{j < W} weight[c][j] x_{t-W+1+j},
 * y_t = act(pre_t), where the positions before the first token are the rows of
 * state_in (oldest first).
 *
 * x, y: [.., C] in dtype dt; weight fp32 [C, W], W in {2, 3, 4}; bias fp32 [C]
 * or NULL; state_in [n_seq, W - 1, C] in dtype dt or NULL for zeros;
 * state_out: same shape, the last W - 1 rows of [state_in; x] (an empty
 * sequence passes its state through); it may alias state_in exactly.
 * Pointers need their element's alignment; x, y and the states 16-byte aligned
 * with C and x_stride multiples of 16 bytes take the vector path.
 */
gdn_status gdn_conv_prefill(const void *x, int64_t x_stride, const float *weight,
                            const float *bias, const void *state_in,
                            const int32_t *cu_seqlens, int n_seq, int T, int C, int W,
                            gdn_dtype dt, gdn_activation act, void *y, void *state_out,
                            void *cuda_stream);

/* gdn_conv_decode - one token for each of n_seq sequences: x, y [n_seq, C];
 * state_inout [n_seq, W - 1, C] moves up by one row in place. */
gdn_status gdn_conv_decode(const void *x, int64_t x_stride, const float *weight,
                           const float *bias, void *state_inout, int n_seq, int C, int W,
                           gdn_dtype dt, gdn_activation act, void *y, void *cuda_stream);

/*
 * gdn_conv_backward - gradients of one gdn_conv_prefill call for dy (shaped
 * like y, contiguous, dtype dt) and dstate_out (shaped like state_out, dtype
 * dt, or NULL for zero): dx (contiguous) and dstate_in in dtype dt, dweight
 * fp32 [C, W], dbias fp32 [C].  workspace: at least
 * gdn_conv_backward_workspace_bytes(..) bytes, 16-byte aligned, scratch.
 */
size_t gdn_conv_backward_workspace_bytes(int n_seq, int T, int C, int W, int packed);
gdn_status gdn_conv_backward(const void *x, int64_t x_stride, const float *weight,
                             const float *bias, const void *state_in,
                             const int32_t *cu_seqlens, int n_seq, int T, int C, int W,
                             gdn_dtype dt, gdn_activation act, const void *dy,
                             const void *dstate_out, void *workspace, size_t workspace_bytes,
                             void *dx, float *dweight, float *dbias, void *dstate_in,
                             void *cuda_stream);

/*
 * gdn_scan_prefill - selective state space scan with one decay a head:
 *   dt_t = softplus(dt_raw_t + dt_bias)
 *   S_t = exp(dt_t A) S_{t-1} + B_t (dt_t x_t)^T,   y_t = S_t^T C_t + D x_t
 *
 * x, y: [.., H, P]; dt_raw: [.., H]; B, C: [.., G, N], head h uses group
 * h / (H / G); all in dtype dtype.  A fp32 [H] (at most 0), D fp32 [H] or NULL
 * for zero, dt_bias fp32 [H] or NULL for zero.  State fp32 [n_seq, H, N, P],
 * the layout of gdn_prefill's (key rows, value columns): state_in or NULL for
 * zeros, state_out may alias state_in exactly; an empty sequence passes its
 * state through.
 * bf16 calls work on 64-token chunks: a NaN or an infinity in x, B or C can
 * reach the outputs of the tokens before it in its chunk, and those behind it;
 * gradients of either type work on such chunks too.  An infinity in a state
 * stays one until a decay of zero.
 * P, N in {64, 128}; H a multiple of G.  x, B, C, y and the states 16-byte
 * aligned, the strides of x, B and C multiples of 16 bytes; dt_raw
 * element-aligned with any stride.
 * workspace: gdn_scan_prefill_workspace_bytes(..) bytes (it can be 0: then
 * NULL will do), 16-byte aligned, scratch.
 */
size_t gdn_scan_prefill_workspace_bytes(int n_seq, int T, int H, int P, int G, int N,
                                        gdn_dtype dtype, int packed);
gdn_status gdn_scan_prefill(const void *x, int64_t x_stride, const void *dt_raw,
                            int64_t dt_stride, const float *A, const void *B, int64_t b_stride,
                            const void *C, int64_t c_stride, const float *D,
                            const float *dt_bias, const float *state_in,
                            const int32_t *cu_seqlens, int n_seq, int T, int H, int P, int G,
                            int N, gdn_dtype dtype, void *workspace, size_t workspace_bytes,
                            void *y, float *state_out, void *cuda_stream);

/* gdn_scan_decode - one token for each of n_seq sequences: x, y [n_seq, H, P],
 * dt_raw [n_seq, H], B, C [n_seq, G, N]; state_inout advanced in place. */
gdn_status gdn_scan_decode(const void *x, int64_t x_stride, const void *dt_raw,
                           int64_t dt_stride, const float *A, const void *B, int64_t b_stride,
                           const void *C, int64_t c_stride, const float *D,
                           const float *dt_bias, float *state_inout, int n_seq, int H, int P,
                           int G, int N, gdn_dtype dtype, void *y, void *cuda_stream);

/*
 * gdn_scan_backward - gradients of one gdn_scan_prefill call (no forward
 * activations are kept; the states are recomputed) for dy (shaped like y,
 * contiguous) and dstate_out (fp32, or NULL for zero).  Contiguous outputs in
 * dtype dtype: dx, ddt (of dt_raw), dB, dC (summed over the heads of a group);
 * fp32: dA [H], dD [H], ddt_bias [H], dstate_in [n_seq, H, N, P].
 * The workspace holds a state and its adjoint for every 64 tokens, 12 bytes an
 * element in bf16 calls and 8 in fp32 ones (4 GB for 8 x 4096 tokens of 80 heads
 * of 128 x 64 in bf16).
 */
size_t gdn_scan_backward_workspace_bytes(int n_seq, int T, int H, int P, int G, int N,
                                         gdn_dtype dtype, int packed);
gdn_status gdn_scan_backward(const void *x, int64_t x_stride, const void *dt_raw,
                             int64_t dt_stride, const float *A, const void *B, int64_t b_stride,
                             const void *C, int64_t c_stride, const float *D,
                             const float *dt_bias, const float *state_in,
                             const int32_t *cu_seqlens, int n_seq, int T, int H, int P, int G,
                             int N, gdn_dtype dtype, const void *dy, const float *dstate_out,
                             void *workspace, size_t workspace_bytes, void *dx, void *ddt,
                             float *dA, void *dB, void *dC, float *dD, float *ddt_bias,
                             float *dstate_in, void *cuda_stream);

/*
 * gdn_norm - root-mean-square norm of rows of d elements:
 *   s = x + residual, rounded to dtype (s = x without a residual)
 *   y = s / sqrt(mean(s^2) + eps) * weight * silu(gate)     (no gate: 1)
 *
 * x, residual, gate: [tokens, heads, d] in dtype dt (heads > 1: a token's
 * heads are contiguous); weight fp32 [d].  residual_out: s, contiguous, given
 * exactly when residual is; it may alias a contiguous residual or x exactly.
 * y by `out`:
 *   GDN_NORM_SAME           dtype dt;
 *   GDN_NORM_FP8_ROW        E4M3 bytes, scales fp32 [tokens * heads]:
 *                           scale = amax / 448 of the row (the W codec's);
 *   GDN_NORM_INT8_GROUP*    int8 codes, scales fp32 [tokens * heads, d / group]:
 *                           scale = amax / 127 (the state codec's).
 * The codes are those of y before any rounding to dt; a zero row or group has
 * scale 0 and codes 0; a row or group that holds a NaN has a NaN scale.
 * The mean is fp32: a row of which mean(s^2) + eps is 0 there (eps = 0 and
 * values below 1e-22 at most) has y = 0 and gradients of zero but for
 * dresidual; one whose sum of squares passes 3e38 has y = 0.
 * d: up to 4096 vectors of 16 bytes, or 8192 elements where pointers, strides
 * or d do not allow vectors; the INT8 groups need them (and d a multiple of
 * the group).
 */
typedef enum {
    GDN_NORM_SAME = 0,
    GDN_NORM_FP8_ROW = 1,
    GDN_NORM_INT8_GROUP32 = 2,
    GDN_NORM_INT8_GROUP16 = 3,
    GDN_NORM_INT8_GROUP64 = 4
} gdn_norm_out;
gdn_status gdn_norm(const void *x, int64_t x_stride, const void *residual,
                    int64_t residual_stride, const void *gate, int64_t gate_stride,
                    const float *weight, int64_t tokens, int heads, int d, float eps,
                    gdn_dtype dt, gdn_norm_out out, void *y, float *scales,
                    void *residual_out, void *cuda_stream);

/*
 * gdn_norm_backward - gradients of gdn_norm at x = s (the residual_out of the
 * forward call, or its x) for dy and for dresidual, the gradient that reaches
 * residual_out from elsewhere (NULL for zero): dx in dtype dt (of s, hence of
 * x and of residual alike), dweight fp32 [d], dgate in dtype dt (given exactly
 * when gate is).  An 8-bit output passes its gradient straight through.
 * workspace as for the others.
 */
size_t gdn_norm_backward_workspace_bytes(int64_t tokens, int heads, int d);
gdn_status gdn_norm_backward(const void *x, int64_t x_stride, const void *gate,
                             int64_t gate_stride, const float *weight, const void *dy,
                             int64_t dy_stride, const void *dresidual,
                             int64_t dresidual_stride, int64_t tokens, int heads, int d,
                             float eps, gdn_dtype dt, void *workspace, size_t workspace_bytes,
                             void *dx, float *dweight, void *dgate, void *cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_LAYER_H_ */
