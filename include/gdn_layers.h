/*
 * gdn_layers.h — C ABI of the layer operators around the delta rule, in the same
 * library (libgdn_gb300.so, sm_103a): the short causal convolution ahead of
 * q, k, v, the selective state space scan of the layers that hybrid stacks mix
 * with the delta rule, and the RMS norm with its output gate or its residual sum.
 *
 * Token arrays are passed as dn_view: a base pointer and element strides of the
 * batch, head and time axes; the feature axis is contiguous.  So the projection's
 * token-major [B][T][H*d], the delta rule's head-major [B][H][T][d] and a slice of
 * a wider projection are all read and written in place.  A view may have any
 * strides (0 in an input repeats it along that axis); outputs must not overlap
 * each other or the inputs.  Vector accesses need every view of the call aligned to
 * them (pointer and strides), else the kernels move one element at a time; 16-byte
 * alignment is always enough.  The norm and the single-token convolution move 16
 * bytes an access, the convolution over tokens 8, the scan 4 elements (one above
 * 32 states, and of x, dt, z and y for single tokens).
 *
 * Dtypes: shape->dtype (DN_F32 or DN_BF16) is that of every token array and of the
 * convolution's taps; parameters (weights, A, D, biases), scan states and their
 * gradients are float32.  Arithmetic is float32; a result is rounded once, when it
 * is stored.
 *
 * Packed variable-length input, ownership, streams, errors: as in gdn.h.  B == 1,
 * T = total tokens, cu_seqlens = device int32 offsets [num_seqs + 1]; nothing
 * crosses a sequence boundary and empty sequences are allowed.  Malformed offsets
 * are found on the device: the call then treats every sequence as empty and sets
 * the status word of the workspace (dn_device_status: DN_ERR_INVALID_ARG).
 * Pointers need the alignment of their element type; workspaces and saved
 * buffers 16 bytes.
 */
#ifndef GDN_GB300_LAYERS_H
#define GDN_GB300_LAYERS_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A token array [B][H][T][d] with element strides; the feature index has stride 1.
 * data == NULL: absent. */
typedef struct {
    void *data;
    int64_t batch, head, time;
} dn_view;

/* ---------------------------------------------------------------- convolution
 * Depthwise, causal, `width` taps (2..4), channel c = h * d + j:
 *     pre[t][c] = bias[c] + sum_k w[c][k] x[t - (width - 1) + k][c]
 *     y = silu ? pre * sigmoid(pre) : pre
 * Inputs before a sequence's first token come from s0 (zero where NULL).
 *   w [H*d][width], bias [H*d] or NULL (float32)
 *   s0, sT [N][width-1][H*d] (dtype): the width - 1 inputs before the first token
 *   (oldest first), and after the last one; N = B or num_seqs; either may be NULL. */
typedef struct {
    int32_t B, H, T, d;
    int32_t width;                /* taps, 2..4                                   */
    int32_t dtype;                /* dn_dtype                                     */
    int32_t silu;                 /* 1: y = silu(pre)                             */
    int32_t num_seqs;             /* packed sequences (ignored without cu_seqlens) */
    const int32_t *cu_seqlens;    /* device, [num_seqs + 1], or NULL              */
} dn_conv_shape;

/* Bytes of device workspace (0 on bad arguments). */
size_t dn_conv_workspace_size(const dn_conv_shape *shape, int for_backward);

dn_status dn_conv_fwd(const dn_conv_shape *shape, const dn_view *x, const float *w,
                      const float *bias, const void *s0, const dn_view *y, void *sT, void *ws,
                      size_t ws_bytes, void *stream);

/* Gradients of <y, dy> + <sT, dsT>.  dsT, ds0 like s0 (NULL: zero / not written); dw and
 * dbias as w and bias (dbias may be NULL).  Sums over tokens are taken in a fixed order. */
dn_status dn_conv_bwd(const dn_conv_shape *shape, const dn_view *x, const float *w,
                      const float *bias, const void *s0, const dn_view *dy, const void *dsT,
                      const dn_view *dx, float *dw, float *dbias, void *ds0, void *ws,
                      size_t ws_bytes, void *stream);

/* One token for each of B sequences (T must be 1, no packing): y from x and state_in,
 * state_out = state_in moved on by x; state_out may be state_in.  No workspace. */
dn_status dn_conv_step(const dn_conv_shape *shape, const dn_view *x, const float *w,
                       const float *bias, const void *state_in, void *state_out, const dn_view *y,
                       void *stream);

/* ------------------------------------------------------- selective state space scan
 * D channels with N states each; B and C are shared by the D / G channels of a group:
 *     delta = dt_softplus ? softplus(dt + dt_bias) : dt + dt_bias
 *     h_t[c][n] = exp(delta A[c][n]) h_{t-1}[c][n] + delta x_t[c] B_t[g][n]
 *     o_t[c]    = sum_n C_t[g][n] h_t[c][n] + D[c] x_t[c]
 *     y_t[c]    = z ? o_t[c] silu(z_t[c]) : o_t[c]
 * A <= 0 and delta >= 0 in use (a decay); nothing checks either.                  */
typedef struct {
    int32_t B, T, D;              /* batch rows, tokens per row, channels          */
    int32_t N, G;                 /* states per channel 1..128, groups (D % G == 0) */
    int32_t dtype, dt_softplus;
    int32_t num_seqs;
    const int32_t *cu_seqlens;
} dn_scan_shape;

typedef struct {
    dn_view x, dt, b, c;          /* [B][T][D] (no head axis), [B][G][T][N] (head = group) */
    dn_view z, y;                 /* [B][T][D]; z.data == NULL: no gate             */
    const float *A;               /* [D][N]                                        */
    const float *D, *dt_bias;     /* [D] or NULL (zero)                            */
    const float *h0;              /* [N_seq][D][N] initial states or NULL (zero)    */
    float *hT;                    /* final states or NULL                          */
} dn_scan_io;

typedef struct {
    dn_view dy;                   /* gradient of y                                 */
    dn_view dx, ddt, db, dc;      /* all written                                   */
    dn_view dz;                   /* written when io.z is given                     */
    const float *dhT;             /* gradient of hT or NULL (zero)                 */
    float *dA;                    /* [D][N]                                        */
    float *dD, *ddt_bias;         /* [D] or NULL (not written)                     */
    float *dh0;                   /* [N_seq][D][N] or NULL (not written)           */
} dn_scan_grads;

size_t dn_scan_workspace_size(const dn_scan_shape *shape, int for_backward);

/* Bytes of the buffer that dn_scan_fwd fills for dn_scan_bwd: the state entering every 8th token
 * (every 16th for N > 32), float32: N / 2 (N / 4) bytes a token and channel. */
size_t dn_scan_saved_size(const dn_scan_shape *shape);

/* saved may be NULL (nothing kept). */
dn_status dn_scan_fwd(const dn_scan_shape *shape, const dn_scan_io *io, void *saved,
                      size_t saved_bytes, void *ws, size_t ws_bytes, void *stream);

/* Gradients of <y, dy> + <hT, dhT>, from the buffer that dn_scan_fwd filled for the same
 * arguments (the library does not check that they are the same). */
dn_status dn_scan_bwd(const dn_scan_shape *shape, const dn_scan_io *io, const dn_scan_grads *grads,
                      const void *saved, size_t saved_bytes, void *ws, size_t ws_bytes,
                      void *stream);

/* One token for each of B sequences (T must be 1, no packing), states io->h0 -> io->hT, which
 * may be the same buffer.  No workspace. */
dn_status dn_scan_step(const dn_scan_shape *shape, const dn_scan_io *io, void *stream);

/* --------------------------------------------------------------------------- norm
 * Per row of d features:
 *     r = residual ? residual + res_scale * x : x     (res_scale [d] or NULL: 1)
 *     y = r / sqrt(mean(r^2) + eps) * w * (z ? silu(z) : 1)
 * w [d], or [H][d] with w_per_head.  sum receives r where given.                   */
typedef struct {
    int32_t B, H, T, d;           /* d <= 16384 */
    int32_t dtype, w_per_head;
    float eps;
    int32_t reserved;
} dn_norm_shape;

dn_status dn_norm_fwd(const dn_norm_shape *shape, const dn_view *x, const float *w,
                      const dn_view *z, const dn_view *residual, const float *res_scale,
                      const dn_view *y, const dn_view *sum, void *stream);

/* Gradients of <y, dy> + <sum, dsum>, with r read from `sum` (as dn_norm_fwd wrote it), or from
 * x when sum is NULL (no residual).  dx = res_scale * dr (dr when there is no res_scale);
 * dresidual = dr, dres_scale = sum over rows of dr * x; both optional, as are dz (z only) and dsum.
 * dx may be NULL when dresidual is given. */
size_t dn_norm_workspace_size(const dn_norm_shape *shape);
dn_status dn_norm_bwd(const dn_norm_shape *shape, const dn_view *x, const float *w,
                      const dn_view *z, const float *res_scale, const dn_view *sum,
                      const dn_view *dy, const dn_view *dsum, const dn_view *dx, float *dw,
                      const dn_view *dz, const dn_view *dresidual, float *dres_scale, void *ws,
                      size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* GDN_GB300_LAYERS_H */
