/*
 * sequence_ops.h - C ABI of the sequence operators of libconv2d_fused for MI355X (gfx950):
 * the short causal convolution, the selective state space scan and the gated linear
 * recurrence, for prompts and for single tokens, the recurrence's gradient, products of a few
 * token rows with 4-bit weights, and products of any number of them in 8-bit integers.
 *
 * The conventions of conv2d_fused.h hold (device pointers owned by the caller, work only
 * enqueued on `stream`, arguments validated on the host before anything is launched, status
 * codes, conv2d_last_error(), the workspace of conv2d_set_workspace, the dtype and
 * activation codes), with these differences:
 *  - Arguments come in a struct, which the call does not keep.
 *  - Activations are channel-last: the channels of one token are contiguous. Where a struct
 *    has strides (in elements), one token's row and one batch entry's first row may stand
 *    anywhere, so a slice of a wider projection is read in place. Strides may not be negative.
 *    The output may not overlap an input or the state anywhere between its first and its last
 *    value (CONV2D_EINVAL), so it is no slice of a tensor of which an input is another slice,
 *    nor the residual.
 *  - Offsets into memory are 64-bit; a call may cover up to 2^30 tokens of up to 2^30 channels
 *    (inputs and outputs of a product, whose weights may number 2^40), and where it would
 *    need 2^32 GPU threads or more (many short sequences of many channels) it returns
 *    CONV2D_EUNSUPPORTED and has to be made in parts.
 *
 * Sequences of a prompt call. Without `offsets` there are nseq sequences of `tokens` tokens
 * each, one batch entry each. With `offsets` (device, int32 [nseq + 1], not decreasing, from
 * 0 to `tokens`) the sequences are packed one after the other: sequence i has the token rows
 * offsets[i] <= t < offsets[i + 1], batch strides are ignored and `tokens` counts all rows. A
 * sequence may be empty. Offsets are read on the device and clamped to [0, tokens] there, so
 * wrong ones give wrong results but touch no other memory.
 *
 * States. Sequence i (or row i of a single-token call) continues from, and leaves its state
 * in, state row slots[i] (device, int32 [nseq]; NULL: row i). A slot outside
 * [0, state_rows) means no state: the sequence starts from zeros and keeps nothing, as with
 * a NULL state (padding rows of a batch). Two sequences of one call may not share a slot.
 * With `fresh` every sequence starts from zeros and the state rows are only written.
 */
#ifndef SEQUENCE_OPS_H
#define SEQUENCE_OPS_H

#include <stddef.h>

#include "conv2d_fused.h"

#ifdef __cplusplus
extern "C" {
#endif

/* y[t, c] = act(bias[c] + sum_j w[c, j] * x[t - (width - 1) + j, c]), j = 0 .. width - 1:
 * a depthwise correlation over a token and the width - 1 before it. The tokens before a
 * sequence's first one are its state row's, [width - 1, channels] in the storage type, the
 * oldest first; afterwards the row holds the sequence's last width - 1 inputs. */
typedef struct causal_conv1d_args {
    const void *x;         /* token rows of `channels` values */
    const void *w;         /* [channels, width], contiguous */
    const float *bias;     /* [channels] or NULL */
    const float *alpha;    /* [channels], needed by CONV2D_ACT_PRELU */
    void *state;           /* [state_rows, width - 1, channels], contiguous, or NULL */
    void *y;               /* token rows of `channels` values */
    const int *offsets;    /* see above */
    const int *slots;      /* see above */
    long long x_batch, x_token, y_batch, y_token; /* strides in elements */
    long long tokens;
    int nseq, state_rows, channels;
    int width;             /* 2, 3 or 4 */
    int act;               /* CONV2D_ACT_* */
    int dtype;             /* of x, w, state and y */
    int fresh;
} causal_conv1d_args;

int causal_conv1d(const causal_conv1d_args *args, void *stream);

/* The same for one token of each of nseq sequences: x and y have nseq rows x_token and
 * y_token apart. `offsets` is NULL and `tokens` 1; batch strides are ignored. */
int causal_conv1d_step(const causal_conv1d_args *args, void *stream);

/* With d = dt[t, c] + dt_bias[c], or log(1 + exp(of that)) with `softplus`, g the group of
 * channel c (channels / groups channels each), and h the state of the sequence:
 *     h[c, n] = exp(d * a[c, n]) * h[c, n] + d * u[t, c] * b[t, g, n]
 *     y[t, c] = sum_n h[c, n] * c[t, g, n] + skip[c] * u[t, c]
 *     y[t, c] *= gate[t, c] / (1 + exp(-gate[t, c]))     (with a gate)
 * The state and every intermediate are fp32; y is rounded once. A finite a counts as at most
 * 2.36e38 in magnitude; where one is -infinity, a state forgets at every step that is not zero.
 * An infinity or NaN in an input may make y, and through the state the later y, infinite or NaN
 * in the channels and the sequence that read it, and in no others. */
typedef struct selective_scan_args {
    const void *u, *dt;    /* token rows of `channels` values */
    const float *a;        /* [channels, states], contiguous */
    const void *b, *c;     /* token rows of groups * states values */
    const float *skip;     /* [channels] or NULL */
    const void *gate;      /* token rows of `channels` values, or NULL */
    const float *dt_bias;  /* [channels] or NULL */
    float *state;          /* [state_rows, channels, states], contiguous, or NULL */
    void *y;               /* token rows of `channels` values */
    const int *offsets;    /* see above */
    const int *slots;      /* see above */
    long long u_batch, u_token, dt_batch, dt_token, b_batch, b_token, c_batch, c_token; /* strides in elements */
    long long gate_batch, gate_token, y_batch, y_token;
    long long tokens;
    long long longest;     /* tokens of the longest sequence where the caller knows it, or 0: it only
                            * steers how the work is split */
    int nseq, state_rows, channels, groups;
    int states;            /* 1 .. 256 */
    int softplus;
    int dtype;             /* of u, dt, b, c, gate and y */
    int fresh;
} selective_scan_args;

int selective_scan(const selective_scan_args *args, void *stream);

/* A long sequence, or one of few channels, is cut into chunks that run side by side where the
 * calling thread's workspace (conv2d_set_workspace) holds this many bytes for the chunks'
 * states; 0: the call is not split. Without it the call gives the same results up to
 * rounding, slower. Host only. */
int selective_scan_workspace_size(const selective_scan_args *args, size_t *bytes);

/* The same for one token of each of nseq sequences, as causal_conv1d_step. */
int selective_scan_step(const selective_scan_args *args, void *stream);

/* With f = 1 / (1 + exp(-(forget[t, c] + forget_bias[c]))) and h the state of the sequence:
 *     h[c] = f * h[c] + (1 - f) * x[t, c]                (coupled), or f * h[c] + x[t, c]
 *     y[t, c] = h[c] * gate[t, c] / (1 + exp(-gate[t, c])), or h[c] without a gate
 * The state and every intermediate are fp32; y is rounded once. An infinity or NaN in an input
 * may make y, and through the state the later y, infinite or NaN in the channels and the
 * sequence that read it, and in no others. */
typedef struct gated_recurrence_args {
    const void *x, *forget; /* token rows of `channels` values */
    const void *gate;       /* token rows of `channels` values, or NULL */
    const float *forget_bias; /* [channels] or NULL */
    float *state;           /* [state_rows, channels], contiguous, or NULL */
    void *y;                /* token rows of `channels` values */
    const int *offsets;     /* see above */
    const int *slots;       /* see above */
    long long x_batch, x_token, forget_batch, forget_token, gate_batch, gate_token, y_batch, y_token; /* in elements */
    long long tokens;
    long long longest;      /* as for selective_scan */
    int nseq, state_rows, channels;
    int coupled;
    int dtype;              /* of x, forget, gate and y */
    int fresh;
} gated_recurrence_args;

/* Long sequences are cut into chunks that run side by side where the calling thread's
 * workspace holds gated_recurrence_workspace_size() bytes (0: the call is not split). Without
 * it the call gives the same results up to rounding, slower. The size is host only. */
int gated_recurrence(const gated_recurrence_args *args, void *stream);
int gated_recurrence_workspace_size(const gated_recurrence_args *args, size_t *bytes);

/* The same for one token of each of nseq sequences, as causal_conv1d_step. */
int gated_recurrence_step(const gated_recurrence_args *args, void *stream);

/* The gradient of gated_recurrence. Given grad, the gradient of a loss with respect to y, it
 * writes those with respect to x, forget, gate (with a gate) and forget_bias (unless
 * grad_forget_bias is NULL). With g_t the gradient with respect to h_t, which is grad times
 * silu(gate) plus f_{t+1} g_{t+1}:
 *     grad_x = g (1 - f) or g,    grad_forget = g (h_{t-1} - x or h_{t-1}) f (1 - f),
 *     grad_gate = grad h_t silu'(gate),    grad_forget_bias = sum of grad_forget over all tokens
 * States: `state` holds the rows that the sequences started from (NULL, or a slot outside it:
 * zeros) and is only read; the forward call has updated its own in place, so the caller keeps a
 * copy. grad_state, [state_rows, channels], holds for each sequence the gradient with respect to
 * the state that it left (NULL: zero) and afterwards that with respect to the state, or the
 * zeros, that it started from.
 * Everything is fp32 but the values read and, rounded once each, grad_x, grad_forget and
 * grad_gate. The sum over tokens has a fixed order. The outputs may be slices of one tensor with
 * the same strides, their rows between each other's, as long as they share no value; they may overlap
 * no input. Needs gated_recurrence_backward_workspace_size() bytes of workspace, and returns
 * CONV2D_EUNSUPPORTED where the thread's is smaller. */
typedef struct gated_recurrence_backward_args {
    const void *grad, *x, *forget; /* token rows of `channels` values */
    const void *gate;       /* token rows of `channels` values, or NULL */
    const float *forget_bias; /* [channels] or NULL */
    const float *state;     /* [state_rows, channels], contiguous, or NULL */
    float *grad_state;      /* [state_rows, channels], contiguous, or NULL */
    void *grad_x, *grad_forget; /* token rows of `channels` values */
    void *grad_gate;        /* token rows of `channels` values; NULL without a gate */
    float *grad_forget_bias; /* [channels] or NULL */
    const int *offsets;     /* see above */
    const int *slots;       /* see above */
    long long grad_batch, grad_token, x_batch, x_token, forget_batch, forget_token, gate_batch, gate_token; /* in elements */
    long long grad_x_batch, grad_x_token, grad_forget_batch, grad_forget_token, grad_gate_batch, grad_gate_token;
    long long tokens;
    long long longest;      /* as for selective_scan */
    int nseq, state_rows, channels;
    int coupled;
    int dtype;              /* of the token rows */
} gated_recurrence_backward_args;

int gated_recurrence_backward(const gated_recurrence_backward_args *args, void *stream);
int gated_recurrence_backward_workspace_size(const gated_recurrence_backward_args *args, size_t *bytes);

/* 4-bit weights: weight (o, k) is (code - zero) * scale with a code of 0 .. 15 and, for each
 * run of `group` inputs (32, 64 or 128; the last one may be shorter) of an output, a scale
 * and a zero point of 0 .. 15 (8 where zeros is NULL). matvec_w4_pack lays them out once for
 * matvec_w4: codes [out_features, ceil(in_features / 2)] bytes, the even input in the low
 * half; scales [out_features, ceil(in_features / group)] in `dtype` (bf16 or f16); zeros the
 * same shape in bytes or NULL. `packed` is 16-byte aligned, matvec_w4_packed_bytes() long. */
int matvec_w4_packed_bytes(int out_features, int in_features, int group, int has_zeros, size_t *bytes);
int matvec_w4_pack(const void *codes, const void *scales, const void *zeros, void *packed, int out_features,
                   int in_features, int group, int dtype, void *stream);

/* y[r, o] = epilogue(sum_k x[r, k] * weight(o, k)) for `rows` token rows, the epilogue that of
 * conv2d_fused: bias, activation, and a residual before or after it. Sums are fp32. A row
 * of x with an infinity or NaN gives NaN. Made for the rows of single tokens: the weights are
 * read again for every 32 rows, and from some 64 to 128 rows on conv2d_fused is faster, as a 1x1
 * convolution with the weights' values in 16 bits. */
typedef struct matvec_w4_args {
    const void *x;         /* [rows, in_features], rows x_row elements apart */
    const void *packed;    /* from matvec_w4_pack, with the same sizes, group, zeros and dtype */
    const float *bias;     /* [out_features] or NULL */
    const float *alpha;    /* [out_features], needed by CONV2D_ACT_PRELU */
    const void *residual;  /* [rows, out_features], rows residual_row elements apart, or NULL */
    void *y;               /* [rows, out_features], rows y_row elements apart */
    long long x_row, residual_row, y_row;
    int rows, in_features, out_features, group, has_zeros;
    int act;               /* CONV2D_ACT_*, CONV2D_RES_BEFORE_ACT */
    int dtype;             /* bf16 or f16: of x, the scales, residual and y */
} matvec_w4_args;

int matvec_w4(const matvec_w4_args *args, void *stream);

/* Rows in 8 bits: value (r, k) is scale[r] * code, with a code of -128 .. 127. They are laid out
 * for matmul_q8, which takes activations (a row for each token) and weights (a row for each
 * output) alike: `packed` is 16-byte aligned and q8_packed_bytes() long, and depends on the
 * number of rows. in_features is at most 2^17 - 1, so that sums of products fit 32 bits.
 * quantize_rows chooses, for each row, the scale max(|x|) / 127 (rounded to fp32, at least
 * 2^-126) and the codes x / scale, rounded to the nearest whole number, ties to even, with no
 * error but that. A row with an infinity or a NaN gets a scale of NaN and codes of 0.
 * q8_pack lays out given codes (int8 [rows, in_features], contiguous) and scales (fp32 [rows]);
 * q8_unpack gives both back. */
typedef struct quantize_rows_args {
    const void *x;         /* [rows, in_features], rows x_row elements apart */
    void *packed;
    long long x_row;
    int rows, in_features;
    int dtype;             /* of x */
} quantize_rows_args;

int q8_packed_bytes(int rows, int in_features, size_t *bytes);
int quantize_rows(const quantize_rows_args *args, void *stream);
int q8_pack(const void *codes, const float *scales, void *packed, int rows, int in_features, void *stream);
int q8_unpack(const void *packed, void *codes, float *scales, int rows, int in_features, void *stream);

/* y[r, o] = epilogue(scale_x[r] * scale_w[o] * sum_k code_x[r, k] * code_w[o, k]) for `rows` token
 * rows, the epilogue that of conv2d_fused: bias, activation, and a residual before or after it.
 * The sums are exact; what follows is fp32, rounded once to y. The rows are x, quantized by the
 * call as quantize_rows does (it needs matmul_q8_workspace_size() bytes of workspace, 0 for a few
 * rows, or returns CONV2D_EUNSUPPORTED), or x_packed, for several products of the same rows. A
 * row or an output whose scale is NaN is NaN before the activation, which keeps it but for ReLU's 0. */
typedef struct matmul_q8_args {
    const void *x;         /* [rows, in_features], rows x_row elements apart, or NULL */
    const void *x_packed;  /* where x is NULL: packed rows, with the same sizes */
    const void *weights;   /* out_features packed rows of in_features */
    const float *bias;     /* [out_features] or NULL */
    const float *alpha;    /* [out_features], needed by CONV2D_ACT_PRELU */
    const void *residual;  /* [rows, out_features], rows residual_row elements apart, or NULL */
    void *y;               /* [rows, out_features], rows y_row elements apart */
    long long x_row, residual_row, y_row;
    int rows, in_features, out_features;
    int act;               /* CONV2D_ACT_*, CONV2D_RES_BEFORE_ACT */
    int dtype;             /* of x, residual and y */
} matmul_q8_args;

int matmul_q8(const matmul_q8_args *args, void *stream);
int matmul_q8_workspace_size(const matmul_q8_args *args, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif
