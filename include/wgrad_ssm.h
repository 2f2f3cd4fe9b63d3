/*
 * wgrad_ssm.h -- C ABI of the selective state space operators of the MI355X
 * (gfx950) library (libwgrad.so): the short causal depthwise convolution and
 * the selective scan, each for whole sequences, backward, and for single
 * tokens. Errors, streams, ownership and wgrad_last_error() are those of
 * wgrad.h: every entry point returns a wgrad_status, the caller owns every
 * device buffer and the stream, nothing is synchronised, no device memory is
 * allocated, and no C++ exception crosses the boundary.
 *
 * Rows. Activations are rows of channels (one row per token, channels last),
 * given as a pointer and the distance between rows in elements, so that x may
 * be one half of a wider matrix. Consecutive elements of a row are adjacent.
 * A sequence is a run of rows:
 *   dense  (packed = 0): N sequences of L rows; sequence n starts at row n*L;
 *   packed (packed = 1): T rows in all; sequence n is rows seq_start[n] to
 *     seq_start[n+1] - 1, with seq_start a device array of N + 1 int32 that
 *     does not decrease, from 0 to T, and no sequence longer than L. Lengths
 *     of 0 are allowed. The array is read on the device only: a value out of
 *     range cannot make a kernel leave its buffers (starts and ends are
 *     clamped to 0..T and the length to L) but gives meaningless results.
 * Pointers need the alignment of their element type, workspaces and saved
 * states 16 bytes. Runs over sequences use accesses of up to 16 bytes at any
 * such alignment; the runs for single tokens use them where pointers, row
 * strides and channels come in whole ones. Row strides are at least the row's
 * width and at most 2^23 elements (of a convolution 2^20). Outputs must not
 * overlap inputs or each other, except where an entry point updates a state in
 * place.
 */
#ifndef WGRAD_SSM_H
#define WGRAD_SSM_H

#include "wgrad.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows of elements: element (r, c) is at ptr[r * stride + c]. */
typedef struct {
    void* ptr;
    int64_t stride;
} wgrad_rows;

/* ------------------------------------------------------------ causal convolution
 *
 *   p[r,c] = bias[c] + sum_{k=0}^{W-1} w[c,k] * x[r - (W-1) + k, c]
 *   y      = p                      (WGRAD_ACT_NONE)
 *   y      = p / (1 + exp(-p))      (WGRAD_ACT_SILU)
 *
 * for each row r of a sequence; the W-1 rows before its first row are
 * init_state[n][0..W-2], or zeros where init_state is NULL. final_state[n]
 * receives the last W-1 rows of (init_state[n], the sequence), so that a
 * later call can go on from there. It is the depthwise (C/G = K/G = 1) 1D
 * convolution of wgrad.h with pad_lo = W-1, pad_hi = 0, and w and dw have
 * that convolution's weight layout [C][W].
 */
typedef enum { WGRAD_ACT_NONE = 0, WGRAD_ACT_SILU = 1 } wgrad_activation;

typedef struct {
    int32_t dtype;      /* wgrad_dtype of x, w, bias, y, dy, dx and the states */
    int32_t activation; /* wgrad_activation */
    int32_t W;          /* filter taps, 1 to 8 */
    int32_t packed;     /* 0 or 1 */
    int64_t N, L;       /* sequences >= 0, rows per sequence (packed: at most) >= 0 */
    int64_t T;          /* packed: rows in all, at most N*L; dense: 0 or N*L */
    int64_t C;          /* channels >= 1 */
} wgrad_cconv_problem;

/* One block for all entry points; each reads the fields its comment names. */
typedef struct {
    wgrad_rows x, y, dy, dx;
    const void* w;             /* [C][W] */
    const void* bias;          /* [C], or NULL: no bias */
    const void* init_state;    /* [N][W-1][C], or NULL: zeros */
    void* final_state;         /* [N][W-1][C], or NULL: not wanted */
    const int32_t* seq_start;  /* [N+1], packed only (else NULL) */
    float* dw;                 /* [C][W] fp32 */
    float* dbias;              /* [C] fp32, or NULL: not wanted */
    const void* dfinal_state;  /* [N][W-1][C], or NULL: zeros */
    void* dinit_state;         /* [N][W-1][C], or NULL: not wanted */
    void* state;               /* step: pool of states [num_slots][W-1][C], updated in place */
    const int32_t* slots;      /* step: device array [rows], or NULL: row i uses state i */
    int64_t rows, num_slots;   /* step */
    void* ws;                  /* backward: workspace of wgrad_cconv_workspace_bytes */
    size_t ws_bytes;
} wgrad_cconv_args;

typedef struct wgrad_cconv_plan_s wgrad_cconv_plan_t;

/* Validate a problem and choose the launch shapes (host only). hip_device as
 * in wgrad_plan. Errors: WGRAD_ERR_INVALID_ARG for sizes or codes out of the
 * ranges above, and for N, L, or rows in all beyond 2^30 or C beyond 2^20. */
int wgrad_cconv_plan(const wgrad_cconv_problem* problem, int hip_device, wgrad_cconv_plan_t** out);
void wgrad_cconv_plan_destroy(wgrad_cconv_plan_t* plan);

/* Bytes of workspace the backward run needs (fp32 partial sums of dw and
 * dbias); a NULL plan gives 0. */
size_t wgrad_cconv_workspace_bytes(const wgrad_cconv_plan_t* plan);

/* y (and final_state) from x, w, bias, init_state, seq_start. One kernel. */
int wgrad_cconv_run(const wgrad_cconv_plan_t* plan, const wgrad_cconv_args* args, void* stream);

/* dx, dw, dbias, dinit_state from x, w, bias, init_state, dy, dfinal_state,
 * seq_start. The value before the activation is recomputed. dw and dbias are
 * summed in fp32 in one fixed order (no atomics): the same plan on the same
 * inputs gives the same bits. Two kernels. */
int wgrad_cconv_backward_run(const wgrad_cconv_plan_t* plan, const wgrad_cconv_args* args, void* stream);

/* One token for each of args->rows rows: row i takes its W-1 previous inputs
 * from state[slots[i]], writes y row i and moves that state on by its x row,
 * in place. Only W, C, dtype and the activation of the plan matter. A slot
 * outside 0..num_slots-1 (padding of a batch) leaves every state alone and
 * gives a y row of zeros. Two rows must not name the same slot. */
int wgrad_cconv_step_run(const wgrad_cconv_plan_t* plan, const wgrad_cconv_args* args, void* stream);

/* ------------------------------------------------------------ selective scan
 *
 * Per row r of a sequence, channel c (of group g = c / (C/G)) and state s:
 *   d      = softplus(delta[r,c] + delta_bias[c])     (softplus = 0: without it)
 *   h[c,s] = exp(d * A[c,s]) * h[c,s] + d * x[r,c] * B[r,g,s]
 *   y[r,c] = (sum_s C[r,g,s] * h[c,s] + D[c] * x[r,c]) * silu(z[r,c])
 * h starts as init_state[n] (or 0) and ends as final_state[n]. delta_bias, D
 * and z are optional (0, 0 and no gate). Rows of B and C hold G groups of S
 * values. States, exponentials and sums are fp32; an exponential below 2^-126
 * counts as 0, and a rate A below -2.3e38 (-infinity too) as -2.3e38.
 */
typedef struct {
    int32_t dtype;     /* wgrad_dtype of x, delta, B, C, z, y and their gradients */
    int32_t softplus;  /* 0 or 1 */
    int32_t packed;    /* 0 or 1 */
    int32_t reserved;  /* must be 0 */
    int64_t N, L, T;   /* as in wgrad_cconv_problem */
    int64_t C, G, S;   /* channels, groups of B and C (C a multiple of G, G at most 2^16), states
                          per channel 1 to 128 */
} wgrad_scan_problem;

typedef struct {
    wgrad_rows x, delta, B, C, z, y;                 /* z.ptr may be NULL */
    const float* A;                                  /* [C][S] */
    const float* D;                                  /* [C] or NULL */
    const float* delta_bias;                         /* [C] or NULL */
    const float* init_state;                         /* [N][C][S] or NULL */
    float* final_state;                              /* [N][C][S] or NULL */
    const int32_t* seq_start;                        /* [N+1], packed only */
    void* saved;                                     /* wgrad_scan_saved_bytes, or NULL: no backward run follows */
    wgrad_rows dy, dx, ddelta, dB, dC, dz;           /* backward; dz if z */
    float *dA, *dD, *ddelta_bias;                    /* fp32; dD and ddelta_bias may be NULL */
    const float* dfinal_state;                       /* [N][C][S] or NULL: zeros */
    float* dinit_state;                              /* [N][C][S] or NULL: not wanted */
    float* state;                                    /* step: [num_slots][C][S], updated in place */
    const int32_t* slots;                            /* step: device array [rows], or NULL: row i uses state i */
    int64_t rows, num_slots;                         /* step */
    void* ws;                                        /* wgrad_scan_workspace_bytes of the direction */
    size_t ws_bytes;
} wgrad_scan_args;

/* What a plan decided, for logging and tests. */
typedef struct {
    int32_t lanes;              /* lanes that share a channel's states */
    int32_t states_per_lane;
    int32_t segments;           /* pieces a sequence of L rows is split into, forward */
    int32_t segments_backward;
    int64_t segment_rows, segment_rows_backward;
    int64_t chunk_rows;         /* rows between two saved states */
    int64_t workspace_bytes, workspace_bytes_backward, saved_bytes;
} wgrad_scan_plan_info;

/* Overrides for tests and benchmarks; 0 means "the plan decides". Production
 * callers pass NULL. */
typedef struct {
    int32_t segments;           /* forward pieces of a sequence of L rows, at least 32 rows each */
    int32_t segments_backward;
} wgrad_scan_overrides;

typedef struct wgrad_scan_plan_s wgrad_scan_plan_t;

/* Validate a problem and choose the split of the sequences (host only).
 * Errors as wgrad_cconv_plan, with C up to 2^23. */
int wgrad_scan_plan(const wgrad_scan_problem* problem, const wgrad_scan_overrides* overrides, int hip_device,
                    wgrad_scan_plan_t** out);
void wgrad_scan_plan_destroy(wgrad_scan_plan_t* plan);
int wgrad_scan_plan_query(const wgrad_scan_plan_t* plan, wgrad_scan_plan_info* info);

/* Workspace of the forward (backward = 0) or backward run, and the size of
 * the saved states that a forward run leaves for the backward run of the same
 * plan (the state before every chunk_rows-th row of each sequence; the format
 * is the library's own). A NULL plan gives 0. */
size_t wgrad_scan_workspace_bytes(const wgrad_scan_plan_t* plan, int backward);
size_t wgrad_scan_saved_bytes(const wgrad_scan_plan_t* plan);

/* y, final_state and saved from x, delta, A, B, C, D, z, delta_bias,
 * init_state, seq_start. */
int wgrad_scan_run(const wgrad_scan_plan_t* plan, const wgrad_scan_args* args, void* stream);

/* dx, ddelta, dA, dB, dC, dD, dz, ddelta_bias, dinit_state from the forward
 * run's inputs, its saved states (which hold init_state), dy and
 * dfinal_state. All sums are fp32 in one fixed order (no atomics): the same
 * plan on the same inputs gives the same bits. */
int wgrad_scan_backward_run(const wgrad_scan_plan_t* plan, const wgrad_scan_args* args, void* stream);

/* One token for each of args->rows rows, from and into state[slots[i]], in
 * place; y row i. Slots as in wgrad_cconv_step_run. Only C, G, S, dtype and
 * softplus of the plan matter. */
int wgrad_scan_step_run(const wgrad_scan_plan_t* plan, const wgrad_scan_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* WGRAD_SSM_H */
