/*
 * miconv_lm.h -- C ABI of the sequence operators of language models: the short
 * causal convolution, the selective state space scan and products with 4-bit
 * weights, for gfx950.  Same library, dtypes, descriptors and status codes as
 * miconv.h.
 *
 * Two calls: lm_plan checks tensor descriptors and arguments and fills a plan
 * (no device call); lm_run checks the pointers and enqueues the kernels on the
 * caller's stream (no synchronisation, no device allocation).  A plan serves
 * every later call with the same descriptors and arguments.  The library keeps
 * no state of its own between calls.
 *
 * Logical layouts follow miconv.h: activations are [N, C, L] with any element
 * strides; fastest are channels-last rows (C fastest).  A packed batch is
 * [1, C, T] with an LM_OFFSETS tensor (int32 [sequences + 1], on the device,
 * ascending from 0 to T): sequence s is the rows offsets[s] .. offsets[s+1]-1,
 * of any length, zero included.  Offsets are clamped to 0..T by the kernels;
 * outputs at rows that no sequence covers mean nothing.
 *
 * Formulas (f32 arithmetic and sums, one rounding to the output's type):
 *
 * LM_CONV, LM_CONV_BWD, LM_CONV_STEP
 *   p[c,t] = bias[c] + sum_{k<K} w[c,k] xx[c, t-K+1+k],   y = act(p),
 *   xx = x for indices >= 0 and state_in[c, K-1+i] for i = -(K-1) .. -1 (zero
 *   without state_in); state_out[c, j] = xx[c, L-(K-1)+j].  K is 1 .. 8;
 *   x, w, bias, y and the states share one dtype.
 *   Gradients: g = gy * act'(p), dx[t] = sum_k w[k] g[t+K-1-k] (g = 0 past the
 *   end; indices below 0 give dstate), dw[k] = sum g[t] xx[t-K+1+k],
 *   dbias = sum g; gstate, the gradient of state_out, adds to dx and dstate.
 *
 * LM_SCAN, LM_SCAN_BWD, LM_SCAN_STEP
 *   d = dt + dt_bias, or log(1 + exp(dt + dt_bias)) with LM_SOFTPLUS
 *   h[c,s] <- exp(d A[c,s]) h[c,s] + d x[c] B[g,s],   g = c / (C / G)
 *   y[c] = (sum_s C[g,s] h[c,s] + D[c] x[c]) * silu(z[c])
 *   x, dt, z, y, B and C share one dtype; A [C, S], D, dt_bias [C] and the
 *   states [N, C, S] are f32; B and C are [N, G, S, L].  S is 1 .. 64.
 *   Gradients have the types of what they are gradients of.  d = 0 (dt the
 *   type's lowest value, with softplus) leaves a state as it is, also for an
 *   infinite A, which counts as the largest number: A = -inf forgets the state
 *   at every step of d > 0.  A state that has overflowed to infinity may turn
 *   into NaN where the axis is split.
 *   LM_SAVED (f32, lm_plan_t.saved_floats elements): the states every few
 *   steps, written by LM_SCAN and read by LM_SCAN_BWD.
 *
 * LM_MV4
 *   y[m,n] = bias[n] + sum_k x[m,k] scales[n,k/group] (q[n,k] - zeros[n,k/group])
 *   q: uint8 [N, K/2], the low four bits the even k; zeros default to 8;
 *   scales and zeros [N, K/group] in x's dtype.  group = K / (columns of
 *   scales), a multiple of 32.  A row of x whose sums pass f32's range at 256
 *   times x (one with an infinity does) gives infinities or NaN.
 */
#ifndef MICONV_LM_H
#define MICONV_LM_H

#include "miconv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further element types of descriptors. */
#define LM_I32 16
#define LM_U8 17

typedef enum lm_op {
    LM_CONV = 0,
    LM_CONV_BWD = 1,
    LM_CONV_STEP = 2,
    LM_SCAN = 3,
    LM_SCAN_BWD = 4,
    LM_SCAN_STEP = 5,
    LM_MV4 = 6
} lm_op;

/* The tensors of a call, by place in lm_plan's and lm_run's arrays.  A place
 * with rank 0 (and a NULL pointer) is absent. */
typedef enum lm_slot {
    LM_X = 0,       /* CONV*, SCAN*: [N, C, L]; *_STEP: [N, C]; MV4: [M, K] */
    LM_W,           /* CONV*: [C, K]; MV4: uint8 [N, K/2] */
    LM_BIAS,        /* optional; CONV*: [C]; MV4: [N] */
    LM_Y,           /* output; optional in SCAN (only states wanted) */
    LM_STATE_IN,    /* optional in CONV*, SCAN*: [sequences, C, K-1] or f32 [sequences, C, S] */
    LM_STATE_OUT,   /* optional output; *_STEP: the state, read and updated in place */
    LM_OFFSETS,     /* optional: int32 [sequences + 1] */
    LM_GY,          /* *_BWD: the output's gradient */
    LM_GSTATE,      /* *_BWD: optional gradient of STATE_OUT */
    LM_DX, LM_DW, LM_DBIAS, LM_DSTATE,  /* *_BWD outputs; each optional except SCAN_BWD's DX */
    LM_DT,          /* SCAN*: as X */
    LM_A, LM_B, LM_C,
    LM_D, LM_Z, LM_DT_BIAS,             /* optional */
    LM_DDT, LM_DA, LM_DB, LM_DC,        /* SCAN_BWD outputs */
    LM_DD, LM_DZ, LM_DDT_BIAS,          /* SCAN_BWD outputs, present with D, Z, DT_BIAS */
    LM_SAVED,       /* SCAN: optional output; SCAN_BWD: input */
    LM_ROWS,        /* *_STEP: optional int32 [N], the state row of each batch row (distinct;
                       a row outside the state is left out: its y is zero) */
    LM_SCALES, LM_ZEROS,
    LM_NSLOT
} lm_slot;

/* lm_args.flags */
#define LM_SILU 1      /* CONV*: act is silu (else the identity) */
#define LM_SOFTPLUS 2  /* SCAN* */

typedef struct lm_args {
    int32_t flags;
    int32_t reserved;
    int64_t max_len;   /* packed calls: a length that few sequences pass (0: T); it only
                          decides how the work is split, results hold for any value and the
                          workspace follows T and the number of sequences */
    int64_t chunk;     /* 0: chosen; else rows per chunk of the long axis (rounded up as the kernel needs) */
} lm_args;

typedef struct lm_plan_t {
    int32_t op, dtype;
    lm_args args;
    conv_tensor t[LM_NSLOT];
    int64_t seqs;      /* sequences (batch rows of a *_STEP, products' rows of x for MV4) */
    int64_t C, L;      /* channels (MV4: outputs), rows of one x row */
    int64_t K;         /* taps; MV4: columns of x */
    int64_t S, G;      /* states, groups; MV4: G = groups of columns (K / G columns each) */
    int64_t chunk, chunks;       /* rows per chunk, chunks per sequence (packed: of max_len rows) */
    int64_t saved_floats;        /* SCAN*: elements of LM_SAVED */
    int64_t workspace_bytes;
    int64_t flops, bytes;        /* algorithmic work of one call (packed calls: of T rows) */
} lm_plan_t;

/*
 * lm_plan -- check a call's descriptors and arguments and fill a plan.
 *   tensors  LM_NSLOT descriptors.
 *   err, err_len  optional buffer for a message on failure.
 * Returns CONV_OK, CONV_EINVAL (shapes, types, missing or surplus tensors), or
 * CONV_EUNSUPPORTED (K, S or group outside the kernels' range, or a call of 2^32
 * or more threads in one launch).
 */
MICONV_API int lm_plan(int32_t op, const conv_tensor *tensors, const lm_args *args, lm_plan_t *out, char *err,
                       size_t err_len);

/*
 * lm_run -- enqueue the planned call on the stream.
 *   ptrs       LM_NSLOT device pointers, NULL where the plan's tensor is absent or empty.
 *   workspace  workspace_bytes of device memory, 256-byte aligned; its content before and
 *              after means nothing.
 * An output must not overlap an input, except for the in-place state of a step.
 * Returns CONV_OK, CONV_EINVAL (a missing pointer, a small workspace),
 * CONV_EALIGN (a pointer off its element size; LM_MV4: weights off 16 bytes),
 * or CONV_EDEVICE.
 */
MICONV_API int lm_run(const lm_plan_t *plan, void *const *ptrs, void *workspace, size_t workspace_bytes,
                      void *stream);

#ifdef __cplusplus
}
#endif
#endif /* MICONV_LM_H */
