/*
 * miconv_lm.h -- C ABI of the sequence operators of language models: the short
 * causal convolution, the selective state space scan, the gated linear
 * recurrence, the RMS norm with the residual's addition, products with 4-bit
 * weights and adapters of many requests, for gfx950.  Same library, dtypes,
 * descriptors and status codes as miconv.h.
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
 *
 * LM_GATED, LM_GATED_BWD, LM_GATED_STEP
 *   k[c] = value log(1 + exp(decay[c])),  a = exp(-k sigmoid(r)),
 *   h[c] <- a h[c] + sqrt(1 - a^2) sigmoid(i) x[c],   y = h
 *   r is LM_A and i LM_B, both as x; decay is LM_D, f32 [C]; lm_args.value is
 *   finite and not negative; states f32 [sequences, C].  x, r, i and y share
 *   one dtype, and gradients have the types of what they are gradients of.
 *   With g_t = gy_t + a_{t+1} g_{t+1} (gstate behind the last step), s =
 *   sqrt(1 - a^2) and q = g (a h_{t-1} - sigmoid(i) x a^2 / s):
 *   dx = g s sigmoid(i), di = g s x sigmoid'(i), dr = -k q sigmoid'(r),
 *   ddecay = -value sigmoid(decay) sum q sigmoid(r).  Where a is 1 (r or decay
 *   far below zero) what is divided by s counts as zero, its limit.
 *   LM_SAVED (f32, lm_plan_t.saved_floats elements): the state in front of
 *   every 64th step, written by LM_GATED and read by LM_GATED_BWD.
 *
 * LM_NORM, LM_NORM_BWD
 *   v = x + residual (in f32; residual is LM_STATE_IN, zero without it),
 *   rstd = 1 / sqrt(mean over C of v^2 + value),  y = v rstd w
 *   x, y and the residual are [N, C, L] or [N, C]; LM_STATE_OUT, present with
 *   the residual, is v rounded to x's dtype; LM_SAVED is rstd, f32 [N, L] or
 *   [N].  A row whose squares' sum passes f32's range has rstd 0.
 *   With y in LM_F8 (e4m3: 4 bits of exponent, 3 of mantissa, largest value
 *   448) LM_SCALES, f32 [N, G, L] or [N, G], has a scale for each group of
 *   C / G channels -- one group, or groups of 32, 64 or 128: top / 448, top the
 *   largest |y| of the group, and what is stored is y 448 / top rounded to
 *   nearest even.  top counts as 2^-112 at least; a group of zeros has scale 1,
 *   one with a NaN has scale NaN.
 *   LM_NORM_BWD: x is v as LM_NORM rounded it or, with LM_STATE_IN, both are what
 *   LM_NORM had and v is their sum in f32.  With u = v rstd:
 *   dx = gstate + rstd (w gy - u mean(w gy u)),  dw = sum over rows of gy u;
 *   gstate (optional) is the gradient of LM_STATE_OUT.  dx is the gradient of x
 *   and of the residual.
 *
 * LM_ADAPTERS
 *   y[m,n] = base[m,n] + scaling[e] scales[m] sum_r (sum_k x[m,k] A[e,r,k]) B[e,n,r],
 *   e = index[m], for rows with an e of 0 .. E-1; y = base for the others.
 *   x is [M, K] or [N, K, L] (row m = n L + l), in A's dtype or LM_F8, the latter
 *   with LM_SCALES f32 [M, 1] or [N, 1, L]; A [E, R, K], B [E, N', R]; index is
 *   LM_ROWS, int32 [M] or [N, L]; base (zero without it) is LM_Z, [M, N'] or
 *   [N, N', L], and may be y itself; scaling (one without it) is LM_D, f32 [E].
 *   R is 1 .. 256.  The inner sums stay in f32.
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
#define LM_F8 18       /* float8 e4m3 (finite and NaN) */

typedef enum lm_op {
    LM_CONV = 0,
    LM_CONV_BWD = 1,
    LM_CONV_STEP = 2,
    LM_SCAN = 3,
    LM_SCAN_BWD = 4,
    LM_SCAN_STEP = 5,
    LM_MV4 = 6,
    LM_GATED = 7,
    LM_GATED_BWD = 8,
    LM_GATED_STEP = 9,
    LM_NORM = 10,
    LM_NORM_BWD = 11,
    LM_ADAPTERS = 12
} lm_op;

/* The tensors of a call, by place in lm_plan's and lm_run's arrays.  A place
 * with rank 0 (and a NULL pointer) is absent.  What GATED*, NORM* and ADAPTERS
 * put where is said with their formulas. */
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
    float value;       /* GATED*: the factor of k; NORM*: what is added to the mean; else not looked at */
    int64_t max_len;   /* packed calls: a length that few sequences pass (0: T); it only
                          decides how the work is split, results hold for any value and the
                          workspace follows T and the number of sequences */
    int64_t chunk;     /* 0: chosen; else rows per chunk of the long axis (rounded up as the kernel needs);
                          NORM*, ADAPTERS: 0 */
} lm_args;

typedef struct lm_plan_t {
    int32_t op, dtype;
    lm_args args;
    conv_tensor t[LM_NSLOT];
    int64_t seqs;      /* sequences (batch rows of a *_STEP or NORM*, products' rows of x for MV4, ADAPTERS) */
    int64_t C, L;      /* channels (MV4, ADAPTERS: outputs), rows of one x row */
    int64_t K;         /* taps; MV4, ADAPTERS: columns of x */
    int64_t S, G;      /* states, groups; MV4, NORM: G = groups of columns; ADAPTERS: rank, adapters */
    int64_t chunk, chunks;       /* rows per chunk, chunks per sequence (packed: of max_len rows);
                                    ADAPTERS: rows per tile, parts of the columns */
    int64_t saved_floats;        /* SCAN*, GATED*: elements of LM_SAVED */
    int64_t workspace_bytes;
    int64_t flops, bytes;        /* algorithmic work of one call (packed calls: of T rows) */
} lm_plan_t;

/*
 * lm_plan -- check a call's descriptors and arguments and fill a plan.
 *   tensors  LM_NSLOT descriptors.
 *   err, err_len  optional buffer for a message on failure.
 * Returns CONV_OK, CONV_EINVAL (shapes, types, missing or surplus tensors), or
 * CONV_EUNSUPPORTED (K, S, group, rank or a norm's channels outside the kernels'
 * range, or a call of 2^32 or more threads in one launch).
 */
MICONV_API int lm_plan(int32_t op, const conv_tensor *tensors, const lm_args *args, lm_plan_t *out, char *err,
                       size_t err_len);

/*
 * lm_run -- enqueue the planned call on the stream.
 *   ptrs       LM_NSLOT device pointers, NULL where the plan's tensor is absent or empty.
 *   workspace  workspace_bytes of device memory, 256-byte aligned; its content before and
 *              after means nothing.
 * An output must not overlap an input, except for the in-place state of a step
 * and a base of ADAPTERS that is y itself (same pointer and strides).
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
