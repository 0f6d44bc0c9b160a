/*
 * ssm.h -- C ABI of the MI355X (gfx950) S6 selective-scan library.
 *
 * The method (pages: "mamba, live", section "what is actually running";
 * "the s6 cell", section "the recurrence"; TensorViz "Carry context through a
 * selective state", explorer page and manifest steps "local", "select",
 * "state", "read"):
 *
 *   u      = SiLU(causal_depthwise_conv_W(x))         (optional, fused)
 *   dt     = softplus(dt_raw + dt_bias)                per (b, t, d)
 *   A      = -exp(A_log)                               per (d, n)
 *   h[n]  <- exp(dt*A[n]) * h[n] + coef(dt, A[n]) * B[t, n] * u
 *            coef = dt                 (SSM_DISC_DELTA_B, the dt*B form)
 *            coef = expm1(dt*A) / A    (SSM_DISC_ZOH, exact zero-order hold)
 *   y      = (sum_n C[t, n] * h[n] + Dskip * u) * SiLU(z)   (C reads the
 *            updated state; the gate only when z is given)
 *
 * The same diagonal cell h <- a*h + b*u with the decay fixed per channel
 * instead of computed per token ("the s6 cell", section "one cell, two
 * architectures"; the fixed-decay side) is selected with
 * disc = SSM_DECAY_CONST:
 *   h[n]  <- exp(A[n]) * h[n] + B[t, n] * u,   A = -exp(A_log)
 * with no step size: dt_raw and dt_bias are not read (they may be NULL) and
 * the backward produces no d_dt_raw / d_dt_bias (those outputs are not
 * written).  State width is dstate (1 for a scalar state per channel).
 *
 * Conventions shared by every call
 *  - Layouts are row-major and channel-last:
 *      x, u, dt_raw, z, y and their gradients       [B, L, D]
 *      B, C and their gradients                     [B, L, N]  (shared by all channels)
 *      A_log, dA_log                                [D, N]
 *      dt_bias, Dskip, conv_b and their gradients   [D]
 *      conv_w                                       [D, W]  (tap W-1 multiplies the current input)
 *      h0, hT, dh0, dhT                             [B, D, N]
 *      conv_state_in / conv_state_out               [B, W-1, D]  (oldest input first)
 *  - Tensors marked "io" hold SSM_F32 or SSM_BF16 values as chosen by the
 *    descriptor's io_dtype; every parameter, state and parameter gradient is
 *    float32.  bf16 results are rounded to nearest, ties to even.
 *  - Every pointer is a DEVICE pointer, except the descriptor pointers, which
 *    are host pointers read before the call returns.  The caller owns all
 *    memory: the library never allocates, frees or keeps a pointer after a
 *    call returns.  Every tensor must start on a 16-byte boundary.
 *  - A NULL optional pointer means "absent": dt_bias, Dskip, conv_b read as 0;
 *    z means "no gate"; h0 and conv_state_in read as zeros; a NULL output is
 *    not written.
 *  - Work is enqueued on `stream` (a hipStream_t; NULL = the default stream)
 *    and is asynchronous: nothing synchronises inside a call.  Calls are
 *    reentrant; concurrent calls on different streams must use different
 *    workspaces and outputs.
 *  - Errors: every call returns an ssm_status.  Argument errors are detected
 *    on the host before any HIP call is made, and then nothing is enqueued.
 *    SSM_ERR_HIP reports a failed launch; a fault inside a kernel surfaces at
 *    the caller's next synchronisation.
 *  - Inputs must be finite.  Outputs may not overlap inputs or each other,
 *    except the exact in-place pairs named below.
 */
#ifndef SSM_AMD_SSM_H
#define SSM_AMD_SSM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SSM_ABI_VERSION 2

typedef int32_t ssm_status;
#define SSM_OK 0
#define SSM_ERR_NULL_ARG 1     /* a required pointer is NULL */
#define SSM_ERR_BAD_SHAPE 2    /* a size is out of range or inconsistent, or needs a launch grid
                                  above 2^31 - 1 workgroups */
#define SSM_ERR_UNSUPPORTED 3  /* a valid request the library does not implement */
#define SSM_ERR_WORKSPACE 4    /* workspace NULL or smaller than the queried size */
#define SSM_ERR_ALIGNMENT 5    /* a tensor does not start on a 16-byte boundary */
#define SSM_ERR_ALIAS 6        /* buffers overlap in a way the call does not allow */
#define SSM_ERR_HIP 7          /* a HIP launch failed */
#define SSM_ERR_SCRATCH_LIMIT 8  /* the request needs more than the static scratch buffer holds */
#define SSM_ERR_HOST_MEMORY 9    /* the host had no memory for the call's checks */

#define SSM_F32 0
#define SSM_BF16 1

#define SSM_DISC_DELTA_B 0     /* write = dt * B * u ("mamba, live"; "the s6 cell") */
#define SSM_DISC_ZOH 1         /* write = expm1(dt*A)/A * B * u (TensorViz explorer) */
#define SSM_DECAY_CONST 2      /* decay exp(A) fixed per (channel, state), write = B * u,
                                  no step size ("the s6 cell", "one cell, two architectures") */

#define SSM_MAX_DSTATE 64
#define SSM_MAX_CONV_WIDTH 8
#define SSM_MAX_SCAN_DIM ((1 << 24) - 1)   /* channels of a sequence scan: a 64-token tile of one
                                             [B, L, D] float32 tensor, and one backward state
                                             checkpoint (D * N <= 64 * D floats), stay under 2^32
                                             bytes, the reach of the kernels' 32-bit offsets */
#define SSM_STATIC_SCRATCH_BYTES (16u << 20)   /* ssm_scan_fwd_static's device buffer, per GPU */

/* Descriptor of a sequence scan (forward or backward). */
typedef struct ssm_scan_desc {
    int64_t batch;       /* B >= 1 */
    int64_t seqlen;      /* L >= 0 */
    int64_t dim;         /* D in [1, SSM_MAX_SCAN_DIM], inner channels */
    int64_t dstate;      /* N in [1, SSM_MAX_DSTATE] */
    int32_t conv_width;  /* 0: x already is the scan input u; 1..8: fused causal conv + SiLU */
    int32_t io_dtype;    /* SSM_F32 or SSM_BF16 */
    int32_t disc;        /* SSM_DISC_DELTA_B, SSM_DISC_ZOH or SSM_DECAY_CONST */
    int32_t chunk_len;   /* 0: library's choice; > 0: split time into chunks of this
                            length (two-level scan); -1: never split time */
} ssm_scan_desc;

/* Descriptor of one streaming step for a stack of independent blocks. */
typedef struct ssm_step_desc {
    int64_t nblocks;     /* >= 1; every per-block tensor gains a leading [nblocks] axis */
    int64_t nstreams;    /* S >= 1 concurrent sequences */
    int64_t dim;         /* D >= 1 */
    int64_t dstate;      /* N in [1, SSM_MAX_DSTATE] */
    int32_t conv_width;  /* 0: x is u; 1..8: causal conv over the carried history + SiLU */
    int32_t io_dtype;    /* SSM_F32 or SSM_BF16 for x, dt_raw, B, C, z, y */
    int32_t disc;        /* SSM_DISC_DELTA_B, SSM_DISC_ZOH or SSM_DECAY_CONST */
    int32_t state_dtype; /* storage of h: SSM_F32 (0), or SSM_BF16 (updated in float32 and
                            rounded to nearest, ties to even, when stored) */
} ssm_step_desc;

/* Descriptor of a causal depthwise convolution. */
typedef struct ssm_conv_desc {
    int64_t batch;       /* B >= 1 */
    int64_t seqlen;      /* L >= 0 */
    int64_t dim;         /* D >= 1 */
    int32_t width;       /* W in [1, SSM_MAX_CONV_WIDTH] */
    int32_t fuse_silu;   /* 1: y = SiLU(conv), 0: y = conv */
    int32_t io_dtype;    /* SSM_F32 or SSM_BF16 for x and y */
    int32_t reserved;    /* must be 0 */
} ssm_conv_desc;

/* Shape of a whole Mamba-style language model (ssm_model_decode_step). */
typedef struct ssm_model_desc {
    int64_t nstreams;    /* S >= 1 independent token streams decoded together */
    int32_t vocab;       /* V >= 1 tokens; the head is tied to the embedding */
    int32_t d_model;     /* residual width, 1 .. SSM_MAX_D_MODEL */
    int32_t n_layers;    /* blocks, >= 1 */
    int32_t d_inner;     /* inner channels per block, >= 1 */
    int32_t d_state;     /* N in [1, SSM_MAX_DSTATE] */
    int32_t dt_rank;     /* rank of the step-size projection, >= 1 */
    int32_t conv_width;  /* W in [1, SSM_MAX_CONV_WIDTH] */
    int32_t reserved;    /* must be 0 */
} ssm_model_desc;
#define SSM_MAX_D_MODEL 8192

/* One block's weights, all float32 device pointers (PyTorch Linear layout,
 * [out_features, in_features]).  NULL optionals: norm_w 1, norm_b 0,
 * conv_b 0, dt_proj_b 0, Dskip 0. */
typedef struct ssm_layer_weights {
    const float *norm_w, *norm_b;      /* [d_model] LayerNorm (eps 1e-5), optional */
    const float *in_proj;              /* [2*d_inner, d_model]: rows 0..d_inner-1 give xin, the rest z */
    const float *conv_w;               /* [d_inner, W], tap W-1 on the current input */
    const float *conv_b;               /* [d_inner], optional */
    const float *x_proj;               /* [dt_rank + 2*d_state, d_inner]: rows give dt, B, C in that order */
    const float *dt_proj_w;            /* [d_inner, dt_rank] */
    const float *dt_proj_b;            /* [d_inner], optional (the scan's dt_bias) */
    const float *A_log;                /* [d_inner, d_state] */
    const float *Dskip;                /* [d_inner], optional */
    const float *out_proj;             /* [d_model, d_inner] */
} ssm_layer_weights;

/* Library version (SSM_ABI_VERSION * 100 + minor). */
int32_t ssm_version(void);

/* Static English text of a status code (never NULL). */
const char *ssm_status_string(ssm_status status);

/*
 * conv1d_causal -- causal depthwise convolution, optionally followed by SiLU
 * ("mamba, live": xc = SiLU(depthwise_conv4(xin)), 4-tap causal, per channel;
 * TensorViz manifest step "local": left padded, reads the current and W-1
 * earlier inputs).
 *   y[b,t,d] = act(b[d] + sum_{k<W} w[d,k] * xt[b, t-(W-1)+k, d])
 * with xt = x for index >= 0 and the carried history state_in (or 0) before.
 *   x         io  [B, L, D]     input
 *   w         f32 [D, W]        taps (required)
 *   b         f32 [D]           bias, optional
 *   state_in  f32 [B, W-1, D]   history before x, optional (zeros)
 *   state_out f32 [B, W-1, D]   the last W-1 inputs after x, optional; must not
 *                               overlap state_in (SSM_ERR_ALIAS)
 *   y         io  [B, L, D]     output (required when L > 0)
 */
ssm_status conv1d_causal(const ssm_conv_desc *desc, const void *x, const float *w,
                         const float *b, const float *state_in, float *state_out,
                         void *y, void *stream);

/* Bytes of device workspace ssm_scan_fwd needs for this descriptor (0 when
 * time is not split). */
ssm_status ssm_scan_fwd_workspace_size(const ssm_scan_desc *desc, size_t *bytes);

/*
 * ssm_scan_fwd -- the selective scan over a whole sequence (the recurrence
 * above, run for t = 0 .. L-1 from h0).  Long sequences with little batch and
 * channel parallelism are split in time into chunks whose end states are
 * combined by the associative rule (P1, W1) then (P2, W2) = (P1*P2, P2*W1 + W2)
 * and then re-scanned from their exact starting states; the result equals the
 * sequential recurrence up to rounding.
 *   x              io  [B, L, D]   u, or the conv input when conv_width > 0 (required)
 *   dt_raw         io  [B, L, D]   required (not read with SSM_DECAY_CONST)
 *   dt_bias        f32 [D]         optional
 *   A_log          f32 [D, N]      required
 *   B, C           io  [B, L, N]   required
 *   Dskip          f32 [D]         optional
 *   z              io  [B, L, D]   gate input, optional
 *   conv_w         f32 [D, W]      required when conv_width > 0, else ignored
 *   conv_b         f32 [D]         optional
 *   conv_state_in  f32 [B, W-1, D] optional
 *   conv_state_out f32 [B, W-1, D] optional (may be exactly conv_state_in)
 *   h0             f32 [B, D, N]   optional
 *   hT             f32 [B, D, N]   optional (may be exactly h0)
 *   y              io  [B, L, D]   required when L > 0
 *   workspace      device memory of ssm_scan_fwd_workspace_size bytes (may be
 *                  NULL when that size is 0)
 */
ssm_status ssm_scan_fwd(const ssm_scan_desc *desc, const void *x, const void *dt_raw,
                        const float *dt_bias, const float *A_log, const void *B,
                        const void *C, const float *Dskip, const void *z,
                        const float *conv_w, const float *conv_b,
                        const float *conv_state_in, float *conv_state_out,
                        const float *h0, float *hT, void *y,
                        void *workspace, size_t workspace_bytes, void *stream);

/*
 * ssm_scan_fwd_static -- ssm_scan_fwd without a workspace argument, for
 * callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc).  Arguments,
 * results and errors are those of ssm_scan_fwd; the chunk summaries of a
 * time split go to a buffer of SSM_STATIC_SCRATCH_BYTES that the library
 * holds on every GPU it runs on (a static device array, kept until the
 * process ends).  The call allocates nothing.
 *   Returns SSM_ERR_SCRATCH_LIMIT, before any HIP call, when
 *   ssm_scan_fwd_workspace_size for the same descriptor exceeds
 *   SSM_STATIC_SCRATCH_BYTES (pass a shorter chunk_len, or -1, or use
 *   ssm_scan_fwd with a workspace).
 *   Every call on one GPU shares that GPU's buffer: calls that overlap on a
 *   GPU (on different streams, or from different host threads without
 *   ordering) race on it and must be serialised by the caller.  Calls on one
 *   stream are ordered and safe.  The buffer keeps the last call's contents;
 *   every value a call reads from it is written earlier in the same call.
 *   The first call on a device looks up the buffer's device address (a HIP
 *   call that is not capturable): make one call on each device before any
 *   graph capture.
 */
ssm_status ssm_scan_fwd_static(const ssm_scan_desc *desc, const void *x, const void *dt_raw,
                               const float *dt_bias, const float *A_log, const void *B,
                               const void *C, const float *Dskip, const void *z,
                               const float *conv_w, const float *conv_b,
                               const float *conv_state_in, float *conv_state_out,
                               const float *h0, float *hT, void *y, void *stream);

/* Bytes of device workspace ssm_scan_bwd needs for this descriptor. */
ssm_status ssm_scan_bwd_workspace_size(const ssm_scan_desc *desc, size_t *bytes);

/*
 * ssm_scan_bwd -- gradients of ssm_scan_fwd for the loss
 * sum(y * dy) + sum(hT * dhT).  The pages state that the selection maps
 * receive gradients (TensorViz explorer, numerical checks) but give no
 * backward; this is the reverse-mode adjoint of the recurrence: with
 * g = dLoss/dh_t, g_{t-1} = exp(dt_t*A) * g_t + C_{t-1} * dyv_{t-1}.  With
 * conv_width > 0 the conv + SiLU prologue ("mamba, live": the 4-tap causal
 * conv before the scan; TensorViz manifest step "local") is differentiated
 * in the same pass: u is recomputed from x, and the gradient of u flows on
 * through SiLU and the taps to x, conv_w, conv_b and conv_state_in.
 *   x, dt_raw, B, C, z, dy    io  as in ssm_scan_fwd (dy [B, L, D] required)
 *   dt_bias, A_log, Dskip, h0 f32 as in ssm_scan_fwd
 *   conv_w, conv_b, conv_state_in  f32 as in ssm_scan_fwd (conv_w required
 *                             when conv_width > 0; all ignored when it is 0)
 *   dhT        f32 [B, D, N]  optional upstream gradient of hT
 *   dx, d_dt_raw, dz   io [B, L, D]  optional outputs (dx is dLoss/dx: the
 *                                    scan input u when conv_width is 0; dz
 *                                    needs z)
 *   dB, dC             io [B, L, N]  optional outputs (summed over channels)
 *   d_dt_bias, dDskip  f32 [D]       optional outputs (summed over batch and time)
 *                                    (d_dt_raw and d_dt_bias are not written with
 *                                    SSM_DECAY_CONST, which has no step size)
 *   dA_log             f32 [D, N]    optional output (summed over batch and time)
 *   dh0                f32 [B, D, N] optional output
 *   dconv_w   f32 [D, W]      optional output (summed over batch and time)
 *   dconv_b   f32 [D]         optional output (summed over batch and time)
 *   dconv_state_in f32 [B, W-1, D]  optional output, the gradient of the
 *                             carried history (written whether or not
 *                             conv_state_in was given)
 *   The three conv outputs must be NULL when conv_width is 0.
 *   workspace  device memory of ssm_scan_bwd_workspace_size bytes (required)
 * Time chunks (desc->chunk_len: 0 the library's choice, -1 never, > 0 this
 * length rounded up to a multiple of 64): with few channel workgroups the
 * sequence is split in time.  The forward's chunk scan and carry give every
 * chunk its exact start state; a reverse walk over chunk summaries gives its
 * end adjoint (over a chunk the adjoint is affine, g_start = prod(exp(dt*A))
 * * g_end + R); every chunk then runs the backward sweep independently.  The
 * result equals the unsplit backward up to rounding.
 */
ssm_status ssm_scan_bwd(const ssm_scan_desc *desc, const void *x, const void *dt_raw,
                        const float *dt_bias, const float *A_log, const void *B,
                        const void *C, const float *Dskip, const void *z,
                        const float *conv_w, const float *conv_b, const float *conv_state_in,
                        const float *h0, const void *dy, const float *dhT,
                        void *dx, void *d_dt_raw, float *d_dt_bias, float *dA_log,
                        void *dB, void *dC, float *dDskip, void *dz, float *dh0,
                        float *dconv_w, float *dconv_b, float *dconv_state_in,
                        void *workspace, size_t workspace_bytes, void *stream);

/*
 * ssm_step -- one token of batched streaming decode ("mamba, live": one token
 * in, one token out, constant work; the whole memory is h plus a (W-1)-token
 * conv history per channel).  For every block k, stream s and channel d:
 *   u = SiLU(conv_b + sum_{j<W-1} conv_w[j] * hist[j] + conv_w[W-1] * x)   (conv_width > 0)
 *   hist <- [hist[1..W-2], x]
 *   then one recurrence step of the scan with u, updating h in place.
 * y reads the updated state; with state_dtype SSM_BF16 what is kept for the
 * next token is its bfloat16 rounding (the pages keep the state in float32;
 * bf16 storage halves the state traffic that bounds a decode step).
 * Tensors (each with a leading [nblocks] axis, block-major):
 *   h          f32 or bf16 [S, D, N]   state (state_dtype), in/out (required)
 *   conv_state f32 [S, W-1, D] history, in/out (required when conv_width > 1)
 *   x, dt_raw  io  [S, D]      required (dt_raw not read with SSM_DECAY_CONST)
 *   B, C       io  [S, N]      required
 *   z          io  [S, D]      optional gate input
 *   conv_w     f32 [D, W]      required when conv_width > 0
 *   conv_b, dt_bias, Dskip  f32 [D]  optional
 *   A_log      f32 [D, N]      required
 *   y          io  [S, D]      output (required)
 */
ssm_status ssm_step(const ssm_step_desc *desc, void *h, float *conv_state, const void *x,
                    const void *dt_raw, const void *B, const void *C, const void *z,
                    const float *conv_w, const float *conv_b, const float *dt_bias,
                    const float *A_log, const float *Dskip, void *y, void *stream);

/*
 * ssm_model_decode_step -- one token of every stream through a whole
 * Mamba-style language model ("mamba, live", section "what is actually
 * running": the streaming form, one token in, one token out):
 *   x = emb[token]
 *   for each block:  hn = LayerNorm(x);  [xin, z] = in_proj(hn)
 *                    u = SiLU(causal conv of xin over the carried history)
 *                    [dt, B, C] = x_proj(u);  dt_raw = dt_proj_w dt
 *                    one ssm_step of the block's state with u, dt_raw,
 *                    dt_bias = dt_proj_b, B, C and the gate z -> y
 *                    x += out_proj(y)
 *   logits = LayerNorm_out(x) emb^T          (head tied to the embedding)
 * The projections run on the matrix cores in float32.  Everything is float32.
 *   desc        host pointer, the model's shape
 *   emb         f32 [V, d_model]   embedding and head (required)
 *   norm_f_w, norm_f_b  f32 [d_model]  final LayerNorm, optional (1, 0)
 *   layers      HOST array of n_layers ssm_layer_weights (device pointers inside),
 *               read before the call returns
 *   tokens      int32 [S]           device; a token outside [0, V) makes that
 *                                   stream's logits and state NaN
 *   h           f32 [n_layers, S, d_inner, d_state]   state, in/out (zeros to start)
 *   conv_state  f32 [n_layers, S, W-1, d_inner]       conv history, in/out (oldest
 *                                   first; may be NULL when W = 1)
 *   logits      f32 [S, V]          output
 *   workspace   ssm_model_decode_workspace_size bytes (required)
 * Every pointer must be 16-byte aligned, except tokens (4-byte aligned);
 * outputs may not overlap the inputs, the workspace or each other.
 */
ssm_status ssm_model_decode_workspace_size(const ssm_model_desc *desc, size_t *bytes);
ssm_status ssm_model_decode_step(const ssm_model_desc *desc, const float *emb, const float *norm_f_w,
                                 const float *norm_f_b, const ssm_layer_weights *layers,
                                 const int32_t *tokens, float *h, float *conv_state, float *logits,
                                 void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * The rest of a training step around ssm_scan_bwd: the layer norm of the
 * residual stream ("mamba, live": LayerNorm before every block and before the
 * tied head), the log-probabilities of the head's tokens, a policy loss on
 * them, and clipping of the gradients.  The pages give no training code; the
 * formulas are stated at each call.
 *
 * Rows: T rows of a [.., D] or [.., V] tensor whose values are contiguous and
 * whose rows lie `stride` values apart (0: contiguous rows; otherwise at least
 * the row's length).  Values between two rows are not read or written, but
 * count as part of the tensor where overlap is checked.  T = 0 is allowed.
 * A tensor here may be a slice of a larger one: it needs its own element's
 * alignment only (2 or 4 bytes; vectors start on 16 bytes where the tensor
 * does, which is faster).  Workspaces start on 16 bytes.
 * -------------------------------------------------------------------------- */

/* Descriptor of a layer norm, forward or backward. */
typedef struct ssm_norm_desc {
    int64_t rows;        /* T >= 0 */
    int64_t dim;         /* D in [1, SSM_MAX_NORM_DIM] */
    int64_t x_stride;    /* rows of x */
    int64_t r_stride;    /* rows of residual; backward: dresidual */
    int64_t s_stride;    /* rows of residual_out; backward: dx */
    int64_t y_stride;    /* rows of y; backward: dy */
    int32_t io_dtype;    /* SSM_F32 or SSM_BF16 */
    float eps;           /* > 0, finite (checked, not used, by the backward) */
} ssm_norm_desc;
#define SSM_MAX_NORM_DIM 16384

/*
 * ssm_layer_norm_fwd -- per row, with s = x + residual in float32,
 *   mean = mean(s),  rstd = 1 / sqrt(mean((s - mean)^2) + eps)
 *   y = (s - mean) * rstd * weight + bias
 * s is normalised before it is rounded to io for residual_out.  Sums are
 * float32: rows reaching past 1e18 either way may overflow their squares.
 *   x            io  [T, D]  required when T > 0
 *   residual     io  [T, D]  optional
 *   weight, bias f32 [D]     optional (1, 0)
 *   residual_out io  [T, D]  optional, s (may be exactly x or exactly residual)
 *   y            io  [T, D]  required when T > 0
 *   mean, rstd   f32 [T]     optional (what the backward takes)
 */
ssm_status ssm_layer_norm_fwd(const ssm_norm_desc *desc, const void *x, const void *residual,
                              const float *weight, const float *bias, void *residual_out,
                              void *y, float *mean, float *rstd, void *stream);

/* Bytes of device workspace ssm_layer_norm_bwd needs for this descriptor. */
ssm_status ssm_layer_norm_bwd_workspace_size(const ssm_norm_desc *desc, size_t *bytes);

/*
 * ssm_layer_norm_bwd -- gradients of ssm_layer_norm_fwd, with
 * xh = (x - mean) * rstd and g = dy * weight:
 *   dx = rstd * (g - mean(g) - xh * mean(g * xh)) + dresidual
 *   dweight = sum over rows of dy * xh,  dbias = sum over rows of dy
 * dx is the gradient of s, so of both x and residual of the forward.
 *   x          io  [T, D]  the normalised tensor (the forward's residual_out
 *                          where it had a residual)
 *   mean, rstd f32 [T]     from the forward
 *   dy         io  [T, D]  upstream gradient of y
 *   dresidual  io  [T, D]  optional upstream gradient of s itself
 *   weight     f32 [D]     optional (1)
 *   dx         io  [T, D]  optional output (may be exactly dy or exactly dresidual)
 *   dweight, dbias f32 [D] optional outputs (zeros when T = 0); the order of
 *                          their sums is fixed for a shape: float32 over at
 *                          most 512 rows and 16 such groups, 64-bit above
 *   workspace  ssm_layer_norm_bwd_workspace_size bytes (required)
 * x, mean, rstd and dy are required when T > 0.
 */
ssm_status ssm_layer_norm_bwd(const ssm_norm_desc *desc, const void *x, const float *weight,
                              const float *mean, const float *rstd, const void *dy,
                              const void *dresidual, void *dx, float *dweight, float *dbias,
                              void *workspace, size_t workspace_bytes, void *stream);

/* Descriptor of the token log-probabilities, forward or backward. */
typedef struct ssm_logp_desc {
    int64_t rows;            /* T >= 0 tokens */
    int64_t vocab;           /* V in [1, SSM_MAX_VOCAB] */
    int64_t logits_stride;   /* rows of logits (V padded to a wider row, say) */
    int64_t dlogits_stride;  /* rows of dlogits */
    int32_t io_dtype;        /* SSM_F32 or SSM_BF16 for logits and dlogits */
    int32_t reserved;        /* must be 0 */
} ssm_logp_desc;
#define SSM_MAX_VOCAB (1 << 24)

/*
 * ssm_token_logp_fwd -- log softmax of each row at its target:
 *   m = max_j z_j,  l = log(sum_j exp(z_j - m)),  logp = z_target - m - l
 * A logit may be -infinity or the type's lowest value (a token ruled out): it
 * adds nothing to the sum; a target ruled out by -infinity has logp
 * -infinity, and a row of nothing but -infinity gives NaN.
 *   logits   io    [T, V]
 *   targets  int32 [T]     a negative target means the row has none: its
 *                          logits are not read and logp and stats are 0; a
 *                          target >= V gives NaN
 *   logp     f32   [T]     output
 *   stats    f32   [T, 2]  optional output (m, l), what the backward takes
 */
ssm_status ssm_token_logp_fwd(const ssm_logp_desc *desc, const void *logits, const int32_t *targets,
                              float *logp, float *stats, void *stream);

/*
 * ssm_token_logp_bwd -- gradient of sum(logp * dlogp):
 *   dlogits_j = dlogp * ([j = target] - exp(z_j - m - l))
 *   dlogp    f32 [T]     upstream gradient; where it is 0, or the target is
 *                        negative, the row's logits are not read and its
 *                        gradient is exactly 0
 *   dlogits  io  [T, V]  output (may be exactly logits, with its stride)
 * All pointers are required when T > 0.  A target >= V gives a NaN row.
 */
ssm_status ssm_token_logp_bwd(const ssm_logp_desc *desc, const void *logits, const int32_t *targets,
                              const float *stats, const float *dlogp, void *dlogits, void *stream);

#define SSM_REDUCE_MEAN 0   /* divide by the counted tokens' summed weights */
#define SSM_REDUCE_SUM 1

/* Descriptor of the policy loss. */
typedef struct ssm_policy_desc {
    int64_t rows;            /* T >= 0 tokens */
    int64_t vocab;           /* V in [1, SSM_MAX_VOCAB] */
    int64_t logits_stride, dlogits_stride;
    double clip_low;         /* in [0, 1]: ratios are held above 1 - clip_low */
    double clip_high;        /* >= 0 (infinity: no upper bound): ... below 1 + clip_high */
    double kl_beta;          /* weight of the KL term, >= 0, finite */
    double grad_scale;       /* factor on dlogits alone (loss scaling, accumulation), finite */
    int32_t io_dtype;        /* SSM_F32 or SSM_BF16 for logits and dlogits */
    int32_t reduction;       /* SSM_REDUCE_MEAN or SSM_REDUCE_SUM */
} ssm_policy_desc;

/* Bytes of device workspace ssm_policy_loss needs for this descriptor. */
ssm_status ssm_policy_loss_workspace_size(const ssm_policy_desc *desc, size_t *bytes);

/*
 * ssm_policy_loss -- clipped policy loss with a KL term, and its gradient.
 * Per token, with logp as in ssm_token_logp_fwd, r = exp(logp - old_logp),
 * A = advantage and d = ref_logp - logp:
 *   policy = -min(r * A, clip(r, 1 - clip_low, 1 + clip_high) * A)
 *   kl     = exp(d) - 1 - d                      (>= 0; 0 when d = 0)
 *   loss   = sum over tokens of weight * (policy + kl_beta * kl)  / norm
 * norm is the sum of the counted tokens' weights (SSM_REDUCE_MEAN; with
 * nothing counted the loss is 0) or 1 (SSM_REDUCE_SUM).  A token counts when
 * its target is not negative and its weight is not 0; of a token that does not
 * count nothing else is read, its logp is 0 and its row of dlogits exactly 0,
 * whatever its logits hold.  A target >= V, or a row of -infinity, makes the
 * loss and its own row NaN.  A token exactly on a bound of r is not clipped.
 *   logits     io    [T, V]  required when T > 0
 *   targets    int32 [T]     required when T > 0
 *   old_logp   f32   [T]     the policy the tokens were drawn from, optional
 *                            (absent: the present one, r = 1 with its gradient)
 *   ref_logp   f32   [T]     the reference of the KL term, optional (no term)
 *   advantages f32   [T]     required when T > 0
 *   weights    f32   [T]     optional (1); 0 leaves a token out
 *   loss       f32   [4]     output (required): the loss; its policy and KL
 *                            terms, without kl_beta; the share of clipped
 *                            tokens; each summed with the weights and divided
 *                            by norm
 *   logp       f32   [T]     optional output
 *   dlogits    io    [T, V]  optional output, grad_scale * dloss/dlogits (may be
 *                            exactly logits, with its stride)
 *   workspace  ssm_policy_loss_workspace_size bytes (required)
 * The order of the sums is fixed for a shape and the rows' places within 16
 * bytes.
 */
ssm_status ssm_policy_loss(const ssm_policy_desc *desc, const void *logits, const int32_t *targets,
                           const float *old_logp, const float *ref_logp, const float *advantages,
                           const float *weights, float *loss, float *logp, void *dlogits,
                           void *workspace, size_t workspace_bytes, void *stream);

/* One tensor of ssm_clip_grad_norm (a slice of a flat buffer, say). */
typedef struct ssm_grad {
    const void *grad;    /* numel values (device) */
    void *out;           /* numel values (device): grad clipped; exactly grad (with its type): in
                            place; NULL: the tensor counts in the norm and is not written */
    int64_t numel;       /* >= 0 */
    int32_t grad_dtype;  /* SSM_F32 or SSM_BF16 */
    int32_t out_dtype;   /* SSM_F32 or SSM_BF16 */
} ssm_grad;
#define SSM_MAX_GRADS (1 << 16)

/*
 * ssm_clip_grad_norm -- global norm of a list of gradients, and clipping:
 *   norm = sqrt(sum over every value of g^2)
 *   factor = min(1, max_norm / (norm + 1e-6)),   out = factor * g
 * Squares and sums are 64-bit.  A NaN among the gradients makes norm, factor
 * and every output NaN; an infinity makes the norm infinite and the factor 0.
 * With factor 1 a tensor clipped in place is not written.
 *   grads      HOST array of `count` ssm_grad (0 <= count <= SSM_MAX_GRADS),
 *              read before the call returns; at most 2^40 values together
 *   max_norm   >= 0; infinity measures and leaves every value as it is (the
 *              factor is 1, also with a norm that is not finite)
 *   norm       f32 [2]  output (required): norm (infinite above float32's range,
 *                       the factor is still right), factor
 *   workspace  ssm_clip_grad_norm_workspace_size bytes (required)
 * Outputs may not overlap each other or any other tensor's gradient.  The
 * order of the sums is fixed for a list's sizes.
 */
ssm_status ssm_clip_grad_norm_workspace_size(const ssm_grad *grads, int64_t count, size_t *bytes);
ssm_status ssm_clip_grad_norm(const ssm_grad *grads, int64_t count, double max_norm, float *norm,
                              void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_AMD_SSM_H */
