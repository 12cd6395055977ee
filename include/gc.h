/*
 * gc.h -- C ABI of libgc: 2-D convolution forward, d_input and wgrad as
 * im2col-free implicit GEMMs on AMD Instinct MI355X (gfx950).
 *
 * The operation is the one benchmarked in "Speedups to gemm_conv_forward and
 * gemm_conv_backward kernels" (PufferLib pull request #522): a forward conv
 * with an optional fused ReLU (the relu=1/relu=0 flag of its layer-1 and
 * layer-2 benchmark lines), and a backward pass that produces the weight
 * gradient ("wgrad") and the input gradient ("d_input"), in fp32 or bf16
 * (its precision=fp32 / precision=bf16 runs).  Stride S, no padding, dilation
 * 1, one group.  Output size: OH = (H-KH)/S + 1, OW = (W-KW)/S + 1 (integer
 * division; the page's layer 1 maps 11x15, K=5, S=3 to 3x4).  The same page
 * also times a separate bias-gradient kernel for these layers; the bias
 * entry points below add a per-channel bias to the forward pass and compute
 * its gradient.
 *
 *   y [b,oc,oh,ow] = f( sum_{ic,kh,kw} x[b,ic,oh*S+kh,ow*S+kw] * w[oc,ic,kh,kw] )
 *   dz             = relu ? dy * (y > 0) : dy          (derivative 0 at 0)
 *   dx [b,ic,ih,iw] = sum over (oc,oh,ow,kh,kw) with oh*S+kh = ih and
 *                     ow*S+kw = iw of dz[b,oc,oh,ow] * w[oc,ic,kh,kw]
 *   dw [oc,ic,kh,kw] = sum_{b,oh,ow} dz[b,oc,oh,ow] * x[b,ic,oh*S+kh,ow*S+kw]
 *
 * Layouts: x, dx NCHW [B][IC][H][W]; w, dw OIHW [OC][IC][KH][KW]; y, dy NCHW
 * [B][OC][OH][OW]; all dense and contiguous.  Storage type GC_F32 (IEEE fp32)
 * or GC_BF16 (bfloat16, 16-bit words); every tensor of a call has that type.
 * Products are accumulated in fp32; bf16 outputs are rounded to nearest even.
 *
 * Conventions common to every entry point:
 *   - Pointers are device pointers (HBM), owned by the caller, at least
 *     4-byte aligned for fp32 and 2-byte aligned for bf16.  The library
 *     never allocates, frees or synchronises; it enqueues kernels on
 *     `stream` (a hipStream_t; NULL means the default stream) and returns.
 *   - Outputs are overwritten, never accumulated into; every element is
 *     written, including exact zeros (input pixels no window covers).
 *   - Scratch memory, where an operation needs it, is passed in as
 *     `workspace` of `ws_bytes` bytes (device memory, 256-byte aligned);
 *     gc_conv_workspace_bytes() gives the size.  NULL/0 is fine when that
 *     size is 0.  Calls that overlap in time must not share a workspace.
 *   - Errors: an invalid descriptor, flag, dtype or a NULL pointer returns
 *     GC_ERR_INVALID_ARG before any HIP call; a workspace that is too small
 *     returns GC_ERR_WORKSPACE; shapes the kernels cannot tile return
 *     GC_ERR_UNSUPPORTED; a failed launch returns GC_ERR_HIP.  Nothing is
 *     enqueued when an error is returned before the launch.
 *   - Every element count (B*IC*H*W, B*OC*OH*OW, OC*IC*KH*KW) must be below
 *     2^31; larger tensors are rejected with GC_ERR_INVALID_ARG.
 *   - Entry points are reentrant.  The only state is an internal,
 *     thread-safe cache of kernel plans per problem shape.
 */
#ifndef GC_H
#define GC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GC_OK = 0,
    GC_ERR_INVALID_ARG = 1,
    GC_ERR_UNSUPPORTED = 2,
    GC_ERR_WORKSPACE = 3,
    GC_ERR_HIP = 4
} gc_status;

typedef enum { GC_F32 = 0, GC_BF16 = 1 } gc_dtype;

typedef enum {
    GC_OP_FWD = 0,          /* gc_conv_fwd and gc_conv_fwd_bias */
    GC_OP_BWD_DATA = 1,     /* gc_conv_bwd_data */
    GC_OP_BWD_WEIGHT = 2,   /* gc_conv_bwd_weight */
    GC_OP_BWD_BIAS = 3,     /* gc_conv_bwd_bias */
    GC_OP_BWD = 4,          /* gc_conv_bwd */
    GC_OP_BWD_WEIGHT_BIAS = 5   /* gc_conv_bwd_weight_bias */
} gc_op;

/* Problem size.  No padding, dilation 1, one group. */
typedef struct {
    int B, IC, H, W;   /* input  [B][IC][H][W] */
    int OC, KH, KW;    /* weight [OC][IC][KH][KW] */
    int stride;        /* S >= 1, the same along h and w */
} gc_conv_desc;

/* Output extent (pure host arithmetic).  Returns GC_OK and sets *OH, *OW, or
 * GC_ERR_INVALID_ARG for a descriptor with any dimension < 1, H < KH, W < KW,
 * stride < 1, or an element count of 2^31 or more. */
int gc_conv_out_dims(const gc_conv_desc *d, int *OH, int *OW);

/* Bytes of workspace that operation `op` needs for this problem and dtype
 * (0 if none).  Returns 0 as well for an invalid descriptor. */
size_t gc_conv_workspace_bytes(int op, const gc_conv_desc *d, int dtype);

/* Forward pass: y = f(conv(x, w)), f = ReLU when relu == 1, identity when
 * relu == 0.  x [B][IC][H][W], w [OC][IC][KH][KW] in, y [B][OC][OH][OW] out. */
int gc_conv_fwd(const void *x, const void *w, void *y,
                void *workspace, size_t ws_bytes,
                const gc_conv_desc *d, int relu, int dtype, void *stream);

/* The forward pass of gc_conv_fwd, for callers that cannot allocate memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the same arguments without a workspace, the same results bit
 * for bit.  Its scratch memory (the packed weights) is a static device array
 * of 2 MiB per GPU, held by each GPU the library runs on until the process
 * ends; it covers both layer shapes of the PR page at every batch size, and
 * a problem whose gc_conv_workspace_bytes(GC_OP_FWD, ...) exceeds it returns
 * GC_ERR_WORKSPACE before anything is enqueued.  Every call on one GPU shares that
 * GPU's array, so calls that may overlap in time on one GPU (on different
 * streams, or from different threads) race and must not be issued; calls
 * on one stream are ordered and safe.  It never allocates or frees memory. */
int gc_conv_fwd_noalloc(const void *x, const void *w, void *y,
                        const gc_conv_desc *d, int relu, int dtype, void *stream);

/* Forward pass with a bias: y = f(conv(x, w) + bias[oc]).  bias [OC] has the
 * storage type and is added in fp32 before the ReLU; everything else is as in
 * gc_conv_fwd (same workspace size).  bias must not be NULL. */
int gc_conv_fwd_bias(const void *x, const void *w, const void *bias, void *y,
                     void *workspace, size_t ws_bytes,
                     const gc_conv_desc *d, int relu, int dtype, void *stream);

/* Bias gradient: db[oc] = sum_{b,oh,ow} dz[b,oc,oh,ow], dz = dy masked by
 * (y_mask > 0) when relu == 1 (y_mask NULL when relu == 0).  db [OC] out.
 * Summed in fp32 in two stages whose order is fixed by the shape (partials
 * per chunk of images in `workspace`, then an ordered sum), so the result is
 * bit-identical from run to run. */
int gc_conv_bwd_bias(const void *dy, const void *y_mask, void *db,
                     void *workspace, size_t ws_bytes,
                     const gc_conv_desc *d, int relu, int dtype, void *stream);

/* d_input: dx from dy and w.  With relu == 1, dy is masked by (y_mask > 0),
 * y_mask being the forward output y; y_mask must be NULL when relu == 0.
 * dy [B][OC][OH][OW], w [OC][IC][KH][KW], y_mask like dy; dx [B][IC][H][W]
 * out (gather form, no atomics: each dx element is written once). */
int gc_conv_bwd_data(const void *dy, const void *w, const void *y_mask, void *dx,
                     void *workspace, size_t ws_bytes,
                     const gc_conv_desc *d, int relu, int dtype, void *stream);

/* wgrad: dw from x and dy (masked by y_mask > 0 when relu == 1; y_mask NULL
 * when relu == 0).  The sum over B*OH*OW is split across workgroups into fp32
 * partials in `workspace` and finished by a fixed-order reduction, so the
 * result is bit-identical from run to run. */
int gc_conv_bwd_weight(const void *x, const void *dy, const void *y_mask, void *dw,
                       void *workspace, size_t ws_bytes,
                       const gc_conv_desc *d, int relu, int dtype, void *stream);

/* wgrad and the bias gradient together: dw as gc_conv_bwd_weight computes it
 * and db[oc] = sum_{b,oh,ow} dz[b,oc,oh,ow] as gc_conv_bwd_bias does (db [OC]
 * in the storage type; dz = dy masked by y_mask > 0 when relu == 1).  The PR
 * page times the bias gradient as a kernel of its own (its bias-grad lines);
 * here db is one more column of the wgrad tiles, whose x operand is 1, so
 * it is summed from the dz already staged for wgrad and finished by the same
 * fixed-order reduction (bit-identical from run to run).  Shapes whose wgrad
 * kernel has no such column run gc_conv_bwd_weight and gc_conv_bwd_bias.
 * Workspace: gc_conv_workspace_bytes(GC_OP_BWD_WEIGHT_BIAS, ...), 256-byte
 * aligned.  db must not be NULL. */
int gc_conv_bwd_weight_bias(const void *x, const void *dy, const void *y_mask, void *dw,
                            void *db, void *workspace, size_t ws_bytes,
                            const gc_conv_desc *d, int relu, int dtype, void *stream);

/* The whole backward of a layer in one call: dx as gc_conv_bwd_data and dw
 * as gc_conv_bwd_weight compute them, with the same arguments and the same
 * results bit for bit.  The PR page times d_input and wgrad together as one
 * "backward"; this entry point runs them with fewer launches: for bf16
 * shapes with a fused plan, one pre-pass launch (dz regrouping for wgrad and
 * weight packing for d_input), then the two main kernels -- in one launch
 * holding both grids side by side where the d_input grid fits the chip in
 * one round, else one after the other -- and the fixed-order reduction of
 * wgrad's partials; for fp32 shapes with a fused plan, one launch holding the
 * d_input and wgrad grids side by side, then the reduction; for other shapes
 * the two calls one after the other.  The workspace
 * (gc_conv_workspace_bytes(GC_OP_BWD, ...)) must be 256-byte aligned. */
int gc_conv_bwd(const void *x, const void *w, const void *dy, const void *y_mask, void *dx,
                void *dw, void *workspace, size_t ws_bytes,
                const gc_conv_desc *d, int relu, int dtype, void *stream);

/* Which kernels an operation would run for this problem (pure host; the
 * same selection the entry point makes, under the current kernel policy).
 * Writes a NUL-terminated description -- the kernel family and its tiling
 * parameters, e.g. "fwd_ws_bf16 G=4 NBW=2 ..." -- into buf (truncated to
 * buf_bytes - 1 characters).  op is a gc_op value.  Returns GC_OK, or
 * GC_ERR_INVALID_ARG for an invalid descriptor, op or dtype, a NULL buf or
 * buf_bytes == 0.  Enqueues nothing. */
int gc_conv_plan_name(int op, const gc_conv_desc *d, int dtype, char *buf, size_t buf_bytes);

/* ------------------------------------------------------------------------
 * The operators a policy network's training step has around its
 * convolutions.  The conventions above hold, except that element counts may
 * pass 2^31 where a limit below says so, and the workspace, where one is
 * needed, is 256-byte aligned.  Inputs and outputs of a call must not
 * overlap unless a call says that they may.
 * ------------------------------------------------------------------------ */

/* Embedding: the discrete features of an observation (the encoder the PR
 * page times embeds 47 of them into rows of 32 values) or any other tokens.
 *
 *   out[r,t,:]    = scale * table[tok[r,t],:]     (zeros for an empty token)
 *   dtable[v,:]   = scale * sum over (r,t) with tok[r,t] == v of dout[r,t,:]
 *
 * A token outside [0, V) is empty: its output row is zeros and its gradient
 * goes nowhere.  tok has `rows` rows of `tokens` values, ld_tok >= tokens
 * elements apart; out and dout rows of tokens*D elements, ld >= tokens*D
 * elements apart (so the embedding can be part of a wider feature row; the
 * elements between are not touched).  table and dtable are dense [V][D].
 * scale is finite.  rows and tokens may be 0; rows*tokens and tokens*D are below 2^31. */
typedef enum { GC_I32 = 0, GC_I64 = 1, GC_U8 = 2 } gc_index_type;
typedef struct {
    int64_t rows;
    int tokens, V, D;
    int itype;             /* gc_index_type of tok */
    int64_t ld, ld_tok;
} gc_embed_desc;

int gc_embed_fwd(const void *tokens, const void *table, void *out, const gc_embed_desc *d, float scale, int dtype,
                 void *stream);

/* Every row of dtable is written, rows without a token as zeros.  Sums run in
 * fp32, over the tokens sorted by value or, for small tables, as a product with
 * the tokens' one-hot matrix, in an order that the call's sizes and tokens alone
 * fix (and, in a small table's columns beside a non-finite value, that value's
 * place), and are rounded once: the result is bit-identical from run to run. */
size_t gc_embed_workspace_bytes(const gc_embed_desc *d, int dtype);
int gc_embed_bwd(const void *tokens, const void *dout, void *dtable, void *workspace, size_t ws_bytes,
                 const gc_embed_desc *d, float scale, int dtype, void *stream);

/* Group norm with an activation, per image over groups of C/groups channels:
 *
 *   hat = (x - mean) * rstd,  rstd = 1 / sqrt(var + eps)   (var biased)
 *   y   = act(gamma[c] * hat + beta[c])
 *
 * layout GC_NCHW ([B][C][H][W], what the convolutions read and write) or
 * GC_NHWC ([B][H][W][C]).  x, y, dy, dx have the storage type dtype; gamma,
 * beta, dgamma and dbeta [C] have param_dtype, GC_F32 or dtype; gamma == NULL
 * stands for ones, beta == NULL for zeros.  mean and rstd are fp32
 * [B][groups]; the forward writes them where they are not NULL, the backward
 * reads them.  C is at most 2^23, C*H*W and B at most 2^30; B*C*H*W may be
 * larger: GC_ERR_UNSUPPORTED only where a launch would need 2^32 threads. */
typedef enum { GC_NCHW = 0, GC_NHWC = 1 } gc_layout;
typedef enum {
    GC_ACT_NONE = 0,
    GC_ACT_RELU = 1,
    GC_ACT_SILU = 2,       /* z / (1 + exp(-z)) */
    GC_ACT_GELU = 3        /* z * Phi(z), Phi the normal distribution function */
} gc_act;
typedef struct {
    int B, C, H, W;
    int groups;            /* divides C */
    int layout;            /* gc_layout */
    int act;               /* gc_act */
    float eps;             /* >= 0 */
} gc_norm_desc;

/* op GC_OP_FWD or GC_OP_BWD; 0 if none is needed, or for an invalid descriptor. */
size_t gc_group_norm_workspace_bytes(int op, const gc_norm_desc *d, int dtype);
int gc_group_norm_fwd(const void *x, const void *gamma, const void *beta, void *y, float *mean, float *rstd,
                      void *workspace, size_t ws_bytes, const gc_norm_desc *d, int dtype, int param_dtype,
                      void *stream);

/* Which kernels a group norm or an embedding's gradient would run (pure host, as
 * gc_conv_plan_name): op GC_OP_FWD or GC_OP_BWD. */
int gc_group_norm_plan_name(int op, const gc_norm_desc *d, int dtype, char *buf, size_t buf_bytes);
int gc_embed_plan_name(const gc_embed_desc *d, int dtype, char *buf, size_t buf_bytes);

/* With g = dy * act'(gamma*hat + beta) (relu's derivative is 0 at 0):
 *   dbeta = sum g,  dgamma = sum g*hat  (over images and positions)
 *   dx = rstd * (gamma*g - mean(gamma*g) - hat * mean(gamma*g*hat))  (means over the group)
 * The activation's argument is recomputed from x, mean and rstd.  dgamma and
 * dbeta may be NULL.  Sums have a fixed order: bit-identical from run to run. */
int gc_group_norm_bwd(const void *x, const void *gamma, const void *beta, const void *dy, const float *mean,
                      const float *rstd, void *dx, void *dgamma, void *dbeta, void *workspace, size_t ws_bytes,
                      const gc_norm_desc *d, int dtype, int param_dtype, void *stream);

/* The global norm of a list of gradients, and their clipping by it:
 *
 *   norm = |prescale| * sqrt(sum over all elements of src^2)
 *   dst  = prescale * min(1, max_norm / (norm + eps)) * src
 *
 * The list is host memory, read during the call; a captured graph keeps its
 * own copy.  Tensors may differ in type and size (n may be 0, the list
 * empty), and together hold up to 2^42 elements; dst may be src.  Squares are
 * added in fp64 in a fixed order.  norm (fp32, one value) is written in any
 * case.  A norm that is NaN makes every dst NaN, an infinite one makes finite
 * elements 0 and the others NaN, as the formula says; gc_grad_norm writes the
 * norm alone and leaves dst unread. */
typedef struct {
    const void *src;
    void *dst;
    int64_t n;
    int dtype;
} gc_tensor;

size_t gc_grad_clip_workspace_bytes(int count);
int gc_grad_norm(const gc_tensor *list, int count, float prescale, float *norm, void *workspace, size_t ws_bytes,
                 void *stream);
int gc_grad_clip(const gc_tensor *list, int count, float max_norm, float prescale, float eps, float *norm,
                 void *workspace, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * The recurrent core that a policy has behind its encoder, and the loss of its
 * head.  The conventions of the operators above hold.
 * ------------------------------------------------------------------------ */

/* Layer norm of rows, with the residual stream's addition in the same pass:
 *
 *   s     = x + residual                 (x alone where residual is NULL)
 *   y     = gamma * (s - mean) * rstd + beta,  rstd = 1 / sqrt(var + eps)  (var biased, over the row)
 *   total = s                            (where total is not NULL)
 *
 * s is added in fp32 and normed as it is; total and y are each rounded once.
 * Rows have D values and lie ld elements apart (ld >= D: parts of wider rows;
 * the elements between are not touched).  gamma, beta, dgamma and dbeta [D]
 * have param_dtype, GC_F32 or dtype; gamma == NULL stands for ones, beta ==
 * NULL for zeros.  mean and rstd [rows] are fp32; the forward writes them where
 * they are not NULL.  total may be residual or x, with the same row distance.
 * rows may be 0 and is at most 2^31 - 1; D is at most 2^23. */
typedef struct {
    int64_t rows;
    int D;
    float eps;                                   /* >= 0 */
    int64_t ld_x, ld_residual, ld_total, ld_y;   /* elements between rows */
} gc_layer_norm_desc;

int gc_layer_norm_fwd(const void *x, const void *residual, const void *gamma, const void *beta, void *y, void *total,
                      float *mean, float *rstd, const gc_layer_norm_desc *d, int dtype, int param_dtype, void *stream);

/* With x the normed rows (the forward's total where it had a residual), hat =
 * (x - mean) * rstd and w = gamma * dy:
 *
 *   dx     = dtotal + rstd * (w - mean of w - hat * mean of w*hat)   (means over the row)
 *   dgamma = sum over rows of dy*hat,  dbeta = sum over rows of dy
 *
 * dtotal, the gradient that reaches the residual stream past the norm, may be
 * NULL; dx is the gradient of x and of the residual alike, and may be dtotal or
 * dy, with the same row distance.  Row distances: x ld_x, dy ld_y, dtotal ld_total, dx
 * ld_residual.  dgamma and dbeta may be NULL; with rows == 0 they are zeros.
 * Sums have a fixed order: bit-identical from run to run. */
size_t gc_layer_norm_workspace_bytes(const gc_layer_norm_desc *d, int dtype);
int gc_layer_norm_bwd(const void *x, const void *gamma, const void *dy, const void *dtotal, const float *mean,
                      const float *rstd, void *dx, void *dgamma, void *dbeta, void *workspace, size_t ws_bytes,
                      const gc_layer_norm_desc *d, int dtype, int param_dtype, void *stream);

/* The gated linear recurrence over B sequences of up to T steps of D channels:
 *
 *   a = sigmoid(gate),  i = coupled ? 1 - a : 1
 *   h[b,t,:] = a[b,t,:] * (reset[b,t] ? 0 : h[b,t-1,:]) + i[b,t,:] * value[b,t,:],   out = h
 *
 * a and i are each right in their own size, to (1.5|gate| + 8) * 2^-24 (0 where below 1e-38): a gate that is
 * open keeps a state over any number of steps, one that closes leaves the value beside a state of any size.
 *
 * h before the first step is h0 [B][D] (fp32; NULL for zeros), after the last
 * one it is written to last [B][D] (fp32, may be NULL, may be h0).  reset, one
 * byte a step (not 0: the step starts anew, as after an episode's end or at the
 * start of a sequence in a packed row; whatever the state held, also if it was
 * not finite), and lengths [B] (int32; values are taken into [0, T]) may be NULL.
 * Steps at and behind a sequence's length are not read; its out there is zeros,
 * its last the state at its length.  T == 1 is the step of a policy that acts.
 *
 * gate, value, out and their gradients have the storage type, D dense channels,
 * and two distances each (elements; reset: bytes): any order of batch and time,
 * and parts of wider rows.  Distances of inputs may be 0; elements of outputs
 * must not overlap.  States are fp32.  states, where it is not NULL, is what the
 * backward needs: [B][ceil(T/16)][D] fp32, h before every sixteenth step.
 * B and T may be 0; T is at most 2^30, GC_ERR_UNSUPPORTED where B*D is 2^31
 * or more. */
enum { GC_RECURRENCE_BLOCK = 16 };      /* steps between two kept states */
typedef struct {
    int64_t batch, step;                /* distance of two sequences, of two steps */
} gc_strides;
typedef struct {
    int B, T, D;
    int coupled;                        /* 0 or 1 */
    gc_strides gate, value, out, dgate, dvalue, reset;
} gc_recurrence_desc;

size_t gc_recurrence_workspace_bytes(int op, const gc_recurrence_desc *d, int dtype);
int gc_recurrence_fwd(const void *gate, const void *value, const float *h0, const uint8_t *reset, const int32_t *lengths,
                      void *out, float *last, float *states, void *workspace, size_t ws_bytes,
                      const gc_recurrence_desc *d, int dtype, void *stream);

/* With g the gradient of h[b,t,:], which is dout and what comes back from the
 * step after it (dlast [B][D], NULL for zeros, behind the last step), and h' the state
 * a step starts from (0 at a reset):
 *
 *   dvalue = i * g,   dgate = a * (1 - a) * (h' - (coupled ? value : 0)) * g,   dh0 = h0's share
 *
 * h' is computed anew from states, so out is not read.  dout has the distances
 * of out.  dgate and dvalue are zeros behind a sequence's length.  dh0 [B][D]
 * fp32 may be NULL, and may be dlast.  Every sum has a fixed order. */
int gc_recurrence_bwd(const void *gate, const void *value, const float *states, const uint8_t *reset,
                      const int32_t *lengths, const void *dout, const float *dlast, void *dgate, void *dvalue, float *dh0,
                      void *workspace, size_t ws_bytes, const gc_recurrence_desc *d, int dtype, void *stream);

/* Distillation of a head from a teacher's K top logits a row, at a temperature t:
 *
 *   p = softmax(teacher / t) over the row's entries,  q = softmax(logits / t) over its V logits
 *   loss     = t^2 * sum over entries of p * (log p - log q[index])
 *   dlogits  = dloss * t * (q - sum of the p of the entries at that place)
 *
 * An entry whose index is outside [0, V) is empty, and an entry of p == 0 adds
 * nothing; several entries may have one index.  A row without any entry of a
 * teacher's logit above -inf has loss 0 and gradient 0, whatever its logits
 * hold.  A logit of -inf has q == 0 (its loss is infinite where p is not 0), in a
 * row of nothing else as well.
 * The forward also writes peak, the largest logit, and mass, the sum of
 * exp((logits - peak) / t) (either may be NULL); the backward reads them.  dloss,
 * loss, peak and mass are fp32 [rows].  logits and dlogits have the storage
 * type, rows ld and ld_grad elements apart (>= V), index and teacher rows
 * ld_index and ld_teacher elements apart (>= K).  dlogits may be logits, with the
 * same row distance.  rows may be 0; rows and V are below 2^31, K is from 1 to 1024. */
typedef struct {
    int64_t rows;
    int V, K;
    int itype;              /* GC_I32 or GC_I64 */
    int teacher_dtype;      /* gc_dtype of teacher */
    float temperature;      /* from 1e-18 to 1e18 */
    int64_t ld, ld_grad, ld_index, ld_teacher;
} gc_distill_desc;

int gc_distill_fwd(const void *logits, const void *index, const void *teacher, float *loss, float *peak, float *mass,
                   const gc_distill_desc *d, int dtype, void *stream);
int gc_distill_bwd(const void *logits, const void *index, const void *teacher, const float *peak, const float *mass,
                   const float *dloss, void *dlogits, const gc_distill_desc *d, int dtype, void *stream);
/* Both at once, where dloss is known before the loss (a mean over rows, say):
 * one read of the logits where a row fits a workgroup's registers. */
int gc_distill_step(const void *logits, const void *index, const void *teacher, const float *dloss, float *loss,
                    void *dlogits, const gc_distill_desc *d, int dtype, void *stream);

/* Which kernels these would run (pure host, as gc_conv_plan_name): op is GC_OP_FWD or GC_OP_BWD
 * (the layer norm's without a residual, or a gradient past it; the recurrence's without lengths, with which each of
 * the sequences begins with a wave), for the distillation also GC_OP_STEP, both at once. */
enum { GC_OP_STEP = 6 };
int gc_layer_norm_plan_name(int op, const gc_layer_norm_desc *d, int dtype, char *buf, size_t buf_bytes);
int gc_recurrence_plan_name(int op, const gc_recurrence_desc *d, int dtype, char *buf, size_t buf_bytes);
int gc_distill_plan_name(int op, const gc_distill_desc *d, int dtype, char *buf, size_t buf_bytes);

/* Human-readable name of a status code. */
const char *gc_status_string(int status);

/* Index-mapper self-check (pure host): builds the magic-number divider for
 * `divisor` exactly as the kernels use it (Granlund & Montgomery, "Division
 * by invariant integers using multiplication", 1994), applies it to every
 * n in [0, n_end) with the same arithmetic the device performs, and returns
 * the number of quotients or remainders that differ from n / divisor and
 * n % divisor.  Requires 1 <= divisor and n_end <= 2^31; returns -1 otherwise. */
int64_t gc_fastdiv_selfcheck(uint32_t divisor, uint32_t n_end);

/* Kernel selection policy, process-wide.  GC_POLICY_AUTO (the default) runs
 * the image-group kernels wherever a shape fits them and the shape-generic
 * kernels elsewhere; GC_POLICY_GENERIC runs the shape-generic kernels for
 * every shape (used to test both families on the same problems).  Returns
 * the previous policy, or -1 for an unknown value (nothing changes).  Calls
 * already enqueued are not affected; set it only while no other thread is
 * issuing calls. */
enum { GC_POLICY_AUTO = 0, GC_POLICY_GENERIC = 1 };
int gc_set_kernel_policy(int policy);

/* Library version, as major*10000 + minor*100 + patch. */
int gc_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GC_H */
