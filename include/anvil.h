/*
 * anvil.h -- C ABI of libanvil, the ANVIL bank step on GB300 (sm_103a).
 *
 * The operation is the one defined on the page "modded-nanogpt
 * track_1_short/optim/anvil.py", function `anvil_cascade` and the constants
 * above it (ANVIL_MAPS, RAIL_FAST_BETA / RAIL_SLOW_BETA / RAIL_FAST_WEIGHT,
 * FROBENIUS_MARGIN / FROBENIUS_EPS).  For every matrix G of a bank [g, m, n]:
 *
 *   v0 <- v0 + (1 - fast_beta) (G - v0)          fast rail   (velocity[0])
 *   v1 <- v1 + (1 - slow_beta) (G - v1)          slow rail   (velocity[1])
 *   blend = w v0 + (1 - w) v1                    w = fast_weight
 *   X  = bf16(G + momentum (blend - G))          Nesterov lookahead
 *   tall (m > n): A = X^T X, update X <- a X + X B
 *   wide (m <= n, square included): A = X X^T, update X <- a X + B X
 *   d  = sqrt(trace of the bf16 first Gram) * margin + eps
 *   X  <- bf16(X / d), A <- bf16(A / d^2)
 *   for each map (a, b, c): [A = bf16(Gram(X)) after the first]
 *       B = bf16(b A + c A A);  X <- bf16(a X + X B  |  a X + B X)
 *   out = X
 *
 * Every number is computed on the GPU by this library's own kernels; there is
 * no CPU path.  All calls are asynchronous on the given stream (a
 * cudaStream_t / CUstream handle passed as void*; NULL = legacy default
 * stream).  A step is four kernels on that stream: momentum + cast, the normaliser d,
 * the normalisation X / d, and one persistent kernel for every product of every map.
 * No call below allocates, frees or synchronises, except anvil_bank_step on its first
 * use of a size (documented there), the error reads anvil_last_device_error (waits for
 * its stream) and anvil_device_error (waits for the device).  Errors are returned as
 * status codes; no exception crosses the ABI.
 */
#ifndef ANVIL_H
#define ANVIL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ANVIL_OK = 0,
    ANVIL_ERR_INVALID_ARG = 1,       /* null pointer, g/m/n < 1, nmaps out of range, ... */
    ANVIL_ERR_UNSUPPORTED_SHAPE = 2, /* a dimension above ANVIL_MAX_DIM / ANVIL_MAX_BATCH, or a
                                        call of over 2^40 padded elements (terabytes of workspace) */
    ANVIL_ERR_ALIGNMENT = 3,         /* pointer not aligned to its element size / workspace to 256 B */
    ANVIL_ERR_ALIAS = 4,             /* a written buffer overlaps another buffer of the call */
    ANVIL_ERR_WORKSPACE = 5,         /* workspace too small, or cannot be allocated during capture */
    ANVIL_ERR_CUDA = 6,              /* a CUDA runtime/driver call or a launch failed */
    ANVIL_ERR_TIMEOUT = 7,           /* a bounded device-side wait gave up (see anvil_last_device_error) */
    ANVIL_ERR_DEVICE = 8,            /* current device is not sm_103 (the kernels are sm_103a only) */
    ANVIL_ERR_UNAVAILABLE = 9        /* a diagnostic this build of the library does not include */
} anvil_status;

/* One quintic spectral map f(s) = a s + b s^3 + c s^5 (an ANVIL_MAPS entry). */
typedef struct { float a, b, c; } anvil_map;

/* Per-step scalars of one bank (the page's AnvilBank momentum / fast_beta /
 * fast_weight, plus the slow rail's beta, RAIL_SLOW_BETA there). */
typedef struct { float momentum, fast_beta, fast_weight, slow_beta; } anvil_scalars;

/* One bank of g matrices of m x n.  All pointers are DEVICE pointers, row-major,
 * caller-owned:
 *   grad      [g, m, n]    fp32, or bf16 bits when grad_bf16 != 0 (the page's bank
 *                          gradient is bf16); read only (never written)
 *   velocity  [2, g, m, n] fp32, read and written in place; rail 0 fast, rail 1 slow
 *   out       [g, m, n]    bf16 bits, written
 *   tail_link  optional DEVICE buffer of anvil_tail_link_bytes(g, m, n) bytes, 256-byte
 *              aligned, or NULL: the step also writes there the sign of every slow-rail
 *              value (2 bits per element: the sign, and whether the tail must read the
 *              value itself), so that anvil_update_tail given the same buffer gates its
 *              decay without reading the fp32 slow rail (0.25 instead of 4 bytes per element)
 * grad must be aligned to its element size, velocity to 4 bytes, out to 2 bytes; out
 * and tail_link must not overlap grad, velocity or any buffer of another bank in the
 * same call.  `scalars` is used when the call's device scalar array is NULL. */
typedef struct {
    const void* grad;
    float* velocity;
    uint16_t* out;
    int g, m, n;
    anvil_scalars scalars;
    int grad_bf16;
    void* tail_link;
} anvil_bank_desc;

/* Bytes of the step-to-tail link buffer of one bank of g matrices of m x n (0 if the
 * shape is invalid).  Its contents are internal to the library: written by the step
 * (anvil_multi_bank_step, anvil_bank_step_traced), read by anvil_update_tail, valid
 * until the bank's next step. */
size_t anvil_tail_link_bytes(int g, int m, int n);

#define ANVIL_MAX_MAPS 16     /* maps per call */
#define ANVIL_MAX_BANKS 8     /* banks per anvil_multi_bank_step call */
#define ANVIL_MAX_DIM 16384   /* largest m or n */
#define ANVIL_MAX_BATCH 65535 /* largest g */

/* Writes the page's six ANVIL_MAPS into maps[0..5] (if cap >= 6) and returns 6. */
int anvil_default_maps(anvil_map* maps, int cap);

/* Bytes of device workspace anvil_multi_bank_step needs for these banks
 * (0 if the descriptors are invalid).  Depends only on g, m, n of each bank. */
size_t anvil_workspace_bytes(const anvil_bank_desc* banks, int nbanks);

/* One ANVIL step over nbanks banks, every kernel grouped across the banks.
 *   banks      host array of nbanks descriptors (1 <= nbanks <= ANVIL_MAX_BANKS)
 *   d_scalars  DEVICE array of nbanks anvil_scalars read by the momentum kernel
 *              when it runs (so a captured CUDA graph sees the current values),
 *              or NULL to use banks[i].scalars, fixed at launch/capture time
 *   maps       host array of nmaps maps (1 <= nmaps <= ANVIL_MAX_MAPS), applied in order
 *   margin, eps  the normaliser d = sqrt(tr) * margin + eps (page: 1.05, 1e-6)
 *   workspace  DEVICE scratch of at least anvil_workspace_bytes(banks, nbanks)
 *              bytes, 256-byte aligned, owned by the caller; its contents on
 *              entry do not matter, and two calls that overlap on the GPU must
 *              not share it
 * Allocates nothing and never synchronises, so it may be captured in a CUDA graph. */
anvil_status anvil_multi_bank_step(const anvil_bank_desc* banks, int nbanks,
                                   const anvil_scalars* d_scalars,
                                   const anvil_map* maps, int nmaps, float margin, float eps,
                                   void* workspace, size_t workspace_bytes, void* stream);

/* One bank with host scalars: the page's anvil_cascade signature with the slow
 * beta, the maps, margin and eps made parameters.  Uses a workspace owned by the
 * library, cached per device and grown on demand: a call that needs more than
 * the cached size frees and allocates it (cudaFree / cudaMalloc, which
 * synchronise the device), so make one call of the largest size before
 * capturing this function in a CUDA graph; a call that would have to grow it
 * while the stream is capturing returns ANVIL_ERR_WORKSPACE.  Every call on a
 * device uses that one workspace: two calls whose work can overlap on the GPU
 * (different streams, or threads) corrupt each other's results, so serialise
 * them, or give each stream its own workspace through anvil_multi_bank_step.
 * maps = NULL selects the page's six ANVIL_MAPS. */
anvil_status anvil_bank_step(const float* grad, float* velocity, int g, int m, int n,
                             float momentum, float fast_beta, float fast_weight, float slow_beta,
                             const anvil_map* maps, int nmaps, float margin, float eps,
                             uint16_t* out, void* stream);

/* anvil_bank_step for callers that must not allocate device memory.  The page has no
 * counterpart: this is a deployment convenience.  Some hosts cannot call cudaMalloc
 * from the code that runs the optimizer step: an application whose device memory is
 * all handed out by its own pool or budget, or a latency-bound loop where cudaMalloc /
 * cudaFree, which synchronise the device, are not allowed.  This variant takes the same arguments as
 * anvil_bank_step but keeps its scratch in a fixed array of
 * ANVIL_STATIC_SCRATCH_BYTES bytes of device memory that the library declares
 * statically: each GPU that loads the library holds that array until the process
 * exits.  It calls no cudaMalloc, cudaFree or other allocating routine.
 *   - Sizes whose scratch (anvil_workspace_bytes of the one bank) exceeds
 *     ANVIL_STATIC_SCRATCH_BYTES are rejected with ANVIL_ERR_WORKSPACE, and
 *     anvil_last_cuda_error() says how many bytes the call needed.  32 MiB holds,
 *     e.g., 22 matrices of 256 x 768 or 3 of 2816 x 768.
 *   - The first call on each GPU looks up the array's device address on that GPU
 *     (cudaGetSymbolAddress, with that GPU current); make that first call before
 *     any stream capture.
 *   - All calls on a GPU share the one array, which keeps whatever the last call
 *     left in it; the step writes every scratch byte before reading it, so nothing
 *     needs clearing.  Two calls whose work overlaps on the GPU (different streams,
 *     or threads) race on the array and corrupt each other's results: serialise them. */
#define ANVIL_STATIC_SCRATCH_BYTES (32u << 20)
anvil_status anvil_bank_step_noalloc(const float* grad, float* velocity, int g, int m, int n,
                                     float momentum, float fast_beta, float fast_weight,
                                     float slow_beta, const anvil_map* maps, int nmaps,
                                     float margin, float eps, uint16_t* out, void* stream);

/* ---- the update tail: anvil_bank_update's steps after the cascade on the page
 * (`_rail_equalizer`, then `_sign_aligned_decay_update`).  For every matrix, with the
 * bank step's output as the update v and lanes along the longer dimension (the rows
 * when m >= n, else the columns), each lane reduced over the other dimension:
 *   P[l] = mean over lane l of v^2;  lane_energy <- lerp(lane_energy, P, 1 - beta2)
 *   gain = rsqrt(max(lane_energy, 1e-10));  scale[l] = gain[l] * (||v||_F / post_norm),
 *   post_norm^2 = sum_l P[l] * lane_len * gain[l]^2   (post_norm clamped at 1e-10)
 *   u = bf16(v * bf16(scale[lane]))
 *   w = fp32 master weight (param bits << 16 | mantissa)
 *   w <- (w - w * [slow rail * w >= 0] * eff_wd * eff_lr[mat]) - u * eff_lr[mat]
 *   param, mantissa <- high and low 16 bits of w.
 * DEVICE pointers, row-major, caller-owned:
 *   update      [g, m, n] bf16 bits, read (the out of anvil_bank_step)
 *   velocity    [2, g, m, n] fp32, read (rail 1, the slow rail, gates the decay)
 *   lane_energy [g, m] fp32 if m >= n, else [g, n]; read and written
 *   param       [g, m, n] bf16 bits of the parameter; read and written
 *   mantissa    [g, m, n] uint16, the low half of the fp32 master weight; read and written
 *   eff_lr      [g] fp32 per-matrix learning rate, read when the kernels run
 *   tail_link   NULL, or the link buffer the step that produced `update` (its out) and
 *               `velocity` was given: the tail then takes the slow rail's signs from it,
 *               with the same results
 * Written buffers must not overlap any other buffer of the call. */
typedef struct {
    const uint16_t* update;
    const float* velocity;
    float* lane_energy;
    uint16_t* param;
    uint16_t* mantissa;
    const float* eff_lr;
    int g, m, n;
    float eff_wd, beta2;
    const void* tail_link;
} anvil_tail_desc;

/* Bytes of device workspace anvil_update_tail needs (0 if the descriptors are invalid). */
size_t anvil_tail_workspace_bytes(const anvil_tail_desc* banks, int nbanks);

/* The update tail over nbanks banks (1 <= nbanks <= ANVIL_MAX_BANKS), three grouped
 * launches on the stream;
 * workspace as for anvil_multi_bank_step (256-byte aligned, caller-owned, contents on
 * entry irrelevant).  Allocates nothing, never synchronises. */
anvil_status anvil_update_tail(const anvil_tail_desc* banks, int nbanks, void* workspace,
                               size_t workspace_bytes, void* stream);

/* The page's Adam step for the parameters outside the ANVIL banks (`_adam_update_step`:
 * bias-corrected Adam with cautious weight decay), elementwise over count fp32 values,
 * DEVICE pointers, caller-owned, read and written in place except grad:
 *   exp_avg    = exp_avg * beta1 + (1 - beta1) * grad
 *   exp_avg_sq = exp_avg_sq * beta2 + ((1 - beta2) * grad) * grad
 *   u = (exp_avg / (sqrt(exp_avg_sq) + eps)) * step_size
 *   u = u + (eff_wd * param) * [u * param > 0];   param = param - u
 * step_size (lr * sqrt(1 - beta2^t) / (1 - beta1^t)) and eff_wd are the caller's, as on
 * the page.  Buffers 4-byte aligned; param, exp_avg and exp_avg_sq must not overlap any
 * other buffer of the call.  One launch on the stream; allocates nothing. */
anvil_status anvil_adam_step(float* param, const float* grad, float* exp_avg, float* exp_avg_sq,
                             size_t count, float beta1, float beta2, float eps, float step_size,
                             float eff_wd, void* stream);

/* AdamW over many tensors in one call, in place: for every tensor, elementwise, with t = step,
 *   g = grad * grad_scale
 *   exp_avg    = exp_avg * beta1 + g * (1 - beta1)
 *   exp_avg_sq = exp_avg_sq * beta2 + (g * (1 - beta2)) * g
 *   param = param * decay - (exp_avg / (sqrt(exp_avg_sq) * root + eps)) * step_size
 * with step_size = lr / (1 - beta1^t), root = 1 / sqrt(1 - beta2^t), decay = 1 - lr * weight_decay
 * (in double, rounded to fp32), in fp32 with one rounding per operation in the order written.
 * param [count] is fp32, bf16 or fp16 (rounded once, to nearest even), or bf16 with mantissa: the
 * two halves of an fp32 value, as anvil_tail_desc has them.  grad is fp32 or of param's type (for
 * an fp32 param any type).
 * scales NULL: exp_avg and exp_avg_sq are fp32.  Else they are 8-bit codes, one byte a value, and
 * scales [2, ceil(count / ANVIL_ADAMW_BLOCK)] fp32 holds a factor per block of consecutive values,
 * for exp_avg and then for the root of exp_avg_sq:
 *   exp_avg = e4m3 code * factor;  exp_avg_sq = (c < 16 ? c : (16 + c % 16) 2^(c / 16 - 1))^2 * factor^2
 * (the root's code is c, and at least 1 where the root is not 0).  The factor is the block's largest
 * magnitude times 1 / 448 (1 / 507904 for the root, the largest codes; 0 for a magnitude below 2^-100), the
 * code the nearest, ties to the even one, of the value times 448 (507904) / that magnitude.  All zeros are states of 0.  The
 * parameter's step uses the unrounded moments.  An infinite or NaN moment makes its block NaN.
 * count may be 0.  Pointers are aligned to their elements' size; arrays on boundaries of four
 * elements are faster.  A written array must not overlap any other array of the call; gradients may
 * overlap each other. */
#define ANVIL_ADAMW_BLOCK 256
#define ANVIL_MAX_TENSORS (1 << 20)
#define ANVIL_MAX_COUNT (1ll << 40)
typedef struct {
    void* param;
    uint16_t* mantissa;
    const void* grad;
    void* exp_avg;
    void* exp_avg_sq;
    float* scales;
    int64_t count;
    int param_dtype, grad_dtype; /* anvil_dtype, below */
} anvil_adamw_tensor;
/* 0 <= beta < 1, eps >= 0, step >= 1, grad_scale what every gradient is multiplied by (1, or what a
 * loss scale or a norm's bound asks for). */
typedef struct {
    double lr, beta1, beta2, eps, weight_decay, grad_scale;
    int64_t step;
} anvil_adamw_config;
/* d_scalars: NULL, or a DEVICE array of four fp32 that is read when the step runs in place of
 * config's lr, weight_decay, grad_scale and step: step_size, root, decay, grad_scale, as
 * anvil_adamw_scalars (host only) gives them; a captured graph then follows the schedule.  One
 * launch per kind of tensor (types, codes, all its arrays on boundaries of four elements or not; few of those
 * that are go with those that are not) and 448 tensors; allocates no device memory. */
anvil_status anvil_adamw_step(const anvil_adamw_tensor* tensors, int ntensors, const anvil_adamw_config* config,
                              const float* d_scalars, void* stream);
anvil_status anvil_adamw_scalars(const anvil_adamw_config* config, float* scalars);

/* The values that 8-bit states stand for, as fp32: m = exp_avg, v = exp_avg_sq, [count] each. */
typedef struct {
    const void* exp_avg;
    const void* exp_avg_sq;
    const float* scales;
    float* m;
    float* v;
    int64_t count;
} anvil_adamw_state;
anvil_status anvil_adamw_values(const anvil_adamw_state* states, int nstates, void* stream);

/* ---- operators around the banks: the layers whose gradients a bank or Adam step takes,
 * and the loss.  Layer norm, the linear layer with its bias, activation and residual, and
 * the log probabilities of given tokens, each forward and backward.
 *
 * Common rules.  DEVICE pointers, caller-owned.  A matrix argument is row-major with
 * contiguous rows and a row stride ld* in elements (at least the row's length; not read
 * when there is at most one row), so a view of wider rows is fine.  Pointers are aligned
 * to their element size; rows on 16-byte boundaries are faster.  Sums, statistics and
 * accumulators are fp32; a result is rounded to its type once, to nearest even.  rows
 * may be 0: forward calls then do nothing, gradients of parameters become 0.  Results
 * are the same bits on every call with the same arguments (no sum's order depends on
 * timing).  Written buffers must not overlap any other buffer of the call except where
 * said; views that interleave in one buffer without sharing an element are fine if their
 * row strides are the same.  Calls allocate nothing and never synchronise, so they may
 * be captured in a CUDA graph; where a call needs scratch, its workspace is as for
 * anvil_multi_bank_step. */
typedef enum { ANVIL_F32 = 0, ANVIL_BF16 = 1, ANVIL_F16 = 2 } anvil_dtype;

#define ANVIL_MAX_ROWS (1 << 30)     /* largest rows of these operators */
#define ANVIL_MAX_WIDTH 16384        /* largest layer-norm width */
#define ANVIL_MAX_FEATURES (1 << 20) /* largest n or k of a linear layer */
#define ANVIL_MAX_VOCAB (1 << 24)    /* largest vocabulary */
#define ANVIL_MAX_TOP 32             /* most alternatives per row */

/* Layer norm of every row of x [rows, width]:
 *   mean = sum x / width,  rstd = 1 / sqrt(sum (x - mean)^2 / width + eps),
 *   y = (x - mean) rstd weight + bias.
 * x and y have type dtype; weight and bias [width] have type weight_dtype, fp32 or dtype,
 * or are NULL (1 and 0).  mean and rstd [rows] fp32 are written for the backward pass, or
 * NULL.  y may be x itself (same pointer and stride). */
typedef struct {
    const void* x;
    const void* weight;
    const void* bias;
    void* y;
    float* mean;
    float* rstd;
    int64_t rows;
    int64_t ldx, ldy;
    int width;
    int dtype, weight_dtype;
    float eps;
} anvil_layernorm_desc;
anvil_status anvil_layernorm_forward(const anvil_layernorm_desc* desc, void* stream);

/* Its gradient, for dy = dL/dy and the mean and rstd of the forward pass; with
 * h = (x - mean) rstd and g = dy weight:
 *   dx = rstd (g - mean(g) - h mean(g h)) [+ residual_grad],
 *   dweight = sum over rows of dy h,  dbias = sum over rows of dy.
 * residual_grad [rows, width] of type dtype, or NULL: the gradient that reaches x past the
 * norm.  dx, dweight and dbias may each be NULL (not computed); dweight and dbias are fp32.
 * dx may be dy, x or residual_grad itself (same pointer and stride). */
typedef struct {
    const void* dy;
    const void* x;
    const float* mean;
    const float* rstd;
    const void* weight;
    const void* residual_grad;
    void* dx;
    float* dweight;
    float* dbias;
    int64_t rows;
    int64_t lddy, ldx, ldr, lddx;
    int width;
    int dtype, weight_dtype;
} anvil_layernorm_grad_desc;
size_t anvil_layernorm_backward_workspace_bytes(const anvil_layernorm_grad_desc* desc);
anvil_status anvil_layernorm_backward(const anvil_layernorm_grad_desc* desc, void* workspace, size_t workspace_bytes,
                                      void* stream);

typedef enum {
    ANVIL_ACT_NONE = 0,
    ANVIL_ACT_RELU = 1,      /* max(z, 0), the slope 0 at 0 */
    ANVIL_ACT_RELU2 = 2,     /* max(z, 0)^2 */
    ANVIL_ACT_GELU = 3,      /* z Phi(z) */
    ANVIL_ACT_GELU_TANH = 4, /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2 */
    ANVIL_ACT_SILU = 5       /* z / (1 + e^-z) */
} anvil_activation;

/* The linear layer:  z = x W^T + bias,  y = act(z) + residual.
 * x [rows, k], residual and y [rows, n], W: [n, k], or stored as its transpose [k, n] when
 * weight_transposed != 0 (one bank of one shape can hold both projections of a block), all
 * of type dtype (ANVIL_BF16 or ANVIL_F16).  bias [n] of type bias_dtype (fp32 or dtype) or
 * NULL; residual may be NULL.  preact [rows, n], or NULL, receives z (rounded; y comes from
 * the unrounded z) for the backward pass.  From one row to many: few rows read the weight
 * once.  y may be residual itself (same pointer and stride). */
typedef struct {
    const void* x;
    const void* weight;
    const void* bias;
    const void* residual;
    void* y;
    void* preact;
    int64_t rows;
    int64_t ldx, ldw, ldr, ldy, ldz;
    int n, k;
    int dtype, bias_dtype;
    int activation;
    int weight_transposed;
} anvil_linear_desc;
/* Scratch of a call (0 for invalid descriptors and where none is needed): copies of
 * operands whose rows are not on 16-byte boundaries, and fp32 parts of products split along
 * the contraction.  Depends on the pointers' alignment. */
size_t anvil_linear_workspace_bytes(const anvil_linear_desc* desc);
anvil_status anvil_linear_forward(const anvil_linear_desc* desc, void* workspace, size_t workspace_bytes, void* stream);

/* Added to the gradient's activation: dz in two parts, see below. */
#define ANVIL_DZ_TWO_PARTS 256

/* Its gradient, for dy = dL/dy and z = preact (not read for ANVIL_ACT_NONE):
 *   dz = dy act'(z),  dx = dz W,  dweight = dz^T x,  dbias = sum over rows of dz.
 * dx [rows, k] of type dtype; dweight in W's layout (weight_transposed), of type
 * dweight_dtype: dtype or ANVIL_F32 (what the bank step takes); dbias [n] fp32.  Each may be
 * NULL (not computed); x is read for dweight only, weight for dx only.  dz is rounded to
 * dtype as the products' operand (in fp16 one beyond 65504 becomes infinite, as do dx and dweight
 * where it takes part); dbias sums the unrounded dz.  With activation + ANVIL_DZ_TWO_PARTS what
 * the rounding drops is kept as a second operand, rounded itself: dz is off by 2^-16 of itself at
 * most (fp16 2^-22) instead of 2^-8 (2^-11), the products take twice the time, and rows is at most
 * ANVIL_MAX_ROWS / 2.  Without an activation dz is dy and nothing is rounded.  accumulate != 0:
 * dweight and dbias are added to what they hold.  The residual's gradient is dy itself. */
typedef struct {
    const void* dy;
    const void* x;
    const void* weight;
    const void* preact;
    void* dx;
    void* dweight;
    float* dbias;
    int64_t rows;
    int64_t lddy, ldx, ldw, ldz, lddx, lddw;
    int n, k;
    int dtype, dweight_dtype;
    int activation;
    int weight_transposed;
    int accumulate;
} anvil_linear_grad_desc;
size_t anvil_linear_backward_workspace_bytes(const anvil_linear_grad_desc* desc);
anvil_status anvil_linear_backward(const anvil_linear_grad_desc* desc, void* workspace, size_t workspace_bytes,
                                   void* stream);

/* The gated layer:  g = x G^T,  u = x U^T,  y = act(g) * u, elementwise.
 * x [rows, k], y [rows, n], G and U: [n, k] each, or both stored as their transposes [k, n] when
 * weight_transposed != 0, all of type dtype (ANVIL_BF16 or ANVIL_F16); views of one matrix that
 * holds both are fine.  preact_gate and preact_up [rows, n], or NULL, receive g and u (rounded; y comes
 * from the unrounded values) for the backward pass.  From one row to many: few rows read the
 * weights once. */
typedef struct {
    const void* x;
    const void* gate;
    const void* up;
    void* y;
    void* preact_gate;
    void* preact_up;
    int64_t rows;
    int64_t ldx, ldgate, ldup, ldy, ldzg, ldzu;
    int n, k;
    int dtype;
    int activation;
    int weight_transposed;
} anvil_gated_desc;
/* Scratch of a call, as anvil_linear_workspace_bytes. */
size_t anvil_gated_linear_workspace_bytes(const anvil_gated_desc* desc);
anvil_status anvil_gated_linear_forward(const anvil_gated_desc* desc, void* workspace, size_t workspace_bytes, void* stream);

/* Its gradient, for dy = dL/dy and the forward pass's g and u:
 *   dg = dy u act'(g),  du = dy act(g),  dx = dg G + du U,  dgate = dg^T x,  dup = du^T x.
 * dx [rows, k] of type dtype, or NULL; dgate and dup in the weights' layout, of type dweight_dtype: dtype
 * or ANVIL_F32, both or neither NULL; x is read for them only, the weights for dx only.  dg and
 * du are rounded to dtype as operands, or kept in two parts with activation + ANVIL_DZ_TWO_PARTS, as the
 * linear layer's dz is.  accumulate != 0: dgate and dup are added to what they hold.  rows is at most
 * ANVIL_MAX_ROWS / 4. */
typedef struct {
    const void* dy;
    const void* x;
    const void* gate;
    const void* up;
    const void* preact_gate;
    const void* preact_up;
    void* dx;
    void* dgate;
    void* dup;
    int64_t rows;
    int64_t lddy, ldx, ldgate, ldup, ldzg, ldzu, lddx, lddgate, lddup;
    int n, k;
    int dtype, dweight_dtype;
    int activation;
    int weight_transposed;
    int accumulate;
} anvil_gated_grad_desc;
size_t anvil_gated_linear_backward_workspace_bytes(const anvil_gated_grad_desc* desc);
anvil_status anvil_gated_linear_backward(const anvil_gated_grad_desc* desc, void* workspace, size_t workspace_bytes,
                                         void* stream);

/* Log probabilities of given tokens under logits [rows, vocab] of type dtype:
 *   lse = log sum_j e^x_j,  logprob = x_target - lse,  entropy = lse - sum_j p_j x_j,
 *   and the `top` (0..ANVIL_MAX_TOP, at most vocab) largest x_j - lse with their columns,
 *   largest first, equal values by the lower column.
 * targets [rows] int32 (int64 when targets_int64 != 0), or NULL with logprob NULL.  A negative target
 * marks a position that does not count: its log probability is 0; one of vocab or more
 * gives NaN.  logprob, entropy and lse [rows] fp32 may each be NULL; top_logprob fp32 and
 * top_index int32 are [rows, top], contiguous.  A logit of -inf is a token that cannot be;
 * a row of nothing else has lse, logprob and top_logprob -inf and entropy 0.  A row with a
 * NaN or +inf comes out NaN (its top_index then means nothing). */
typedef struct {
    const void* logits;
    const void* targets;
    float* logprob;
    float* entropy;
    float* lse;
    float* top_logprob;
    int32_t* top_index;
    int64_t rows;
    int64_t ld;
    int vocab, top;
    int dtype, targets_int64;
} anvil_logprob_desc;
anvil_status anvil_token_logprobs(const anvil_logprob_desc* desc, void* stream);

/* Their gradient, for u = dL/dlogprob (NULL: 0) and v = dL/dentropy (NULL: 0) [rows] fp32
 * and the lse (and entropy, with v) of the forward pass, p_j = e^(x_j - lse):
 *   dlogits_j = u ([j = target] - p_j) - v p_j (x_j - lse + entropy),
 * of type dtype [rows, vocab]; a p_j below 2^-126 counts as 0.  u is taken as 0 where the
 * target is negative; a row whose lse is -inf has the gradient 0.  dlogits may be logits itself
 * (same pointer and stride). */
typedef struct {
    const void* logits;
    const void* targets;
    const float* lse;
    const float* entropy;
    const float* grad_logprob;
    const float* grad_entropy;
    void* dlogits;
    int64_t rows;
    int64_t ld, ldd;
    int vocab;
    int dtype, targets_int64;
} anvil_logprob_grad_desc;
anvil_status anvil_token_logprobs_backward(const anvil_logprob_grad_desc* desc, void* stream);

/* Softmax cross entropy of a head, without its logits in memory:  z = x W^T,
 *   lse = log sum_j e^z_j,  loss = lse - z_target.
 * x [rows, k], W: [vocab, k], or its transpose [k, vocab] when weight_transposed != 0, both of type
 * dtype (ANVIL_BF16 or ANVIL_F16); loss and lse [rows] fp32, or NULL.  targets [rows] int32 (int64 when
 * targets_int64 != 0), or NULL with loss NULL.  A negative target marks a position that does not
 * count: its loss is 0 (its lse is computed); one of vocab or more gives NaN.  A logit of -inf is a
 * token that cannot be; a row of nothing else has lse -inf and loss inf.  A row with a NaN or +inf
 * logit comes out NaN.  Logits are fp32 sums: of up to 1024 terms as the tensor cores add them, which cuts off
 * (1e-6 of a logit's magnitude, towards 0), and of those sums rounded to nearest. */
typedef struct {
    const void* x;
    const void* weight;
    const void* targets;
    float* loss;
    float* lse;
    int64_t rows;
    int64_t ldx, ldw;
    int vocab, k;
    int dtype, targets_int64;
    int weight_transposed;
} anvil_head_desc;
/* Scratch: 8 bytes per row and 64 columns of the vocabulary, 4 per row, and copies of operands off the
 * 16-byte boundaries. */
size_t anvil_linear_cross_entropy_workspace_bytes(const anvil_head_desc* desc);
anvil_status anvil_linear_cross_entropy(const anvil_head_desc* desc, void* workspace, size_t workspace_bytes, void* stream);

/* Its gradient, for grad_loss = dL/dloss [rows] and the forward pass's lse [rows], both fp32:
 *   d_j = grad_loss (e^(z_j - lse) - [j = target]),  dx = d W,  dweight = d^T x.
 * The logits are computed again, a piece of the vocabulary at a time; d over the largest finite |grad_loss| is
 * rounded to dtype as the products' operand (in fp16 with 2^13 more, so that small values are held), sums are fp32.  dx
 * [rows, k] of type dtype; dweight in W's layout, of type dweight_dtype: dtype or ANVIL_F32.  Each may be
 * NULL.  grad_loss is taken as 0 where the target is negative; a target of vocab or more is no column's
 * (d_j = grad_loss e^(z_j - lse)); a row whose lse is -inf has the gradient 0.  accumulate != 0: dweight
 * is added to what it holds. */
typedef struct {
    const void* x;
    const void* weight;
    const void* targets;
    const float* lse;
    const float* grad_loss;
    void* dx;
    void* dweight;
    int64_t rows;
    int64_t ldx, ldw, lddx, lddw;
    int vocab, k;
    int dtype, targets_int64, dweight_dtype;
    int weight_transposed;
    int accumulate;
} anvil_head_grad_desc;
/* Scratch: d for a piece (512 MB, or 512 bytes a row where that is more), dx's fp32 sum where there are
 * several pieces, copies as above, and parts of products split along the contraction. */
size_t anvil_linear_cross_entropy_backward_workspace_bytes(const anvil_head_grad_desc* desc);
anvil_status anvil_linear_cross_entropy_backward(const anvil_head_grad_desc* desc, void* workspace, size_t workspace_bytes,
                                                 void* stream);

/* Per-stage dumps of one bank step, for parity testing (not the hot path).
 * DEVICE pointers, each optional (NULL = skip), in the page's layout:
 *   X_raw [g, m, n] bf16            bf16 cast of the momentum lookahead
 *   d     [g]       fp32            normaliser per matrix
 *   X     [nmaps+1, g, m, n] bf16   normalised X, then X after each map
 *   A, B  [nmaps, g, s, s] bf16     per map (s = min(m, n)); A[0] is the
 *                                   normalised first Gram */
typedef struct {
    uint16_t* X_raw;
    float* d;
    uint16_t* X;
    uint16_t* A;
    uint16_t* B;
} anvil_trace;

/* anvil_multi_bank_step for one bank, plus the dumps.  Same arguments and
 * workspace rules; out receives the same result as without tracing.  The cascade
 * runs one phase per launch here (with the dumps copied out in between); a trace
 * with every pointer NULL gives that phase-by-phase run without dumps. */
anvil_status anvil_bank_step_traced(const anvil_bank_desc* bank, const anvil_scalars* d_scalars,
                                    const anvil_map* maps, int nmaps, float margin, float eps,
                                    void* workspace, size_t workspace_bytes,
                                    const anvil_trace* trace, void* stream);

/* Reads (and, if clear != 0, resets) the current device's error word, which a
 * kernel sets when one of its bounded waits gives up instead of hanging.
 * Synchronises the device.  Returns ANVIL_OK, ANVIL_ERR_TIMEOUT or ANVIL_ERR_CUDA. */
anvil_status anvil_device_error(int clear);

/* The error word as the work queued so far on `stream` leaves it: waits for that stream
 * only (cudaStreamSynchronize), then reads and resets the word with one atomic exchange
 * on the device, so a timeout is reported once.  The word belongs to the device, not to
 * the stream: a wait that gave up in work on another stream shows here too if it gave up
 * before this read, and otherwise in a later read.  Returns ANVIL_OK, ANVIL_ERR_TIMEOUT,
 * ANVIL_ERR_CUDA or ANVIL_ERR_DEVICE. */
anvil_status anvil_last_device_error(void* stream);

/* Self-test of the bounded waits: launches one block that waits on a barrier
 * nothing will ever complete, for at most timeout_us microseconds, after which
 * it records a timeout in the device error word and returns.  It neither
 * faults nor hangs the GPU. */
anvil_status anvil_selftest_wait_timeout(unsigned timeout_us, void* stream);

/* Per-launch timing for benchmarks.  Between anvil_profile_begin and
 * anvil_profile_end, every kernel launch of anvil_multi_bank_step, anvil_bank_step,
 * anvil_update_tail, anvil_adam_step and the operators around the banks in the process is
 * bracketed by two CUDA events
 * recorded on the call's stream (at most max_records launches; later ones are
 * not timed).  begin creates the events (a host call: do not begin, or step
 * with profiling on, while a stream is capturing).  end synchronises, writes up
 * to cap records in launch order, destroys the events and returns how many
 * launches were timed (negative on a CUDA error). */
/* Kinds 3-7 are the cascade's phases, each its own launch in traced steps only; an
 * untraced step runs them all in one ANVIL_KERNEL_CASCADE launch. */
typedef enum {
    ANVIL_KERNEL_MOMENTUM = 0,     /* momentum + cast + diagonal partials */
    ANVIL_KERNEL_NORM_D = 1,       /* d per matrix */
    ANVIL_KERNEL_NORMALIZE = 2,    /* X <- bf16(X / d) */
    ANVIL_KERNEL_GRAM_NORM = 3,    /* first Gram, A = bf16(bf16(X X^T) / d^2) */
    ANVIL_KERNEL_GRAM = 4,         /* A = bf16(X X^T) */
    ANVIL_KERNEL_SQPOLY = 5,       /* B = bf16(b A + c A A) */
    ANVIL_KERNEL_XUPDATE = 6,      /* X <- bf16(a X + B X) */
    ANVIL_KERNEL_XUPDATE_OUT = 7,  /* the last map's X-update, written to out */
    ANVIL_KERNEL_TAIL_POWER = 8,   /* update tail: lane powers */
    ANVIL_KERNEL_TAIL_SCALE = 9,   /* update tail: lane energies and scales */
    ANVIL_KERNEL_TAIL_APPLY = 10,  /* update tail: equalise + sign-aligned decay update */
    ANVIL_KERNEL_ADAM = 11,        /* Adam step */
    ANVIL_KERNEL_CASCADE = 12,     /* the whole cascade (every product of every map) */
    ANVIL_KERNEL_NORM_FORWARD = 13,      /* layer norm */
    ANVIL_KERNEL_NORM_BACKWARD = 14,     /* its row pass: dx and partial column sums */
    ANVIL_KERNEL_NORM_GRADS = 15,        /* dweight and dbias from the partial sums */
    ANVIL_KERNEL_LINEAR_PREPARE = 16,    /* copies of unaligned operands; dz = dy act'(z) and its partial column sums */
    ANVIL_KERNEL_LINEAR_PRODUCT = 17,    /* a product of the linear layer */
    ANVIL_KERNEL_LINEAR_SUM = 18,        /* sums of split products and of dbias */
    ANVIL_KERNEL_LOGPROB = 19,           /* token log probabilities */
    ANVIL_KERNEL_LOGPROB_BACKWARD = 20,  /* their gradient */
    ANVIL_KERNEL_ADAMW = 21,             /* AdamW over many tensors, and the values of its states */
    ANVIL_KERNEL_GATED_PREPARE = 22,     /* the gated layer: dg and du */
    ANVIL_KERNEL_GATED_PRODUCT = 23,     /* both products, activation and product */
    ANVIL_KERNEL_GATED_SUM = 24,         /* sums of its split products */
    ANVIL_KERNEL_HEAD_PREPARE = 25,      /* the head's cross entropy: the scale of its gradient */
    ANVIL_KERNEL_HEAD_PRODUCT = 26,      /* its logits, and what becomes of them */
    ANVIL_KERNEL_HEAD_SUM = 27           /* rows' statistics joined; dx rounded */
} anvil_kernel_kind;

typedef struct { int kind; float ms; } anvil_profile_record;

anvil_status anvil_profile_begin(int max_records);
int anvil_profile_end(anvil_profile_record* records, int cap);

/* Diagnostic, host only (no CUDA call, no GPU needed): the order in which the cascade
 * kernel of anvil_multi_bank_step walks its work items for these banks and nmaps maps.
 * Items are 256 x 256 output tiles; the kernel's phases are the first Gram, then per
 * map the Gram (after the first map), B = bA + cA^2 and the X-update (the normalisation
 * X / d is its own kernel, before the cascade).  The order is a list of runs, each one phase of a range of matrices of one
 * bank, matrix by matrix; every phase of a matrix comes after the phases it reads.
 * Writes up to cap runs and returns how many there are (-1 on invalid arguments). */
typedef struct {
    int phase;  /* phase index, 0 = the first Gram */
    int op;     /* 0 Gram, 1 first Gram, 2 B = bA + cA^2, 3 X-update, 4 last X-update */
    int bank;   /* index of the bank in the call */
    int mat0;   /* first matrix of the run */
    int nmat;   /* matrices in the run */
    int begin;  /* index of the run's first item in the walk */
    int tiles;  /* items per matrix in this phase */
} anvil_schedule_run;
int anvil_schedule_runs(const anvil_bank_desc* banks, int nbanks, int nmaps, anvil_schedule_run* runs, int cap);

/* Per-item timeline of the cascade kernel, for performance work.  Only a library built
 * with the timeline option (build.py --timeline, which writes libanvil_timeline.so)
 * records it; this library returns ANVIL_ERR_UNAVAILABLE.  Item t (0-based, in the
 * order of anvil_schedule_runs) of the latest cascade launch owns 16 64-bit words
 * starting at word 16 t, for t < ANVIL_TIMELINE_ITEMS:
 *   0 pair | (op | bank << 8 | phase << 16) << 16 | matrix << 48;  1 block row | block
 *   column << 16 | k-blocks << 32;  then %globaltimer nanoseconds when 2 the pair's
 *   scheduler took it, 3 its input phases were complete, 4 its entry was handed out,
 *   5 the first operand load was armed, 6 the MMA issuer read it, 7 its accumulator was
 *   free, 8 its first k-block landed, 9 its last MMAs were issued, 10 the epilogue found
 *   the accumulator complete, 11 the epilogue was done;  12 and 13: SM cycles (clock64)
 *   at 8 and 9;  14 SM cycles the MMA issuer waited for k-blocks after the first to
 *   land;  15 SM cycles the producer waited for free operand stages.
 * anvil_timeline_read copies min(bytes, the buffer) to host memory (synchronous; call
 * after the launch has completed).  anvil_timeline_clear zeroes the buffer. */
#define ANVIL_TIMELINE_ITEMS 16384
anvil_status anvil_timeline_read(void* host, size_t bytes);
anvil_status anvil_timeline_clear(void);

/* Human-readable name of a status. */
const char* anvil_status_string(anvil_status status);

/* Text of the last CUDA error this library saw on this thread ("" if none). */
const char* anvil_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* ANVIL_H */
