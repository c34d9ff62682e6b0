/*
 * libmuon — the Muon optimizer step (momentum orthogonalised by quintic
 * Newton–Schulz) for the 2-D weight matrices of a GPT-2-style body, on one
 * AMD Instinct MI355X (gfx950).
 *
 * Sources, cited by page title and section:
 *  [P4] "modded-nanogpt 50B-token 长时程训练实验解析：Muon vs Adam 与数据复用策略的实证对比",
 *       section "从源码看 Muon 的分布式正交化实现" (Muon's orthogonalisation, from
 *       the source) and section "超参配置解析" (hyper-parameters).
 *  [P2] "2025-10-27_FixMuonLR" record analysis, sections "改动一" (per-matrix
 *       lr_mul / wd_mul, the Muon learning rate) and "改动二" (the vectorised
 *       step, the lerp momentum buffer owned by the group, reset(), the early
 *       qkvo reshape, NorMuon's per-lane second moment).
 *  [P3] "2024-11-19 FlexAttention" record analysis, optimizer section
 *       (Muon on 2-D params, 5 NS steps, momentum warm-up 0.85 -> 0.95).
 *
 * Conventions for every entry point:
 *  - Plain C: pointers and sizes only. Device pointers are HIP device
 *    addresses; `stream` is a hipStream_t passed as void* (NULL = the
 *    default stream of the current device).
 *  - Ownership: the caller owns params, grads, momentum and the workspace.
 *    A handle owns only host memory. The library never allocates device
 *    memory; muon_init uploads its descriptor tables into the caller's
 *    workspace and zeroes its state there, blocking; muon_step and
 *    muon_reset only enqueue work on `stream` and never synchronise.
 *  - Errors: every call returns a muon_status; nothing aborts or throws
 *    across the ABI (a host allocation failure inside the library returns
 *    MUON_E_HOST). Validation happens before any HIP call. A kernel fault
 *    surfaces at the caller's next synchronisation. Handles are not
 *    thread-safe; use one stream per handle per call. muon_step allocates
 *    no memory, host or device (unless muon_profile_enable turned on its
 *    event records).
 */
#ifndef LIBMUON_H
#define LIBMUON_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum muon_status {
    MUON_OK = 0,
    MUON_E_INVALID_ARG = -1, /* null pointer, bad enum, non-finite / out-of-range scalar */
    MUON_E_SHAPE = -2,       /* rows, cols or count < 1 */
    MUON_E_LAYOUT = -3,      /* negative offset, overlap, extent beyond the buffers */
    MUON_E_NO_DEVICE = -4,   /* no HIP device, or the device is not gfx950 */
    MUON_E_HIP = -5,         /* a HIP runtime call failed (see muon_last_error) */
    MUON_E_STATE = -6,       /* misuse of a handle (wrong device current, ...) */
    MUON_E_WORKSPACE = -7,   /* workspace null, misaligned (256 B) or too small */
    MUON_E_HOST = -8         /* host-side failure: out of host memory (the message says what failed) */
} muon_status;

/* One table entry: `count` contiguous row-major [rows, cols] float32 matrices
 * starting at element `offset` of the flat params / grads / momentum buffers
 * (count = 4 expresses the fused qkvo weight as its four [d, d] matrices,
 * [P2] change 2). Only 2-D weights belong here ([P4] Muon source).
 * lr_mul / wd_mul scale lr and weight decay for these matrices ([P2] change 1).
 * frozen != 0: params and momentum of these matrices are never touched. */
typedef struct muon_matrix {
    int64_t rows;
    int64_t cols;
    int64_t count;
    int64_t offset;
    float lr_mul;
    float wd_mul;
    int32_t frozen;
    int32_t reserved; /* must be 0 */
} muon_matrix;

#define MUON_MAX_NS_STEPS 16

enum { MUON_NS_BF16 = 0, MUON_NS_FP32 = 1 };
enum { MUON_MOMENTUM_LERP = 0, MUON_MOMENTUM_HEAVY_BALL = 1 };

/* Hyper-parameters ([P4] hyper-parameter and Muon source sections):
 *  momentum 0.95, nesterov 1, ns_steps 5 with (a, b, c) = (3.4445, -4.7750,
 *  2.0315) per iteration, ns_eps 1e-7, weight_decay 0, NorMuon off
 *  (beta2 0.95, eps 1e-10 when on). ns_coeffs[k] holds (a, b, c) of
 *  iteration k, so a per-iteration schedule can replace the fixed quintic.
 *  momentum_kind LERP: m <- beta m + (1-beta) g, Nesterov u = (1-beta) g + beta m
 *  ([P2] change 2); HEAVY_BALL: m <- beta m + g, Nesterov u = g + beta m
 *  ([P4] Muon source). ns_precision BF16: bf16 MFMA operands with fp32
 *  accumulation; FP32: fp32 throughout (debug / reference mode).
 *  stream_groups (not a method parameter; 0 .. 4, default 0): G > 1 lets
 *  muon_step split the tiled matrices into up to G cost-balanced groups, at
 *  least 2 matrices per group, when their update output is at most 262144
 *  tiles of 64 x 64 (a few tile rounds of the GPU per launch). 0 lets the
 *  library choose: 3 when the update output is at least 4096 such tiles
 *  (one round of 256 x 256 tiles on 256 CUs), 1 for smaller steps, whose
 *  launches are latency-bound. Each group
 *  runs its chain (momentum, Newton–Schulz, NorMuon, update) on its own
 *  stream: group 0 on the caller's stream, group g > 0 on a default-priority
 *  stream the handle owns, started after group g - 1's momentum and joined
 *  back into the caller's stream at the end, so one group's kernels fill
 *  the others' tails and launch gaps. 1 keeps every launch on the caller's
 *  stream. Results are bit-identical for every value. */
typedef struct muon_hparams {
    float momentum;
    int32_t nesterov;
    int32_t momentum_kind;
    int32_t ns_steps;
    float ns_coeffs[MUON_MAX_NS_STEPS][3];
    float ns_eps;
    int32_t ns_precision;
    int32_t normuon;
    float normuon_beta2;
    float normuon_eps;
    float weight_decay;
    int32_t stream_groups;
} muon_hparams;

/* Opaque handle: the host-side plan for one table on one device. */
typedef struct muon_handle muon_handle;

/* Fill *hp with the defaults above. */
void muon_hparams_default(muon_hparams* hp);

/* Bytes of device workspace muon_init needs for this table and hp.
 * Host-only; validates the table (same errors as muon_init).
 * Library plumbing: the pages have no counterpart (their optimizer keeps its
 * buffers in PyTorch tensors). */
muon_status muon_workspace_bytes(const muon_matrix* table, int32_t n, const muon_hparams* hp,
                                 size_t* out_bytes);

/* Validate the host table, build the plan (short-side frame per matrix:
 * matrices with rows > cols run transposed, [P4] Muon source; same-shape
 * matrices batched per launch, [P2] change 2), upload descriptors into
 * `workspace` (device, caller-owned, >= muon_workspace_bytes, 256-B aligned,
 * kept for the handle's lifetime and not written by the caller), and zero
 * the NorMuon state and the Newton–Schulz input buffer (whose padding beyond
 * the matrices' 64 x 64 tiles no step writes again). Blocking: returns after
 * these copies and fills are done. `device` is the HIP device index; it must
 * be current in every later call.
 * n = 0 is allowed (every step is then a no-op). On error *out is NULL. */
muon_status muon_init(muon_handle** out, const muon_matrix* table, int32_t n, const muon_hparams* hp,
                      void* workspace, size_t ws_bytes, int32_t device);

/* Size of the library's own device workspace (64 MiB per GPU). */
#define MUON_STATIC_WORKSPACE_BYTES ((size_t)64 << 20)

/* muon_init without a caller workspace, for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid allocation): the handle's workspace is a file-scope device
 * array of MUON_STATIC_WORKSPACE_BYTES inside the library, one per GPU, held
 * from the library's first use of that GPU until the process ends. Everything
 * else is muon_init's: the same plan, uploads and zeroing (the array keeps
 * the previous handle's contents, so the state that must start at zero is
 * cleared here), blocking, and the returned handle works with muon_step,
 * muon_reset and the views as usual. No device memory is allocated and no
 * stream or event is created: hp->stream_groups is taken as 1.
 * Tables whose muon_workspace_bytes exceed MUON_STATIC_WORKSPACE_BYTES are
 * rejected with MUON_E_WORKSPACE. All handles made this way on one GPU share
 * its array: a later muon_init_static on that GPU takes it over (an earlier
 * handle on the GPU must not be stepped afterwards), and calls on such
 * handles that overlap in time race. */
muon_status muon_init_static(muon_handle** out, const muon_matrix* table, int32_t n, const muon_hparams* hp,
                             int32_t device);

/* One Muon step ([P4] Muon source; [P2] change 2), enqueued on `stream`:
 * momentum + Nesterov, Frobenius normalisation, hp.ns_steps Newton–Schulz
 * iterations, optional NorMuon, and
 *   p <- p (1 - lr lr_mul wd wd_mul) - lr lr_mul max(1, rows/cols)^0.5 O.
 * params, momentum: float32 device buffers of `numel` elements, updated in
 * place; grads: float32 device buffer of `numel` elements, read only. All
 * three share the table's layout and must not alias each other.
 * momentum_coef < 0 uses hp.momentum (a per-call value supports momentum
 * warm-up, [P3]); lr is the per-call learning rate (schedules live with the
 * caller). Errors: MUON_E_LAYOUT if numel < the table's extent,
 * MUON_E_INVALID_ARG for null buffers or non-finite lr. */
muon_status muon_step(muon_handle* h, float* params, const float* grads, float* momentum, int64_t numel,
                      float lr, float momentum_coef, void* stream);

/* Zero the momentum of every non-frozen matrix in `momentum` (numel
 * elements, may be NULL to skip) and the NorMuon second moment, on
 * `stream` ([P2] change 2: reset() after warm-up / capture dirtied them). */
muon_status muon_reset(muon_handle* h, float* momentum, int64_t numel, void* stream);

/* Free the handle (host memory only). NULL is a no-op. Library plumbing,
 * not defined by the pages. */
void muon_destroy(muon_handle* h);

/* Static description of a status code. Library plumbing, not defined by the
 * pages. */
const char* muon_status_string(muon_status s);

/* Detail of the handle's last error ("" if none); NULL handle -> the last
 * error of a failed muon_init / muon_workspace_bytes on this thread. Library
 * plumbing, not defined by the pages. */
const char* muon_last_error(const muon_handle* h);

/* ---- introspection (tests and tools) ------------------------------------
 * Library plumbing, not defined by the pages: these expose the library's own
 * buffers and plan so that tests can compare each stage with an oracle. */

/* Where matrix `index` (0-based over the table with counts expanded) lives
 * in the workspace: short-side shape m <= n, row stride ld (elements) of the
 * padded canonical buffers, element offsets into the X buffers and into the
 * per-row NorMuon arrays, transposed = stored rows > cols, active = !frozen,
 * gram_offset = element offset of its m_pad x m_pad Gram / polynomial
 * buffers (MUON_VIEW_GRAM / MUON_VIEW_POLY; -1 if frozen). */
typedef struct muon_layout {
    int64_t x_offset;
    int64_t row_offset;
    int32_t m, n, ld, m_pad;
    int32_t transposed;
    int32_t active;
    int32_t stored_rows, stored_cols;
    int64_t param_offset;
    int64_t gram_offset;
} muon_layout;

muon_status muon_matrix_layout(const muon_handle* h, int32_t index, muon_layout* out);

/* Number of matrices (counts expanded). */
int32_t muon_num_matrices(const muon_handle* h);

enum {
    MUON_VIEW_XTILDE = 0,  /* momentum kernel output: canonical, padded X~ (bf16 or fp32) */
    MUON_VIEW_NS_OUT = 1,  /* final Newton–Schulz output, same layout */
    MUON_VIEW_SUMSQ = 2,   /* float32 [num_matrices]: sum of u^2 */
    MUON_VIEW_SCALE = 3,   /* float32 [num_matrices]: s = 1/(sqrt(sumsq) + ns_eps) */
    MUON_VIEW_V = 4,       /* float32 per canonical row: NorMuon second moment */
    MUON_VIEW_F = 5,       /* float32 per canonical row: NorMuon row factor */
    MUON_VIEW_STATUS = 6,  /* int32 [num_matrices]: bit 0 = non-finite u seen this step */
    MUON_VIEW_GRAM = 7,    /* the last iteration's A = X X^T: m_pad x m_pad per matrix at its gram_offset
                              (tiled and one-panel matrices; the short-side <= 64 path keeps A in LDS, its
                              region is unspecified) */
    MUON_VIEW_POLY = 8     /* the last iteration's B = b A + c A A, same layout as MUON_VIEW_GRAM */
};

/* Device pointer and byte size of an internal buffer, valid after the
 * stream work of the last muon_step has completed. */
muon_status muon_debug_view(const muon_handle* h, int32_t which, void** dev_ptr, size_t* bytes);

/* ---- host-side schedules (scalars for muon_step's lr and momentum_coef) ---
 * Pure host functions; no handle, no device. Out-of-range arguments give NaN. */

/* Warmup-stable-decay LR multiplier ([P4] hyper-parameter section, and the
 * [P3] FlexAttention record's schedule): for step it in [0, num_iterations),
 * (it + 1) / warmup_iters while it < warmup_iters, then 1, and from
 * num_iterations - warmdown_iters on (num_iterations - it) / warmdown_iters,
 * i.e. linear to 0 at the end. The Muon group uses warmup_iters = 0. */
float muon_lr_wsd(int64_t it, int64_t num_iterations, int64_t warmup_iters, int64_t warmdown_iters);

/* Cool-down-to-floor LR multiplier ([P2] change 3, reading stated in the
 * design notes): with x = min(step / main_iterations, 1), the multiplier is
 * floor + (1 - floor) * min(1, (1 - x) / cooldown_frac): 1 until the last
 * cooldown_frac of the main phase, then linear down to floor, and flat at
 * floor for every extension step past main_iterations ([P2]: 0.80, 0.30). */
float muon_lr_cooldown_floor(int64_t step, int64_t main_iterations, float cooldown_frac, float floor);

/* Momentum warm-up ([P3] training loop): frac = min(step / warmup_steps, 1),
 * momentum = (1 - frac) start + frac end ([P3]: 500 steps, 0.85 -> 0.95). */
float muon_momentum_warmup(int64_t step, int64_t warmup_steps, float start, float end);

/* ---- layer operators ------------------------------------------------------
 * The pass that makes the gradients muon_step reads, for the weight matrices
 * its table holds: the linear layer (matrix product with bias, activation and
 * residual in its epilogue) with its two gradients, on 16-bit and on 8-bit
 * operands and for the experts of a mixture, and layer norm and root-mean-square
 * norm with their backward passes. Library plumbing, not defined by the pages.
 *
 * These calls take no handle and keep no state: everything they need is in
 * their arguments, and they only enqueue kernels on `stream` of the current
 * device (they may be captured into a graph, and calls on different streams
 * may run at once as long as they share neither outputs nor workspace). Device
 * pointers belong to the current device. Row strides are in elements; 0 means
 * the row length. Sizes 0 of tokens / rows are allowed (the gradients of
 * weights are then 0, or unchanged when accumulating, and tensors without
 * elements may be NULL). Outputs may not overlap inputs, other outputs or the
 * workspace, except that y / dx may be the very tensor of `add` (same address
 * and stride) where no other input lies: the sum then replaces it. (Column
 * ranges side by side in one buffer's rows do not overlap; with unlike strides
 * their extents must not.) Elements between rows (stride beyond the row length)
 * are left as they were. Products and sums are held in fp32 (those of 8-bit
 * operands partly in less: muon_linear_scaled_forward says where) and rounded
 * once to each output's type; no atomics are used, so the same call gives the
 * same bits. Errors are muon_status codes, with the detail in
 * muon_op_last_error; validation comes before any HIP call. */

enum { MUON_TYPE_BF16 = 0, MUON_TYPE_FP16 = 1, MUON_TYPE_FP32 = 2 };
enum {
    MUON_WEIGHT_IN_OUT = 0, /* W [in_features, out_features], as the body's c_fc [d, 4d] */
    MUON_WEIGHT_OUT_IN = 1  /* W [out_features, in_features] */
};
enum {
    MUON_ACT_NONE = 0,
    MUON_ACT_RELU = 1,
    MUON_ACT_RELU2 = 2,     /* max(z, 0)^2 */
    MUON_ACT_GELU = 3,      /* z (1 + erf(z / sqrt 2)) / 2 */
    MUON_ACT_GELU_TANH = 4, /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2 */
    MUON_ACT_SILU = 5       /* z / (1 + e^-z) */
};
enum { MUON_LINEAR_FORWARD = 0, MUON_LINEAR_GRAD_INPUT = 1, MUON_LINEAR_GRAD_WEIGHT = 2 };

/* One linear layer on one batch. dtype (bf16 or fp16) is the type of X, W, Y
 * and of their gradients dX, dY; bias and the weight gradients are float32.
 * tokens < 2^24, features and strides at most 2^21, and an output holds fewer
 * than 2^35 elements (MUON_E_SHAPE). */
typedef struct muon_linear {
    int64_t tokens;
    int64_t in_features;
    int64_t out_features;
    int64_t ld_x; /* X, dX [tokens, in_features] */
    int64_t ld_w; /* W, dW in weight_layout */
    int64_t ld_y; /* Y, dY [tokens, out_features] */
    int32_t dtype;
    int32_t weight_layout;
} muon_linear;

/* What happens to a product before its one rounding. */
typedef struct muon_epilogue {
    int32_t activation;
    int32_t reserved;  /* must be 0 */
    const float* bias; /* forward: [out_features], or NULL */
    const void* add;   /* forward: residual [tokens, out_features]; grad input: another gradient of X
                          [tokens, in_features]; or NULL */
    int64_t ld_add;
    void* z;           /* forward: where the pre-activation X W + bias goes, rounded [tokens, out_features], or
                          NULL; grad input: read, the pre-activation [tokens, in_features] whose activation X
                          was (NULL with MUON_ACT_NONE) */
    int64_t ld_z;
} muon_epilogue;

/* Bytes of device workspace (256-byte aligned) the call `op` needs; often 0,
 * and NULL is then accepted. a, b: the addresses of its two operands (forward:
 * x, w; grad input: dy, w; grad weight: x, dy), of which only the alignment is
 * looked at: operands whose rows do not start 16-byte aligned or whose length
 * is no multiple of 8 are first copied to aligned rows in the workspace, except
 * for small products and few tokens, which read them as they are (and up to 7
 * elements of the gap between two rows, whose values do not matter).
 * Host-only. */
muon_status muon_linear_workspace_bytes(const muon_linear* d, int32_t op, const void* a, const void* b,
                                        size_t* out_bytes);

/* Y = act(X W + bias) + add; e NULL: Y = X W. The activation is taken of the
 * unrounded sum. */
muon_status muon_linear_forward(const muon_linear* d, const void* x, const void* w, const muon_epilogue* e, void* y,
                                void* workspace, size_t ws_bytes, void* stream);

/* dX = (dY W^T) * act'(z) + add: with an activation this is the gradient of
 * the previous layer's pre-activation, in one pass. act'(0) = 0 for relu. */
muon_status muon_linear_grad_input(const muon_linear* d, const void* dy, const void* w, const muon_epilogue* e,
                                   void* dx, void* workspace, size_t ws_bytes, void* stream);

/* dW (+)= the product of X and dY over the tokens, in the weight's layout and
 * float32: `dw` may point into the flat gradient buffer of muon_step. dbias
 * [out_features] (+)= the sum of dY over the tokens, or NULL. accumulate != 0
 * adds to what is there. */
muon_status muon_linear_grad_weight(const muon_linear* d, const void* x, const void* dy, float* dw, float* dbias,
                                    int32_t accumulate, void* workspace, size_t ws_bytes, void* stream);

/* One layer norm on one batch of rows. dtype (any of the three) is the type
 * of x, y and of their gradients; weight, bias, their gradients and the row
 * statistics are float32. rows < 2^24, cols and strides at most 2^21. */
typedef struct muon_layernorm {
    int64_t rows;
    int64_t cols;
    int64_t ld_x;   /* x */
    int64_t ld_y;   /* y, dy */
    int64_t ld_dx;  /* dx */
    int64_t ld_add; /* add */
    int32_t dtype;
    float eps;
} muon_layernorm;

/* y = (x - mean) rstd weight + bias per row, rstd = 1 / sqrt(var + eps) with
 * the variance over the row (its elements' number as divisor). weight, bias
 * [cols] or NULL (1, 0); mean, rstd [rows] are written. */
muon_status muon_layernorm_forward(const muon_layernorm* d, const void* x, const float* weight, const float* bias,
                                   void* y, float* mean, float* rstd, void* stream);

/* Bytes of device workspace muon_layernorm_backward needs when it reduces a
 * weight or bias gradient. Host-only. */
muon_status muon_layernorm_workspace_bytes(const muon_layernorm* d, size_t* out_bytes);

/* dx = the gradient of x from dy, + add (or NULL); dweight, dbias [cols] (+)=
 * the sums over rows of dy (x - mean) rstd and of dy, each or NULL (with both
 * NULL no workspace is needed). mean, rstd as the forward pass wrote them. */
muon_status muon_layernorm_backward(const muon_layernorm* d, const void* dy, const void* x, const float* weight,
                                    const float* mean, const float* rstd, const void* add, void* dx, float* dweight,
                                    float* dbias, int32_t accumulate, void* workspace, size_t ws_bytes, void* stream);

/* One root-mean-square norm on one batch of rows. dtype (any of the three) is the
 * type of x, residual, sum, y and of their gradients; weight, its gradient and the
 * row statistics are float32. rows < 2^24, cols and strides at most 2^21. */
typedef struct muon_rmsnorm {
    int64_t rows;
    int64_t cols;
    int64_t ld_x;   /* x; backward: what the norm was taken of */
    int64_t ld_add; /* residual; backward: add */
    int64_t ld_sum; /* sum */
    int64_t ld_y;   /* y, dy */
    int64_t ld_dx;  /* dx */
    int32_t dtype;
    float eps;
} muon_rmsnorm;

/* A matrix [rows, cols] in 8-bit floating point, its values in blocks of 128 columns
 * that share a float32 scale: an element stands for its 8-bit value times its block's
 * scale. Rows start 16-byte aligned: data, and ld in bytes (a multiple of 16; 0: the
 * row length rounded up to one); what writes such a matrix writes zeros from cols to
 * the next multiple of 16, what reads one may read these bytes, whose values do not
 * matter. Activations and gradients have a scale for each 128 columns of each row,
 * scale [ceil(cols / 128), rows] (one block's scales of all rows side by side, as the
 * products read them); weights for each 128 x 128, scale [ceil(rows / 128),
 * ceil(cols / 128)]. A scale is the largest magnitude of its block, taken as 2^-110 at
 * least, divided by the format's largest number; values are rounded to nearest, ties
 * to even. A block that holds an infinity or a NaN has it for a scale, and so stands
 * for no finite number anywhere. */
enum { MUON_EIGHT_E4M3 = 0 /* up to 448 */, MUON_EIGHT_E5M2 = 1 /* up to 57344 */ };
typedef struct muon_eight {
    void* data;
    float* scale;
    int64_t ld;
    int32_t format;   /* weights: MUON_EIGHT_E4M3 */
    int32_t reserved; /* must be 0 */
} muon_eight;

/* y = r rstd weight per row, rstd = 1 / sqrt(mean(r^2) + eps), of r = x, or with a
 * residual of r = sum = x + residual rounded to dtype, which is written as the new
 * residual stream (residual and sum come together; sum may be the very tensor of x
 * or residual, same address and stride). y: in dtype, or NULL; q: in 8 bits, from
 * the unrounded values, or NULL (one of the two is given, or both). weight [cols] or
 * NULL (1); rstd [rows] is written. Squares beyond float32 make y 0; with eps 0, a row
 * whose squares all vanish in float32 (zeros among them) has no finite y. */
muon_status muon_rmsnorm_forward(const muon_rmsnorm* d, const void* x, const void* residual, const float* weight,
                                 void* sum, void* y, const muon_eight* q, float* rstd, void* stream);

/* Bytes of device workspace muon_rmsnorm_backward needs when it reduces a weight
 * gradient. Host-only. */
muon_status muon_rmsnorm_workspace_bytes(const muon_rmsnorm* d, size_t* out_bytes);

/* dx = the gradient of x (what the norm was taken of) from dy, + add (or NULL);
 * dweight [cols] (+)= the sums over rows of dy x rstd, or NULL (then no workspace is
 * needed). rstd as the forward pass wrote it. */
muon_status muon_rmsnorm_backward(const muon_rmsnorm* d, const void* dy, const void* x, const float* weight,
                                  const float* rstd, const void* add, void* dx, float* dweight, int32_t accumulate,
                                  void* workspace, size_t ws_bytes, void* stream);

/* x [rows, cols] (row stride ld_x, any of the three types) to 8 bits, activations' or
 * gradients' blocks. rows < 2^24, cols and strides at most 2^21, and rows times cols,
 * as the next multiple of 512, at most 2^35 - 2^11. */
muon_status muon_quantize(int64_t rows, int64_t cols, int64_t ld_x, int32_t dtype, const void* x, const muon_eight* q,
                          void* stream);

/* A weight [rows, cols] (any of the three types; muon_step's params as they are) to
 * 8 bits, weights' blocks: q in its own order, q_t the other one [cols, rows], with
 * the same values and scales; either NULL. rows, cols and strides at most 2^21, and
 * fewer than 2^23 blocks. */
muon_status muon_quantize_weight(int64_t rows, int64_t cols, int64_t ld_w, int32_t dtype, const void* w,
                                 const muon_eight* q, const muon_eight* q_t, void* stream);

/* The linear layer on 8-bit operands: Y = act(X W^T + bias) + add with X [tokens, in]
 * and W [out, in] (d->weight_layout MUON_WEIGHT_OUT_IN), and dX = (dY W^T) * act'(z) +
 * add with dY [tokens, out] and W [in, out] (MUON_WEIGHT_IN_OUT): both operands lie
 * with the sum's index contiguous, so a layer that is trained keeps its weight in both
 * orders (muon_quantize_weight writes them). d->dtype is the type of the output, add
 * and z; of d's strides only the output's is looked at (ld_y; ld_x), the operands'
 * must be 0, as their own are in the muon_eight. A block's products are summed by the
 * matrix unit: each 8 of consecutive k in fixed point, where what lies below 2^-13 of
 * the largest one's power of two is cut off each, so that the 8 are off by less than
 * 7 2^-13 of the largest product; the sums of the 8s in fp32. A block's sum is multiplied
 * by the product of its two scales and added in fp32. Operands of random sign cost 2^-12
 * of the results at most (root mean square); where large products of the same 8 cancel,
 * a result made of the small ones has no such relative bound. The weight's gradient is
 * muon_linear_grad_weight's, of the 16-bit tensors. */
muon_status muon_linear_scaled_forward(const muon_linear* d, const muon_eight* x, const muon_eight* w,
                                       const muon_epilogue* e, void* y, void* stream);
muon_status muon_linear_scaled_grad_input(const muon_linear* d, const muon_eight* dy, const muon_eight* w,
                                          const muon_epilogue* e, void* dx, void* stream);

/* The linear layers of a mixture of experts on rows that lie grouped by expert:
 * expert e has rows offsets[e] .. offsets[e + 1] - 1 of X, Y and their gradients, and
 * weight e of W, `stride_w` elements after the one before (0: back to back, as `count`
 * matrices of one table entry are). bias and dbias are [experts, out_features].
 * offsets [experts + 1] are int32 on the device, ascending, in [0, rows]; they are read
 * there, so that a captured call serves later offsets. Others are taken as the nearest
 * that are in range and ascending: rows are then of unspecified values, and nothing
 * outside the tensors is read or written. Rows before the first and behind the last
 * expert's are not read and left as they are. rows < 2^24, experts at most 2^16,
 * features from 8 to 2^21. An output of fewer than 2^24 tiles of 64 x 64 is taken, and
 * larger ones may be refused (MUON_E_SHAPE): of rows, counted as rows / 64 rounded down
 * and one for each expert (each row, of fewer rows); of weight gradients, an expert's as
 * the next multiple of 8. */
typedef struct muon_grouped {
    int64_t rows;
    int64_t experts;
    int64_t in_features;
    int64_t out_features;
    int64_t ld_x; /* X, dX [rows, in_features] */
    int64_t ld_w; /* each expert's W, dW in weight_layout */
    int64_t ld_y; /* Y, dY [rows, out_features] */
    int64_t stride_w;
    int32_t dtype; /* bf16 or fp16, as muon_linear's */
    int32_t weight_layout;
} muon_grouped;

/* Y = act(X W_e + bias_e) + add per expert. */
muon_status muon_grouped_linear_forward(const muon_grouped* d, const void* x, const void* w, const int32_t* offsets,
                                        const muon_epilogue* e, void* y, void* stream);

/* dX = (dY W_e^T) * act'(z) + add per expert. */
muon_status muon_grouped_linear_grad_input(const muon_grouped* d, const void* dy, const void* w,
                                           const int32_t* offsets, const muon_epilogue* e, void* dx, void* stream);

/* Bytes of device workspace (256-byte aligned) that the weight gradient needs: often 0,
 * and NULL is then accepted; where few experts of few features have many rows, room for
 * the sums of pieces of them. Of x and dy only the alignment is looked at. Host-only. */
muon_status muon_grouped_linear_workspace_bytes(const muon_grouped* d, const void* x, const void* dy,
                                                size_t* out_bytes);

/* dW_e (+)= the product of X and dY over the expert's rows, float32, and dbias_e (+)=
 * the sum of dY over them, or NULL: zeros (or unchanged, when accumulating) for an
 * expert without rows. */
muon_status muon_grouped_linear_grad_weight(const muon_grouped* d, const void* x, const void* dy,
                                            const int32_t* offsets, float* dw, float* dbias, int32_t accumulate,
                                            void* workspace, size_t ws_bytes, void* stream);

/* Detail of the last failed layer operator call on this thread ("" if none). */
const char* muon_op_last_error(void);

/* ---- measurement (benchmarks) -------------------------------------------
 * Library plumbing, not defined by the pages. */

enum {
    MUON_KERNEL_MOMENTUM = 0, /* momentum + Nesterov + cast + sum of squares */
    MUON_KERNEL_GRAM = 1,     /* A = X X^T (upper tiles, mirrored) */
    MUON_KERNEL_POLY = 2,     /* B = b A + c A^2 (upper tiles, mirrored) */
    MUON_KERNEL_UPDATE = 3,   /* X <- a X + B X (a X added in fp32 before rounding) */
    MUON_KERNEL_NORMUON = 4,  /* NorMuon row factors */
    MUON_KERNEL_APPLY = 5,    /* parameter update */
    MUON_KERNEL_NS_SMALL = 6, /* every Newton-Schulz iteration of the bf16 matrices whose
                               * short side is at most 64 (one workgroup per matrix) */
    MUON_KERNEL_NS_PANEL = 7, /* every Newton-Schulz iteration of the bf16 matrices whose
                               * short side is 256 and long side at most 4096 (one
                               * workgroup per matrix, A and B kept in LDS) */
    MUON_KERNEL_COUNT = 8
};

/* Algorithmic work of one muon_step for this plan (frozen matrices excluded).
 * flops[k]: floating-point operations of kernel class k per step, counting a
 * symmetric product (Gram, A^2) as m(m+1)k; bytes[k]: bytes a kernel class
 * must move per step (momentum: g, m read, m, X~ written; apply: O, p read,
 * p written; NorMuon: row partials, v, f); launches[k]: launches per step. */
typedef struct muon_work {
    double flops[MUON_KERNEL_COUNT];
    double bytes[MUON_KERNEL_COUNT];
    int64_t launches[MUON_KERNEL_COUNT];
    int64_t active_elements;
} muon_work;

muon_status muon_work_stats(const muon_handle* h, muon_work* out);

/* on != 0: every later muon_step records a pair of HIP events around each
 * kernel launch on its stream (host-side records only, no device memory).
 * on == 0 stops recording; recorded pairs are kept until read. */
muon_status muon_profile_enable(muon_handle* h, int32_t on);

/* Wait for the recorded events and return, for kernel class `kernel`, the
 * number of recorded launches and their summed duration in milliseconds.
 * clear != 0 drops every record afterwards. */
muon_status muon_profile_read(muon_handle* h, int32_t kernel, int32_t clear, int64_t* launches, double* total_ms);

#ifdef __cplusplus
}
#endif

#endif /* LIBMUON_H */
