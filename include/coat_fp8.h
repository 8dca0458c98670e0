/*
 * coat_fp8.h - C ABI of the MI355X (gfx950) FP8-optimizer-state AdamW step.
 *
 * The method is COAT's optimizer with FP8-compressed Adam state as described
 * in "COAT: FP8 training, 40% less memory, 1.4x faster" (blob.wenxiaobai.com),
 * sections "FP8 optimizer states" and "Solution: dynamic range expansion",
 * and in its mirror on zhanchiexpo.com (per-group quantization of the states).
 * The FP8 bit layouts are those of the FP8 guide on maplevalley.com.cn,
 * section "format choice" (E4M3 = 1+4+3 bits, E5M2 = 1+5+2 bits), with OCP
 * E4M3FN / E5M2 semantics.
 *
 * State layout (everything flat, row-major, owned by the caller):
 *   - a tensor of n parameters is cut into groups of G consecutive elements
 *     (the last group may be shorter); groups never span tensors;
 *   - for each of the two Adam moments (m: first, v: second) the state is
 *       q[n]            uint8 FP8 codes (sign bit | magnitude code),
 *       s[ceil(n/G)]    fp64 per-group scale,
 *       k[ceil(n/G)]    fp32 per-group expansion exponent,
 *     and a stored code decodes to x = sign(q) * (|q| * s)^(1/k);
 *   - requantizing a group takes amax = max|x| and amin = min over nonzero |x|,
 *     k = ln(R_fp8) / ln(amax/amin) (k = 1 if amax/amin <= 1 + 1e-6, if the
 *     group is all zero, or with COAT_FMT_NO_EXPAND), s = amax^k / fpmax, and
 *     rounds fpmax * (|x| / amax)^k to the FP8 grid, nearest, ties to even,
 *     saturating at fpmax. R_fp8 = fpmax / min subnormal: 448 / 2^-9 for E4M3,
 *     57344 / 2^-16 for E5M2. k is lowered when needed so that amax^k and
 *     amax^k / R_fp8 stay within [2^-1022, 2^1023]. A group holding a
 *     non-finite moment is stored with s = NaN, k = 1 and every code 0x7F.
 *
 * Conventions for every entry point:
 *   - all array pointers are device pointers (HIP device memory) owned by the
 *     caller; the library allocates nothing and keeps no state between calls,
 *     except the device table array of coat_fp8_adamw_step_multi_static;
 *   - work is enqueued on `stream` (a hipStream_t; NULL = the null stream) and
 *     the call returns without waiting; device-side faults surface at the
 *     caller's next synchronization;
 *   - arrays must not overlap one another; in/out arrays are updated in place;
 *   - the byte arrays (codes), fp32 and bf16 arrays must start on a 16-byte
 *     boundary; s and k arrays need their natural alignment;
 *   - group G must be a power of two in [16, 1024];
 *   - return value: COAT_OK, or a negative status (see coat_strerror); on
 *     error nothing has been enqueued, except where COAT_EHIP is said to
 *     leave earlier launches of the same call.
 */
#ifndef COAT_FP8_H
#define COAT_FP8_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as hipStream_t, declared here so that this header needs no HIP include. */
typedef struct ihipStream_t* coat_stream_t;

enum {
    COAT_FMT_E4M3 = 0,          /* OCP E4M3FN: bias 7, max 448, NaN 0x7F/0xFF, no Inf */
    COAT_FMT_E5M2 = 1,          /* OCP E5M2: bias 15, max 57344, Inf 0x7C/0xFC */
    COAT_FMT_NO_EXPAND = 0x100  /* flag OR-ed into a format: force k = 1 (plain absmax) */
};

enum {
    COAT_OK = 0,
    COAT_EINVAL = -1, /* null pointer with n > 0, n < 0, bad group or format, step < 1,
                         non-finite hyperparameter, workspace too small */
    COAT_EALIGN = -2, /* a pointer does not meet the alignment stated above */
    COAT_EHIP = -3,   /* the HIP runtime refused the launch */
    COAT_ERANGE = -4  /* more tensors than COAT_STATIC_MAX_TENSORS (static-table entry point) */
};

/*
 * One AdamW step over FP8-compressed moments of one tensor (COAT's optimizer
 * step, article section "FP8 optimizer states"; the update is decoupled
 * weight decay AdamW with bias correction at t = step):
 *   m' = b1 m + (1 - b1) g,  v' = b2 v + (1 - b2) g^2,
 *   p' = p (1 - lr wd) - (lr / (1 - b1^t)) m' / (sqrt(v' / (1 - b2^t)) + eps),
 * where m, v are the dequantized stored moments; then m', v' are requantized
 * group by group with dynamic range expansion.
 *
 *   params       fp32 master weights, n, in/out
 *   params_bf16  bf16 copy of the new master weights (RNE), n, out; may be NULL
 *   grads        bf16 gradients, n, in
 *   m_q,m_s,m_k  first-moment codes (n), scales and exponents (ceil(n/G)), in/out
 *   v_q,v_s,v_k  second-moment state, same shapes, in/out
 *   fmt_m/fmt_v  COAT_FMT_E4M3 or COAT_FMT_E5M2, optionally | COAT_FMT_NO_EXPAND
 *   step         t >= 1, the step being taken
 * The stored moments are states written by coat_fp8_quantize or by an earlier
 * step (an all-zero group stores s = 0 with signed-zero codes, a poisoned
 * group s = NaN with NaN codes). For states neither writes (an Inf code under
 * a zero or NaN scale, a scale of +Inf) the result is unspecified.
 */
int coat_fp8_adamw_step(float* params, uint16_t* params_bf16, const uint16_t* grads,
                        uint8_t* m_q, double* m_s, float* m_k,
                        uint8_t* v_q, double* v_s, float* v_k,
                        int64_t n, int32_t group, int32_t fmt_m, int32_t fmt_v,
                        float lr, float beta1, float beta2, float eps, float weight_decay,
                        int64_t step, coat_stream_t stream);

/* One tensor of a parameter list for the multi-tensor step; fields as above. */
typedef struct coat_tensor {
    float* params;
    uint16_t* params_bf16; /* may be NULL */
    const uint16_t* grads;
    uint8_t* m_q;
    double* m_s;
    float* m_k;
    uint8_t* v_q;
    double* v_s;
    float* v_k;
    int64_t n;            /* 0 allowed: the tensor is skipped */
} coat_tensor;

/* Bytes of device workspace a plan over `count` tensors needs. */
size_t coat_multi_workspace_bytes(int32_t count);

/*
 * A parameter list prepared for repeated multi-tensor steps: the descriptor
 * table and the tile table live in caller-owned device workspace.
 */
typedef struct coat_multi_plan {
    void* workspace;    /* device memory holding the tables */
    int32_t count;      /* tensors */
    int64_t tiles;      /* 1024-element tiles across all tensors */
    int64_t n_total;    /* parameters across all tensors */
    int32_t n_partial;  /* tensors whose size is not a multiple of 1024 */
} coat_multi_plan;

/*
 * Validate `count` descriptors (host array) and enqueue on `stream` their copy,
 * with a tile table, into `workspace` (device memory, 256-byte aligned, at
 * least coat_multi_workspace_bytes(count) bytes). The tables travel in the
 * arguments of small copy launches, one per 3 KB of tables (11 for the 363
 * tensors of a Llama-2-13B list), so the call neither stages through host
 * memory nor waits: it returns once they are enqueued, and the host array
 * `tensors` is read during the call only. Steps
 * enqueued after it on the same stream see the tables; a step on another
 * stream must be ordered after them by the caller. The plan stays valid while
 * the tensors' buffers and the workspace do. COAT_EHIP (a refused launch) may
 * leave the copies before it enqueued.
 */
int coat_multi_plan_init(coat_multi_plan* plan, const coat_tensor* tensors, int32_t count,
                         void* workspace, size_t workspace_bytes, coat_stream_t stream);

/*
 * One step over every tensor of a plan, asynchronous: one kernel launch over
 * the whole list (for G >= 128 a second, small one when some tensor ends
 * inside a 1024-element tile: its last tile). The result equals calling
 * coat_fp8_adamw_step on each tensor in turn, bit for bit.
 */
int coat_fp8_adamw_step_planned(const coat_multi_plan* plan, int32_t group, int32_t fmt_m,
                                int32_t fmt_v, float lr, float beta1, float beta2, float eps,
                                float weight_decay, int64_t step, coat_stream_t stream);

/*
 * Convenience: coat_multi_plan_init followed by coat_fp8_adamw_step_planned
 * (it enqueues the table copies, then the step, all on `stream`, and returns
 * without waiting).
 */
int coat_fp8_adamw_step_multi(const coat_tensor* tensors, int32_t count, int32_t group,
                              int32_t fmt_m, int32_t fmt_v, float lr, float beta1, float beta2,
                              float eps, float weight_decay, int64_t step, void* workspace,
                              size_t workspace_bytes, coat_stream_t stream);

/* Largest parameter list coat_fp8_adamw_step_multi_static accepts. */
#define COAT_STATIC_MAX_TENSORS 4096

/*
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation): the
 * multi-tensor step of coat_fp8_adamw_step_multi with its plan tables kept in
 * a device array inside the library instead of a caller workspace. It takes
 * the same arguments minus the workspace, calls no allocator (no hipMalloc,
 * no hipFree, no host staging buffer) and does not synchronize: it enqueues a
 * few small copy launches that carry the tables in their kernel arguments,
 * then the step, all on `stream`, and returns. The result equals
 * coat_fp8_adamw_step_multi's bit for bit.
 *   - count <= COAT_STATIC_MAX_TENSORS (4096), else COAT_ERANGE before anything
 *     is enqueued; other errors as for coat_fp8_adamw_step_multi;
 *   - each GPU holds one copy of the table array (about 377 KB) from its
 *     first call until the process ends; it is looked up once per device with
 *     that device current, so `stream` must belong to the current device;
 *   - every call on a GPU rewrites that GPU's one array: calls that may
 *     overlap on one GPU (other streams, other host threads without ordering)
 *     race, so they must be serialized, e.g. issued on one stream; the array
 *     keeps the last call's tables, and every entry the step reads is
 *     written by the call itself, so nothing has to start cleared;
 *   - the host array `tensors` is read during the call only;
 *   - COAT_EHIP (a refused launch) may leave the copies before it enqueued.
 */
int coat_fp8_adamw_step_multi_static(const coat_tensor* tensors, int32_t count, int32_t group,
                                     int32_t fmt_m, int32_t fmt_v, float lr, float beta1,
                                     float beta2, float eps, float weight_decay, int64_t step,
                                     coat_stream_t stream);

/*
 * Quantize an fp32 array into FP8 state (q, s, k) with per-group dynamic
 * range expansion, exactly as the step requantizes a moment (article section
 * "Solution: dynamic range expansion"). Used to initialise or import state.
 *   x in (n), q out (n), s/k out (ceil(n/G)).
 */
int coat_fp8_quantize(const float* x, int64_t n, int32_t group, int32_t fmt, uint8_t* q,
                      double* s, float* k, coat_stream_t stream);

/*
 * Dequantize FP8 state to fp32: x = sign(q) (|q| s)^(1/k), the value the step
 * starts from (in fp64), to within one fp32 ulp (the power is evaluated to
 * about 2^-28 before the rounding to fp32). Used to export state.
 */
int coat_fp8_dequantize(const uint8_t* q, const double* s, const float* k, int64_t n,
                        int32_t group, int32_t fmt, float* x, coat_stream_t stream);

/*
 * Plain FP8 codec on fp32 values (no scaling, no expansion): encode rounds to
 * nearest, ties to even, saturating at the largest finite value, NaN -> 0x7F;
 * decode is exact. Formats as in the FP8 guide, section "format choice".
 */
int coat_fp8_encode(const float* y, int64_t n, int32_t fmt, uint8_t* q, coat_stream_t stream);
int coat_fp8_decode(const uint8_t* q, int64_t n, int32_t fmt, float* y, coat_stream_t stream);

/*
 * FP8 activation codec with per-tensor or per-group granularity (article
 * section "Solution: mixed-granularity FP8 precision flow": layer inputs are
 * kept in FP8 for the backward pass, the quantization granularity varying
 * between layers; which layer takes which granularity is the caller's
 * choice). Plain absmax scaling of bf16 values, no expansion:
 *   group == 0: one scale for the whole array (scale[1]);
 *   group = G, a power of two in [16, 1024]: one scale per G consecutive
 *   values (scale[ceil(n/G)], the last group may be short);
 *   s = RN32(amax / fpmax); code = encode(RN32(x / s)) rounded to nearest,
 *   ties to even, saturating (for s = 0, an all-zero group, the sign alone);
 *   a tensor or group holding a NaN or Inf: s = NaN and every code 0x7F.
 * Dequantize writes RN_bf16(RN32(decode(code) * s)).
 *   x bf16 in (n), q out (n), scale out; fmt COAT_FMT_E4M3 or COAT_FMT_E5M2
 *   (no flags). x, q 16-byte aligned (COAT_EALIGN), scale 4-byte aligned.
 * Per tensor, the quantizer uses scale[0] as its accumulator while it runs
 * (it enqueues four small launches); the caller must not read it until the
 * stream reaches the end of the call.
 */
int coat_fp8_act_quantize(const uint16_t* x, int64_t n, int32_t group, int32_t fmt, uint8_t* q,
                          float* scale, coat_stream_t stream);
int coat_fp8_act_dequantize(const uint8_t* q, const float* scale, int64_t n, int32_t group,
                            int32_t fmt, uint16_t* x, coat_stream_t stream);

/* Element types of the entry points below. */
enum { COAT_BF16 = 0, COAT_FP32 = 1 };

/*
 * Microscaled 4-bit floating point (OCP MX, E2M1 elements): a row is cut into
 * blocks of 32 consecutive values; each block has one scale byte b and stands
 * for code * 2^(b - 127), a code being a sign bit and one of the magnitudes
 * 0, 0.5, 1, 1.5, 2, 3, 4, 6.
 *   - quantizing a block: e = floor(log2(amax)) - 2, at least -127; b = e + 127;
 *     code = x / 2^e rounded to nearest, ties to the even code, magnitudes over
 *     6 cut to 6. An all-zero block has b = 0 and signed-zero codes; a block
 *     holding a NaN or Inf has b = 0xFF and codes 0, and reads back as NaN.
 *   - a matrix of `rows` rows of k values is stored as
 *       q[rows][coat_mx4_code_bytes(k)]   two codes a byte, the first in the low
 *                                         half; k rounded up to 128 values,
 *       s[rows][coat_mx4_scale_bytes(k)]  one byte a block, rounded up to 16,
 *     both without gaps, the values, blocks and bytes past k zero.
 */
int64_t coat_mx4_code_bytes(int64_t k);  /* 64 ceil(k / 128) */
int64_t coat_mx4_scale_bytes(int64_t k); /* 16 ceil(k / 512) */

/*
 * Quantize a matrix along its rows, its columns, or both in one pass.
 *   x      rows x cols, bf16 or fp32 (dtype), row i at x + i ld, in
 *   q, s   x's rows quantized (rows of cols values), out; both NULL to skip
 *   q_t, s_t  x's columns quantized: the transposed matrix, cols rows of
 *          `rows` values each, out; both NULL to skip
 * ld >= cols counts elements. x needs its type's alignment, the byte arrays 16
 * (COAT_EALIGN). rows = 0 or cols = 0 writes nothing. The sizes are limited to
 * 2^31 - 1 each (COAT_EINVAL).
 */
int coat_mx4_quantize(const void* x, int64_t rows, int64_t cols, int64_t ld, int32_t dtype,
                      uint8_t* q, uint8_t* s, uint8_t* q_t, uint8_t* s_t, coat_stream_t stream);

/*
 * Read a quantized matrix back: x (rows x cols, bf16 or fp32, row i at
 * x + i ld) gets each code's value, rounded once (bf16 and fp32 hold every
 * value of a matrix that coat_mx4_quantize wrote exactly). Elements of x
 * between cols and ld are left as they are.
 */
int coat_mx4_dequantize(const uint8_t* q, const uint8_t* s, int64_t rows, int64_t cols, void* x,
                        int64_t ld, int32_t dtype, coat_stream_t stream);

/*
 * Product of two quantized matrices on the matrix units:
 *   y[i][j] = sum over k of A[i][k] B[j][k],  A m x k, B n x k, y m x n.
 * With row-quantized activations X and weights W (out x in) a linear layer is
 * Y = X W^T; with the column-quantized forms of coat_mx4_quantize its backward
 * products are dX = dY (W^T)^T and dW = dY^T (X^T)^T. Sums are held in fp32,
 * in an order that depends on (m, n, k) alone; y is rounded once.
 *   y      bf16 or fp32 (dtype), row i at y + i ld, ld >= n, out
 *   workspace  device memory, 256-byte aligned, at least
 *          coat_mx4_matmul_workspace_bytes(m, n, k) bytes (may be NULL if that
 *          is 0); calls that may overlap in time need one each.
 * m = 0 or n = 0 writes nothing; k = 0 writes zeros. The byte arrays are
 * 16-byte aligned, y has its type's alignment (COAT_EALIGN). m, n and k are
 * limited to 2^31 - 1 (COAT_EINVAL). Elements of y between n and ld are left
 * as they are.
 */
size_t coat_mx4_matmul_workspace_bytes(int64_t m, int64_t n, int64_t k);
int coat_mx4_matmul(const uint8_t* a_q, const uint8_t* a_s, int64_t m, const uint8_t* b_q,
                    const uint8_t* b_s, int64_t n, int64_t k, void* y, int64_t ld, int32_t dtype,
                    void* workspace, size_t workspace_bytes, coat_stream_t stream);

/*
 * The border between two blocks of a transformer: the norm after a block, the
 * gated and scaled residual addition, and the norm before the next block,
 * whose result is that block's layer input. Per token (row) t, with
 * N(a) = a / sqrt(mean(a^2) + eps) over the row and g the gate's row
 * t / rows_per_gate,
 *   z  = w_post N(y)            (z = y if post = 0)
 *   r' = r + scale g z          rounded to the stream's type
 *   h  = w_pre N(r')            computed from the rounded r'
 * A missing weight or gate counts as ones.
 */
typedef struct coat_border {
    int64_t rows;          /* tokens */
    int64_t cols;          /* channels, 1 .. COAT_BORDER_MAX_COLS */
    int64_t rows_per_gate; /* >= 1; the gate has ceil(rows / rows_per_gate) rows (1: one per token, rows: one for all) */
    float eps;             /* at least 2^-126 (the smallest normal fp32), finite */
    float scale;           /* the residual scale, finite (its products with a row's factor and with D are formed in fp32) */
    int32_t post;          /* 1: y is normalised, 0: it is not */
    int32_t stream_type;   /* COAT_BF16 or COAT_FP32: r, r_out, dr_out, dr */
    int32_t param_type;    /* of w_post, w_pre and gate */
    int32_t grad_type;     /* of dw_post, dw_pre and dgate */
} coat_border;

#define COAT_BORDER_MAX_COLS 16384

enum { COAT_FMT_MX4 = 2 }; /* a layer input stored as coat_mx4_quantize stores it */

/*
 * Forward. All matrices are rows x cols without gaps.
 *   y      bf16, the block's output; NULL: no addition (the first block), r' = r
 *   r      the residual stream
 *   w_post, w_pre  cols values, may be NULL; w_post only with post
 *   gate   ceil(rows / rows_per_gate) x cols, may be NULL; only with y
 *   r_out  r', out; may be NULL, may be r itself
 *   h      bf16 layer input, out; may be NULL
 *   q, q_scale  the layer input in a stored form, out; both may be NULL. It is
 *          exactly that of the bf16 h:
 *          fmt COAT_FMT_E4M3 / COAT_FMT_E5M2: as coat_fp8_act_quantize with
 *          `group` a power of two in [16, 512] that divides cols, fp32 scales;
 *          fmt COAT_FMT_MX4: as coat_mx4_quantize along the rows, group = 32,
 *          q_scale its scale bytes.
 * With h and q both NULL there is no norm before the next block (w_pre NULL);
 * at least one output is needed. Matrices of bf16 and fp32 need their type's
 * alignment, q 16 bytes, q_scale 4, and 16 for COAT_FMT_MX4 (COAT_EALIGN).
 * Sums of squares are held in fp32. A row that holds a NaN has a norm of NaN. A row
 * that holds an Inf, or whose sum of squares passes fp32 (a root mean square over
 * 1.8e19 / sqrt(cols)), is divided by infinity: N is NaN where the Inf stands and 0
 * elsewhere, so that h is 0 there, and r' = r after such a row of y. Other rows do
 * not change.
 */
int coat_block_norm(const coat_border* b, const uint16_t* y, const void* r, const void* w_post,
                    const void* w_pre, const void* gate, void* r_out, uint16_t* h, uint8_t* q,
                    void* q_scale, int32_t group, int32_t fmt, coat_stream_t stream);

/*
 * Backward, from the stored r' (the forward's r_out, or r if there was no
 * addition). With D the whole gradient of r',
 *   D  = dr_out + N'(r')^T (w_pre dh)     dw_pre  = sum_t dh N(r')
 *   dr = D                                dgate   = sum over a gate row's tokens of scale z D
 *   dy = N'(y)^T (w_post scale g D)       dw_post = sum_t scale g D N(y)
 * (N'^T the transposed derivative of N; without the post-norm dy = scale g D).
 *   dr_out  gradient of r' from later blocks; NULL: zero
 *   dh      bf16 gradient of h; NULL: there was no norm before the next block
 *   dr      out, the stream's type; may be dr_out itself
 *   dy      bf16, out, with y; NULL without y
 *   dw_post, dw_pre, dgate  out, grad_type; each may be NULL, and is only
 *           allowed with its weight or gate; rows = 0 gives zeros. The sums are
 *           held in fp32, in an order that depends on the sizes alone.
 *   workspace  device memory, 256-byte aligned, at least
 *           coat_block_norm_backward_workspace_bytes(b) bytes; calls that may
 *           overlap in time need one each.
 * A row of r' (with dh) or of y (with post) that holds a NaN or Inf gives NaN in all of
 * its dr and dy, or its dy, and in the sums over tokens that those values enter. For a
 * finite row whose sum of squares passes fp32 what goes through that norm is 0, or NaN
 * if the sum of its products with the gradient passes fp32 too.
 */
size_t coat_block_norm_backward_workspace_bytes(const coat_border* b);
int coat_block_norm_backward(const coat_border* b, const uint16_t* y, const void* r_out,
                             const void* dr_out, const uint16_t* dh, const void* w_post,
                             const void* w_pre, const void* gate, void* dr, uint16_t* dy,
                             void* dw_post, void* dw_pre, void* dgate, void* workspace,
                             size_t workspace_bytes, coat_stream_t stream);

/*
 * The products of a training step, over the bf16 weights that the optimizer step
 * writes (one row per output feature): a linear layer with its epilogue, dropout
 * without a stored mask, and the softmax cross entropy of a vocabulary projection
 * without stored logits. All matrices have one row per token, row i at p + i ld,
 * ld >= the columns, counting elements; elements between the columns and ld are
 * neither read nor written. Sizes are limited to 2^31 - 1 each. Matrices need
 * their type's alignment (COAT_EALIGN).
 *
 * Dropout. rng points to two 64-bit numbers in device memory, (seed, step), read
 * when the work runs, so that a captured graph draws anew after they changed.
 * Element (i, j) of a matrix with `cols` columns takes 16 bits of the Philox 4x32
 * generator with 10 rounds (Salmon et al., "Parallel random numbers: as easy as 1,
 * 2, 3"): key seed, counter (i ceil(cols / 8) + j / 8, step + offset), 64 bits
 * each with the low words first; half word j % 8 of the four output words, low
 * halves first. It is dropped if they are under t = round(65536 p), at most 65535;
 *   D(v) = v 65536 / (65536 - t) where kept, 0 where dropped
 * (whatever v was). offset tells the uses of one (seed, step) apart: a layer's
 * number, say, with step advanced by the number of layers. p = 0 needs no rng.
 */
enum { COAT_ACT_NONE = 0, COAT_ACT_RELU = 1, COAT_ACT_GELU = 2, COAT_ACT_GELU_TANH = 3, COAT_ACT_SILU = 4 };

typedef struct coat_epilogue {
    int32_t act;        /* COAT_ACT_*: max(z, 0); z Phi(z); z sigmoid(sqrt(8 / pi) (z + 0.044715 z^3)); z sigmoid(z) */
    float scale;        /* finite, also times the factor of D */
    float p;            /* dropout, 0 <= p < 1 */
    int64_t offset;     /* added to the step */
    const int64_t* rng; /* (seed, step) in device memory, 8-byte aligned; may be NULL if p = 0 */
} coat_epilogue;

/*
 * Linear layer: z = x w^T + bias, y = residual + scale D(act(z)).
 *   x      bf16, m x k      w  bf16, n x k
 *   bias   n values of bias_type, may be NULL
 *   residual  m x n, the type of y; may be NULL, may be y itself (same ld)
 *   z      bf16, m x n, out: kept for the backward pass; may be NULL
 *   y      m x n, bf16 or fp32 (y_type), out
 * Sums are held in fp32, in an order that depends on the sizes and on whether x and
 * w are aligned (below) alone; y and z are each rounded once from them.
 *   workspace  device memory, 256-byte aligned, at least
 *          coat_linear_workspace_bytes(m, n, k, aligned) bytes (may be NULL if that
 *          is 0); calls that may overlap in time need one each. aligned: whether x
 *          and w are 16-byte aligned and k, ldx and ldw multiples of 8, ldx and ldw
 *          under 2^22.
 * m = 0 or n = 0 writes nothing; k = 0 gives z = bias.
 */
size_t coat_linear_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t aligned);
int coat_linear(const uint16_t* x, int64_t m, int64_t k, int64_t ldx, const uint16_t* w, int64_t n, int64_t ldw,
                const coat_epilogue* e, const void* bias, int32_t bias_type, const void* residual,
                int64_t ldr, uint16_t* z, int64_t ldz, void* y, int64_t ldy, int32_t y_type,
                void* workspace, size_t workspace_bytes, coat_stream_t stream);

/*
 * Its backward pass, with the forward's epilogue and random numbers:
 *   dz = scale D(dy) act'(z),  dx = dz w,  dw = dz^T x,  dbias = sum of dz over the tokens
 * (the gradient of residual is dy). act' is taken at the stored z; that of the
 * first activation is 0 at 0. Where D(dy) is 0 so is dz, whatever z holds.
 *   dy     m x n, bf16 or fp32 (dy_type)
 *   z      the forward's; needed with an activation, may be NULL without
 *   dx     bf16, m x k, dw bf16, n x k, dbias n values of dbias_type: out, each may
 *          be NULL, one at least is needed; x may be NULL without dw, w without dx
 * The products take dz rounded to bf16, without the factors scale and 1 / (1 - p),
 * which their sums are multiplied by; dbias adds dz as it was before. Up to 2048
 * values of dz are taken as two bf16 terms. m = 0 gives dw and dbias of zeros, n = 0
 * a dx of zeros.
 *   workspace  as above, at least coat_linear_backward_workspace_bytes(m, n, k,
 *          aligned) bytes; aligned: whether x and w are, as above.
 */
size_t coat_linear_backward_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t aligned);
int coat_linear_backward(const void* dy, int64_t lddy, int32_t dy_type, const uint16_t* x, int64_t m, int64_t k,
                         int64_t ldx, const uint16_t* w, int64_t n, int64_t ldw, const coat_epilogue* e,
                         const uint16_t* z, int64_t ldz, uint16_t* dx, int64_t lddx, uint16_t* dw, int64_t lddw,
                         void* dbias, int32_t dbias_type, void* workspace, size_t workspace_bytes,
                         coat_stream_t stream);

/*
 * Dropout of a matrix: y = residual + scale D(x).
 *   x      rows x cols, bf16 or fp32 (x_type)
 *   residual  the type of y; may be NULL
 *   y      rows x cols, bf16 or fp32 (y_type), out; may be x or residual itself (same
 *          type and ld)
 * Its backward pass is the same call on dy, without the residual: dx = scale D(dy).
 */
int coat_dropout(const void* x, int64_t rows, int64_t cols, int64_t ldx, int32_t x_type, const void* residual,
                 int64_t ldr, float scale, float p, const int64_t* rng, int64_t offset, void* y, int64_t ldy,
                 int32_t y_type, coat_stream_t stream);

/*
 * Softmax cross entropy of a vocabulary projection, the logits never stored:
 *   l = x w^T,  lse = log sum_v exp(l_v),  loss = lse - l_label   per token.
 *   x      bf16, tokens x cols      w  bf16, vocab x cols, vocab >= 1
 *   labels tokens 64-bit numbers; a token whose label is ignore_index is left out:
 *          loss 0, lse 0, and its row of x is not used. Any other label outside
 *          [0, vocab) makes that token's loss NaN (and its gradients).
 *   loss, lse  tokens fp32, out
 * The logits are sums in fp32 and are not rounded further.
 *   workspace  as above, coat_linear_cross_entropy_workspace_bytes(tokens, vocab,
 *          cols, aligned); aligned: whether x and w are, as for the linear layer, and
 *          tokens ldx is under 2^31.
 */
size_t coat_linear_cross_entropy_workspace_bytes(int64_t tokens, int64_t vocab, int64_t cols, int32_t aligned);
int coat_linear_cross_entropy(const uint16_t* x, int64_t tokens, int64_t cols, int64_t ldx, const uint16_t* w,
                              int64_t vocab, int64_t ldw, const int64_t* labels, int64_t ignore_index,
                              float* loss, float* lse, void* workspace, size_t workspace_bytes,
                              coat_stream_t stream);

/*
 * Its backward pass, from the forward's lse and loss:
 *   g = dloss (softmax(l) - onehot(label)),  dx = g w,  dw = g^T x,
 * the logits computed again in pieces of the vocabulary.
 *   loss   the forward's, tokens fp32; the label's own g is dloss expm1(-loss), good to
 *          the digits that loss has. May be NULL, as in the form without it: that g is
 *          then dloss (exp(l_label - lse) - 1), off by about 2^-23 |lse| dloss, which is
 *          much of it for a token that the model is sure of.
 *   dloss  fp32, the gradient of each token's loss (dloss_count = tokens), or one
 *          value for all of them (dloss_count = 1)
 *   dx     bf16, tokens x cols, dw bf16, vocab x cols: out, each may be NULL, one
 *          at least is needed. A token that is left out has zeros in dx and no part
 *          in dw, whatever its x holds.
 * The products take g rounded to bf16, without dloss's largest finite magnitude
 * among the tokens that count, which their sums are multiplied by; sums are held in
 * fp32. A dloss under 2^-100 of that magnitude loses digits of its g, and one under
 * 2^-126 of it may count as zero, also in its own row of dx. Up to 16 tokens, or
 * 2048 logits, have their g taken as two bf16 terms. tokens = 0 gives a dw of zeros.
 * The workspace holds the g of a piece: of up to 2^27 logits, or 2048 columns.
 *   workspace  as above, coat_linear_cross_entropy_backward_workspace_bytes(tokens,
 *          vocab, cols, aligned).
 */
size_t coat_linear_cross_entropy_backward_workspace_bytes(int64_t tokens, int64_t vocab, int64_t cols, int32_t aligned);
int coat_linear_cross_entropy_backward_loss(const uint16_t* x, int64_t tokens, int64_t cols, int64_t ldx, const uint16_t* w,
                                            int64_t vocab, int64_t ldw, const int64_t* labels, int64_t ignore_index,
                                            const float* lse, const float* loss, const float* dloss,
                                            int64_t dloss_count, uint16_t* dx, int64_t lddx, uint16_t* dw,
                                            int64_t lddw, void* workspace, size_t workspace_bytes,
                                            coat_stream_t stream);
int coat_linear_cross_entropy_backward(const uint16_t* x, int64_t tokens, int64_t cols, int64_t ldx, const uint16_t* w,
                                       int64_t vocab, int64_t ldw, const int64_t* labels, int64_t ignore_index,
                                       const float* lse, const float* dloss, int64_t dloss_count, uint16_t* dx,
                                       int64_t lddx, uint16_t* dw, int64_t lddw, void* workspace,
                                       size_t workspace_bytes, coat_stream_t stream);

/* Static description of a status code. */
const char* coat_strerror(int status);

/* ABI version of this library (major * 100 + minor). */
int coat_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* COAT_FP8_H */
