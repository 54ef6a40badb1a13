/*
 * paro.h - C ABI of the MI355X (gfx950) rotated W4G128 linear library.
 *
 * The library implements the inference hot path of ParoQuant (pairwise
 * rotation quantization, arXiv 2511.10645):
 *
 *   Y = X W + b = (X T^-1)(T W) + b                     (CSDN article, section 2.1)
 *   T = (prod_{t=1..K} R(P_t, Theta_t)) diag(alpha)     (paper notes, "关键设计")
 *
 * R(P_t, Theta_t) is one stage of independent Givens rotations: every channel
 * of a quantization group belongs to exactly one pair (i, j) of the stage, and
 * the pair is rotated by its own angle theta with the 2x2 matrix
 * [[cos, -sin], [sin, cos]] acting on (v_i, v_j) (CSDN article, section 2.2):
 *
 *   v_i <- cos(theta) v_i - sin(theta) v_j,   v_j <- sin(theta) v_i + cos(theta) v_j
 *
 * Conventions fixed by this library (the pages leave them open):
 *   - stage 0 of the arrays is applied first;
 *   - activations are divided by alpha and then go through the SAME stages in
 *     the SAME order with the SAME update (this equals x T^-1 for a row x);
 *     weights are multiplied by alpha and then go through the stages;
 *   - W4G128 quantization (paper notes, "主实验"; per-group s and z:
 *     "损失函数 / 训练策略") is asymmetric min/max round-to-nearest-even over
 *     15 steps with the range widened to include 0, an fp16 scale and an
 *     integer zero in [0, 15].
 *
 * Types: fp16 tensors are passed as uint16_t* (IEEE binary16 bit patterns).
 * Every tensor is row-major and contiguous. Device pointers are HIP device
 * memory (for example torch.Tensor.data_ptr() of a ROCm tensor); host
 * pointers are ordinary memory. The caller owns every tensor; a rotation
 * handle owns only the device tables it allocates in paro_rotation_create and
 * frees in paro_rotation_destroy.
 *
 * Errors: every int-returning function returns PARO_OK (0) or a negative
 * paro_status and never throws or aborts. Argument checks run on the host
 * before anything is enqueued, so a failed check enqueues nothing. A failed
 * kernel launch returns PARO_ERR_HIP. Asynchronous device faults surface at
 * the caller's next synchronisation, as with any HIP library.
 * paro_last_error() returns a thread-local message for the last failure.
 *
 * Threads and streams: hot calls (paro_rotate, paro_w4_linear) allocate
 * nothing, do not synchronise and write no global state (they may be captured
 * into a HIP graph); a handle may be used from several threads and streams at
 * once. Per-device set-up that needs allocation and synchronisation happens in
 * paro_device_init, which paro_rotation_create also runs.
 */
#ifndef PARO_H
#define PARO_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h> /* hipStream_t */

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PARO_OK = 0,
  PARO_ERR_NULL = -1,        /* a required pointer is NULL */
  PARO_ERR_SHAPE = -2,       /* sizes inconsistent (d % group, N % 16, negative sizes, ...) */
  PARO_ERR_PAIRING = -3,     /* a stage is not a perfect pairing inside every group */
  PARO_ERR_VALUE = -4,       /* alpha <= 0 or non-finite, theta non-finite, non-finite weights */
  PARO_ERR_ALIGN = -5,       /* a tensor pointer is not 16-byte aligned */
  PARO_ERR_UNSUPPORTED = -6, /* a valid request the library does not implement */
  PARO_ERR_WORKSPACE = -7,   /* workspace missing or too small */
  PARO_ERR_HIP = -8          /* a HIP runtime call failed */
} paro_status;

/* Static string naming a status code. Never NULL. */
const char* paro_status_string(int status);

/* Thread-local detail message of the last failing call on this thread ("" if none). */
const char* paro_last_error(void);

/*
 * Per-device set-up (synchronous; allocates, launches and synchronises on the
 * null stream, so not inside a stream capture). Checks once per device how
 * workgroups are dispatched to the XCDs (the small-batch linear splits k over
 * workgroups that must meet in one XCD's L2) and records the result;
 * idempotent and thread-safe. paro_rotation_create calls it for its device.
 * A device on which it never ran still gives correct results: the
 * small-batch linear then exchanges its partial sums through memory-side
 * (system-scope) accesses, about 15% slower.
 * Errors: PARO_ERR_HIP (nothing is recorded; a later call tries again),
 * PARO_ERR_UNSUPPORTED (device ordinal >= 64).
 */
int paro_device_init(void);

/* Opaque rotation plan: the K stages of pairs/angles plus alpha for one layer,
 * validated and turned into device tables. Immutable after creation. */
typedef struct paro_rotation paro_rotation;

/*
 * Create a rotation plan on the current HIP device (synchronous).
 *
 *   d      number of input channels; d % group == 0; d % 128 == 0;
 *          d <= 2^24.
 *   group  rotation group size: 64, 128 or 256 (pairs never leave a group,
 *          paper notes "关键设计").
 *   K      number of stages, 0 <= K <= 32 (the pages' default is 8).
 *   pairs  host int32 [K][d/2][2], global channel ids. In every stage each
 *          channel appears exactly once and i / group == j / group. The
 *          order of pairs inside a stage is free; the order (i, j) inside a
 *          pair selects the sign as in the update above (swapping i and j is
 *          the same as negating theta). Partial and sparse pairings (only
 *          some pairs rotate; paper notes "核心观察") are expressed with
 *          theta = 0, an exact identity; the activation side then skips the
 *          identities and runs fewer stages where the remaining rotations
 *          allow it (see paro_rotation_plan_host's layout[4]).
 *   theta  host float [K][d/2], radians, finite. The library evaluates
 *          c = (float)cos((double)theta), s = (float)sin((double)theta) on the
 *          host.
 *   alpha  host float [d], finite and > 0.
 *   out    receives the handle.
 *
 * Runs paro_device_init for the current device.
 * Errors: PARO_ERR_NULL, PARO_ERR_SHAPE, PARO_ERR_PAIRING, PARO_ERR_VALUE,
 * PARO_ERR_UNSUPPORTED (group not in {64,128,256}, K > 32, d % 128 != 0,
 * d > 2^24),
 * PARO_ERR_HIP (device allocation or copy failed). The host arrays are only
 * read during the call.
 */
int paro_rotation_create(int64_t d, int32_t group, int32_t K, const int32_t* pairs,
                         const float* theta, const float* alpha, paro_rotation** out);

/* Free the plan's device tables (synchronous). NULL is a no-op. The caller
 * must make sure no enqueued work still uses the handle. */
void paro_rotation_destroy(paro_rotation* r);

/* Read back plan properties (host only; any pointer may be NULL). */
int paro_rotation_info(const paro_rotation* r, int64_t* d, int32_t* group, int32_t* K);

/*
 * Online activation transform X' = X T^-1, row by row
 * (paper notes, "关键设计" and "亮点与洞察": one fused launch for all stages).
 *
 *   x, y   device fp16 [M][d], 16-byte aligned. y == x (in place) is allowed;
 *          any other overlap is undefined.
 *   M      number of token rows, 0 <= M <= 2^31 - 1; M == 0 is a no-op.
 *   stream HIP stream the kernel is enqueued on (0 = the null stream).
 *
 * Arithmetic: fp32 inside, one fp16 round-to-nearest-even per output.
 * Errors: PARO_ERR_NULL, PARO_ERR_SHAPE (M out of range), PARO_ERR_ALIGN,
 * PARO_ERR_HIP.
 */
int paro_rotate(const paro_rotation* r, const uint16_t* x, uint16_t* y, int64_t M,
                hipStream_t stream);

/*
 * Offline weight transform and int4 group quantization: Q(T W) (r != NULL)
 * or Q(W) (r == NULL, plain W4).
 *
 *   w        device fp16 [N][d] (the nn.Linear [out][in] layout, i.e. the
 *            transpose of the math W whose rows are input channels).
 *   group    quantization group along d: 64, 128 or 256; with r != NULL it
 *            must equal the plan's group.
 *   qweight  device uint8 [N][d/2]: each 4 bytes (a little-endian 32-bit
 *            word) hold the codes c0 .. c7 of 8 consecutive channels, the even
 *            channels in the low 16 bits and the odd ones in the high 16 bits,
 *            4 bits each in channel order: bytes c0 | c2 << 4, c4 | c6 << 4,
 *            c1 | c3 << 4, c5 | c7 << 4 (so that two codes at a time unpack
 *            into an fp16 pair with one AND-OR).
 *   scales   device fp16 [N][d/group].
 *   zeros    device uint8 [N][d/group], values 0..15.
 *
 * The result is bit-exact with this arithmetic, in fp32 with every operation
 * rounded on its own (no fused multiply-add):
 *   u_k = w_k * alpha_k; for each stage and pair: a = u_i, b = u_j,
 *   u_i = c*a - s*b, u_j = s*a + c*b (c, s as in paro_rotation_create);
 *   per group: mn = min(0, min u), mx = max(0, max u), s32 = (mx - mn) / 15,
 *   s16 = fp16(s32) (round to nearest even; 0 becomes 1.0),
 *   z = clamp(rint(-mn / s16), 0, 15), q = clamp(rint(u / s16) + z, 0, 15).
 * Synchronises the stream to read a device error flag and returns
 * PARO_ERR_VALUE if some transformed weight or some scale is not finite
 * (the outputs are then unspecified). Allocates a 4-byte flag per call.
 * Errors: also PARO_ERR_NULL, PARO_ERR_SHAPE, PARO_ERR_ALIGN,
 * PARO_ERR_UNSUPPORTED, PARO_ERR_HIP.
 */
int paro_quantize_weights(const paro_rotation* r, const uint16_t* w, int64_t N, int64_t d,
                          int32_t group, uint8_t* qweight, uint16_t* scales, uint8_t* zeros,
                          hipStream_t stream);

/* Bytes of device workspace with which paro_w4_linear runs its fastest
 * kernels for this plan (NULL: plain W4) and these sizes; 0 means the call
 * uses no workspace. For M > 64 on layers with fewer than 256 output tiles of
 * 256 x 256 whose k-tiles can be shared out among the workgroups (stream-K)
 * this includes 128 MiB of fp32 partial tiles (two of 256 KB per workgroup),
 * and on layers whose 64 x 128 tiles leave CUs idle 32 KB per tile and k
 * split; paro_w4_linear also runs, with the smaller-tile kernel unsplit, on
 * the minimum: 16 KiB + M d 2 bytes (rounded up to 256) with a plan, none
 * without. */
size_t paro_w4_linear_workspace_size(const paro_rotation* r, int64_t M, int64_t N, int64_t d);

/*
 * The W4 linear layer on rotated activations (W4G128 in the paper notes'
 * main experiments; groups of 64 and 256 as well, the sizes the CSDN
 * article's section 5.2 compares):
 *   Y[m][n] = sum_k X'[m][k] * (q[n][k] - z[n][k/G]) * s[n][k/G] + bias[n]
 * with X' = X T^-1 when r != NULL (rotated inside the call) and X' = X when
 * r == NULL (plain W4, or activations the caller rotated already).
 *
 *   x        device fp16 [M][d]; qweight/scales/zeros as produced by
 *            paro_quantize_weights with the same group; bias device fp16 [N]
 *            or NULL;
 *   y        device fp16 [M][N] (must not overlap x).
 *   group    G = 64, 128 or 256; other values return PARO_ERR_UNSUPPORTED.
 *            A plan r must have the same d and group (the pairs stay inside
 *            quantization groups), else PARO_ERR_SHAPE, and belong to the
 *            current device, else PARO_ERR_VALUE.
 *   N % 16 == 0, d % 128 == 0, d % G == 0, M >= 0 (M == 0 is a no-op); N <= 2^30,
 *   d <= 2^22, M < 2^30, else PARO_ERR_UNSUPPORTED.
 *   workspace, workspace_bytes: device memory of
 *            paro_w4_linear_workspace_size(r, M, N, d) bytes, or of at least
 *            the minimum given there (M > 64: then without stream-K),
 *            256-byte aligned (may be NULL when the size in use is 0;
 *            smaller than the minimum: PARO_ERR_WORKSPACE). Its first 16 KiB hold
 *            arrival counters that must be zero before the first call that
 *            uses the workspace (zero-fill it once after allocating it); every
 *            call leaves them zero again. The rest is scratch. Calls that may
 *            run at the same time (different streams) need different
 *            workspaces.
 *
 * Execution: M <= 64 runs one kernel that streams the packed weights (token
 * columns in blocks of 16) and, for plans of group 64 or 128 that execute at
 * most 8 stages, applies the transform to the activations inside the same
 * kernel; other plans rotate into the workspace first. M > 64 rotates into
 * the workspace and then runs
 * a matrix-core kernel: 256 x 256 tiles from 256 such tiles, one per
 * workgroup; with fewer, when every XCD holds n-blocks and k is long enough,
 * the same kernel with each XCD's k-tiles shared out in equal ranges among 16
 * to 32 of its workgroups (stream-K): partial tiles meet through fp32 partial
 * tiles in the workspace (the last piece to arrive adds them in k order),
 * when the workspace holds them; else a kernel with 128 x 256 tiles, or
 * 64 x 256 or 64 x 128 (k split two or four ways inside the workgroup) for
 * layers with few tiles, the latter with k also split across 2 or 4
 * workgroups per tile when the tiles leave CUs idle and the workspace holds
 * their partial tiles.
 *
 * Arithmetic: X' exactly as paro_rotate computes it (fp16); fp32 accumulation
 * of exact fp16 products against the fp16 rounding of each dequantized weight
 * (q - z) * s, in an order that depends on the sizes (and for M > 64 on
 * whether the workspace holds the stream-K partial tiles) but not on timing;
 * fp16 output.
 * Errors: PARO_ERR_NULL, PARO_ERR_SHAPE, PARO_ERR_VALUE, PARO_ERR_ALIGN,
 * PARO_ERR_UNSUPPORTED, PARO_ERR_WORKSPACE, PARO_ERR_HIP.
 */
int paro_w4_linear(const paro_rotation* r, const uint16_t* x, const uint8_t* qweight,
                   const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias,
                   uint16_t* y, int64_t M, int64_t N, int64_t d, int32_t group,
                   void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * paro_w4_linear for callers that cannot allocate device memory (code under
 * HIP-graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * the same kernels, arguments and result as paro_w4_linear, with the
 * workspace taken from a static device array inside the library instead of a
 * caller's buffer. The call allocates and frees nothing.
 *
 *   Scratch: (64 MiB + 16 KiB) per device, held from the library's load until
 *            the process ends; its address is looked up and its arrival
 *            counters cleared by paro_device_init (paro_rotation_create runs
 *            it), and every completed call leaves the counters zero again.
 *   Limit:   the minimum workspace of paro_w4_linear (see
 *            paro_w4_linear_workspace_size) must not exceed that size (for
 *            example M x d <= 32 Mi elements for a rotated layer with
 *            M > 64), else PARO_ERR_WORKSPACE and nothing is enqueued; the
 *            stream-K partial tiles are used when they fit as well.
 *   Sharing: every call on one device uses that device's single array, so
 *            calls that may run at the same time on one device (several
 *            streams or threads) race and give wrong results: serialise them,
 *            or use paro_w4_linear with a workspace per stream.
 * Errors: those of paro_w4_linear, PARO_ERR_WORKSPACE (too large, see
 * above), PARO_ERR_UNSUPPORTED (paro_device_init has not run on the current
 * device).
 */
int paro_w4_linear_noalloc(const paro_rotation* r, const uint16_t* x, const uint8_t* qweight,
                           const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias,
                           uint16_t* y, int64_t M, int64_t N, int64_t d, int32_t group,
                           hipStream_t stream);

/* Activations of the products with an epilogue. */
typedef enum {
  PARO_ACT_NONE = 0,
  PARO_ACT_SILU = 1,      /* z / (1 + e^-z) */
  PARO_ACT_GELU = 2,      /* z (1 + erf(z / sqrt 2)) / 2 */
  PARO_ACT_GELU_TANH = 3, /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2 */
  PARO_ACT_RELU = 4       /* max(z, 0) */
} paro_activation;

/* Element types of tensors that are not fp16 alone. */
typedef enum { PARO_TYPE_F32 = 0, PARO_TYPE_F16 = 1, PARO_TYPE_BF16 = 2 } paro_type;

/* Which transform paro_rotation_backward differentiates. */
typedef enum {
  PARO_SIDE_ACTIVATION = 0, /* X' = X T^-1, as paro_rotate computes it */
  PARO_SIDE_WEIGHT = 1      /* the rows of T W in the [N][d] layout, as the quantizer transforms them */
} paro_side;

/* Bytes of device scratch paro_rotation_backward needs for M rows (0 when
 * M <= 0). */
size_t paro_rotation_backward_workspace_size(const paro_rotation* r, int64_t M);

/*
 * Gradients of the transform with respect to its input, its angles and its
 * channel scales: the step that learns theta and alpha by minimising the
 * layer-wise output loss (paper notes, "损失函数 / 训练策略"). For every row r
 * of x (a token for PARO_SIDE_ACTIVATION; a weight row, [N][d] layout, for
 * PARO_SIDE_WEIGHT) the transform is v_0 = r / alpha (activation) or
 * r * alpha (weight), then the K stages in order with the pair update
 * (v_i, v_j) <- (c v_i - s v_j, s v_i + c v_j) (CSDN article, section 2.2).
 * Given gy = dL/d(output):
 *   gx[m][k]     = dL/dr: gy walked back through the transposed stages, then
 *                  divided (activation) or multiplied (weight) by alpha;
 *   dtheta[t][p] = sum over rows of g'_j v'_i - g'_i v'_j, with (i, j) the
 *                  stored pair p of stage t, v' that stage's outputs and g'
 *                  their gradient (d v'_i / d theta = -v'_j,
 *                  d v'_j / d theta = v'_i); pairs with theta = 0 included;
 *   dalpha[k]    = sum over rows of g_0[k] * d v_0[k] / d alpha[k], i.e.
 *                  -g_0 r / alpha^2 (activation) or g_0 r (weight),
 * with g_0 the gradient of v_0.
 *
 *   side     PARO_SIDE_ACTIVATION or PARO_SIDE_WEIGHT, else PARO_ERR_VALUE.
 *   x        device fp16 [M][d] (4-byte aligned): the transform's input.
 *   gy       device fp32 [M][d] (8-byte aligned): gradient of its output.
 *   gx       device fp32 [M][d] (8-byte aligned) or NULL (not computed); may
 *            be gy itself (in place).
 *   dtheta   device fp32 [K][d/2] (may be NULL when K == 0), overwritten.
 *   dalpha   device fp32 [d], overwritten.
 *   M        rows, 0 <= M < 2^31 (M == 0 writes zero gradients).
 *   workspace, workspace_bytes: device scratch of at least
 *            paro_rotation_backward_workspace_size(r, M) bytes, 256-byte
 *            aligned (NULL when that size is 0); calls that may overlap need
 *            different workspaces.
 *
 * Arithmetic: fp32. The stages' inputs are recovered from their outputs by
 * the transposed update instead of being stored. The sums over rows are taken
 * per chunk of rows and the chunks added in a fixed order: the result does
 * not depend on scheduling.
 * Errors: PARO_ERR_NULL, PARO_ERR_VALUE, PARO_ERR_SHAPE, PARO_ERR_ALIGN,
 * PARO_ERR_WORKSPACE, PARO_ERR_HIP.
 */
int paro_rotation_backward(const paro_rotation* r, int32_t side, const uint16_t* x,
                           const float* gy, float* gx, float* dtheta, float* dalpha, int64_t M,
                           void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of device workspace paro_layer_loss needs (0 for M <= 0, or d not the plan's). */
size_t paro_layer_loss_workspace_size(const paro_rotation* r, int64_t M, int64_t N, int64_t d,
                                      int32_t with_gradients);

/*
 * Layer-wise output loss of the quantized, transformed layer (paper notes,
 * "损失函数 / 训练策略": L = ||Q(D)(X') - D(X)||, minimised per layer to learn
 * the angles and scales), as the squared Frobenius norm
 *   L = sum_{m,n} (Y_q[m][n] - Y[m][n])^2,
 *   Y_q = paro_w4_linear's output (fp16) on X' = paro_rotate(x) with the
 *         4-bit weights (qweight, scales, zeros: Q(T W) from
 *         paro_quantize_weights with this plan), i.e. fp32 sums of X' times
 *         the fp16 rounding of each dequantized weight,
 *   Y   = x w^T with w the original fp16 weights [N][d] (fp32 accumulation).
 * With dtheta and/or dalpha non-NULL also the gradients, passing through the
 * quantizer and the fp16 roundings unchanged (straight-through):
 * dY = 2 (Y_q - Y), dL/dX' = dY W_hat, dL/d(T W) = dY^T X', then both
 * transforms' gradients as paro_rotation_backward computes them (activation
 * side with x, weight side with w), summed. Since X' (T W)^T = X W^T for all
 * angles and scales, that sum equals the activation side's gradient for
 * dL/dX' = dY E, E = W_hat - T W (T W in the quantizer's fp32), which is how
 * it is computed: the two sides' other terms cancel and are each tens of
 * times larger than the result. E comes from the quantizer's own pass over
 * T W, with W_hat from the codes that pass produces; these equal qweight,
 * scales and zeros bit for bit when those are Q(T W) of this plan, as
 * required above. dY and E enter that product rounded to fp16, with fp32
 * sums.
 *
 *   x        device fp16 [M][d], w device fp16 [N][d] (16-byte aligned);
 *   qweight, scales, zeros: as for paro_w4_linear, with the plan's group;
 *   loss     device fp32 [1] (per-tile sums in a fixed order, fp64 at the end);
 *   dtheta   device fp32 [K][d/2] or NULL; dalpha device fp32 [d] or NULL;
 *   N % 16 == 0, 0 <= M, N < 2^30; M == 0 writes zeros.
 *   workspace: at least paro_layer_loss_workspace_size(r, M, N, d, dtheta ||
 *            dalpha) bytes, 256-byte aligned, zero-filled once after
 *            allocation (its first 16 KiB hold paro_w4_linear's arrival
 *            counters for M <= 64, which every call leaves zero, whatever M
 *            and N the workspace is reused with). Calls that may run at the
 *            same time need different workspaces.
 * Every step runs in this library's kernels (the dense products on the
 * matrix cores); the call allocates nothing and does not synchronise.
 * Errors: PARO_ERR_NULL, PARO_ERR_SHAPE, PARO_ERR_ALIGN, PARO_ERR_WORKSPACE,
 * PARO_ERR_HIP, and those of paro_w4_linear.
 */
int paro_layer_loss(const paro_rotation* r, const uint16_t* x, const uint16_t* w,
                    const uint8_t* qweight, const uint16_t* scales, const uint8_t* zeros, int64_t M,
                    int64_t N, int64_t d, int32_t group, float* loss, float* dtheta, float* dalpha,
                    void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * The W4 linear with its bias, an activation and a residual in the epilogue:
 *   Y[m][n] = act(Z[m][n]) + R[m][n],
 *   Z[m][n] = sum_k X'[m][k] W_hat[n][k] + bias[n],
 * X', W_hat, sizes, alignment and workspace (paro_w4_linear_workspace_size;
 * without a plan and with M <= 64 its first 16 KiB are enough) as for
 * paro_w4_linear; Z, the activation and the sum in fp32, one rounding
 * to fp16. Up to a few hundred tokens the product runs in kernels of its own
 * (where the transform is not fused into it), whose fp32 sums run in another
 * order: Z may differ from paro_w4_linear's in the last places.
 *   residual  device fp16 [M][N], 16-byte aligned, or NULL; may be y itself
 *             (each value is read before it is replaced), no other overlap.
 *   act       a paro_activation.
 * Errors: those of paro_w4_linear, PARO_ERR_VALUE (unknown activation).
 */
int paro_w4_linear_act(const paro_rotation* r, const uint16_t* x, const uint8_t* qweight,
                       const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias,
                       const uint16_t* residual, int32_t act, uint16_t* y, int64_t M, int64_t N,
                       int64_t d, int32_t group, void* workspace, size_t workspace_bytes,
                       hipStream_t stream);

/*
 * The gated feed-forward product, both projections and their product in one
 * kernel:
 *   Y[m][n] = act(Zg[m][n]) Zu[m][n],
 *   Zg[m][n] = sum_k X'[m][k] W_hat[n][k] + bias[n],
 *   Zu[m][n] = sum_k X'[m][k] W_hat[N + n][k] + bias[N + n].
 * The weight block has 2 N rows, the gate projection's first, then the up
 * projection's: what paro_quantize_weights makes of the two [N][d] weights
 * laid one after the other. Both projections read the same X', so a plan r is
 * shared by them.
 *   qweight [2N][d/2], scales and zeros [2N][d/group], bias [2N] or NULL,
 *   y fp16 [M][N]; N % 16 == 0 and N d < 2^31, else as paro_w4_linear with
 *   2 N rows, the workspace (paro_w4_gated_workspace_size; without a plan and
 *   with M <= 64 its first 16 KiB are enough) included.
 * Errors: those of paro_w4_linear, PARO_ERR_VALUE (unknown activation).
 */
size_t paro_w4_gated_workspace_size(const paro_rotation* r, int64_t M, int64_t N, int64_t d);
int paro_w4_gated(const paro_rotation* r, const uint16_t* x, const uint8_t* qweight,
                  const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias, int32_t act,
                  uint16_t* y, int64_t M, int64_t N, int64_t d, int32_t group, void* workspace,
                  size_t workspace_bytes, hipStream_t stream);

/*
 * Gradients of the two products above with respect to their pre-activations
 * and to X', for learning through them (the transform's own gradients follow
 * from dX' by paro_rotation_backward; the 4-bit weights are constants).
 * paro_w4_linear_act_backward, for dY = dL/dY:
 *   dZ = dY act'(Z),  dX' = dZ W_hat  (and dL/dR is dY itself).
 * paro_w4_gated_backward:
 *   dZg = dY Zu act'(Zg),  dZu = dY act(Zg),  dX' = [dZg dZu] W_hat.
 * Z is computed again from X' rather than kept by the forward call: a kept Z
 * would cost 2 M (2) N bytes and its fp16 rounding. dZ is the bias gradient
 * before its sum over the tokens, and dZ^T X' would be the weights'.
 *   x     device fp16 [M][d]: X', the transformed activations (not needed,
 *         may be NULL, for a linear without activation);
 *   dy    device fp16 [M][N];
 *   dz    device fp16 [M][N], gated [M][2N] (gate, then up), overwritten; for a
 *         linear without activation, where dZ is dY, it may be NULL or dy (else
 *         dY is copied there);
 *   dx    device fp16 [M][d], overwritten, or NULL (dz alone);
 *   all 16-byte aligned and not overlapping; act, bias, sizes as for the
 *   forward calls, at most 2^21 weight rows; M == 0 is a no-op.
 *   workspace: at least the ..._workspace_size bytes (beyond 128 tokens W_hat
 *         transposed in fp16, 2 d (2) N bytes, is the largest part; not
 *         always less for fewer tokens; 0 for sizes that the call refuses or
 *         has nothing to do for), 256-byte aligned,
 *         zero-filled once after allocation (its first 16 KiB hold arrival
 *         counters, which every call leaves zero).
 * Arithmetic: fp32 sums and epilogues. dZ is rounded to fp16, which is what
 * dX' is then summed from, so gradients far below fp16's normal range
 * (6e-5) lose accuracy: scale the loss, as is usual with fp16 gradients.
 * relu'(0) is 0. Results do not depend on timing.
 * Errors: those of paro_w4_linear, PARO_ERR_VALUE (unknown activation).
 */
size_t paro_w4_linear_act_backward_workspace_size(int64_t M, int64_t N, int64_t d, int32_t act);
int paro_w4_linear_act_backward(const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
                                const uint8_t* zeros, const uint16_t* bias, int32_t act,
                                const uint16_t* dy, uint16_t* dz, uint16_t* dx, int64_t M, int64_t N,
                                int64_t d, int32_t group, void* workspace, size_t workspace_bytes,
                                hipStream_t stream);
size_t paro_w4_gated_backward_workspace_size(int64_t M, int64_t N, int64_t d);
int paro_w4_gated_backward(const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
                           const uint8_t* zeros, const uint16_t* bias, int32_t act, const uint16_t* dy,
                           uint16_t* dz, uint16_t* dx, int64_t M, int64_t N, int64_t d, int32_t group,
                           void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Mixture of experts: every token goes through k of E experts. A routing says
 * which: M tokens, R = M k pairs p = m k + s of a token m and its slot s. The
 * rows of the experts' products are the pairs in expert order: first those of
 * expert 0 in the order of their numbers, then those of expert 1, and so on; the
 * pairs without an expert come last and have no row.
 *   ids      device int32 [M][k]: the expert of each pair; one outside 0 .. E - 1
 *            (-1) means none.
 *   offsets  device int32 [E + 1]: expert e has rows offsets[e] .. offsets[e + 1] - 1.
 *   order    device int32 [R]: the pair of each row; -1 from offsets[E] on.
 *   place    device int32 [R]: the row of each pair; -1 without an expert.
 *   weights  device fp32 [R]: the pairs' weights (read by the combining calls).
 * The tables are those of paro_experts_route or paro_experts_sort: tables that
 * contradict each other give wrong results, but no access outside the tensors.
 */
typedef struct paro_routing {
  int64_t M;
  int32_t E, k;
  const int32_t *ids, *offsets, *order, *place;
  const float* weights;
} paro_routing;

/*
 * The router: for every token the k largest of its E logits l, the lower expert
 * first where two are equal, with p = softmax(l) and
 *   w_s = p_s / (sum of p over the k)  (normalize != 0),  else  w_s = p_s;
 * and the tables of the routing. An expert with logit -inf or NaN is never
 * taken: a token with fewer than k others has pairs without an expert (id -1,
 * weight 0), and a token whose mask leaves none has no expert at all. A NaN
 * among a token's logits makes its weights NaN. fp32 arithmetic; the logits'
 * order is exact.
 *   logits   device [M][E] of a paro_type, aligned to it.
 *   ids, weights, offsets, order, place: outputs, as above (M == 0: offsets = 0).
 *   1 <= k <= E <= 1024, k <= 16, R < 2^24.
 *   workspace: paro_experts_route_workspace_size(M, E, k) bytes (0 up to 128
 *            tokens), 256-byte aligned; scratch, not shared by calls that may
 *            run at the same time. The size never shrinks with M: one for the
 *            largest batch serves every smaller one.
 * paro_experts_sort makes the tables of given ids (a router of the caller's, or
 * the experts e0 .. e0 + E - 1 that one device holds, from ids - e0).
 * Errors: PARO_ERR_NULL, PARO_ERR_SHAPE, PARO_ERR_VALUE (unknown type),
 * PARO_ERR_ALIGN, PARO_ERR_UNSUPPORTED (limits), PARO_ERR_WORKSPACE, PARO_ERR_HIP.
 */
size_t paro_experts_route_workspace_size(int64_t M, int32_t E, int32_t k);
int paro_experts_route(const void* logits, int32_t type, int64_t M, int32_t E, int32_t k, int32_t normalize,
                       int32_t* ids, float* weights, int32_t* offsets, int32_t* order, int32_t* place,
                       void* workspace, size_t workspace_bytes, hipStream_t stream);
int paro_experts_sort(const int32_t* ids, int64_t M, int32_t E, int32_t k, int32_t* offsets, int32_t* order,
                      int32_t* place, void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Gradient of the router at its logits, for dw = dL/dw (the choice of the experts
 * is constant): with normalize dl_i = w_i (dw_i - sum_s w_s dw_s) for the token's
 * experts and 0 for the others (logits may be NULL), else
 * dl_j = p_j (dw_j [j is one of them] - sum_s p_s dw_s). Pairs without an expert
 * take no part, and a token without experts has a gradient of 0. Where a logit of
 * a token with experts is NaN or +inf, the p are NaN, and so is the gradient at
 * every expert (normalize: at the token's).
 *   ids, weights, normalize: the forward call's; dweights device fp32 [M][k];
 *   dlogits device [M][E], of the logits' type, overwritten (may be logits).
 * Errors: as paro_experts_route, without a workspace.
 */
int paro_experts_route_backward(const void* logits, int32_t type, int64_t M, int32_t E, int32_t k, int32_t normalize,
                                const int32_t* ids, const float* weights, const float* dweights, void* dlogits,
                                hipStream_t stream);

/*
 * The experts' products on 4-bit weights, each row by its expert's:
 *
 * paro_w4_experts_gated, for row r of expert e and its token m:
 *   H[r][n] = act(Zg) Zu,  Zg = sum_k X'[m][k] W_hat[e][n][k] + bias[e][n],
 *   Zu the same with row N + n: the weights of an expert are a block of 2 N rows
 *   as for paro_w4_gated.
 * paro_w4_experts_combine, over the slots s of a token with row r_s, expert e_s:
 *   Y[m][n] = residual[m][n]
 *             + sum_s w[m][s] (sum_k H[r_s][k] W_hat[e_s][n][k] + bias[e_s][n]).
 *
 *   x        device fp16 [M][d]: X', transformed activations (paro_rotate; the
 *            experts of a layer share the transform);
 *   h        device fp16 [R][N] (gated's output; rows from offsets[E] on are left
 *            as they were) and [R][d] (combine's input, transformed if its
 *            weights are: like X's, one transform for all experts of a layer).
 *   qweight  device uint8 [E][P][d/2], scales [E][P][d/group], zeros likewise,
 *            bias fp16 [E][P] or NULL, with P = 2 N (gated) or N (combine): what
 *            paro_quantize_weights makes of the E [P][d] weights, one after the
 *            other;
 *            Rows from offsets[E] on and a transform of h: how many there are is
 *            known on the device alone, and paro_rotation_backward over h and dh
 *            sums all R rows. A caller that makes it zero-fills h and dh before
 *            the calls that write them (which leave those rows as they were).
 *            paro_rotate may be run over all rows, whatever those hold.
 *   residual device fp16 [M][N] or NULL; may be y itself, no other overlap;
 *   y        device fp16 [M][N]; tokens without an expert get the residual, or 0.
 *   N % 16 == 0, d % 128 == 0, d % group == 0, P and d <= 2^21, P d < 2^31; the
 *   tokens times their channels (gated d, combine N) < 2^30, R max(P, d) < 2^34,
 *   E max(P, d) < 2^27;
 *   tensors 16-byte aligned. M == 0 is a no-op.
 *   workspace: at least the ..._workspace_size bytes (combine: its rows in fp32,
 *   4 R N bytes, so that a token's sum is rounded once), 256-byte aligned;
 *   scratch, not shared by calls that may run at the same time. The sizes, those of
 *   the gradients below too, never shrink with M: for the same E, k, N and d a
 *   workspace for the largest batch serves every smaller one.
 * Arithmetic: fp32 sums of exact fp16 products, one rounding to fp16; results do
 * not depend on timing, nor a row's on the other rows' values.
 * The calls read the numbers of rows on the device: they do not synchronise, and
 * a captured call follows the routing that its replay finds.
 * Errors: PARO_ERR_NULL, PARO_ERR_SHAPE, PARO_ERR_VALUE (unknown activation),
 * PARO_ERR_ALIGN, PARO_ERR_UNSUPPORTED, PARO_ERR_WORKSPACE, PARO_ERR_HIP.
 */
size_t paro_w4_experts_gated_workspace_size(int64_t M, int32_t E, int32_t k, int64_t N, int64_t d);
int paro_w4_experts_gated(const paro_routing* routing, const uint16_t* x, const uint8_t* qweight,
                          const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias, int32_t act,
                          uint16_t* h, int64_t N, int64_t d, int32_t group, void* workspace, size_t workspace_bytes,
                          hipStream_t stream);
size_t paro_w4_experts_combine_workspace_size(int64_t M, int32_t E, int32_t k, int64_t N, int64_t d);
int paro_w4_experts_combine(const paro_routing* routing, const uint16_t* h, const uint8_t* qweight,
                            const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias,
                            const uint16_t* residual, uint16_t* y, int64_t N, int64_t d, int32_t group,
                            void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Their gradients (the 4-bit weights are constants):
 * paro_w4_experts_gated_backward, for dH = dL/dH (fp16 [R][N], by row):
 *   dZg = dH Zu act'(Zg), dZu = dH act(Zg) (dz fp16 [R][2N], rows from offsets[E]
 *   on left as they were), Z computed again, and
 *   dX'[m] = sum over the token's rows r of dZ[r] W_hat[e] (dx fp16 [M][d], 0 for a
 *   token without an expert; NULL: not computed).
 * paro_w4_experts_combine_backward, for dY = dL/dY (fp16 [M][N]), with
 * U[r] = dY[m] W_hat[e] (fp32):
 *   dH[r] = w U[r] (dh fp16 [R][d], rows from offsets[E] on left as they were),
 *   dw[m][s] = U[r] . H[r] + dY[m] . bias[e] (dweights fp32 [M][k], 0 without an
 *   expert); the residual's gradient is dY itself.
 * Arguments, limits and errors as for the forward calls. dX' is summed from dZ
 * rounded to fp16, as it is returned; a bias gradient is the sum of an expert's
 * rows of dZ, or of w dY. A row of dZ or dY that is not finite makes gradients of
 * its own token that are not finite: NaN also where the sum is an infinity.
 */
size_t paro_w4_experts_gated_backward_workspace_size(int64_t M, int32_t E, int32_t k, int64_t N, int64_t d);
int paro_w4_experts_gated_backward(const paro_routing* routing, const uint16_t* x, const uint8_t* qweight,
                                   const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias, int32_t act,
                                   const uint16_t* dh, uint16_t* dz, uint16_t* dx, int64_t N, int64_t d,
                                   int32_t group, void* workspace, size_t workspace_bytes, hipStream_t stream);
size_t paro_w4_experts_combine_backward_workspace_size(int64_t M, int32_t E, int32_t k, int64_t N, int64_t d);
int paro_w4_experts_combine_backward(const paro_routing* routing, const uint16_t* h, const uint8_t* qweight,
                                     const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias,
                                     const uint16_t* dy, uint16_t* dh, float* dweights, int64_t N, int64_t d,
                                     int32_t group, void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Distillation loss from a teacher's top logits, the objective of learning through
 * a whole model (the layer-wise one is paro_layer_loss). Per row, with
 * q = softmax(z / T) over the V logits of the student and the teacher's entries i
 * (logit t_i at index j_i):
 *   lse NULL: p_i = exp(t_i / T) / sum over the entries,  P = 0;
 *   else:     p_i = exp(t_i / T - lse), lse the log of the sum of exp(t / T) over
 *             all the teacher's logits, and P = max(0, 1 - sum p): the rest of its
 *             mass, compared with the student's outside the entries, Q, as one
 *             more class;
 *   L = w T^2 [sum_i p_i (log p_i - log q_ji) + P (log P - log Q)],
 *   dL/dz_j = w T (A q_j - sum of p_i with j_i = j), outside the entries with a
 *   rest w T q_j (A - P / Q); A = sum p + P.
 *   z        device [M][V] of a paro_type, 16-byte aligned; student logits of
 *            -inf are classes that it cannot take, finite ones may be of any size
 *            (a mask of the type's lowest number), and a NaN or +inf makes its row's
 *            loss NaN.
 *   values   device [M][K] of a paro_type (t), index device int32 [M][K] (j): an
 *            index outside 0 .. V - 1 (-1) means no entry, a value of -inf an
 *            entry of mass 0; an index that comes twice adds its masses.
 *   lse, row_weight  device fp32 [M] or NULL (w = 1). A row with w = 0 is left
 *            out whatever it holds, and so is (lse NULL) one without an entry
 *            above -inf: loss 0, gradient 0. With a rest and no student mass
 *            outside the entries, those logits have no gradient.
 *   loss     device fp32 [M].
 *   dz       device [M][V] of z's type, 16-byte aligned: grad_scale dL/dz (the
 *            scale keeps fp16 gradients normal), or NULL; may be z itself.
 *   M < 2^22, 1 <= V <= 2^20, 1 <= K <= 1024; T > 0 with log2(e) / T finite in fp32.
 * Arithmetic: exponentials and their sums over the row in fp32, the entries in
 * fp64; results do not depend on timing. One launch, no workspace.
 * Errors: PARO_ERR_NULL, PARO_ERR_SHAPE, PARO_ERR_VALUE, PARO_ERR_ALIGN,
 * PARO_ERR_UNSUPPORTED, PARO_ERR_HIP.
 */
int paro_distill_loss(const void* z, int32_t z_type, const void* values, int32_t value_type, const int32_t* index,
                      const float* lse, const float* row_weight, int64_t M, int64_t V, int64_t K, double temperature,
                      double grad_scale, float* loss, void* dz, hipStream_t stream);

/* Plan of an AdamW step over a fixed list of tensors. Immutable after creation. */
typedef struct paro_adamw paro_adamw;

/* Values of each moment for `count` tensors of n[i] values: every tensor's
 * moments start at a multiple of 256, so this is the sum of n[i] rounded up to
 * 256. -1 for a bad list (a negative or too large size). */
int64_t paro_adamw_moments(int32_t count, const int64_t* n);

/*
 * AdamW over many tensors at once, the optimizer of the angles and scales
 * (paper notes, "损失函数 / 训练策略"), for step t:
 *   m <- beta1 m + (1 - beta1) g,  v <- beta2 v + (1 - beta2) g^2,
 *   p <- p (1 - lr weight_decay)
 *        - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * in fp32; p is rounded once to its type (with fp16 or bf16 parameters an
 * update below half a step of the value is lost).
 *
 * paro_adamw_create (synchronous) makes the plan of a list of tensors; the
 * caller owns the tensors and keeps them where they are. Lists of more than
 * 120 tensors are put into a table in the current device's memory (so not
 * inside a stream capture), which paro_adamw_destroy frees; no enqueued step
 * may still use it then.
 *   count, n            tensors and their values, n[i] >= 0 (0: skipped);
 *   params, grads       host arrays of device pointers, contiguous, aligned to
 *                       their element type (16 bytes: the fast accesses);
 *   param_type, grad_type  a paro_type for all of them;
 *   state_bits          32: m and v device fp32 [paro_adamw_moments]; scales
 *                       unused.
 *                       8: m and v device bytes [paro_adamw_moments], e4m3
 *                       numbers, and m_scale and v_scale device fp32 [moments
 *                       / 256]: block b of 256 consecutive values of a tensor
 *                       stands for m = e4m3 * m_scale[b] and sqrt(v) = e4m3 *
 *                       v_scale[b], scale = largest magnitude / 448 (rounded
 *                       to nearest even; sqrt(v) is not rounded to zero where
 *                       v > 0; a block below 2^-100 is held as zero). A
 *                       gradient that is not finite leaves its block's scale
 *                       infinite or NaN, and the block's moments NaN.
 *                       Zero-fill all of them before the first step, the
 *                       padding between the tensors included.
 * Errors: PARO_ERR_NULL, PARO_ERR_VALUE (unknown type; parameters, moments or
 * scales that overlap each other or a gradient), PARO_ERR_UNSUPPORTED
 * (state_bits, out of host memory), PARO_ERR_SHAPE, PARO_ERR_ALIGN,
 * PARO_ERR_HIP (the table).
 *
 * paro_adamw_step runs step t >= 1 on the current device, in one launch (one
 * for every 2^33 values), without upload, allocation or synchronisation. A
 * captured call replays the t and the rates it was captured with. Steps of one
 * plan must not run at the same time.
 * Errors: PARO_ERR_NULL, PARO_ERR_VALUE (step < 1; lr or weight_decay
 * negative, beta outside [0, 1), eps <= 0, or one of them, or the rates made
 * from them, not finite in fp32), PARO_ERR_HIP.
 */
int paro_adamw_create(int32_t count, const int64_t* n, void* const* params, int32_t param_type,
                      const void* const* grads, int32_t grad_type, int32_t state_bits, void* m,
                      void* v, float* m_scale, float* v_scale, paro_adamw** out);
void paro_adamw_destroy(paro_adamw* h);
int paro_adamw_step(const paro_adamw* h, int64_t step, double lr, double beta1, double beta2,
                    double eps, double weight_decay, hipStream_t stream);

/*
 * Channel-pair selection (host only, synchronous, no GPU): fills pairs
 * [K][d/2][2] with global channel ids in the layout paro_rotation_create
 * takes; every stage is a perfect pairing inside every group of `group`
 * channels (pair p of a stage belongs to group p / (group / 2)).
 *
 * paro_pairs_random: random pairs with de-duplication, the selection the
 * paper notes name ("局限与展望": random plus de-duplication). Reading: for
 * each group in order and each stage in order, draw a uniformly random
 * permutation of the group's channels (Fisher-Yates from the last position
 * down, j = r mod (i + 1) with r the next SplitMix64 output of one stream
 * seeded with `seed`, state += 0x9E3779B97F4A7C15 per output); then for
 * positions i = 0, 2, 4, ... pair the channel at i with the first channel
 * after it not yet paired with it in an earlier stage of the group, which is
 * exchanged with the channel at position i + 1; if none is left, draw the
 * stage again (at most 4096 draws).
 * The pair is stored as (channel at i, its partner). No unordered pair
 * occurs twice in one group. K <= group - 1; near that bound the earlier
 * stages can leave no pairing without repeats (for example 7 stages of a
 * group of 8 need a one-factorization the greedy stages may not extend), and
 * the call returns PARO_ERR_VALUE.
 * Errors: PARO_ERR_NULL, PARO_ERR_SHAPE (group odd or not dividing d, d >
 * 2^24, K out of range), PARO_ERR_VALUE (4096 draws without a pairing).
 */
int paro_pairs_random(int64_t d, int32_t group, int32_t K, uint64_t seed, int32_t* pairs);

/*
 * paro_pairs_by_gap: pairs of channels whose values differ strongly (CSDN
 * article, section 2.2: pairs with a large numeric difference are preferred).
 * score: host float [d], one value per input channel (for example the
 * largest |W| over the output rows). Reading: in each group, rank the
 * channels by score, largest first (ties: lower channel first); stage t
 * pairs the i-th largest with the ((i + t) mod (group / 2))-th smallest, for
 * i = 0 .. group / 2 - 1, stored as (larger, smaller). Stage 0 pairs the
 * largest with the smallest; every pair joins the top and the bottom half of
 * the ranking, which is the largest total score difference a perfect
 * pairing can have, and no pair repeats across stages. K <= group / 2.
 * Errors: PARO_ERR_NULL, PARO_ERR_SHAPE, PARO_ERR_VALUE (non-finite score).
 */
int paro_pairs_by_gap(int64_t d, int32_t group, int32_t K, const float* score, int32_t* pairs);

/*
 * paro_sparsify_angles: keep only the strongest rotations of a plan (paper
 * notes, "核心观察": a sparse rotation keeping the top 10% of the channel
 * pairs matches the full one). theta, theta_out: host float [K][d/2] (may
 * be the same array). Reading: the n_keep pairs with the largest |theta| over
 * the whole plan keep their angle (ties: the earlier stage and pair first),
 * every other pair gets theta = 0, an exact identity. For angles in
 * [-pi, pi], |theta| orders the rotations by their distance from the
 * identity. Errors: PARO_ERR_NULL, PARO_ERR_SHAPE (0 <= n_keep <= K d / 2,
 * d even), PARO_ERR_VALUE (non-finite angle).
 */
int paro_sparsify_angles(int64_t d, int32_t K, const float* theta, int64_t n_keep, float* theta_out);

/*
 * Measurement: a plain device copy dst[0 .. bytes) = src[0 .. bytes) at the
 * rate HBM sustains for one read and one write stream (16-byte buffer loads
 * and stores, 4 per lane in flight, `blocks` workgroups of 256 lanes striding
 * over the buffer). It is the measured ceiling that the memory-bound kernels
 * (paro_rotate, the small-batch paro_w4_linear) are reported against, next to
 * the datasheet peak; it takes no part in the method.
 *   src, dst  device memory, 16-byte aligned, not overlapping;
 *   bytes     a multiple of 16 (0 is a no-op);
 *   blocks    1 .. 2^20.
 * Asynchronous on stream. Errors: PARO_ERR_NULL, PARO_ERR_ALIGN,
 * PARO_ERR_SHAPE, PARO_ERR_HIP.
 */
int paro_stream_copy(const void* src, void* dst, size_t bytes, int32_t blocks, hipStream_t stream);

/*
 * Measurement: fp16 matrix-core throughput with operands in registers. Each
 * of `blocks` workgroups runs one wavefront per SIMD (256 lanes); every
 * wavefront runs `iters` rounds of 16 independent v_mfma_f32_32x32x16_f16
 * (32768 flop each) on operands read once from src, then each lane writes the
 * sum of its 256 fp32 accumulators to out[lane]. With random operands the
 * rate is the ceiling the matrix cores sustain under the chip's power limit,
 * which the prefill linear is reported against next to the datasheet peak; it
 * takes no part in the method. With every operand 1.0, each output is
 * 4096 * iters.
 *   src   device fp16 [n], 16-byte aligned, n a multiple of 8 in [8, 2^30];
 *   out   device float [blocks * 256];
 *   blocks 1 .. 2^16, iters >= 0.
 * Asynchronous on stream. Errors: PARO_ERR_NULL, PARO_ERR_ALIGN,
 * PARO_ERR_SHAPE, PARO_ERR_HIP.
 */
int paro_mfma_loop(const void* src, int64_t n, float* out, int32_t blocks, int32_t iters, hipStream_t stream);

/*
 * Host-only view of the per-segment rotation schedule that
 * paro_rotation_create uploads (for testing the plan logic without a GPU).
 * Fills `out` (host memory of out_bytes) with the exact table image and writes
 * the image size to *needed (out may be NULL to query the size), and the
 * layout descriptor to *layout (may be NULL):
 *   layout[0] = channels per segment (128 or 256),
 *   layout[1] = pairs per lane (1 or 2),
 *   layout[2] = 32-bit words per virtual lane per segment (the schedule's
 *               fields padded to a multiple of 4; the image of a segment is
 *               [layout[2] / 4][virtual lane][4], four consecutive fields of
 *               a lane side by side; after the segments' images comes the
 *               store permutation, [segment][virtual lane][2] words: the LDS
 *               byte offsets at which a lane writes its packed output pair
 *               and from which it reads the natural pair of its own index,
 *               which the activation transform uses for 256-channel
 *               segments),
 *   layout[3] = 1 if the factored two-FMA stage form is used, 0 for the
 *               general 2x2 form,
 *   layout[4] = stages the activation schedule executes: K for a plan
 *               without identities; with pairs of theta == 0 (exact
 *               identities, a partial or sparse pairing) the identities are
 *               dropped and each other rotation goes to the first stage after
 *               the last rotation on either of its channels, which gives the
 *               length of the longest chain of rotations linked by shared
 *               channels (<= K).
 * Runs the same validation as paro_rotation_create and returns its errors;
 * PARO_ERR_WORKSPACE when out is non-NULL and out_bytes is too small.
 */
int paro_rotation_plan_host(int64_t d, int32_t group, int32_t K, const int32_t* pairs,
                            const float* theta, const float* alpha, void* out, size_t out_bytes,
                            size_t* needed, int32_t layout[5]);

#ifdef __cplusplus
}
#endif

#endif /* PARO_H */
