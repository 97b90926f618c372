/*
 * iabn.h -- C ABI of the MI355X (gfx950) In-Place Activated BatchNorm library.
 *
 * The method: "In-Place Activated BatchNorm for Memory-Optimized Training of DNNs"
 * (Rota Bulo, Porzi, Kontschieder), as summarised on the paperlayer page of arXiv
 * 1712.02616v3.  Section 3 ("In-Place Activated Batch Normalization") fuses batch
 * normalisation with an invertible activation into one layer that keeps a single
 * buffer: the forward writes y over x, and the backward rebuilds everything it
 * needs from y by inverting the activation and the scale-and-shift.
 *
 * Conventions shared by every entry point
 *   - Tensors hold N*C*H*W elements of the storage dtype, contiguous, in layout
 *     NCHW (element (n,c,h,w) at ((n*C + c)*H + h)*W + w) or NHWC (at
 *     ((n*H + h)*W + w)*C + c).  Device pointers.  Element pointers must be
 *     aligned to their element size; 16-byte alignment (and H*W, resp. C, a
 *     multiple of 16/element-size) enables the 128-bit vector path, anything
 *     else takes the scalar path with identical results.
 *   - Per-channel vectors (gamma, beta, statistics, gradients) are fp32 device
 *     arrays of length C, for both storage dtypes.  Arithmetic is fp32, with the
 *     per-channel finishing steps in fp64.
 *   - m = N*H*W is the reduction length of one channel.
 *   - The caller owns every buffer, including the workspace.  The library never
 *     allocates or frees, and the compute entry points never synchronise: they
 *     are reentrant and keep no state besides one process-wide setting
 *     (iabn_set_grouped_kernels).  Only iabn_workspace_status synchronises.
 *     Calls are enqueued on `stream` and return once launched.  The status reports
 *     argument validation (done before any HIP call) and launch errors; faults
 *     inside kernels surface at the caller's next synchronisation.
 *   - Results are bitwise deterministic for a given shape, layout, dtype,
 *     pointer alignment and device CU count: no floating-point atomics, fixed
 *     reduction orders.
 *   - Calls that may run at the same time (on different streams) need separate
 *     workspaces; calls in stream order may share one.
 *   - NHWC maps, and NCHW maps whose channels are large or few, may run a
 *     kernel whose workgroups share a slice of channels or one channel and
 *     exchange partial sums through the workspace while all of them are
 *     resident (the grid never exceeds the CU count).  Should the device be held
 *     by other work so long that a partner does not arrive within about a
 *     second, the waiting workgroup gives up and its statistics, and every
 *     output computed from them, become NaN instead of the kernel hanging; it
 *     also records the timeout in the workspace, which iabn_workspace_status
 *     reports.  Callers that share the device with long-running work on other
 *     streams can switch these kernels off (iabn_set_grouped_kernels, or the
 *     environment variable IABN_GROUPED_KERNELS=0): every call then takes
 *     kernels whose workgroups never wait on one another.
 *   - Calls may be captured in a HIP graph (stream capture): they launch
 *     kernels only, with no allocation, memset, copy or synchronisation, and a
 *     replay gives the same bits as the eager call.
 *   - Preconditions that are not checked: gamma_c != 0 in the backward (the
 *     affine step must be invertible), finite inputs (NaN propagates), and no
 *     overlap between buffers other than the aliasing each call allows.
 */
#ifndef IABN_H
#define IABN_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum iabn_status {
    IABN_OK = 0,
    IABN_ERR_INVALID_ARG = 1,   /* a size, enum, scalar or pointer is not acceptable  */
    IABN_ERR_UNSUPPORTED = 2,   /* valid request this build does not implement        */
    IABN_ERR_WORKSPACE = 3,     /* workspace missing or smaller than iabn_workspace_size */
    IABN_ERR_MISALIGNED = 4,    /* a pointer is not aligned to its element size       */
    IABN_ERR_HIP = 5            /* the HIP runtime reported an error at launch        */
} iabn_status;

typedef enum iabn_layout { IABN_NCHW = 0, IABN_NHWC = 1 } iabn_layout;

/* Storage dtype of x / y / dy / dx.  Arithmetic is fp32 (statistics finished in
 * fp64) for every storage dtype; stored results round to nearest even.  fp16
 * keeps IEEE binary16 subnormals and overflows to infinity. */
typedef enum iabn_dtype { IABN_F32 = 0, IABN_BF16 = 1, IABN_F16 = 2 } iabn_dtype;

/* Invertible activations (section 3, "INPLACE-ABN"; section 4, "Experimental
 * setup" uses leaky ReLU with slope 0.01).  act_param is the leaky slope
 * (must be > 0) or the ELU alpha (must be > 0); identity ignores it.
 *   leaky ReLU: y = z > 0 ? z : a*z        ELU: y = z > 0 ? z : alpha*(exp(z)-1) */
typedef enum iabn_act {
    IABN_ACT_IDENTITY = 0,
    IABN_ACT_LEAKY_RELU = 1,
    IABN_ACT_ELU = 2
} iabn_act;

/* Human-readable name of a status code (static storage). */
const char *iabn_status_string(iabn_status status);

/* Library ABI version: major*10000 + minor*100 + patch. */
int iabn_version(void);

/* Process-wide switch of the kernels whose workgroups wait on one another
 * (the exchanging kernels described above).  enabled = 1 allows them (the
 * default unless the environment variable IABN_GROUPED_KERNELS is "0" when the
 * library first plans a call), 0 forbids them: NHWC maps then take one
 * workgroup per slice of channels or the split kernels, NCHW maps one
 * workgroup per channel or the split kernels, with results equal within the
 * parity tolerances (the reduction order differs).  enabled < 0 changes
 * nothing.  Returns the setting in force before the call.  Calls planned
 * after it follow the new setting; iabn_workspace_size does not depend on it.
 * This is the only state the library keeps across calls besides per-device
 * caches of the CU count. */
int iabn_set_grouped_kernels(int enabled);

/* Reads the exchange status word that every workspace carries in its first
 * 256 bytes: *timed_out = 1 if an exchanging kernel that used this workspace
 * gave up waiting for a partner (its outputs then hold NaN) since the word was
 * last cleared, else 0.  clear != 0 resets the word after reading it.  Unlike
 * every other entry point this one synchronises `stream` (it copies the word
 * to the host); call it after the work to check, not inside graph capture.
 * A workspace whose contents were never written by the library reads as 0
 * (the recorded value is one fixed 64-bit pattern).
 * Errors: IABN_ERR_INVALID_ARG (timed_out NULL), IABN_ERR_WORKSPACE (NULL or
 * under 256 bytes), IABN_ERR_MISALIGNED, IABN_ERR_HIP (copy failed). */
iabn_status iabn_workspace_status(void *workspace, size_t workspace_bytes, int clear,
                                  int *timed_out, hipStream_t stream);

/* Bytes of device workspace that iabn_forward_train, iabn_forward_stats,
 * iabn_backward, iabn_backward_reduce and iabn_backward_eval need for this
 * shape (0 for an empty problem).  Depends on the arguments and on the current
 * device's CU count (which bounds the exchanging kernels' grid).
 * One buffer serves forward and backward of the same shape.  Returns 0 for
 * invalid arguments too. */
size_t iabn_workspace_size(int64_t N, int64_t C, int64_t H, int64_t W,
                           iabn_layout layout, iabn_dtype dtype);

/* Training forward, in place (section 3, "Batch Normalization Review" and
 * "INPLACE-ABN"; the single stored buffer of section 1):
 *   mu_c, var_c = empirical mean and biased variance of channel c over its m
 *   elements; invstd_c = 1/sqrt(var_c + eps);
 *   y = act(gamma_c * (x - mu_c) * invstd_c + beta_c), written over x.
 *   x_inout      in: x, out: y (same buffer, storage dtype, `layout`)
 *   gamma, beta  in: fp32 [C]
 *   running_mean, running_var  in/out fp32 [C], both or neither may be NULL:
 *                new = (1 - momentum)*old + momentum*batch, where the batch
 *                variance is the unbiased var_c*m/(m-1)
 *   save_mean, save_invstd     out fp32 [C]: mu_c and invstd_c
 *   eps >= 0, 0 <= momentum <= 1; training needs m >= 2.  C == 0 is a no-op.
 *   workspace    device, >= iabn_workspace_size bytes, 16-byte aligned; its
 *                contents on entry do not matter.
 * Equivalent to iabn_forward_stats followed by iabn_forward_apply. */
iabn_status iabn_forward_train(void *x_inout,
                               int64_t N, int64_t C, int64_t H, int64_t W,
                               iabn_layout layout, iabn_dtype dtype,
                               const float *gamma, const float *beta,
                               float *running_mean, float *running_var,
                               float *save_mean, float *save_invstd,
                               iabn_act act, float act_param, float eps, float momentum,
                               void *workspace, size_t workspace_bytes,
                               hipStream_t stream);

/* First stage of iabn_forward_train: reads x, computes the statistics, writes
 * save_mean / save_invstd, updates the running statistics, and leaves the
 * per-channel affine constants in the workspace for iabn_forward_apply.  x is
 * not modified.  Arguments as for iabn_forward_train. */
iabn_status iabn_forward_stats(const void *x,
                               int64_t N, int64_t C, int64_t H, int64_t W,
                               iabn_layout layout, iabn_dtype dtype,
                               const float *gamma, const float *beta,
                               float *running_mean, float *running_var,
                               float *save_mean, float *save_invstd,
                               float eps, float momentum,
                               void *workspace, size_t workspace_bytes,
                               hipStream_t stream);

/* Second stage of iabn_forward_train: y = act(...) written over x, from the
 * constants iabn_forward_stats left in the same workspace, on the same stream,
 * for the same x, shape, layout and dtype. */
iabn_status iabn_forward_apply(void *x_inout,
                               int64_t N, int64_t C, int64_t H, int64_t W,
                               iabn_layout layout, iabn_dtype dtype,
                               iabn_act act, float act_param,
                               void *workspace, size_t workspace_bytes,
                               hipStream_t stream);

/* Inference forward, in place, with the running statistics: section 3, "Batch
 * Normalization Review" normalises with the minibatch statistics in training;
 * at inference the pages state no rule, and the usual one is taken, the
 * running estimates that iabn_forward_train keeps (momentum update, unbiased
 * variance) standing in for the batch statistics:
 *   y = act(gamma_c * (x - running_mean_c) / sqrt(running_var_c + eps) + beta_c)
 * written over x.  All per-channel inputs are fp32 [C] and required.  Needs no
 * workspace.  An empty tensor (any extent 0) is a no-op. */
iabn_status iabn_forward_eval(void *x_inout,
                              int64_t N, int64_t C, int64_t H, int64_t W,
                              iabn_layout layout, iabn_dtype dtype,
                              const float *gamma, const float *beta,
                              const float *running_mean, const float *running_var,
                              iabn_act act, float act_param, float eps,
                              hipStream_t stream);

/* Training backward from the stored output alone (section 3, "INPLACE-ABN" I
 * and II; Appendix, "Derivation of Gradient"):
 *   z = act^-1(y), dz = act'(z)*dy (both from y), xhat = (z - beta_c)/gamma_c,
 *   dbeta_c = sum dz, dgamma_c = sum dz*xhat,
 *   dx = gamma_c*invstd_c*(dz - dbeta_c/m - xhat*dgamma_c/m).
 *   y, dy        in, storage dtype, `layout`; y is never modified
 *   dx           out, storage dtype; may be exactly dy (in place), must not
 *                overlap y, and must not partly overlap dy
 *   gamma, beta  in fp32 [C], the values the forward used (gamma_c != 0)
 *   save_invstd  in fp32 [C], from the forward
 *   dgamma, dbeta out fp32 [C]
 *   Needs m >= 2.  C == 0 is a no-op.  Workspace as for the forward.
 * The ELU inverse clamps y/alpha to at least -1 + 2^-24, which only rounding of
 * the stored y can reach.  Equivalent to iabn_backward_reduce followed by
 * iabn_backward_apply. */
iabn_status iabn_backward(const void *y, const void *dy, void *dx,
                          int64_t N, int64_t C, int64_t H, int64_t W,
                          iabn_layout layout, iabn_dtype dtype,
                          const float *gamma, const float *beta, const float *save_invstd,
                          float *dgamma, float *dbeta,
                          iabn_act act, float act_param,
                          void *workspace, size_t workspace_bytes,
                          hipStream_t stream);

/* First stage of iabn_backward: the per-channel sums, dgamma and dbeta, and the
 * per-channel coefficients of dx left in the workspace. */
iabn_status iabn_backward_reduce(const void *y, const void *dy,
                                 int64_t N, int64_t C, int64_t H, int64_t W,
                                 iabn_layout layout, iabn_dtype dtype,
                                 const float *gamma, const float *beta, const float *save_invstd,
                                 float *dgamma, float *dbeta,
                                 iabn_act act, float act_param,
                                 void *workspace, size_t workspace_bytes,
                                 hipStream_t stream);

/* Second stage of iabn_backward: dx from y, dy and the coefficients that
 * iabn_backward_reduce left in the same workspace (same stream, shapes, act). */
iabn_status iabn_backward_apply(const void *y, const void *dy, void *dx,
                                int64_t N, int64_t C, int64_t H, int64_t W,
                                iabn_layout layout, iabn_dtype dtype,
                                iabn_act act, float act_param,
                                void *workspace, size_t workspace_bytes,
                                hipStream_t stream);

/* Backward through iabn_forward_eval: the running statistics are frozen
 * constants of the layer, as when a pre-trained network is fine-tuned with its
 * normalisation statistics fixed (the "Eval mode" in the "Problem" section of
 * "Efficient ConvBN Blocks for Transfer Learning and Beyond").  The chain rule of
 * the inference forward, taken from the stored output alone:
 *   z = act^-1(y), dz = act'(z)*dy (both from y),
 *   dx = gamma_c * dz / sqrt(running_var_c + eps),
 *   dbeta_c = sum dz, dgamma_c = sum dz*(z - beta_c)/gamma_c.
 *   y, dy, dx    as for iabn_backward (dx may be exactly dy)
 *   gamma, beta, running_var, eps   in: the values iabn_forward_eval used
 *                (gamma_c != 0, eps >= 0)
 *   dgamma, dbeta out fp32 [C], both or neither may be NULL; when NULL the sums
 *                are skipped and only dx is written
 *   Needs m >= 1.  C == 0 is a no-op.  Workspace as for the forward.
 * HBM traffic: 3S for dx (read y, dy; write dx), 2S more for the sums. */
iabn_status iabn_backward_eval(const void *y, const void *dy, void *dx,
                               int64_t N, int64_t C, int64_t H, int64_t W,
                               iabn_layout layout, iabn_dtype dtype,
                               const float *gamma, const float *beta,
                               const float *running_var, float eps,
                               float *dgamma, float *dbeta,
                               iabn_act act, float act_param,
                               void *workspace, size_t workspace_bytes,
                               hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Optimized checkpointing (section 3, "Proposed Checkpointing"): the scheme the
 * pages weigh InPlace-ABN II against.  A BN + activation block keeps the
 * normalised xhat instead of its input x; the layer output y is rebuilt from
 * xhat (scale-and-shift, then the activation) when the following layer's
 * backward needs it, and the BN backward reads xhat itself rather than
 * recomputing it from x.  These run the split kernels (statistics pass, then an
 * elementwise pass; backward sums, then dx), on every layout, dtype and
 * activation, with the workspace of iabn_workspace_size.
 */

/* Training forward of the checkpointing block:
 *   mu_c, var_c, invstd_c, running statistics, save_mean, save_invstd exactly as
 *   iabn_forward_train;
 *   xhat = (x - mu_c)*invstd_c, written over x (the kept buffer);
 *   y = act(gamma_c*xhat' + beta_c) into y, where xhat' is xhat as stored, so
 *   that y equals what iabn_recompute_from_xhat gives from the kept buffer.
 *   y must not overlap x.  Errors as for iabn_forward_train.
 * HBM traffic: read x twice, write xhat and y (4S). */
iabn_status iabn_forward_train_ckpt(void *x_inout, void *y,
                                    int64_t N, int64_t C, int64_t H, int64_t W,
                                    iabn_layout layout, iabn_dtype dtype,
                                    const float *gamma, const float *beta,
                                    float *running_mean, float *running_var,
                                    float *save_mean, float *save_invstd,
                                    iabn_act act, float act_param, float eps, float momentum,
                                    void *workspace, size_t workspace_bytes,
                                    hipStream_t stream);

/* The layer output rebuilt from the kept buffer: y = act(gamma_c*xhat + beta_c).
 * y may be exactly xhat (in place) but must not partly overlap it.  Needs no
 * workspace; an empty tensor is a no-op.  HBM traffic 2S. */
iabn_status iabn_recompute_from_xhat(const void *xhat, void *y,
                                     int64_t N, int64_t C, int64_t H, int64_t W,
                                     iabn_layout layout, iabn_dtype dtype,
                                     const float *gamma, const float *beta,
                                     iabn_act act, float act_param, hipStream_t stream);

/* Training backward of the checkpointing block, from the kept xhat:
 *   z = gamma_c*xhat + beta_c, formed with one fused multiply-add so that the
 *   activation's branch follows the sign of the exact value; dz = act'(z)*dy;
 *   dbeta_c = sum dz, dgamma_c = sum dz*xhat,
 *   dx = gamma_c*invstd_c*(dz - dbeta_c/m - xhat*dgamma_c/m).
 *   Arguments, aliasing (dx may be exactly dy) and errors as for iabn_backward,
 *   with xhat in place of y.  HBM traffic 5S (sums, then dx). */
iabn_status iabn_backward_ckpt(const void *xhat, const void *dy, void *dx,
                               int64_t N, int64_t C, int64_t H, int64_t W,
                               iabn_layout layout, iabn_dtype dtype,
                               const float *gamma, const float *beta, const float *save_invstd,
                               float *dgamma, float *dbeta,
                               iabn_act act, float act_param,
                               void *workspace, size_t workspace_bytes,
                               hipStream_t stream);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the training
 * forward exactly as iabn_forward_train, with the same arguments, results and
 * errors, but no workspace argument.  Its workspace is a static device array of
 * IABN_NOALLOC_SCRATCH_BYTES bytes inside the library, one per device, held from
 * the library's load until the process ends; the call allocates nothing.
 *   - Shapes whose iabn_workspace_size exceeds the array are rejected with
 *     IABN_ERR_WORKSPACE before any HIP call (use iabn_forward_train).
 *   - Every call on a device shares that device's array: calls that may overlap
 *     on one device (different streams, or several host threads) race and give
 *     wrong results.  Calls in stream order are safe; the array keeps the last
 *     call's contents, which no call needs cleared.
 *   - A timeout of the exchanging kernels is recorded in the array, where
 *     iabn_workspace_status cannot reach it; callers that share the device with
 *     long-running work switch those kernels off (iabn_set_grouped_kernels).
 *   - The first call on a device looks up the array's device address (a HIP
 *     runtime query, no allocation); capture a graph after one eager call. */
#define IABN_NOALLOC_SCRATCH_BYTES (8u << 20)
iabn_status iabn_forward_train_noalloc(void *x_inout,
                                       int64_t N, int64_t C, int64_t H, int64_t W,
                                       iabn_layout layout, iabn_dtype dtype,
                                       const float *gamma, const float *beta,
                                       float *running_mean, float *running_var,
                                       float *save_mean, float *save_invstd,
                                       iabn_act act, float act_param, float eps, float momentum,
                                       hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Residual blocks kept in 8 bits.  The same trade for the blocks of a language
 * model (row norms, gated activations, linear layers): what a block keeps for its
 * backward is one byte an element instead of the tensor.
 *
 * Tensors here are rows x cols of the storage dtype, the columns contiguous and the
 * rows `ld` elements apart (ld >= cols), so a slice of a wider buffer is taken as it
 * is.  Any alignment of one element is accepted; where a width is no multiple of 8, the
 * row's end is read by one wide access inside the row and written in smaller pieces.  rows and cols stay below 2^31; offsets are
 * 64-bit.  An output may be exactly an input of the same call (same pointer and
 * ld) unless said otherwise, and must not overlap one in any other way; two slices of
 * one buffer (equal ld, disjoint columns) do not overlap.  No two outputs of a call
 * overlap, and vectors of cols, statistics, codes and workspaces overlap nothing else of
 * it (but a vector's gradient may be exactly a vector that the call reads).  rows == 0 or cols == 0 is
 * a no-op that succeeds (gradients summed over no rows are written as zeros).
 *
 * Codes: a tensor [rows, cols] is kept as
 *   codes  int8  [rows, cols rounded up to 32], 16-byte aligned, and
 *   exps   uint8 [rows, that / 32], one for each group of 32 along the row;
 *   value = q * 2^(E - 127), |q| <= 127, E the smallest exponent (1 to 248) under which
 *   the group's largest magnitude rounds to at most 127; q to nearest, ties to even
 *   (magnitudes of 127.5 * 2^121 and above, which have none, become 127 * 2^121).
 *   E = 0: a group of zeros.  E = 255: a group that held an infinity or a NaN; all
 *   of it reads NaN.  Padding codes are zero.  Values are exact in bf16 (not always in
 *   f16: they round, or overflow to infinity, when unpacked to it).
 */

/* codes and exps of x [rows, cols].  Reads x once. */
iabn_status iabn_codes_pack(const void *x, int64_t ldx, int64_t rows, int64_t cols,
                            iabn_dtype dtype, int8_t *codes, uint8_t *exps, hipStream_t stream);

/* y = scale_c * value + shift_c, rounded once; scale and shift fp32 [cols], either
 * may be NULL (1 and 0). */
iabn_status iabn_codes_unpack(const int8_t *codes, const uint8_t *exps, int64_t rows,
                              int64_t cols, const float *scale, const float *shift, void *y,
                              int64_t ldy, iabn_dtype dtype, hipStream_t stream);

/* Activations of the gated unit: SiLU x*sigmoid(x), GELU x*Phi(x), and GELU with the
 * tanh form of Phi. */
typedef enum iabn_glu_act { IABN_GLU_SILU = 0, IABN_GLU_GELU = 1, IABN_GLU_GELU_TANH = 2 } iabn_glu_act;

/* out = act(gate) * up, or act(gate) without up (NULL), from the tensors as they are;
 * and their codes for the backward: codes_gate / exps_gate with codes_up / exps_up
 * (no codes_up without up), or all NULL (inference).  out may be exactly gate or up. */
iabn_status iabn_glu_forward(const void *gate, int64_t ldgate, const void *up, int64_t ldup,
                             void *out, int64_t ldout, int64_t rows, int64_t cols,
                             iabn_dtype dtype, iabn_glu_act act, int8_t *codes_gate,
                             uint8_t *exps_gate, int8_t *codes_up, uint8_t *exps_up,
                             hipStream_t stream);

/* Backward from the codes, g' and u' their values (u' = 1 without codes_up):
 *   dgate = dout * u' * act'(g'), dup = dout * act(g') (with codes_up),
 *   out   = act(g') * u', when not NULL: the next layer's input rebuilt.
 * dgate, dup and out may each be exactly dout. */
iabn_status iabn_glu_backward(const int8_t *codes_gate, const uint8_t *exps_gate,
                              const int8_t *codes_up, const uint8_t *exps_up, const void *dout,
                              int64_t lddout, void *dgate, int64_t lddgate, void *dup,
                              int64_t lddup, void *out, int64_t ldout, int64_t rows, int64_t cols,
                              iabn_dtype dtype, iabn_glu_act act, hipStream_t stream);

/* Bytes of workspace of iabn_linear_wgrad; 0 when it needs none (and for invalid
 * arguments).  Depends on the arguments and the device's CU count. */
size_t iabn_linear_wgrad_workspace_size(int64_t rows, int64_t n, int64_t k, iabn_dtype dtype);

/* Weight gradient of y = x W^T + bias, W [n, k], from the codes of x [rows, k]:
 *   dw = (dw +) dy^T (scale * x + shift), dbias = (dbias +) sum over rows of dy,
 * the bracketed terms with accumulate != 0.  dy [rows, n] of `dtype`; dw [n, k], rows
 * lddw apart, of dw_dtype; scale, shift fp32 [k] or NULL; dbias fp32 [n] or NULL.
 * k == 0 leaves dbias alone to compute.  dw must not overlap dy.
 * lddy and k stay below 2^26.  Sums are fp32; the products are exact (codes are exact in
 * bf16, and f16 and f32 values of dy enter as two and three bf16 parts).  workspace: device, 16-byte
 * aligned, iabn_linear_wgrad_workspace_size bytes; it carries no status word. */
iabn_status iabn_linear_wgrad(const void *dy, int64_t lddy, iabn_dtype dtype, const int8_t *codes,
                              const uint8_t *exps, const float *scale, const float *shift,
                              void *dw, int64_t lddw, iabn_dtype dw_dtype, float *dbias,
                              int accumulate, int64_t rows, int64_t n, int64_t k,
                              void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Row norms: RMS x * rstd, layer (x - mean) * rstd, rstd = 1/sqrt(mean of squares of
 * what is scaled + eps). */
typedef enum iabn_norm { IABN_NORM_NONE = 0, IABN_NORM_RMS = 1, IABN_NORM_LAYER = 2 } iabn_norm;

/* The boundary between two residual blocks: the block's output b goes through the
 * post-norm, its gate and the residual scale into the residual stream r, and the
 * pre-norm makes the next block's input of it:
 *   r' = r + alpha * g * post(b),   n = pre(r'),   norm(x) = xhat * weight + bias.
 * weights and biases are fp32 [cols], NULL for 1 and 0.  gate: NULL, or
 * [rows / rows_per_gate, cols] contiguous of gate_dtype (f32 or the storage dtype),
 * each gate row for rows_per_gate (a divisor of rows) consecutive rows: rows for a
 * learned vector, a sample's rows, or 1.  rows_per_gate is ignored without a gate.
 * cols <= 16384. */
typedef struct iabn_resnorm {
    int64_t rows, cols;
    iabn_dtype dtype;
    iabn_norm post, pre;
    const float *post_weight, *post_bias, *pre_weight, *pre_bias;
    float alpha, eps;
    const void *gate;
    iabn_dtype gate_dtype;
    int64_t rows_per_gate;
} iabn_resnorm;

/* Forward.  b NULL: r' = r (the first norm of a network).  r_out NULL: r' is not
 * written; n is written unless pre is none.  n is formed from the unrounded r'.
 * post_stats, pre_stats: fp32 [rows, 2], mean and rstd, or NULL.  codes_b / exps_b:
 * codes of post's xhat (of b itself when post is none), codes_n / exps_n: codes of
 * pre's xhat; NULL when the backward will read the tensors themselves.  r_out and n
 * may each be exactly r or b, but not one another (or the gate, if it has a row for each). */
iabn_status iabn_resnorm_forward(const iabn_resnorm *layer, const void *r, int64_t ldr,
                                 const void *b, int64_t ldb, void *r_out, int64_t ldr_out,
                                 void *n, int64_t ldn, float *post_stats, float *pre_stats,
                                 int8_t *codes_b, uint8_t *exps_b, int8_t *codes_n,
                                 uint8_t *exps_n, hipStream_t stream);

/* Bytes of workspace of iabn_resnorm_backward (0 for an empty problem and invalid
 * arguments); rows_per_gate as in the layer, any value >= 1 without a gate. */
size_t iabn_resnorm_workspace_size(int64_t rows, int64_t cols, int64_t rows_per_gate);

/* Backward, from dr_out (gradient of r'; NULL: zero) and dn (of n; NULL: zero), and
 * either the stored r_out and b or the codes (not a mixture), with the forward's
 * statistics:
 *   D  = dr_out + rstd (q - [<q>] - xhat <q xhat>), q = dn * pre_weight   -> dr
 *   dz = alpha * D; dgate = sum dz * post(b); h = g * dz * post_weight
 *   db = rstd_b (h - [<h>] - xhat_b <h xhat_b>)       [.]: layer norms only
 * dr may be NULL; db NULL: the branch gets no gradients (and dpost_*, dgate must be
 * NULL).  dpost_*, dpre_* fp32 [cols], dgate of gate_dtype shaped as gate; each may be
 * NULL.  b (codes_b) is needed with db for a post-norm or dgate only.  dr and db may be
 * exactly dr_out or dn, but not one another, nor the gate; dgate may be exactly the gate.
 * No output overlaps what was saved.
 * rows == 0: dpost_* and dpre_* are written as zeros; dgate has no rows and is not
 * written (a caller whose gate is one vector for every row clears it itself).
 * workspace: device, 16-byte aligned; it carries no status word.  Sums over rows are
 * fp32 within a block of rows and finished in fp64, in a fixed order. */
iabn_status iabn_resnorm_backward(const iabn_resnorm *layer, const void *dr_out,
                                  int64_t lddr_out, const void *dn, int64_t lddn,
                                  const void *r_out, int64_t ldr_out, const void *b, int64_t ldb,
                                  const int8_t *codes_n, const uint8_t *exps_n,
                                  const int8_t *codes_b, const uint8_t *exps_b,
                                  const float *post_stats, const float *pre_stats, void *dr,
                                  int64_t lddr, void *db, int64_t lddb, float *dpost_weight,
                                  float *dpost_bias, float *dpre_weight, float *dpre_bias,
                                  void *dgate, void *workspace, size_t workspace_bytes,
                                  hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Attention, rotary positions and group norm: what a block of an image, video or
 * language model needs next to the norms and gated units above.
 *
 * A tensor of heads [batch, rows, heads, head_dim]: element (b, r, h, d) lies at
 * data + b*batch + r*row + h*head + d (strides in elements, not negative; any alignment
 * of one element).  Slices of a wider projection and layouts with heads before rows
 * are taken as they lie. */
typedef struct iabn_heads {
    void *data;
    int64_t batch, row, head;
} iabn_heads;

/* One attention problem: batch sequences of q_len queries and k_len keys, heads query heads
 * (a multiple of kv_heads: query head h goes with key head h / (heads / kv_heads)) of
 * head_dim elements, a multiple of 8 up to 128.
 *
 * Query i of a sequence of Lq queries and Lk keys sees the keys j < Lk with
 *   i + (Lk - Lq) - left <= j <= i + (Lk - Lq) + right,
 * left or right < 0: unbounded on that side.  right = 0 is causal with the last query at
 * the last key (new tokens behind a cache).  A query that sees no key gets out = 0,
 * lse = -inf, and has no part in any gradient.  Keys behind a sequence's length are not read.
 * Other hidden keys take no part while they are finite; a NaN or an infinity in a key or value
 * (in the backward: in a query or dout too) may reach rows that do not see it, as 0 * NaN.
 *
 * Lengths: q_lens, k_lens int32 [batch] on the device, or NULL (the whole length).  Rows of
 * out and of gradients behind a length are written as zeros (lse: -inf).
 * Packed: q_starts, k_starts int32 [batch + 1] on the device: sequence b is rows
 * starts[b] .. starts[b+1] - 1 of a tensor of q_rows (k_rows) rows, the batch stride is not
 * used, and q_len (k_len) is the most rows that a sequence has; rows in no sequence are
 * left as they were.  Either side may be packed, padded or full by itself.  Values outside
 * the tensors are cut to them.
 *
 * q_len and k_len times heads / kv_heads stay at or below 2^29, and
 * batch * kv_heads * (2 max(q_len * heads / kv_heads, k_len) + 256) below 2^32.  scale > 0. */
typedef struct iabn_attention {
    int64_t batch, heads, kv_heads, head_dim, q_len, k_len;
    iabn_dtype dtype;
    float scale;
    int64_t left, right;
    const int32_t *q_starts, *k_starts;
    int64_t q_rows, k_rows;
    const int32_t *q_lens, *k_lens;
} iabn_attention;

/* Bytes of workspace of iabn_attention_forward (backward == 0) or _backward; 0 when it needs
 * none (and for invalid arguments).  Depends on the arguments and the device's CU count;
 * of lengths and starts on whether there are any, not on their values. */
size_t iabn_attention_workspace_size(const iabn_attention *problem, int backward);

/* out = softmax(scale * q k^T) v over the visible keys; lse: fp32 [batch, heads, q_len]
 * (packed queries: [heads, q_rows]), log of the sum of exp(scale * q k^T), or NULL.  out
 * overlaps none of q, k, v.  Softmax statistics and sums are fp32; for 16-bit types the
 * probabilities are rounded to them before they meet v (float16: raised by a power of two
 * first, so that those down to 2^-25 of a row's largest keep their digits).  workspace: device, 16-byte aligned,
 * iabn_attention_workspace_size(problem, 0) bytes; it carries no status word. */
iabn_status iabn_attention_forward(const iabn_attention *problem, const iabn_heads *q,
                                   const iabn_heads *k, const iabn_heads *v,
                                   const iabn_heads *out, float *lse, void *workspace,
                                   size_t workspace_bytes, hipStream_t stream);

/* Gradients of the forward from its out and lse, the probabilities recomputed:
 *   P = exp(scale * q k^T - lse), delta = sum_d dout * out, dS = P * (dout v^T - delta),
 *   dv = P^T dout, dq = scale * dS k, dk = scale * dS^T q,
 * dk and dv summed over the query heads of a key head.  dq, dk and dv overlap nothing else
 * of the call (slices of one buffer do not overlap).  For 16-bit types P and dS are rounded to
 * them before their products (float16: raised by powers of two first, so that small gradients
 * keep their digits). */
iabn_status iabn_attention_backward(const iabn_attention *problem, const iabn_heads *q,
                                    const iabn_heads *k, const iabn_heads *v,
                                    const iabn_heads *out, const float *lse,
                                    const iabn_heads *dout, const iabn_heads *dq,
                                    const iabn_heads *dk, const iabn_heads *dv, void *workspace,
                                    size_t workspace_bytes, hipStream_t stream);

typedef enum iabn_pos { IABN_POS_I32 = 0, IABN_POS_I64 = 1, IABN_POS_F32 = 2 } iabn_pos;

/* Rotary positions with `axes` coordinates a token: pair p (of `pairs`) of every head turns by
 * angle = position[axis[p]] * inv_freq[p], (a, b) -> (a cos - b sin, b cos + a sin), a and b
 * the head's elements p and pairs + p, or with `interleaved` 2p and 2p + 1; elements from
 * 2*pairs on are copied.  inv_freq float64 [pairs] (radians a step) and axis int32 [pairs]
 * (NULL: all 0; values are cut to [0, axes)) on the device.  positions: coordinate c of token (b, r)
 * at b*pos_batch + r*pos_row + c, of pos_type; pos_batch 0 shares them among the batch.
 * Angles are formed in float64.  rows below 2^30. */
typedef struct iabn_rotary_spec {
    int64_t batch, rows, head_dim, pairs, axes;
    iabn_dtype dtype;
    int interleaved;
    const double *inv_freq;
    const int32_t *axis;
    const void *positions;
    iabn_pos pos_type;
    int64_t pos_batch, pos_row;
} iabn_rotary_spec;

/* q_out = turned q, and k_out = turned k where k_heads > 0 (k, k_out may else be NULL).  With
 * `inverse` by the negative angles: the gradient.  q_out may be exactly q, k_out exactly k. */
iabn_status iabn_rotary(const iabn_rotary_spec *spec, const iabn_heads *q, int64_t q_heads,
                        const iabn_heads *q_out, const iabn_heads *k, int64_t k_heads,
                        const iabn_heads *k_out, int inverse, hipStream_t stream);

/* Activations of the group norm: those of the gated unit, identity, and leaky ReLU with slope
 * act_param for z < 0 (0: ReLU). */
typedef enum iabn_gn_act {
    IABN_GN_SILU = 0, IABN_GN_GELU = 1, IABN_GN_GELU_TANH = 2, IABN_GN_IDENTITY = 3,
    IABN_GN_LEAKY_RELU = 4
} iabn_gn_act;

/* Group norm with an activation, channels last: n samples of hw rows of c channels, rows ld
 * elements apart (ld >= c); groups of c / groups neighbouring channels, groups a divisor of c. */
typedef struct iabn_group_norm {
    int64_t n, hw, c, groups;
    iabn_dtype dtype;
    const float *weight, *bias;          /* fp32 [c], NULL: 1 and 0 */
    iabn_gn_act act;
    float act_param, eps;
} iabn_group_norm;

/* Bytes of workspace of both passes (0 for an empty problem and invalid arguments). */
size_t iabn_group_norm_workspace_size(const iabn_group_norm *layer);

/* y = act(xhat * weight + bias), xhat = (x - mean) * rstd over a sample's group,
 * rstd = 1 / sqrt(biased variance + eps).  stats: fp32 [n, groups, 2], mean and rstd, or NULL.
 * y may be exactly x.  Rows n*hw below 2^31, c below 2^26, groups below 2^24.  workspace: device,
 * 16-byte aligned; it carries no status word. */
iabn_status iabn_group_norm_forward(const iabn_group_norm *layer, const void *x, int64_t ldx,
                                    void *y, int64_t ldy, float *stats, void *workspace,
                                    size_t workspace_bytes, hipStream_t stream);

/* Gradients from x and the forward's stats: dz = act'(z) * dy, dbias_c = sum dz,
 * dweight_c = sum dz * xhat, dx = rstd * (weight dz - <weight dz> - xhat <weight dz xhat>),
 * <.> the mean over the group.  dx, dweight and dbias may each be NULL; dx may be exactly
 * dy or x, dweight exactly weight and dbias exactly bias.  n == 0 or hw == 0: dweight and dbias
 * are written as zeros. */
iabn_status iabn_group_norm_backward(const iabn_group_norm *layer, const void *x, int64_t ldx,
                                     const void *dy, int64_t lddy, void *dx, int64_t lddx,
                                     const float *stats, float *dweight, float *dbias,
                                     void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Describes, as a short text, the kernels that iabn_forward_train and
 * iabn_backward launch for this problem when every tensor pointer is 16-byte
 * aligned (aligned16 != 0) or not, e.g.
 *   "forward=channel_resident(512x49) backward=channel_resident(512x49,dy_streamed)".
 * For logging, benchmarks and tests; it launches nothing.  Writes at most
 * `len` bytes including the terminating NUL into `buf` and returns the length
 * of the full description (like snprintf), or -1 for invalid arguments. */
int iabn_describe_plan(int64_t N, int64_t C, int64_t H, int64_t W,
                       iabn_layout layout, iabn_dtype dtype, iabn_act act,
                       int aligned16, char *buf, size_t len);

#ifdef __cplusplus
}
#endif

#endif /* IABN_H */
