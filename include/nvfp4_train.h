/*
 * nvfp4_train.h — C ABI of libnvfp4.so, second part: the operators of a quantization-aware-
 * distillation training step that stand around nvfp4_fakequant and nvfp4_qad_kl (nvfp4.h):
 * layer norm with the amax that the next quantization needs, its backward pass, the global
 * gradient norm with its clip factor, and an AdamW step over many tensors at once with the
 * states in 32 bits or in 8.
 *
 * The conventions of nvfp4.h hold: device pointers owned by the caller, no allocation, no host
 * synchronization, argument errors returned before anything is enqueued, buffers on the current
 * device, outputs that do not overlap inputs (AdamW updates in place, as stated there). Every
 * result is the same from run to run on one device: no sum depends on the order of atomics.
 * Unlike the quantizer's, these operators' inputs may hold infinities and NaN: they propagate
 * as IEEE arithmetic has it and touch nothing but their own row, column or element (and the
 * 32-element block of an 8-bit state).
 */
#ifndef NVFP4_TRAIN_H
#define NVFP4_TRAIN_H

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of a tensor. An unknown value is refused with NVFP4_ERR_VALUE. */
typedef enum {
    NVFP4_TYPE_BF16 = 0,
    NVFP4_TYPE_F32 = 1
} nvfp4_type;

/* Layer norm over the last dimension of x [rows, cols]. For every row, in binary32:
 *   mean = S x / cols;  var = S (x - mean)^2 / cols;  rstd = 1 / sqrt(var + eps)
 *   y    = (x - mean) * rstd * weight + bias, rounded once to x's type
 *   x       [rows, cols] of x_type                                                  (in)
 *   weight  NULL (all ones), or [cols] of w_type                                    (in)
 *   bias    NULL (all zeros), or [cols] of w_type                                   (in)
 *   y       [rows, cols] of x_type                                                  (out)
 *   mean    NULL, or [rows] float, for the backward pass                            (out)
 *   rstd    NULL, or [rows] float                                                   (out)
 *   amax    NULL, or [1] float: max |y| over the values as stored, exactly: the amax of y's
 *           quantization (nvfp4_quantize, nvfp4_quantize_gemm), which then needs no pass of
 *           nvfp4_amax. NaN if a y is NaN; 0 for an empty tensor                      (out)
 * The variance is the mean square distance from the mean, taken from the row held on chip, so
 * a large mean cancels nothing. Every pointer needs its element's alignment only; x and y are
 * best at the same place within 16 bytes (else rows are read three times by the element, about five
 * times as slow). cols >= 1 and rows >= 0 (else NVFP4_ERR_SHAPE), eps
 * finite and >= 0 (else NVFP4_ERR_VALUE). One kernel, one read of x (rows of more
 * than 65536 columns, and operands that start at different places within 16 bytes, are read
 * again from L2), after a zero-fill of amax where more than one CTA runs. */
NVFP4_API nvfp4_status nvfp4_layer_norm(const void* x, nvfp4_type x_type, const void* weight, const void* bias,
                                        nvfp4_type w_type, int64_t rows, int64_t cols, float eps, void* y,
                                        float* mean, float* rstd, float* amax, cudaStream_t stream);

/* Bytes of workspace that nvfp4_layer_norm_backward needs for this shape on the current device
 * when a weight or bias gradient is asked for; 0 for an empty tensor, -1 for an invalid shape. */
NVFP4_API int64_t nvfp4_layer_norm_workspace(int64_t rows, int64_t cols);

/* Backward pass of nvfp4_layer_norm. With xh = (x - mean) * rstd and h = dy * weight per row:
 *   dx      = rstd * (h - S h / cols - xh * S (h * xh) / cols), rounded once to x's type
 *   dweight = S over rows of dy * xh;   dbias = S over rows of dy
 * Sums in binary32, in an order that depends on the shape and the device alone.
 *   dy, x      [rows, cols] of x_type                                               (in)
 *   weight     NULL (all ones), or [cols] of w_type                                 (in)
 *   mean, rstd [rows] float, as nvfp4_layer_norm wrote them                          (in)
 *   dx         [rows, cols] of x_type                                               (out)
 *   dweight    NULL, or [cols] of w_type                                            (out)
 *   dbias      NULL, or [cols] of w_type                                            (out)
 *   workspace  [nvfp4_layer_norm_workspace(rows, cols)] bytes, 16-byte aligned; may be NULL
 *              when dweight and dbias are. Calls that may overlap on the GPU need workspaces
 *              of their own                                                      (scratch)
 *   workspace_bytes  its size; smaller than needed is refused (NVFP4_ERR_SHAPE)
 * rows == 0 zero-fills dweight and dbias. One kernel over the rows, which leaves each CTA's
 * column sums in the workspace, and one small kernel that adds them. */
NVFP4_API nvfp4_status nvfp4_layer_norm_backward(const void* dy, const void* x, nvfp4_type x_type,
                                                 const void* weight, nvfp4_type w_type, const float* mean,
                                                 const float* rstd, int64_t rows, int64_t cols, void* dx,
                                                 void* dweight, void* dbias, void* workspace,
                                                 int64_t workspace_bytes, cudaStream_t stream);

/* One tensor of a list, as the host describes it to nvfp4_tensor_plan. */
typedef struct {
    void* param;               /* [numel] of param_type, or NULL: gradients only (grad norm)    */
    const void* grad;          /* [numel] of grad_type                                          */
    float* master;             /* NULL, or [numel]: FP32 master of a BF16 param                 */
    void* exp_avg;             /* first moment: [numel] float, or E4M3 codes                    */
    void* exp_avg_sq;          /* second moment: [numel] float, or E4M3 codes of its root       */
    uint8_t* exp_avg_scale;    /* 8-bit states: [ceil(numel / 32)] E8M0 bytes; else NULL        */
    uint8_t* exp_avg_sq_scale; /* likewise                                                      */
    int64_t numel;
    int64_t first;             /* index of element 0 for the random words: a multiple of 8      */
    float weight_decay;
    int32_t param_type;        /* nvfp4_type                                                    */
    int32_t grad_type;         /* nvfp4_type                                                    */
    int32_t state_bits;        /* 32 or 8                                                       */
} nvfp4_opt_tensor;

/* Size in bytes of the plan of a list (0 <= count < 2^24), or -1 for a list that
 * nvfp4_tensor_plan would refuse for its count or lengths. */
NVFP4_API int64_t nvfp4_tensor_plan_bytes(const nvfp4_opt_tensor* tensors, int64_t count);

/* Checks a list and writes its plan to host memory: a table of the tensors and of the equal
 * pieces ("chunks") into which the kernels cut them. The caller copies the image to 16-byte
 * aligned device memory once and keeps it for as long as the pointers in it stay valid.
 *   image   [nvfp4_tensor_plan_bytes] bytes of HOST memory                          (out)
 *   chunks  number of chunks, for the launches below                                (out)
 * A list is either all gradients (every param NULL: for nvfp4_grad_norm) or all optimizer
 * tensors. Refused: a NULL pointer where one is needed (NVFP4_ERR_NULL); a negative length, a
 * total of 2^34 elements or more, `first` not a multiple of 8 (NVFP4_ERR_SHAPE); a pointer that
 * is not aligned to its element (NVFP4_ERR_ALIGN); an unknown type, state_bits other than 32
 * and 8 or not the same in the whole list, a master of a param that is not BF16, a non-finite weight decay, both kinds in one
 * list, or memory that one tensor writes and another one writes or reads (NVFP4_ERR_VALUE). */
NVFP4_API nvfp4_status nvfp4_tensor_plan(const nvfp4_opt_tensor* tensors, int64_t count, void* image,
                                         int64_t image_bytes, int64_t* chunks);

/* Bytes of the workspace of nvfp4_grad_norm. */
#define NVFP4_GRAD_NORM_WORKSPACE 16400

/* Norm of all gradients of a list together, and the factor that clips it:
 *   norm  = sqrt(S over all tensors of g^2);  scale = min(1, max_norm / (norm + 1e-6))
 * scale is NaN when the norm is not finite: nvfp4_adamw then leaves everything as it is.
 *   plan       device copy of a nvfp4_tensor_plan image                             (in)
 *   chunks     as nvfp4_tensor_plan gave it for this plan: the plan is read by it
 *   max_norm   >= 0, infinity allowed (scale = 1); else NVFP4_ERR_VALUE
 *   norm       [1] float                                                            (out)
 *   scale      [1] float                                                            (out)
 *   workspace  [NVFP4_GRAD_NORM_WORKSPACE] bytes, 16-byte aligned, zero before the first call;
 *              each call leaves it ready for the next. Calls that may overlap on the GPU need
 *              workspaces of their own                                           (scratch)
 * Squares are added in binary32 eight at a time and the eights in binary64; an eight whose sum
 * overflows or loses its precision to underflow is added in binary64, so the norm is right
 * over the whole range of its type. One kernel. */
NVFP4_API nvfp4_status nvfp4_grad_norm(const void* plan, int64_t chunks, float max_norm, float* norm, float* scale,
                                       void* workspace, cudaStream_t stream);

/* Device block that counts an optimizer's steps. beta1_t and beta2_t are the coefficients to
 * the power of the steps taken so far (1 before the first). */
typedef struct {
    double beta1_t, beta2_t;
    uint32_t step;       /* steps taken so far                                              */
    uint32_t arrived;    /* 0 between calls                                                 */
    uint32_t reserved[2];
} nvfp4_adamw_control;

/* One AdamW step over a list, in place. With t the steps taken before this one plus one and
 * g = scale * grad, in binary32, fma(a, b, c) = a * b + c rounded once:
 *   m' = fma(m, beta1, (1 - beta1) * g)
 *   v' = fma(v, beta2, (1 - beta2) * (g * g));   u' = sqrt(v')
 *   p' = fma(m' / fma(u', r, eps), -lr / (1 - beta1^t), p * (1 - lr * weight_decay)),  r = 1 / sqrt(1 - beta2^t)
 * where 1 - beta^t is taken in binary64 and rounded once. Beside 8-bit states and with eps in [2^-36, 2^100] the
 * root is the hardware's approximation (2^-23; 0 for a v' below 2^-126) and the quotient the product with its approximate
 * reciprocal (2^-23); any other eps, 0 among them, takes the rounded root and quotient.
 * Parameters. FP32: p. BF16 with a master: p is the master, param = BF16(p'), to nearest even.
 * BF16 without one: p' is rounded stochastically, because an update is mostly far below half a
 * BF16 step, and rounding to nearest would lose it every time.
 * States in 32 bits: m and v. States in 8 bits: m and u = sqrt(v) (half v's range of exponents)
 * as E4M3 codes in blocks of 32 consecutive elements of the tensor, each block with one E8M0
 * byte s: a value is code * 2^(s - 127), and s is the smallest from 1 on that leaves no
 * magnitude of the block above 448. m is rounded to nearest even; u stochastically, because
 * with beta2 near 1 v moves by less than half a step, and rounding to nearest would freeze it;
 * a positive u keeps a positive code, since a zero would leave eps alone in the denominator. The
 * step itself uses m' and u' before that rounding.
 * Random words. Element i of a tensor (k = first + i), t - 1 steps taken, mod 2^32:
 *   word = mix((k >> 3) ^ mix(seed + 0x9E3779B9 * (t - 1))) + (k & 7) * 0x9E3779B9
 *   mix(a): a ^= a >> 16; a *= 0x85EBCA6B; a ^= a >> 13; a *= 0xC2B2AE35; a ^= a >> 16
 *   (the 32-bit finalizer of MurmurHash3, a bijection)
 * Its high half is added to the 16 bits that a BF16 parameter drops; its low half to the upper
 * 16 of the 20 bits that a code of u drops.
 *   plan, chunks  as for nvfp4_grad_norm, of a list of optimizer tensors             (in)
 *   state_bits  32 or 8, as the list's tensors have it (else NVFP4_ERR_VALUE; a list of the other
 *              kind is left alone)
 *   control    device block; the kernel counts the step in it, so a captured call counts on at
 *              every replay                                                      (in/out)
 *   lr         finite, >= 0 (else NVFP4_ERR_VALUE); not used where lr_device is given
 *   lr_device  NULL, or [1] float read by the kernel (a captured call follows it)    (in)
 *   beta1, beta2  in [0, 1); eps finite, >= 0 (else NVFP4_ERR_VALUE)
 *   scale      NULL (1), or [1] float, e.g. from nvfp4_grad_norm. If it is not finite the step
 *              does not take place: only amax is written                             (in)
 *   amax       NULL, or [count] float: max |param| of each tensor as stored, the amax of its next
 *              fake-quantization; zero-filled first in stream order; 0 for an empty tensor (out)
 *   count      number of tensors of the plan, read where amax is given (another number: amax is
 *              zero-filled and nothing else is done)
 * Calls on one control block or one list must not overlap on the GPU. One kernel. */
NVFP4_API nvfp4_status nvfp4_adamw(const void* plan, int64_t chunks, int32_t state_bits,
                                   nvfp4_adamw_control* control, float lr, const float* lr_device, double beta1, double beta2, float eps, uint32_t seed,
                                   const float* scale, float* amax, int64_t count, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* NVFP4_TRAIN_H */
