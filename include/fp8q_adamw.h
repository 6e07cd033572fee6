/*
 * fp8q_adamw.h -- the optimizer step of the C ABI of libfp8q: AdamW over many
 * tensors in one call, with its states in 32 bits or in 8. Conventions and
 * status codes are those of fp8q.h, which includes this header.
 */
#ifndef FP8Q_ADAMW_H
#define FP8Q_ADAMW_H

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FP8Q_ADAMW_BF16 0 /* parameters or gradients in bf16 */
#define FP8Q_ADAMW_F32  1 /* ... in FP32                     */

#define FP8Q_ADAMW_MAX_NUMEL ((1LL << 34) - 1024) /* elements of one tensor with a gradient */

/*
 * One tensor of a step: device arrays of `numel` elements, contiguous.
 *   param      updated in place.
 *   exp_avg, exp_avg_sq  the two moments, updated in place. 32-bit states: FP32.
 *              8-bit states: E4M3 codes, with FP32 scales [ceil(numel / 128)],
 *              one for each 128 consecutive elements; exp_avg_sq then holds the
 *              ROOT of the second moment, whose range E4M3 can hold.
 *   exp_avg_scale, exp_avg_sq_scale  8-bit states only (NULL otherwise).
 *   copy       bf16 copy of an FP32 parameter, written (NULL: none).
 * Arrays need the alignment of their elements only; tensors whose arrays all
 * start on 16-byte boundaries (codes: 4) run faster. No two arrays of a call
 * may overlap.
 */
typedef struct fp8q_adamw_tensor {
    void *param;
    void *exp_avg;
    void *exp_avg_sq;
    float *exp_avg_scale;
    float *exp_avg_sq_scale;
    uint16_t *copy;
    int64_t numel;
} fp8q_adamw_tensor;

/*
 * adamw_step -- one step of AdamW (decoupled weight decay), t = step:
 *   g' = g * grad_scale
 *   m  = beta1 m + (1 - beta1) g'
 *   v  = beta2 v + (1 - beta2) g'^2
 *   p  = p (1 - lr weight_decay) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * in FP32; the factors that depend on the options alone are computed in FP64
 * and rounded once. The parameter takes this step's moments as computed, before
 * they are rounded to their storage. A bf16 parameter is rounded to nearest
 * even, and changes below half its last place are lost: train FP32 parameters
 * with a bf16 copy where that matters.
 *
 * 8-bit states: a block of 128 elements has the scale s = fl32(amax * fl32(1 /
 * 448)), within a last place of the quotient that the quantizers of fp8q.h take,
 * and codes E4M3(fl32(x / s)), rounded STOCHASTICALLY: the code above with the
 * probability of the part that is cut off. (Rounded to nearest, a moment whose
 * step is less than half a code's, as those of beta2 near 1 are, would never
 * move.) The 16 random bits of an element and state are a hash of seed, step,
 * the tensor's place in the call and the element's number, so a step can be
 * repeated exactly. A root of the second moment above zero is never stored as
 * zero: its element would take a far too large step next time. A block of either
 * moment with an infinity or a NaN reads back as NaN; a gradient whose square
 * passes FP32 (from 1.8e19 on) makes the second moment one.
 *
 * tensors     HOST array of `count` entries, read during the call.
 * grads       HOST array of `count` device addresses, read during the call: the
 *             gradient of each tensor, contiguous; NULL: the tensor takes no
 *             part in this step.
 * param_dtype, grad_dtype  FP8Q_ADAMW_*, the same for all tensors of a call.
 * state_bits  32 or 8.
 * lr, step    used where lr_dev, step_dev are NULL; else DEVICE arrays of one
 *             element, read when the kernels run (a captured step that is
 *             replayed takes their values of that time).
 * grad_scale  DEVICE FP32 [1] or NULL for 1. A scale that is not finite makes
 *             the step leave every array as it was.
 * Shapes: count >= 0, 0 <= numel <= FP8Q_ADAMW_MAX_NUMEL, step >= 1 (a device step below 1 acts as 1),
 *         0 <= beta1, beta2 < 1, eps >= 0 (with 0, elements whose moments are
 *         all zero become NaN: 0 / 0; a positive eps that FP32 rounds to 0 or
 *         to infinity is refused).
 * One launch for each 64 tensors (56 with 8-bit states). count == 0, or no elements: FP8Q_OK.
 * Errors: FP8Q_ERR_NULL, FP8Q_ERR_SHAPE (also for the options' ranges),
 *         FP8Q_ERR_ALIGN, FP8Q_ERR_ENUM, FP8Q_ERR_HIP. Everything is checked
 *         before the first launch.
 */
int adamw_step(int32_t count, const fp8q_adamw_tensor *tensors, const void *const *grads, int param_dtype,
               int grad_dtype, int state_bits, double lr, double beta1, double beta2, double eps, double weight_decay,
               int64_t step, const float *lr_dev, const int64_t *step_dev, const float *grad_scale, uint64_t seed,
               hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8Q_ADAMW_H */
