/*
 * gc_train.h -- C ABI of libgc.so for the operators of the training step that fill the
 * gradient bucket: 8-bit activation checkpoints, the MLP activation and the layer norm with
 * backward passes that read such checkpoints, and the weight gradient of a linear layer
 * whose input was kept in 8 bits.
 *
 * Conventions for every call
 *   - As in gc.h: device pointers, work only enqueued on `stream` (a hipStream_t as void*),
 *     nothing synchronized, allocated or read back; the caller owns every buffer and the
 *     workspace; outputs that overlap inputs or each other are refused (slices beside each
 *     other of one wider matrix do not overlap); arguments are checked on the
 *     host before anything is enqueued and a rejected call makes no HIP call (gc_last_error()
 *     has the reason).
 *   - A matrix is rows x cols of one element type (enum gc_dtype) with consecutive columns; a
 *     row starts `ld` elements after the one before, ld >= cols.  Only the natural alignment
 *     of the element type is needed.  rows, cols in [0, 2^31 - 64], rows * ld at most 2^40;
 *     rows == 0 or cols == 0 is a no-op unless a call says otherwise.
 *   - Sums, statistics and products are held in fp32; a result is rounded once, to nearest
 *     even, when it is stored.  Every sum has a fixed order: the same call on the same inputs
 *     gives the same bits.
 *
 * The checkpoint of a rows x cols matrix (the MXINT8 block format of the Open Compute
 * Project's "Microscaling Formats (MX) Specification" v1.0: blocks of 32 with a shared power
 * of two, elements with 6 fraction bits):
 *   ldc   = 32 * ceil(cols / 32), ng = ldc / 32
 *   codes : int8[rows * ldc], 16-byte aligned; column c of row r at r * ldc + c, zero for c >= cols
 *   exps  : uint8[rows * ng]; byte g of row r scales columns [32 g, 32 g + 32)
 *   value = code * 2^(E - 133)
 * Packing: amax = max |x| over the block; E = 127 + floor(log2 amax), at least 7 (bf16, fp32)
 * or 109 (fp16), the least for which every value is an element of the type;
 * code = clamp(round-half-even(x * 2^(133 - E)), -127, 127).  |value - x| is at most half of
 * 2^(E - 133), or one whole step where |x| rounds to 128 steps.  A block that holds an Inf or a NaN
 * has E = 255 and codes 0, and all of its values are NaN, so that an overflow reaches the
 * gradients and is noticed there.
 */
#ifndef GC_TRAIN_H
#define GC_TRAIN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum gc_dtype { GC_F32 = 0, GC_F16 = 1, GC_BF16 = 2 };

enum gc_act_kind {
  GC_ACT_GELU = 0,       /* f(x) = x * Phi(x), Phi the normal distribution function              */
  GC_ACT_GELU_TANH = 1,  /* f(x) = x * (1 + tanh(sqrt(2/pi) * (x + 0.044715 x^3))) / 2          */
  GC_ACT_SILU = 2        /* f(x) = x / (1 + exp(-x))                                             */
};

/* gc_ckpt_pack -- the checkpoint of x. */
int gc_ckpt_pack(int dtype, const void* x, int64_t ldx, int64_t rows, int64_t cols, int8_t* codes,
                 uint8_t* exps, void* stream);

/* gc_ckpt_unpack -- out = the values of a checkpoint, rounded to the type of out (exact for
 * the type it was packed from). */
int gc_ckpt_unpack(int dtype, const int8_t* codes, const uint8_t* exps, int64_t rows, int64_t cols,
                   void* out, int64_t ldo, void* stream);

/* gc_act_forward -- y = f(x), and in the same pass the checkpoint of x (x_codes, x_exps: both
 * or neither) and of y as stored (y_codes, y_exps: both or neither). */
int gc_act_forward(int dtype, int kind, const void* x, int64_t ldx, int64_t rows, int64_t cols, void* y,
                   int64_t ldy, int8_t* x_codes, uint8_t* x_exps, int8_t* y_codes, uint8_t* y_exps,
                   void* stream);

/* gc_act_backward -- dx = dy * f'(x), x given in full (x, ldx) or as its checkpoint (x_codes,
 * x_exps); exactly one of the two. */
int gc_act_backward(int dtype, int kind, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                    const int8_t* x_codes, const uint8_t* x_exps, int64_t rows, int64_t cols, void* dx,
                    int64_t lddx, void* stream);

/*
 * gc_layernorm_forward -- for every row: mean = sum x / cols, rstd = 1 / sqrt(sum (x - mean)^2 / cols + eps),
 * y = (x - mean) * rstd * weight + bias; in the same pass the checkpoints of x and of y as
 * stored, as in gc_act_forward.  weight, bias: [cols] of type wdtype (dtype or GC_F32), either
 * may be NULL (1 and 0).  mean, rstd: float[rows].  cols == 0 is refused when rows > 0.
 */
int gc_layernorm_forward(int dtype, const void* x, int64_t ldx, int64_t rows, int64_t cols, int wdtype,
                         const void* weight, const void* bias, float eps, void* y, int64_t ldy,
                         float* mean, float* rstd, int8_t* x_codes, uint8_t* x_exps, int8_t* y_codes,
                         uint8_t* y_exps, void* stream);

/* Workspace bytes of gc_layernorm_backward (host only). */
int gc_layernorm_backward_workspace(int64_t rows, int64_t cols, size_t* bytes);

/*
 * gc_layernorm_backward -- with xh = (x - mean) * rstd and t = dy * weight, for every row
 *   dx = rstd * (t - sum t / cols - xh * (sum t * xh) / cols),
 * and over all rows dw = sum dy * xh and db = sum dy (fp32; added to what is there when
 * accumulate != 0).  x in full or as its checkpoint, exactly one of the two; mean and rstd as
 * the forward pass wrote them (of the full x in both cases).  weight may be NULL (1); dw and
 * db may be NULL, both or either.  With rows == 0, dw and db are cleared (accumulate == 0).
 */
int gc_layernorm_backward(int dtype, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                          const int8_t* x_codes, const uint8_t* x_exps, int64_t rows, int64_t cols,
                          int wdtype, const void* weight, const float* mean, const float* rstd, void* dx,
                          int64_t lddx, float* dw, float* db, int accumulate, void* workspace,
                          size_t workspace_bytes, void* stream);

/* Workspace bytes of gc_linear_wgrad (host only). */
int gc_linear_wgrad_workspace(int dtype, int64_t rows, int64_t in_features, int64_t out_features,
                              size_t* bytes);

/*
 * gc_linear_wgrad -- the weight gradient of y = x W^T + b, from the checkpoint of x
 * (rows x in_features):
 *   dw[o, i] = sum over rows m of dy[m, o] * value[m, i],   db[o] = sum over m of dy[m, o]
 * dy: rows x out_features of type dtype.  dw: float, row o at o * lddw, lddw >= in_features;
 * db: float[out_features] or NULL.  Both are added to what is there when accumulate != 0 (a
 * view into a gradient bucket over several micro-batches).  An fp32 dy enters whole, except for bits
 * below 2^-133; codes and 16-bit dy are exact, so only the fp32 sums round.  For GC_F16 a checkpoint of another
 * type's values is rounded to fp16 first.  With rows == 0, dw and db are cleared
 * (accumulate == 0).
 */
int gc_linear_wgrad(int dtype, const void* dy, int64_t lddy, const int8_t* codes, const uint8_t* exps,
                    int64_t rows, int64_t in_features, int64_t out_features, float* dw, int64_t lddw,
                    float* db, int accumulate, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GC_TRAIN_H */
