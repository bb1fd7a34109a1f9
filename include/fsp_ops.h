/*
 * fsp_ops.h - C ABI of the operators a rank runs beside the sharded step:
 *
 *   - AdamW over a list of tensors in one launch (parameters that are not
 *     sharded, or a rank's own shards after a reduce-scatter), with its states
 *     in 32 or in 8 bits;
 *   - the embedding lookup with scaling and its gradient by sorted tokens (the
 *     gradient goes straight into a parameter's slice of a main-grad buffer);
 *   - matrices in 8-bit floating point with one scale per block of 128, and
 *     their product (a linear layer's forward pass and both of its gradients).
 *
 * The conventions of fsp.h hold: host-side checks before anything is launched,
 * a status and fsp_last_error() on refusal, buffers and streams owned by the
 * caller, asynchronous on the given stream and current device, nothing
 * allocated on the device except by the *_create functions.  Device pointers
 * must lie in live CUDA allocations that hold the whole buffer.  Kernels that wait
 * (for their own copies and products) give up after about 2 s and set bits of the
 * device error word (fsp_device_error): 1 and 2 the AdamW step's, 32 the products'.
 */
#ifndef FSP_OPS_H
#define FSP_OPS_H

#include "fsp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- AdamW over a list of tensors ------------------------------------------ */

/* Elements that share one scale in the 8-bit states; a block never spans two
 * tensors. */
#define FSP_ADAMW_BLOCK 256

typedef enum {
  FSP_STATE_F32 = 0,   /* exp_avg, exp_avg_sq: fp32                                 */
  /* exp_avg: int8 codes q with m = s q |q| / 127^2, s the block's largest |m|;
   * exp_avg_sq: uint8 codes q with v = s (q / 255)^4, s the block's largest v.
   * Codes are rounded to nearest even; a v above 0 keeps a code of at least 1,
   * so a denominator never loses its second moment.  The update of an element
   * uses m' and v' before they are rounded. */
  FSP_STATE_8BIT = 1
} fsp_state_dtype;

/* A list of tensors registered on the current device. */
typedef struct fsp_adamw_list fsp_adamw_list;

/* Registers n (>= 0) tensors.
 *   numels:       elements of each (>= 0).
 *   params:       n device pointers, contiguous tensors of param_dtypes[i]
 *                 (fsp_dtype): fp32, or bf16 (updated in fp32 and rounded to
 *                 nearest even once).
 *   grads:        n device pointers, contiguous, grad_dtypes[i] (fsp_dtype).
 *   copies:       NULL, or n device pointers (each may be NULL) to bf16 tensors
 *                 that receive the new parameter rounded to nearest even - what
 *                 the next forward, or an all-gather, reads.
 * Pointers need their elements' natural alignment only (tensors whose pointers
 * are all aligned to four elements take vector accesses); no two tensors may
 * overlap.  Tensor i's states are slots [offset_i, offset_i + numel_i) of the
 * state buffers, offset_i being the previous tensor's end rounded up to a
 * multiple of FSP_ADAMW_BLOCK.  Synchronous (allocates and uploads the list's
 * table of work tiles). */
fsp_status fsp_adamw_list_create(int32_t n, const int64_t* numels, void* const* params, const int32_t* param_dtypes,
                                 const void* const* grads, const int32_t* grad_dtypes, void* const* copies,
                                 fsp_adamw_list** out);

/* Slots of each state buffer (a multiple of FSP_ADAMW_BLOCK) and, when offsets
 * is not NULL, the n tensors' first slots. */
fsp_status fsp_adamw_list_info(const fsp_adamw_list* list, int64_t* state_len, int64_t* offsets);

/* Frees the list (its device table); NULL is a no-op.  Must not race with a
 * call or an in-flight step that uses it. */
void fsp_adamw_list_destroy(fsp_adamw_list* list);

/* One AdamW update of every tensor of the list (fsp.h's rule and hparams; with
 * fp32 states and parameters the same bits as fsp_sharded_step on the same
 * gradients with n_d = 1).
 *   exp_avg, exp_avg_sq: state_len elements of state_dtype's types, 16-byte
 *               aligned; slots between tensors are not written.
 *   exp_avg_scale, exp_avg_sq_scale: state_len / FSP_ADAMW_BLOCK fp32 scales
 *               (8-bit states; NULL with fp32 states).
 *   step:       t >= 1, or step_dev: device, 8-byte aligned int64 holding t
 *               (step is then ignored), advanced by one after the update when
 *               `advance` is non-zero - the form to capture in a CUDA graph.
 *   grad_scale: NULL, or a device fp32 that multiplies every gradient (a clip
 *               coefficient, 1 / loss scale).
 * A gradient that is not finite makes its element's states NaN or infinite;
 * with 8-bit states it makes its block's scales, and so the block's states,
 * not finite.  A block of m or v whose largest value is 0 holds zeros.  The list
 * holds the launch's counter of work tiles: steps on one list must be ordered on
 * the device (one stream, or events). */
fsp_status fsp_adamw_list_step(const fsp_adamw_list* list, int32_t state_dtype, void* exp_avg, void* exp_avg_sq,
                               float* exp_avg_scale, float* exp_avg_sq_scale, const fsp_adamw_hparams* hp,
                               int64_t step, int64_t* step_dev, int32_t advance, const float* grad_scale,
                               void* cuda_stream);

/* What 8-bit states stand for, as fp32 (state_len each): for checkpoints. */
fsp_status fsp_adamw_list_state_values(const fsp_adamw_list* list, const void* exp_avg, const void* exp_avg_sq,
                                       const float* exp_avg_scale, const float* exp_avg_sq_scale, float* exp_avg_out,
                                       float* exp_avg_sq_out, void* cuda_stream);

/* The inverse: fp32 states (state_len each; exp_avg_sq >= 0) into 8-bit codes
 * and scales. */
fsp_status fsp_adamw_list_state_load(const fsp_adamw_list* list, const float* exp_avg_in, const float* exp_avg_sq_in,
                                     void* exp_avg, void* exp_avg_sq, float* exp_avg_scale, float* exp_avg_sq_scale,
                                     void* cuda_stream);

/* ---- embedding ---------------------------------------------------------------- */

/* out[i][:] = scale * weight[tokens[i]][:], multiplied in fp32 and rounded once.
 *   tokens:  n_tokens (>= 0) indices, int32 (index_bytes 4) or int64 (8).
 *   weight:  vocab x dim, rows weight_stride (>= dim) elements apart, of
 *            weight_dtype; out: n_tokens x dim, rows out_stride apart.
 * A token outside [0, vocab) gives a row of zeros and sets bit 16 of the device
 * error word. */
fsp_status fsp_embedding(const void* weight, int32_t weight_dtype, int64_t vocab, int64_t dim, int64_t weight_stride,
                         const void* tokens, int32_t index_bytes, int64_t n_tokens, float scale, void* out,
                         int32_t out_dtype, int64_t out_stride, void* cuda_stream);

/* Device workspace, in bytes, of fsp_embedding_backward. */
fsp_status fsp_embedding_backward_workspace_bytes(int64_t vocab, int64_t dim, int64_t n_tokens, size_t* bytes);

/* grad_weight[r][:] = (accumulate: +) scale * sum of grad_out[i][:] over the i
 * with tokens[i] == r: the tokens are sorted (stably), each row's terms are
 * added in fp32 in an order that depends on the tokens alone, multiplied, added
 * to the old value (accumulate) and rounded once.  Without accumulate every row
 * is written (zeros where no token points); with it only rows that tokens point
 * to are touched.
 *   grad_out: n_tokens x dim of grad_dtype, rows grad_stride (>= dim) apart.
 *   grad_weight: vocab x dim of weight_dtype, rows weight_stride apart.
 *   padding_idx: a token whose gradient is dropped (its row gets zeros, or with
 *            accumulate keeps its value); negative: none.
 *   workspace: 16-byte aligned, at least ..._workspace_bytes; free for other use
 *            once the stream has passed this call.
 * n_tokens < 2^31 - 16384, vocab < 2^31 - 1, dim <= 65535 * 32 (four times that where dim, the strides and
 * the pointers allow accesses of four elements).  A token outside [0, vocab) is dropped and sets bit 16 of the
 * device error word. */
fsp_status fsp_embedding_backward(const void* tokens, int32_t index_bytes, int64_t n_tokens, const void* grad_out,
                                  int32_t grad_dtype, int64_t dim, int64_t grad_stride, void* grad_weight,
                                  int32_t weight_dtype, int64_t vocab, int64_t weight_stride, float scale,
                                  int64_t padding_idx, int32_t accumulate, void* workspace, size_t workspace_bytes,
                                  void* cuda_stream);

/* ---- matrices in 8-bit floating point, a scale per block of 128 ----------------- */

/* A matrix of `rows` x `cols` values whose rows are cut into blocks of 128 (the
 * last one filled up with zeros): code e4m3(x / s), round to nearest even, with
 * s = 2^e the smallest power of two for which 448 s >= max|x| of the block (e in
 * [-127, 127]); a block that holds a NaN or an infinity stands for NaN.
 * Layout, in the order the tensor cores read it: the codes as tiles of 128 rows
 * x 128 columns, 16 KB each, tile (i, j) at ((i * ceil(cols / 128)) + j) * 16384,
 * row r of a tile at r * 128 with its 16-byte pieces p at p ^ (r % 8); then, from scale_offset, 512-byte pieces of scale exponents
 * (e + 127, 255 for NaN) for 128 rows x 4 blocks, piece (i, j) at
 * (i * ceil(cols / 512) + j) * 512, row r's block k (mod 4) at
 * (r % 32) * 16 + (r / 32) * 4 + k.  Rows past the matrix (and blocks past the
 * last one in a piece) hold nothing that anything depends on. */
fsp_status fsp_fp8_bytes(int64_t rows, int64_t cols, size_t* bytes, size_t* scale_offset);

/* Writes x (rows x cols of dtype, rows `stride` elements apart) as such a matrix
 * (out) and / or its transpose, cols x rows with blocks along the rows of x
 * (out_t); either may be NULL, not both.  Outputs 16-byte aligned. */
fsp_status fsp_fp8_quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t stride, void* out,
                            void* out_t, void* cuda_stream);

/* The values such a matrix stands for, as fp32 rows x cols (contiguous). */
fsp_status fsp_fp8_values(const void* q, int64_t rows, int64_t cols, float* out, void* cuda_stream);

/* c[m][n] = (accumulate: +) sum over k of a[m][k] b[n][k]: a is m x k, b is
 * n x k, both laid out as above; summed in fp32, rounded once.
 *   c: m x n of dtype (fp32 or bf16; accumulate: fp32 only), rows c_stride
 *   (>= n) elements apart. */
fsp_status fsp_fp8_matmul(const void* a, const void* b, int64_t m, int64_t n, int64_t k, void* c, int32_t dtype,
                          int64_t c_stride, int32_t accumulate, void* cuda_stream);

/* A linear layer's forward pass on 8-bit operands: y = q(x) w^T, with x (rows x
 * in_features of x_dtype, rows x_stride apart) quantised along its rows here and
 * w (out_features x in_features) as fsp_fp8_quantize's `out` laid it out.
 *   y: rows x out_features of y_dtype, rows y_stride apart.
 *   workspace: 16-byte aligned, at least fsp_fp8_linear_workspace_bytes (NULL
 *   where that is 0: up to four rows are quantised on chip). */
fsp_status fsp_fp8_linear(const void* x, int32_t x_dtype, int64_t rows, int64_t in_features, int64_t x_stride,
                          const void* w, int64_t out_features, void* y, int32_t y_dtype, int64_t y_stride,
                          void* workspace, size_t workspace_bytes, void* cuda_stream);

/* Its gradients: grad_x = q(grad_y) wt^T (NULL: not wanted), wt being w's
 * transpose as `out_t` laid it out, and grad_w (+)= q(grad_y^T) q(x^T)^T (fp32;
 * NULL: not wanted; accumulate: added to it).  x and wt are read only where
 * grad_w and grad_x are wanted. */
fsp_status fsp_fp8_linear_backward(const void* x, int32_t x_dtype, int64_t x_stride, const void* grad_y,
                                   int32_t grad_y_dtype, int64_t grad_y_stride, int64_t rows, int64_t in_features,
                                   int64_t out_features, const void* wt, void* grad_x, int32_t grad_x_dtype,
                                   int64_t grad_x_stride, float* grad_w, int64_t grad_w_stride, int32_t accumulate,
                                   void* workspace, size_t workspace_bytes, void* cuda_stream);

/* Device workspace, in bytes, of fsp_fp8_linear (backward 0) and of
 * fsp_fp8_linear_backward (backward 1). */
fsp_status fsp_fp8_linear_workspace_bytes(int64_t rows, int64_t in_features, int64_t out_features, int32_t backward,
                                          size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* FSP_OPS_H */
