/*
 * ss_block.h -- the operators of libss in front of the output head of ss.h:
 * dropout from a counter-based generator, and the gated feed-forward block
 * whose output (plus the residual) is the head's H. Forward and backward, as
 * hand-written CUDA for GB300 (sm_103a).
 *
 * The conventions of ss.h hold here too: device pointers on the current CUDA
 * device, buffers owned by the caller, row-major dense matrices, bf16 passed
 * as uint16_t bit patterns, work enqueued asynchronously on `stream`, argument
 * errors returned before anything is enqueued, no C++ exception across this
 * boundary. No call here synchronises or allocates; every call may be captured
 * into a CUDA graph.
 */
#ifndef SS_BLOCK_H_
#define SS_BLOCK_H_

#include "ss.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SS_MAX_F 65536 /* largest inner width of the feed-forward block */

typedef enum ss_dtype { SS_BF16 = 0, SS_FP32 = 1 } ss_dtype;

/* act(g) of the gated block. SS_ACT_GELU is g Phi(g) with the normal
 * distribution's Phi; SS_ACT_GELU_TANH its usual tanh form
 * g/2 (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))). */
typedef enum ss_act {
  SS_ACT_SILU = 0,
  SS_ACT_GELU = 1,
  SS_ACT_GELU_TANH = 2,
  SS_ACT_RELU = 3
} ss_act;

/*
 * Dropout from a counter-based generator: no mask is stored, the backward
 * makes the same one again from the same fields. Element i of a call is
 * element e = offset + i of the stream; its 32 random bits are half of
 * SplitMix64 output number e >> 1 (Steele, Lea and Flood, OOPSLA 2014; the
 * generator of ss_build_candidates) of the stream seeded with `seed`: the low
 * half where e is even, the high half where e is odd. The element is dropped
 * where its bits are below floor(p 2^32); what is kept is multiplied by
 * 1 / (1 - p) in fp32. A dropped element is 0 whatever x holds there (also
 * infinities and NaN). p = 0 keeps everything, p = 1 drops everything.
 *   p        : in [0, 1]; else SS_ERR_INVALID.
 *   seed     : any. Output k of seed s is output k - 1 of seed
 *              s + 0x9E3779B97F4A7C15: take seeds that do not differ by small
 *              multiples of that constant (consecutive integers are fine).
 *   seed_dev : NULL, or a device word (8-byte aligned) that is added to `seed`
 *              when the kernel runs, so that a captured graph can draw a new
 *              mask at every replay.
 *   offset   : first element of the stream; a tensor processed in pieces gets
 *              the whole tensor's mask when each piece passes its position.
 * A NULL pointer to this struct means p = 0.
 */
typedef struct ss_dropout_spec {
  double p;
  uint64_t seed;
  const uint64_t* seed_dev;
  uint64_t offset;
} ss_dropout_spec;

/*
 * y[i] = residual[i] + (kept ? x[i] / (1 - p) : 0), computed in fp32 and
 * rounded once.
 *   x, y [n] of `dtype` (ss_dtype); residual [n] or NULL (no addend).
 *   y may be x or residual; otherwise the buffers must not overlap.
 *   Pointers need the alignment of their element only (16-byte aligned
 *   pointers run faster).
 * 0 <= n < 2^62. n = 0: nothing is enqueued.
 */
ss_status ss_dropout(const void* x, const void* residual, int64_t n, int dtype,
                     const ss_dropout_spec* drop, void* y, ss_stream stream);

/*
 * The gradient of ss_dropout with respect to x: dx[i] = kept ? dy[i] / (1 - p)
 * : 0 (dx may be dy). The gradient of the residual is dy itself.
 */
ss_status ss_dropout_backward(const void* dy, int64_t n, int dtype, const ss_dropout_spec* drop,
                              void* dx, ss_stream stream);

/*
 * The gated feed-forward block. With Wg, Wu [F, D] and Wd [D, F] (as linear
 * layers hold them):
 *   G = X Wg^T   U = X Wu^T   A = act(G) U   Z = A Wd^T
 *   Y = residual + dropout(Z)
 * Both projections, the activation and the product are one kernel; the down
 * projection, dropout (element t * D + d of the stream, plus drop->offset) and
 * the residual another.
 *
 * Limits: 0 <= T < 2^31; D % 8 == 0, 8 <= D <= SS_MAX_D; F % 8 == 0,
 * 8 <= F <= SS_MAX_F (else SS_ERR_UNSUPPORTED, or SS_ERR_INVALID for values
 * that can never be valid). Every tensor 16-byte aligned.
 *
 * Workspace: ss_ffn_workspace_size bytes, 16-byte aligned, its first 1024
 * bytes (the header of ss.h, with the status word) zero when new. One
 * workspace serves the forward and the backward of a block, in any order, and
 * any smaller T; calls that may run at the same time need one each (two
 * captured graphs that are replayed at the same time too). A device wait that
 * timed out is recorded in the status word (ss_read_status); what that call
 * wrote is unspecified. Later calls on the workspace then do nothing until its
 * header is zeroed (an empty batch's zeroes are written all the same).
 */
size_t ss_ffn_workspace_size(int64_t T, int64_t D, int64_t F); /* 0: invalid sizes */

/*
 *   X [T, D], Wg, Wu [F, D], Wd [D, F] bf16; residual [T, D] bf16 or NULL.
 *   Y [T, D] bf16 out (may be `residual`; else no output may overlap an input
 *   or another output).
 *   G, U, A [T, F] bf16 out: what the backward needs; all three, or all NULL
 *   (no backward follows). A is rounded to bf16 before the down projection,
 *   from G and U in fp32.
 *   R [T, ss_ffn_low_bits_pitch(F)] bytes out, 32-byte aligned, or NULL: the
 *   next four bits of G and of U for the backward, which make the error that
 *   stems from their rounding to bf16 a sixteenth (only with G, U and A). What
 *   lies past column F of a row is unspecified.
 * Sums are held in fp32. T = 0: nothing is enqueued.
 */
ss_status ss_ffn_forward(const uint16_t* X, const uint16_t* Wg, const uint16_t* Wu,
                         const uint16_t* Wd, const uint16_t* residual, int64_t T, int64_t D,
                         int64_t F, int act, const ss_dropout_spec* drop, uint16_t* Y, uint16_t* G,
                         uint16_t* U, uint16_t* A, uint8_t* R, void* workspace,
                         size_t workspace_bytes, ss_stream stream);
int64_t ss_ffn_low_bits_pitch(int64_t F); /* F rounded up to 64; 0 if F <= 0 */

/*
 * From dY [T, D] and the forward's G, U, A (and R, or NULL: G and U as they are):
 *   dZ = dropout'(dY)   dA = dZ Wd   dG = dA U act'(G)   dU = dA act(G)
 *   dX = dG Wg + dU Wu  dWg = dG^T X  dWu = dU^T X  dWd = dZ^T A
 * (the gradient of the residual is dY itself; relu'(0) = 0).
 *   dX [T, D] bf16 out; dWg, dWu [F, D], dWd [D, F] of dw_dtype (ss_dtype).
 *   accumulate: 0 -> the weight gradients are overwritten; 1 -> added to.
 * dG and dU are rounded to bf16 for the products that follow (as dA U act'(G)
 * and dA act(G) in fp32); sums are held in fp32. The same drop fields as in
 * the forward. The outputs must not overlap the inputs or one another.
 * T = 0: the weight gradients are zeroed unless accumulate.
 */
ss_status ss_ffn_backward(const uint16_t* dY, const uint16_t* X, const uint16_t* Wg,
                          const uint16_t* Wu, const uint16_t* Wd, const uint16_t* G,
                          const uint16_t* U, const uint16_t* A, const uint8_t* R, int64_t T,
                          int64_t D, int64_t F, int act, const ss_dropout_spec* drop, int dw_dtype,
                          int accumulate,
                          uint16_t* dX, void* dWg, void* dWu, void* dWd, void* workspace,
                          size_t workspace_bytes, ss_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* SS_BLOCK_H_ */
