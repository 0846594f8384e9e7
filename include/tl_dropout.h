/*
 * tl_dropout.h - C ABI of dropout whose mask is never stored.
 *
 *   y = residual + (kept ? x / (1 - p) : 0)        (without residual: 0)
 *
 * Whether element i (row-major: row * cols + column, whatever the strides) is kept
 * is a function of a key that the device reads, of a site and of i alone, so the
 * backward pass, a recomputed segment and a repeated micro-batch see the forward's
 * mask by naming the same key ("Practical LLM in Rust", chapter 13 "Accumulate
 * gradients and recompute activations": recomputation replays the dropout of its
 * ticket).  The gradient of x is the same call on the gradient of y without a
 * residual; that of the residual is the gradient of y itself.
 *
 * Random numbers.  Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random
 * numbers: as easy as 1, 2, 3", SC 2011) with key (seed mod 2^32, seed >> 32) and
 * counter (b mod 2^32, b >> 32 | (ticket >> 32) << 8, ticket mod 2^32, site) gives
 * eight 16-bit numbers for the elements 8 b .. 8 b + 7, the low half of each word
 * first.  An element is kept where its number is at least P = round(65536 p): p
 * is taken to the nearest multiple of 2^-16, and so is the divisor, 1 - P / 65536, so
 * that the mean is kept exactly.
 *
 * Numbers.  One multiply-add in fp32, rounded once to the tensors' type.  A dropped
 * element is 0 (the residual) whatever x holds, NaN included; p = 1 drops all.
 *
 * Memory.  The caller owns every tensor.  Rows are contiguous, row t starting at
 * element t * ld; any ld >= cols and any element-aligned address is accepted.
 * Where rows begin on 16-byte boundaries (fp32: 32-byte ones) and hold whole blocks
 * of 8 elements, or follow one another without gaps from such a boundary on,
 * accesses are vectors, and so they are for long 16-bit rows at one phase (address
 * modulo 16) in all operands; others are by elements.  y may be x's or the residual's own memory (same address
 * and ld).  Any other overlap of y with an argument is an error.
 *
 * The call is asynchronous on the given stream, keeps no state and no scratch, and
 * can be captured in a CUDA graph, which then reads the key anew in every replay.
 * Make one call with the operands' types and layout before the capture, so that its
 * kernel is loaded.  Status codes are those of tl.h: TL_EINVAL (arguments),
 * TL_ESTATE (another device is current), TL_ECUDA.  A call that returns TL_EINVAL or
 * TL_ESTATE has launched nothing.
 */
#ifndef TL_DROPOUT_H
#define TL_DROPOUT_H

#include "tl.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    const void* x;
    const void* residual;   /* NULL: none */
    void* y;
    int64_t rows, cols;     /* >= 0; rows * cols at most 2^40 */
    int64_t ldx, ldr, ldy;  /* elements, >= cols, < 2^40 where there are several rows (of one row not used) */
    const int64_t* key;     /* device: seed, ticket (0 .. 2^56 - 1) */
    uint32_t site;          /* which dropout of the model */
    int32_t dtype;          /* of x, residual and y: TL_F32, TL_BF16 or TL_F16 */
    float p;                /* 0 .. 1 */
    int32_t device;         /* that holds them; the current one */
} tl_dropout_args;

int tl_dropout(const tl_dropout_args* args, tl_stream stream);

/* The text of the calling thread's last call of tl_dropout that returned an error ("" before the first). */
const char* tl_dropout_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* TL_DROPOUT_H */
