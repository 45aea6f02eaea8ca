/*
 * swiglu_probe.h -- diagnostics of libswiglu: kernels that measure what this
 * device actually sustains, for reading the fused kernel's roofline fraction
 * against more than the datasheet (the datasheet peaks assume the top clock
 * and ideal memory), and the plans of the training calls.  Not part of the
 * fused product.
 *
 * Same conventions as swiglu.h: device pointers, `stream` is a hipStream_t
 * (NULL = default), calls enqueue and return, errors are swiglu_status codes.
 */
#ifndef SWIGLU_PROBE_H_
#define SWIGLU_PROBE_H_

#include <stddef.h>
#include <stdint.h>

#include "swiglu.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Matrix-core ceiling: `blocks` workgroups of 256 threads each run `iters`
 * iterations of 8 independent v_mfma_f32_32x32x16_bf16 per wave on register
 * operands (no memory traffic).  Flops = blocks * 4 waves * iters * 8 * 32768.
 * `sink` (device, >= blocks * 256 floats) receives the accumulators so the
 * work cannot be elided.  blocks >= 1, iters >= 1. */
swiglu_status swiglu_probe_mfma(float *sink, int blocks, int iters, void *stream);

/* HBM read ceiling: streams `bytes` (multiple of 16, >= 16) from `src` with
 * 16-byte loads, grid-stride, and writes one 32-bit checksum per thread to
 * `sink` (device, >= blocks * 256 uint32).  blocks >= 1. */
swiglu_status swiglu_probe_read(const void *src, size_t bytes, uint32_t *sink, int blocks,
                                void *stream);

/* Host call, no launch: how a launch of the training calls is cut into work items at
 * (M,K,N) on the current device.  `launch` is one of swiglu_train_launch; plan
 * receives, for each of its one or two products, the tile's rows and columns
 * (dual products: of both halves), the tiles run whole, the others, the parts
 * each of these is split into over the contraction, and a part's 64-deep blocks.
 * Returns the number of products, 0 for an invalid shape (or M == 0) or launch. */
typedef enum {
    SWIGLU_TRAIN_FORWARD = 0,    /* Y, G, U */
    SWIGLU_TRAIN_RECOMPUTED = 1, /* dG, dU from Gate and Up computed again */
    SWIGLU_TRAIN_DY = 2,         /* dG, dU from dY = dZ W3^T (no weight gradients) */
    SWIGLU_TRAIN_DY_DW3 = 3,     /* the same, and dW3 */
    SWIGLU_TRAIN_DA = 4,
    SWIGLU_TRAIN_DW = 5,         /* dW1 | dW2 */
    SWIGLU_TRAIN_DA_DW = 6,
    SWIGLU_TRAIN_LAUNCHES = 7
} swiglu_train_launch;
int swiglu_probe_train_plan(int launch, int64_t M, int64_t K, int64_t N, int32_t plan[12]);

#ifdef __cplusplus
}
#endif

#endif /* SWIGLU_PROBE_H_ */
