/*
 * fa_rotary.h -- queries and keys on their way into the attention of fa.h:
 * an optional root-mean-square norm of each head and the rotary position, in
 * one pass over q and k, forward and backward.
 *
 * For a head row x of d elements at position p:
 *
 *     y = x / sqrt(mean_j x_j^2 + eps) * w           (norm = 1; else y = x)
 *     a' = s (a cos(p f_i) - b sin(p f_i))           pair i of y, i < r / 2
 *     b' = s (b cos(p f_i) + a sin(p f_i))
 *
 * with r = rotary_dim <= d, f_i = freqs[i] and s = rotary_scale. Pair i is
 * (y_i, y_{i + r/2}), or (y_{2i}, y_{2i+1}) with interleaved = 1; elements
 * r .. d-1 are not turned (and not scaled by s). Arithmetic is fp32, rounded
 * once to bf16 (mean x^2 too: the norm wants rows of an rms below 2^59, and above
 * 2^-59 where eps does not outweigh it). The angle is formed in 64-bit
 * fixed-point fractions of a turn from f_i / 2 pi in fp64: for frequencies up to 1
 * it is off by 2^-24 turns at most at any 32-bit position. Frequencies are finite.
 *
 * Conventions are those of fa.h (device pointers owned by the caller, status
 * codes, errors reported before any CUDA call, asynchronous calls,
 * deterministic results, sm_100 only), with these differences:
 *   - Tensors are views: element (b, h, n, j) of a bf16 [B, heads, N, d]
 *     tensor lies at b * stride_b + h * stride_h + n * stride_n + j elements
 *     from its pointer. Strides are multiples of 8 and >= 0, pointers 16-byte
 *     aligned, so the views of a fused projection's output are read in place.
 *   - An output may be its own input (same pointer and strides): each row is
 *     then replaced. Other overlaps of an output with an input or another
 *     output return FA_ERR_INVALID_ARG, except heads of one token-major
 *     buffer that do not meet (the q and k views of a fused projection).
 *   - The kernels hold no bounded waits: the device status word of
 *     fa_last_device_error is neither read nor written.
 *   - d is 64, 128 or 256 (else FA_ERR_UNSUPPORTED). rotary_dim is a multiple
 *     of 16 in [0, d] (0: the norm alone, freqs may be NULL, positions may
 *     not: they are read all the same); norm_eps is finite and >= 0;
 *     rotary_scale is finite.
 *   - Rows may be given any position, negative ones too.
 */
#ifndef FA_ROTARY_H_
#define FA_ROTARY_H_

#include <stddef.h>
#include <stdint.h>

#include "fa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A bf16 [B, heads, N, d] view; strides in elements, d contiguous. */
typedef struct {
    void *ptr;
    int64_t stride_b, stride_h, stride_n;
} fa_heads_t;

typedef struct {
    const double *freqs;      /* device, rotary_dim / 2: radians per position */
    const void *q_weight;     /* device, d norm weights, or NULL for ones */
    const void *k_weight;
    int32_t rotary_dim;
    int32_t interleaved;      /* 0: pairs (i, i + r/2); 1: pairs (2i, 2i + 1) */
    int32_t norm;             /* 1: norm each head first */
    int32_t weight_f32;       /* weights are fp32 (1) or bf16 (0) */
    float rotary_scale;       /* multiplies cos and sin; 1 where nothing asks otherwise */
    float norm_eps;
} fa_rotary_t;

typedef struct {
    fa_heads_t q, k;          /* in: H and H_kv heads */
    fa_heads_t q_out, k_out;  /* out */
    const int32_t *positions; /* device int32, position of token (b, n) at */
    int64_t pos_stride_b;     /*   b * pos_stride_b + n * pos_stride_n */
    int64_t pos_stride_n;     /*   (0 repeats) */
    fa_rotary_t rotary;
    int32_t B, H, H_kv, N, d, reserved;
} fa_qk_rotary_t;

/* Forward. H need not be a multiple of H_kv; either may be 0. */
int fa_qk_rotary(const fa_qk_rotary_t *args, void *stream);

typedef struct {
    fa_heads_t dq_out, dk_out; /* in: gradients of the outputs */
    fa_heads_t q, k;           /* in: the forward's inputs (norm = 1 only; else unread) */
    fa_heads_t dq, dk;         /* out: gradients of the inputs; may replace dq_out, dk_out */
    const int32_t *positions;
    int64_t pos_stride_b, pos_stride_n;
    fa_rotary_t rotary;        /* as in the forward */
    float *dq_weight;          /* out, fp32 [d] each: gradients of the weights, summed */
    float *dk_weight;          /*   over batch, heads and tokens; norm = 1 only, else NULL */
    int32_t B, H, H_kv, N, d, reserved;
} fa_qk_rotary_bwd_t;

/*
 * Backward: with g the output gradient turned back by the same angles (and
 * scaled by s) and n = x / sqrt(mean x^2 + eps),
 *     dw = sum g * n,     dx = (g w - n mean(g w n)) / sqrt(mean x^2 + eps)
 * (norm = 0: dx = g). Sums are fp32 per thread block and fp64 across blocks,
 * in a fixed order. workspace: device memory owned by the caller, 16-byte
 * aligned, at least fa_qk_rotary_bwd_workspace_bytes(...) bytes, overlapping
 * no other argument, with no initialisation; scratch after the call. It may
 * be NULL where that size is 0.
 */
int fa_qk_rotary_bwd(const fa_qk_rotary_bwd_t *args, void *workspace, size_t workspace_bytes,
                     void *stream);

/* Workspace bytes of fa_qk_rotary_bwd (0 without the norm, or if invalid). */
size_t fa_qk_rotary_bwd_workspace_bytes(int B, int H, int H_kv, int N, int d, int norm);

#ifdef __cplusplus
}
#endif

#endif /* FA_ROTARY_H_ */
