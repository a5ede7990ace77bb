/*
 * hoc_block.h -- what stands between the residual stream and an expert-parallel
 * dispatch (HOCCL section 2.1: EP token dispatch and combine surround the
 * experts), and back: the root-mean-square norm with the residual's addition,
 * rows of 8 bits that an exchange moves in half the bytes, the routing of tokens
 * to experts, dropout, and the gradients of them all.
 *
 * Conventions, beside those of hoc.h:
 *   - Rows are matrices of HOC_BFLOAT16 or HOC_FLOAT32 with a row stride in
 *     elements; sums, statistics and scores are binary32 or wider, each result is
 *     rounded once, when it is stored.
 *   - Everything is stream-ordered, never waits on the host, allocates nothing
 *     and may be captured into a CUDA graph after one call of the same kind.
 *     Results are the same bits every time.  Pointers belong to the current device.
 *   - eps, scale and p point to one host number each, read during the call.
 *   - Any alignment to the element is taken; rows that start on 16-byte boundaries
 *     (and are whole 16-byte vectors) run faster.
 *   - Inputs must not overlap outputs, except as stated.  rows == 0 or
 *     tokens == 0 does nothing (a weight gradient is still written).
 */
#ifndef HOC_BLOCK_H
#define HOC_BLOCK_H

#include <stddef.h>
#include <stdint.h>

#include "hoc.h"
#include "hoc_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The widest row and the most experts of the calls below. */
#define HOC_NORM_MAX_WIDTH 32768
#define HOC_ROUTE_MAX_EXPERTS 1024
#define HOC_ROUTE_MAX_TOPK 31

/* A row of 8 bits, as it goes through an exchange: `width` values in e4m3, from
 * the next multiple of 16 bytes on (*scales_at) one binary32 scale for each 128
 * of them (the last group may be shorter), and up to a multiple of 16 bytes in
 * all (*bytes).  A value stands for q * scale.  A dispatch moves such rows as
 * rows of *bytes / 2 bf16 elements. */
hocResult_t hoc_wire8_row(int width, size_t* bytes, size_t* scales_at);

/* For each of `rows` rows of `width` values
 *   h = x + residual, rounded to dtype;   y = h / sqrt(mean(h^2) + eps) * weight
 * x, residual, h and y are of `dtype`; weight [width] of `weight_dtype`
 * (HOC_BFLOAT16 or HOC_FLOAT32).  residual NULL: h is x and is not stored (h must
 * be NULL); otherwise h may be NULL where it is not wanted.  y is stored in
 * dtype (NULL: not wanted) and in rows of 8 bits to wire ([rows][bytes of
 * hoc_wire8_row], aligned to 16 bytes; NULL: not wanted); one of the two is
 * given.  Those are of y before it is rounded: a group's scale is
 * max(max|y| / 448, 2^-100), its values the binary32 quotients y / scale rounded to
 * the nearest even (a NaN stays one and takes no part in the scale; an infinite y
 * makes its whole group NaN); bytes of a row that hold neither are not written.
 * Squares are binary32: a row whose squares add up to more than that holds gives
 * zeros.  h may be x or residual, and y may be x or, where h is not stored there,
 * residual, each with the same row stride. */
hocResult_t hoc_rms_norm(int rows, int width, hocDataType_t dtype, const void* x, size_t ldx, const void* residual,
                         size_t ldr, const void* weight, hocDataType_t weight_dtype, const float* eps, void* h, size_t ldh,
                         void* y, size_t ldy, void* wire, void* stream);

/* int32 entries of the workspace hoc_rms_norm_grad needs where dw is wanted.  It
 * needs no initial value; calls that run at the same time need one each. */
hocResult_t hoc_rms_norm_workspace(int rows, int width, size_t* ints);

/* Gradients of y = h / sqrt(mean(h^2) + eps) * weight where dy (+ dy2, if it is
 * given: a norm whose output went two ways) is the gradient for y, and dres (NULL:
 * none) one that came to h itself, down the residual stream:
 *   d = dy + dy2;   s = 1 / sqrt(mean(h^2) + eps)
 *   dx = s (d weight - h s^2 mean(d weight h)) + dres     for h, and so for x and the residual
 *   dw (+)= sum over the rows of d h s
 * Rows are of dtype.  dw [width] (NULL: not wanted, and no workspace) is of
 * dw_dtype (HOC_BFLOAT16 or HOC_FLOAT32); accumulate != 0 adds to what it holds
 * (binary32 addition, one rounding).  dx may be dy, dy2, h or dres, with the same
 * row stride. */
hocResult_t hoc_rms_norm_grad(int rows, int width, hocDataType_t dtype, const void* dy, size_t lddy, const void* dy2,
                              size_t lddy2, const void* h, size_t ldh, const void* weight, hocDataType_t weight_dtype,
                              const float* eps, const void* dres, size_t lddres, void* dx, size_t lddx, void* dw,
                              hocDataType_t dw_dtype, int accumulate, int32_t* workspace, size_t workspace_ints,
                              void* stream);

/* Rows of 8 bits that an exchange delivered, widened for the experts' products:
 * y[d][r] = bf16(q * scale) for the rows r of rank buffer d that groups->seg
 * covers, 0 .. seg[d][sources * experts] (cut to [0, capacity[d]]), wire[d]
 * being [capacity[d]][bytes of hoc_wire8_row], aligned to 16 bytes, and y[d]
 * [capacity[d], width] bf16.  Rows behind them are left as they were.  Buffers
 * of a rank with capacity 0 may be NULL.  counts (NULL: none): the device [nranks *
 * nranks] element counts that the dispatch of these rows wrote, in elements of its
 * rows (*bytes / 2 each), which become counts in elements of y, as a combine of
 * rows of `width` takes them. */
hocResult_t hoc_expert_widen(const hocRowGroups_t* groups, const void* const* wire, int width, void* const* y,
                             uint64_t* counts, void* stream);

/* Scores of the experts. */
typedef enum { HOC_SCORE_SOFTMAX = 0, HOC_SCORE_SIGMOID = 1 } hocScore_t;

/* Routing of `tokens` tokens to topk of `experts` experts each; topk is at most
 * HOC_ROUTE_MAX_TOPK and the experts of top_groups groups, groups divides experts and
 * is at most 32.  logits: [tokens,
 * experts] of dtype, row stride ldl; with the score s of an expert (softmax over the
 * token's experts, or sigmoid)
 *   key  = s + bias            bias: [experts] binary32 (NULL: none), for the choice only
 *   groups > 1: the experts form that many groups of neighbours; the top_groups
 *          groups are kept whose two largest keys have the largest sum (of equal
 *          ones the first; a group's only key counts alone)
 *   ids  = the topk largest keys of the kept groups, largest first, of equal ones
 *          the lowest expert        [tokens * topk] int32
 *   gate = scale * s, or with renormalise != 0 scale * s / sum of the chosen s   [tokens * topk] binary32
 * which is what hoc_ep_dispatch_fused and its kin take.  Keys are compared as 64-bit
 * arithmetic has them, without a bias and left-out groups as the logits are.  An
 * expert whose logit is -inf or NaN is masked out: it has no share of a softmax and is
 * never chosen, and neither is one whose bias makes its key -inf or NaN.  Where fewer
 * than topk are left, the last slots get id -1, which a dispatch drops, and gate 0.  A
 * logit of +inf takes a softmax's whole, several of them equal parts. */
hocResult_t hoc_ep_route(int tokens, int experts, int topk, const void* logits, hocDataType_t dtype, size_t ldl,
                         int score, const float* bias, int groups, int top_groups, int renormalise, const float* scale,
                         int32_t* ids, float* gate, void* stream);

/* Gradient for the logits, [tokens, experts] of dtype with row stride ldd, where
 * dgate [tokens * topk] binary32 is that for the gates and logits, ids, score,
 * renormalise and scale are those of the routing; the choice itself has none.  Slots
 * whose id is outside [0, experts), or that of a masked expert, add nothing; masked
 * logits get 0.  dlogits may be logits, with the same row stride. */
hocResult_t hoc_ep_route_grad(int tokens, int experts, int topk, const void* logits, hocDataType_t dtype, size_t ldl,
                              int score, int renormalise, const float* scale, const int32_t* ids, const float* dgate,
                              void* dlogits, size_t ldd, void* stream);

/* y = residual + x * 65536 / (65536 - t) where the element is kept, residual (NULL:
 * 0) where it is dropped, for `rows` rows of `width` values of dtype; t = p * 65536
 * rounded to the nearest (at most 65535; 0 <= p < 1), so that an element is dropped
 * with probability t / 65536.  Nothing of the mask is stored: element i = row *
 * width + column is dropped where its 16 random bits are below t, which are those of
 * Philox4x32-10 (Salmon, Moraes, Dror, Shaw: Parallel random numbers: as easy as 1,
 * 2, 3; 2011) under the key seed[0] for the counter (i / 8, seed[1]), 64 bits each,
 * low word first: word (i % 8) / 2, its low half for even i.  seed: two int64 on the
 * device, read when the call runs (a graph that is replayed draws anew once
 * seed[1] is changed).  The gradient is the same call on the gradient, without a
 * residual.  y may be x or residual, with the same row stride.  p == 0 draws nothing.  There may be
 * 2^31 rows and more (almost 2^43 elements): a run of n elements is n rows of width 1. */
hocResult_t hoc_dropout(size_t rows, int width, hocDataType_t dtype, const void* x, size_t ldx, const void* residual,
                        size_t ldr, const double* p, const int64_t* seed, void* y, size_t ldy, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HOC_BLOCK_H */
