/*
 * hoc_layer.h -- the matrix products that run between the collectives: the
 * products of an expert layer on the rows an expert-parallel dispatch
 * delivered (HOCCL section 2.1: EP token dispatch and combine surround them),
 * grouped by expert with ragged row counts that only the device knows, and a
 * dense linear layer on the same kernels.  Both have their epilogue fused
 * (bias, activation, residual) and both have their gradients.
 *
 * Conventions, beside those of hoc.h:
 *   - Matrices are row-major bf16 (HOC_BFLOAT16) unless stated; products
 *     accumulate in binary32 and are rounded once, when they are stored.
 *   - A weight has shape [experts, out, in] (linear layer: [out, in]).  With
 *     HOC_ACT_SWIGLU its `out` rows of gates come first and the `out` rows of
 *     linear values after them: [experts, 2 * out, in].
 *   - `status` is a device int32; bit 2 (value 4) is set, never cleared, if a
 *     wait inside a kernel gave up after 2 s in which nothing moved (the results are
 *     then undefined).
 *   - Everything is stream-ordered, never waits on the host and may be captured
 *     into a CUDA graph after one call of the same kind.
 *   - Rows of x, dy and the weights that start on 16-byte boundaries (widths and
 *     strides that are multiples of 8, aligned pointers) run as they lie, with
 *     no memory beside the arguments'.  For other rows, products above a small
 *     size copy the operands into scratch that the call allocates and frees in
 *     stream order from a memory pool of this library's own, which keeps what it
 *     was given until hoc_layer_trim; where no scratch is to be had a slower
 *     kernel runs.
 *   - Inputs must not overlap outputs, except as stated.
 */
#ifndef HOC_LAYER_H
#define HOC_LAYER_H

#include <stddef.h>
#include <stdint.h>

#include "hoc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations.  GELU is the tanh form 0.5 z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3)));
 * SILU z / (1 + exp(-z)); SWIGLU silu(gate) * value.  A gradient through RELU is
 * 0 where its input is not above 0, also where dy is infinite or NaN. */
typedef enum {
  HOC_ACT_NONE = 0,
  HOC_ACT_RELU = 1,
  HOC_ACT_GELU = 2,
  HOC_ACT_SILU = 3,
  HOC_ACT_SWIGLU = 4
} hocAct_t;

/* Where each expert's rows lie.  Rank buffer d (0 <= d < nranks, at most
 * HOC_MAX_RANKS) holds `capacity[d]` rows (host array, read during the call)
 * and belongs to `experts` experts; the rows of its expert e that came from
 * source s are the rows seg[d][s * experts + e] .. seg[d][s * experts + e + 1),
 * seg being a device array [nranks][sources * experts + 1] of int64.  This is
 * the layout hoc_ep_dispatch_fused (and hoc_ep_pack + the all-to-all) writes,
 * with the offsets hoc_ep_segments computes; sources = 1 is a buffer sorted
 * by expert.  Ranges are read on the device: a range is cut to
 * [0, capacity[d]), and one that ends before it starts is empty. */
typedef struct {
  int nranks;
  int experts; /* of one rank */
  int sources;
  const int64_t* seg;
  const size_t* capacity;
} hocRowGroups_t;

/* Row ranges of the receive layout of a dispatch: expert_ids[s] as in
 * hoc_ep_dispatch_fused ([tokens * topk] int32 of source rank s; ids outside
 * [0, experts) are dropped pairs), experts over all ranks (a multiple of
 * nranks).  Writes seg, device [nranks][nranks * (experts / nranks) + 1]. */
hocResult_t hoc_ep_segments(int nranks, const int32_t* const* expert_ids, int tokens, int topk, int experts,
                            int64_t* seg, void* stream);

/* Forward product of every rank's experts: for every row r of expert e of rank d
 *   z = W[d][e] x[d][r] + bias[d][e];   y[d][r] = act(z);   pre[d][r] = z
 * x[d]: [capacity[d], in]; weight[d]: [experts, out or 2 out, in]; bias (NULL:
 * none): bias[d] [experts, out or 2 out]; y[d]: [capacity[d], out]; pre (NULL:
 * not wanted): pre[d] [capacity[d], out or 2 out], z rounded to bf16, which
 * the gradients need.  Rows in no range are not written.  Buffers of a rank
 * with capacity 0 may be NULL. */
hocResult_t hoc_expert_mm(const hocRowGroups_t* groups, const void* const* x, const void* const* weight,
                          const void* const* bias, int in, int out, int act, void* const* y, void* const* pre,
                          int32_t* status, void* stream);

/* Gradient for the inputs: dx[d][r] = W[d][e]^T dy[d][r], weight[d] being
 * [experts, out, in] and dy[d] [capacity[d], out].  With act != HOC_ACT_NONE
 * the layer's input came out of that activation, pre[d] is what went into it,
 * and the gradient for pre is written instead: dx * act'(pre), [capacity[d],
 * in] (SWIGLU: pre and dx are [capacity[d], 2 * in], gates first). */
hocResult_t hoc_expert_mm_dgrad(const hocRowGroups_t* groups, const void* const* dy, const void* const* weight,
                                int in, int out, int act, const void* const* pre, void* const* dx, int32_t* status,
                                void* stream);

/* Gradient for the weights and biases:
 *   dw[d][e] = sum over the expert's rows of dy[r]^T x[r]   [experts, out, in]
 *   db[d][e] = sum over the expert's rows of dy[r]          [experts, out]  (db NULL: not wanted)
 * dtype: HOC_BFLOAT16 or HOC_FLOAT32, the type of dw and db.  accumulate != 0
 * adds to what dw and db hold (binary32 addition, one rounding); otherwise
 * they are written, zeros for an expert without rows. */
hocResult_t hoc_expert_mm_wgrad(const hocRowGroups_t* groups, const void* const* dy, const void* const* x, int in,
                                int out, hocDataType_t dtype, int accumulate, void* const* dw, void* const* db,
                                int32_t* status, void* stream);

/* Linear layer: y = act(x W^T + bias) + residual for `rows` rows.  Row strides
 * in elements (ldx >= in, ldy >= out, ldr >= out); weight [out or 2 out, in];
 * bias [out or 2 out], residual [rows, out] (its row stride ldr) and pre
 * [rows, out or 2 out] may be NULL.  residual may be y itself. */
hocResult_t hoc_linear(int rows, const void* x, size_t ldx, const void* weight, const void* bias,
                       const void* residual, size_t ldr, int in, int out, int act, void* y, size_t ldy, void* pre,
                       int32_t* status, void* stream);

/* dx = dy W (through act'(pre) as in hoc_expert_mm_dgrad); dy [rows, out] with
 * row stride lddy, dx and pre contiguous. */
hocResult_t hoc_linear_dgrad(int rows, const void* dy, size_t lddy, const void* weight, int in, int out, int act,
                             const void* pre, void* dx, int32_t* status, void* stream);

/* dw = dy^T x [out, in] and db = column sums of dy [out] (NULL: not wanted). */
hocResult_t hoc_linear_wgrad(int rows, const void* dy, size_t lddy, const void* x, size_t ldx, int in, int out,
                             hocDataType_t dtype, int accumulate, void* dw, void* db, int32_t* status, void* stream);

/* dz = dy * act'(pre) for `rows` rows of `width` outputs: dy [rows, width];
 * pre and dz [rows, width or 2 width].  dz may be pre itself, or dy itself
 * (not with SWIGLU). */
hocResult_t hoc_act_grad(int rows, int width, int act, const void* dy, const void* pre, void* dz, void* stream);

/* Gives scratch of the current device that no call uses any more back to the
 * device, all but `keep` bytes of it.  Calls still under way on a stream keep
 * theirs: wait for the stream first.  Nothing is given back without this call. */
hocResult_t hoc_layer_trim(size_t keep);

#ifdef __cplusplus
}
#endif

#endif /* HOC_LAYER_H */
