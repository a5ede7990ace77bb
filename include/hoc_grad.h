/*
 * hoc_grad.h -- what a data-parallel step does with its gradients once they
 * are reduced (HOCCL section 2.1: DP gradient buckets): the global norm over
 * many tensors, and clipping by it.
 */
#ifndef HOC_GRAD_H
#define HOC_GRAD_H

#include <stddef.h>
#include <stdint.h>

#include "hoc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A list of device tensors of one dtype (HOC_FLOAT32 or HOC_BFLOAT16), kept
 * as a table in device memory so that a call does not pass thousands of
 * pointers again.  ptr[i] and count[i] (elements, 0 allowed) are host arrays
 * read during the call.  Any element alignment; tensors of one list must not
 * overlap.  Creation allocates device memory on the current device and waits
 * for the upload; the tensors stay the caller's.  A list is used with the device
 * current on which it was made (HOC_ERR_INVALID_ARG otherwise). */
typedef struct hocTensorList hocTensorList_t;
hocResult_t hoc_tensor_list_create(hocTensorList_t** list, int n, const void* const* ptr, const size_t* count,
                                   hocDataType_t dtype);
hocResult_t hoc_tensor_list_destroy(hocTensorList_t* list);

/* int32 entries of the workspace the two calls below need for this list.  A
 * workspace needs no initial value; calls that run at the same time need one
 * each. */
hocResult_t hoc_grad_workspace(const hocTensorList_t* list, size_t* ints);

/* norm[0] (device binary32) = sqrt of the sum of squares over all tensors.
 * Squares are binary32, summed in binary32 within a tile of at most 8192
 * elements and in binary64 across tiles, in an order that depends only on the
 * list: the same list and values give the same bits.  A square above
 * the binary32 range makes the norm inf, a NaN makes it NaN; 0 for no elements. */
hocResult_t hoc_grad_norm(const hocTensorList_t* src, float* norm, int32_t* workspace, size_t workspace_ints, void* stream);

/* norm as above, then dst = c * src with c = min(1, max_norm / (norm + 1e-6))
 * in binary32, one rounding to the dtype (NaN if the norm is NaN).  max_norm
 * points to one host float >= 0, read during the call.  dst has
 * the counts and the dtype of src and may be src itself (in place); other
 * overlaps are not allowed.  In place with c == 1 nothing is written. */
hocResult_t hoc_grad_clip(const hocTensorList_t* src, const hocTensorList_t* dst, const float* max_norm, float* norm,
                          int32_t* workspace, size_t workspace_ints, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HOC_GRAD_H */
