// Cross attention: what its kernels share.
//
// For each batch entry and query head, with the keys that take part (index below k_len, key_mask not 0)
//   S = scale q k^T,  P = softmax of S over these keys,  out = P v,  lse = log sum exp S;
// a row without such a key has out = 0 and lse = -inf. Backward, with delta = sum(dout out) per query:
//   dS = scale P (dout v^T - delta),  dq = dS k,  dk = dS^T q,  dv = P^T dout,
// dk and dv summed over the query heads that share a key head.
#pragma once

#include "elem.cuh"
#include "gs_common.cuh"
#include "gs_internal.h"

namespace gs {

__device__ __forceinline__ bool key_valid(const AttnArgs& a, int b, int key, int len) {
    return key < len && (!a.key_mask || a.key_mask[b * a.mask_stride + key] != 0);
}

// Keys of batch entry b below its valid length.
__device__ __forceinline__ int key_count(const AttnArgs& a, int b) {
    return a.k_len ? max(0, min(a.k_len[b], a.len_k)) : a.len_k;
}

template <class T>
__device__ __forceinline__ const T* head_base(const AttnTensor& t, int b, int h) {
    return static_cast<const T*>(t.data) + b * t.batch_stride + h * t.head_stride;
}

}  // namespace gs
