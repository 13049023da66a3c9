// Lists of selected pages, shared by the decode kernels.
#pragma once

#include "fa512_device.cuh"
#include "fa512_internal.h"

namespace fa512 {

// The list of (sequence b, KV head kvh).
__device__ __forceinline__ const int32_t* list_of(const DecodeParams& p, int b, int kvh) {
    return p.listed + (static_cast<size_t>(b) * p.n_kv_heads + kvh) * p.n_listed;
}

// Logical page of entry e; -1 for an entry that names none.  `held`: pages of
// the sequence.  A list that does not rise breaks the order between two
// neighbours somewhere, so looking at the entry before is enough to record it;
// the entry that breaks it is skipped.
__device__ __forceinline__ int list_page(const DecodeParams& p, const int32_t* list, int e, int held) {
    const int page = list[e], before = e > 0 ? list[e - 1] : -1;
    if (page < 0) return -1;
    if (page >= held || (e > 0 && page <= before) || (e > 0 && before < 0)) {
        report_error(p.err, FA512_DEVICE_ERR_INDEX);
        return -1;
    }
    return page;
}

}  // namespace fa512
