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

// End of the positions [v0, v1), counted along the list, after the entries
// without a page at their end are left out.  All lanes of a warp together;
// v0 is a multiple of 16.
__device__ __forceinline__ int list_end(const DecodeParams& p, const int32_t* list, int v0, int v1) {
    const int lane = threadIdx.x & 31;
    const int e0 = v0 / p.page_size, e1 = min(p.n_listed, (v1 + p.page_size - 1) / p.page_size);
    int last = -1;
    for (int e = e0; e < e1; e += 32) {
        const unsigned some = __ballot_sync(0xffffffffu, e + lane < e1 && list[e + lane] >= 0);
        if (some) last = e + 31 - __clz(some);
    }
    return last < 0 ? v0 : min(v1, (last + 1) * p.page_size);
}

}  // namespace fa512
