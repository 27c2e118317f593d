// kv4.cuh -- the 4-bit paged KV cache as its kernels see it.
#pragma once

#include "common.cuh"
#include "host.h"

namespace bitnet {

// Weights are held up to 2^14; sums of weights times values stand over that, so that they pass fp32's range
// no sooner than with weights up to 1.
constexpr float kSumUnit = 0x1p14f;

// Records a status (the first one stays) in the device status word.
__device__ __forceinline__ void record_status(int *status, int code) {
    if (status) atomicCAS(status, 0, code);
}

// Offset of the rows of (page, head) in units of rows: row r of it is at (this + r).
__device__ __forceinline__ int64_t kv4_rows(const Kv4Cache &c, int page, int head) {
    return ((int64_t)page * c.heads + head) << c.page_log2;
}

// The page that holds position pos >= 0 of sequence b, or -1 (and a status) where the
// table has none.
__device__ __forceinline__ int kv4_page(const Kv4Cache &c, const Kv4Batch &bt, int b, int pos, int *status) {
    const int i = pos >> c.page_log2;
    int page = -1;
    if (i < bt.max_pages) page = __ldg(bt.table + (int64_t)b * bt.table_stride + i);
    if ((unsigned)page >= (unsigned)c.pages) {
        record_status(status, (int)BITNET_ERR_INVALID_ARG);
        page = -1;
    }
    return page;
}

// Sequence and position of token row t; false where the row belongs to no sequence.
// The sequence is the last b with q_starts[b] <= t.
__device__ __forceinline__ bool kv4_locate(const Kv4Batch &bt, int t, int &b, int &pos) {
    if (t < __ldg(bt.starts) || t >= __ldg(bt.starts + bt.batch)) return false;
    int lo = 0, hi = bt.batch;  // starts[lo] <= t < starts[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(bt.starts + mid) <= t) lo = mid;
        else hi = mid;
    }
    b = lo;
    pos = __ldg(bt.lens + lo) - (__ldg(bt.starts + lo + 1) - t);
    return true;
}

}  // namespace bitnet
