// kv4_abi.cu -- the C ABI of the 4-bit paged KV cache (declared in include/bitnet.h):
// argument validation and launch.
#include <math.h>

#include "host.h"

namespace bitnet {

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 30;
constexpr int kMaxHeads = 1 << 15;
constexpr int kMaxBatch = 1 << 15;

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bitnet_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? BITNET_OK : BITNET_ERR_CUDA; }

bool valid_dt(bitnet_dtype_t dt) { return dt == BITNET_F32 || dt == BITNET_BF16; }

bitnet_status_t shape_of(const bitnet_kv4_cache_t *c, Kv4Cache *o) {
    if (!c) return BITNET_ERR_INVALID_ARG;
    if (c->dim != 64 && c->dim != 128 && c->dim != 256) return BITNET_ERR_UNSUPPORTED_SHAPE;
    int log2 = 0;
    while ((1 << log2) < c->page_size && log2 < 8) ++log2;
    if (log2 < 4 || (1 << log2) != c->page_size) return BITNET_ERR_UNSUPPORTED_SHAPE;
    if (c->heads < 1 || c->heads > kMaxHeads) return BITNET_ERR_UNSUPPORTED_SHAPE;
    if (c->pages < 0 || c->pages > INT32_MAX) return BITNET_ERR_INVALID_ARG;
    if (c->pages * c->heads >= (((int64_t)1 << 32) - 64) >> log2) return BITNET_ERR_UNSUPPORTED_SHAPE;  // rows are counted in 32 bits
    *o = Kv4Cache{c->k_codes, c->v_codes, c->k_step, c->v_step, c->k_bos, c->v_bos, (int)c->pages, c->heads, log2,
                  c->dim};
    return BITNET_OK;
}

bitnet_status_t arrays_of(const bitnet_kv4_cache_t *c, const bitnet_kv4_batch_t *b, Kv4Batch *o) {
    const void *p[6] = {c->k_codes, c->v_codes, c->k_step, c->v_step, c->k_bos, c->v_bos};
    for (const void *x : p)
        if (c->pages > 0 && (!x || !aligned(x, 16))) return BITNET_ERR_INVALID_ARG;
    if (!b->kv_lens || !b->q_starts || (b->max_pages > 0 && !b->block_table)) return BITNET_ERR_INVALID_ARG;
    if (!aligned(b->kv_lens, 4) || !aligned(b->q_starts, 4) || !aligned(b->block_table, 4)) return BITNET_ERR_INVALID_ARG;
    *o = Kv4Batch{b->block_table, b->kv_lens, b->q_starts, b->table_stride, b->batch, b->max_pages};
    return BITNET_OK;
}

// Sizes of the batch; *empty where the call has no rows at all.
bitnet_status_t sizes_of(const bitnet_kv4_batch_t *b, int64_t T, bool *empty) {
    if (!b || T < 0 || T > kMaxTokens) return BITNET_ERR_INVALID_ARG;
    if (b->batch < 0 || b->batch > kMaxBatch || b->max_pages < 0 || b->table_stride < b->max_pages)
        return BITNET_ERR_INVALID_ARG;
    *empty = T == 0 || b->batch == 0;
    return BITNET_OK;
}

// Row starts of a strided [T][heads][dim] tensor must be 16-byte aligned and not lie before its first.
bool valid_rows(const void *p, bitnet_dtype_t dt, int64_t token_stride, int64_t head_stride) {
    const int64_t unit = dt == BITNET_BF16 ? 8 : 4;
    const int64_t most = (int64_t)1 << 32;
    return p && aligned(p, 16) && token_stride >= 0 && head_stride >= 0 && token_stride <= most && head_stride <= most &&
           token_stride % unit == 0 && head_stride % unit == 0;
}

}  // namespace

}  // namespace bitnet

using namespace bitnet;

extern "C" {

bitnet_status_t bitnet_kv4_write(const void *k, const void *v, bitnet_dtype_t dt, int64_t T, int64_t k_token_stride,
                                 int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                                 const bitnet_kv4_cache_t *cache, const bitnet_kv4_batch_t *batch, int bits, float eps,
                                 void *stream) {
    if (!valid_dt(dt) || (bits != 3 && bits != 4) || !(eps > 0.0f) || isinf(eps)) return BITNET_ERR_INVALID_ARG;
    Kv4Cache c;
    Kv4Batch b;
    bool empty;
    bitnet_status_t st = shape_of(cache, &c);
    if (st == BITNET_OK) st = sizes_of(batch, T, &empty);
    if (st != BITNET_OK || empty) return st;
    if ((st = arrays_of(cache, batch, &b)) != BITNET_OK) return st;
    if (!valid_rows(k, dt, k_token_stride, k_head_stride) || !valid_rows(v, dt, v_token_stride, v_head_stride))
        return BITNET_ERR_INVALID_ARG;
    return from_cuda(launch_kv4_write(k, v, dt == BITNET_BF16, T, k_token_stride, k_head_stride, v_token_stride,
                                      v_head_stride, c, b, bits, eps, static_cast<cudaStream_t>(stream)));
}

bitnet_status_t bitnet_kv4_read(const bitnet_kv4_cache_t *cache, const bitnet_kv4_batch_t *batch, int64_t T,
                                void *k_out, void *v_out, bitnet_dtype_t dt, void *stream) {
    if (!valid_dt(dt)) return BITNET_ERR_INVALID_ARG;
    Kv4Cache c;
    Kv4Batch b;
    bool empty;
    bitnet_status_t st = shape_of(cache, &c);
    if (st == BITNET_OK) st = sizes_of(batch, T, &empty);
    if (st != BITNET_OK || empty || (!k_out && !v_out)) return st;
    if ((st = arrays_of(cache, batch, &b)) != BITNET_OK) return st;
    if (!aligned(k_out, 16) || !aligned(v_out, 16)) return BITNET_ERR_INVALID_ARG;
    return from_cuda(launch_kv4_read(c, b, T, k_out, v_out, dt == BITNET_BF16, static_cast<cudaStream_t>(stream)));
}

size_t bitnet_kv4_attention_workspace_bytes(int64_t T, int64_t q_heads, int64_t heads, int64_t dim, int64_t batch) {
    if (T <= 0 || T > kMaxTokens || heads < 1 || heads > kMaxHeads || q_heads < heads || q_heads > kMaxHeads ||
        q_heads % heads != 0 || T * q_heads > INT32_MAX || (dim != 64 && dim != 128 && dim != 256) || batch < 1 || batch > kMaxBatch)
        return 0;
    return kv4_attention_workspace(T, (int)q_heads, (int)heads, (int)dim, (int)batch);
}

bitnet_status_t bitnet_kv4_attention(const void *q, bitnet_dtype_t dt, int64_t T, int64_t q_heads,
                                     int64_t q_token_stride, int64_t q_head_stride, const bitnet_kv4_cache_t *cache,
                                     const bitnet_kv4_batch_t *batch, float scale, int causal, int64_t window,
                                     int64_t max_q, void *out, float *lse, void *ws, size_t ws_bytes, void *stream) {
    if (!valid_dt(dt) || !isfinite(scale) || (causal != 0 && causal != 1) || window < 0 || (window > 0 && !causal) ||
        max_q < 0)
        return BITNET_ERR_INVALID_ARG;
    Kv4Cache c;
    Kv4Batch b;
    bool empty;
    bitnet_status_t st = shape_of(cache, &c);
    if (st == BITNET_OK) st = sizes_of(batch, T, &empty);
    if (st != BITNET_OK) return st;
    if (q_heads < c.heads || q_heads > kMaxHeads || q_heads % c.heads != 0 || T * q_heads > INT32_MAX)
        return BITNET_ERR_UNSUPPORTED_SHAPE;
    if (empty) return BITNET_OK;
    if ((st = arrays_of(cache, batch, &b)) != BITNET_OK) return st;
    if (!valid_rows(q, dt, q_token_stride, q_head_stride) || !out || !aligned(out, 16) || !aligned(lse, 4))
        return BITNET_ERR_INVALID_ARG;
    if (!ws || !aligned(ws, 256) || ws_bytes < kv4_attention_workspace(T, (int)q_heads, c.heads, c.dim, b.batch))
        return BITNET_ERR_WORKSPACE;
    return from_cuda(launch_kv4_attention(q, dt == BITNET_BF16, T, (int)q_heads, q_token_stride, q_head_stride, c, b,
                                          scale, causal != 0, window, max_q, out, lse, ws,
                                          static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
