// A paged cache of keys and values: its shape, where a row lies, and the checks
// that both of an attention layer's operators make of it. Host code without a CUDA
// call, so that it can be tested without a GPU.
#pragma once

#include <cstdint>

#include "qmv.h"

namespace qmv {

struct CacheShape {
    int pages, page_size, kv_heads, head_dim;
    int64_t page_stride, token_stride, head_stride;
};

// No two rows overlap: sorted by stride, each dimension steps over the whole of the one before.
inline bool rows_apart(const CacheShape &c)
{
    int64_t stride[3] = {c.head_stride, c.token_stride, c.page_stride};
    int64_t count[3] = {c.kv_heads, c.page_size, c.pages};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            // (of equal strides, the dimension of one entry first: it takes no step)
            if (stride[j] > stride[j + 1] || (stride[j] == stride[j + 1] && count[j] > count[j + 1])) {
                const int64_t s = stride[j], n = count[j];
                stride[j] = stride[j + 1], count[j] = count[j + 1];
                stride[j + 1] = s, count[j + 1] = n;
            }
    int64_t span = c.head_dim;
    for (int i = 0; i < 3; ++i) {
        if (count[i] == 1) continue;
        if (stride[i] < span) return false;
        span = stride[i] * (count[i] - 1) + span;
    }
    return true;
}

inline qmv_status check_heads(int T, int heads, int kv_heads, int head_dim)
{
    if (T < 1 || T > QMV_MAX_TOKENS || kv_heads < 1 || kv_heads > QMV_MAX_KV_HEADS || heads < kv_heads ||
        heads % kv_heads != 0 || heads / kv_heads > QMV_MAX_HEAD_GROUP ||
        int64_t(T) * (heads + 2 * kv_heads) >= int64_t(1) << 31)
        return QMV_ERR_COUNT;
    return head_dim == 64 || head_dim == 128 || head_dim == 256 ? QMV_OK : QMV_ERR_SHAPE;
}

inline qmv_status check_cache(const CacheShape &c)
{
    if (c.pages < 1 || c.page_size < 8 || c.page_size % 8 != 0 || c.page_size > 65536) return QMV_ERR_SHAPE;
    // a tensor map's strides stay below 2^40 bytes, and products of stride and count within 63 bits
    const int64_t most = int64_t(1) << 38;
    for (const int64_t s : {c.page_stride, c.token_stride, c.head_stride})
        if (s < c.head_dim || s % 8 != 0 || s > most) return QMV_ERR_SHAPE;
    if (c.page_stride > (int64_t(1) << 46) / c.pages) return QMV_ERR_SHAPE;
    return rows_apart(c) ? QMV_OK : QMV_ERR_SHAPE;
}

}  // namespace qmv
