// qmv_attend_run: attention of new tokens over a paged cache.
//
// The simplest kernel that is right: a warp for each query head of each new token,
// over the keys that it sees one after the other, with the running maximum and sum
// of a softmax. Every key is read once for each query head.
#include <cuda_bf16.h>

#include <cmath>
#include <cstdint>

#include "qmv.h"
#include "qmv_cache.h"
#include "qmv_launch.cuh"

namespace qmv {
namespace {

struct AttendParams {
    const uint16_t *q, *k, *v;
    const int32_t *table, *q_start, *kv_len;
    uint16_t *out;
    float *lse;
    int B, T, max_new, heads, group;
    int page_size, pages, max_pages;
    float scale;
    int window, sinks;
    int64_t ld_q, ld_out, page_stride, token_stride, head_stride;
};

// First row, new tokens and keys of a sequence.
struct Sequence {
    int row, n, keys;
    __device__ __forceinline__ Sequence(const AttendParams &p, int b)
    {
        row = p.q_start ? min(max(__ldg(p.q_start + b), 0), p.T) : b * p.max_new;
        n = p.q_start ? min(max(__ldg(p.q_start + b + 1), row), p.T) - row : p.max_new;
        keys = min(max(__ldg(p.kv_len + b), 0), p.max_pages * p.page_size);
    }
};

template <int D>
__global__ void __launch_bounds__(128) attend_simple(const AttendParams p)
{
    constexpr int E = D / 32;
    grid_dependency_wait();
    const int64_t unit = int64_t(blockIdx.x) * 4 + threadIdx.x / 32;
    const int lane = threadIdx.x & 31, t = int(unit / p.heads), h = int(unit % p.heads);
    if (t >= p.T) return;
    for (int b = 0; b < p.B; ++b) {
        const Sequence s(p, b);
        const int i = t - s.row;
        if (i < 0 || i >= s.n || i >= p.max_new) continue;
        const int pos = s.keys - s.n + i;
        float q[E], o[E], m = -INFINITY, l = 0.0f;
        for (int e = 0; e < E; ++e) {
            q[e] = __fmul_rn(bf16_bits_to_f32(p.q[t * p.ld_q + h * D + lane + 32 * e]), p.scale);
            o[e] = 0.0f;
        }
        const int low = p.window ? max(pos - p.window + 1, 0) : 0;
        for (int j = p.window && p.sinks > 0 ? 0 : low; j <= pos; ++j) {
            if (j < low && j >= p.sinks) j = low;
            const int page = __ldg(p.table + int64_t(b) * p.max_pages + j / p.page_size);
            if (page < 0 || page >= p.pages) continue;
            const int64_t at = page * p.page_stride + j % p.page_size * p.token_stride + h / p.group * p.head_stride + lane;
            float dot = 0.0f;
            for (int e = 0; e < E; ++e) dot = __fmaf_rn(q[e], bf16_bits_to_f32(p.k[at + 32 * e]), dot);
            for (int d = 16; d > 0; d /= 2) dot = __fadd_rn(dot, __shfl_xor_sync(0xffffffffu, dot, d));
            const float top = fmaxf(m, dot);
            const float keep = top == -INFINITY ? 1.0f : expf(m - top), w = top == -INFINITY ? 0.0f : expf(dot - top);
            m = top;
            l = __fmaf_rn(l, keep, w);
            for (int e = 0; e < E; ++e) o[e] = __fmaf_rn(o[e], keep, __fmul_rn(w, bf16_bits_to_f32(p.v[at + 32 * e])));
        }
        for (int e = 0; e < E; ++e) {
            const float y = l == 0.0f ? 0.0f : __fdiv_rn(o[e], l);
            reinterpret_cast<__nv_bfloat16 *>(p.out)[t * p.ld_out + h * D + lane + 32 * e] = __float2bfloat16_rn(y);
        }
        if (p.lse && lane == 0) p.lse[int64_t(t) * p.heads + h] = l == 0.0f ? -INFINITY : __fadd_rn(m, logf(l));
    }
}

template <int D>
cudaError_t launch_attend(const AttendParams &p, cudaStream_t stream)
{
    static std::atomic<int> configured[64] = {};
    Launch l;
    l.grid = dim3(unsigned((int64_t(p.T) * p.heads + 3) / 4));
    l.threads = 128;
    l.smem = 0;
    l.pdl = true;
    return launch_one(attend_simple<D>, configured, l, stream, p);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

qmv_status check_attend(int B, int T, int max_new, int heads, int kv_heads, int head_dim, int page_size, int max_pages, int window, int sinks)
{
    const qmv_status st = check_heads(T, heads, kv_heads, head_dim);
    if (st != QMV_OK) return st;
    if (B < 1 || B > QMV_MAX_SEQUENCES || max_new < 1 || max_new > T) return QMV_ERR_COUNT;
    if (page_size < 8 || page_size % 8 != 0 || page_size > 65536 || max_pages < 1 || int64_t(max_pages) * page_size > (1 << 26) ||
        window < 0 || window > (1 << 30) || sinks < 0 || sinks > (1 << 30))
        return QMV_ERR_SHAPE;
    return QMV_OK;
}

}  // namespace
}  // namespace qmv

extern "C" size_t qmv_attend_workspace_size(int B, int T, int max_new, int heads, int kv_heads, int head_dim, int page_size,
                                            int max_pages, int window, int sinks)
{
    if (qmv::check_attend(B, T, max_new, heads, kv_heads, head_dim, page_size, max_pages, window, sinks) != QMV_OK) return 0;
    return 16;
}

extern "C" qmv_status qmv_attend_run(const uint16_t *q, const uint16_t *k_cache, const uint16_t *v_cache,
                                     const int32_t *page_table, const int32_t *q_start, const int32_t *kv_len,
                                     uint16_t *out, float *lse, int B, int T, int max_new, int heads, int kv_heads,
                                     int head_dim, int page_size, int pages, int max_pages, float scale, int window,
                                     int sinks, int64_t ld_q, int64_t ld_out, int64_t page_stride, int64_t token_stride,
                                     int64_t head_stride, void *workspace, size_t workspace_bytes, unsigned flags,
                                     qmv_stream_t stream)
{
    using namespace qmv;
    if (!q || !k_cache || !v_cache || !page_table || !kv_len || !out) return QMV_ERR_NULL;
    qmv_status st = check_attend(B, T, max_new, heads, kv_heads, head_dim, page_size, max_pages, window, sinks);
    if (st != QMV_OK) return st;
    if (!q_start && int64_t(B) * max_new != T) return QMV_ERR_COUNT;
    st = check_cache({pages, page_size, kv_heads, head_dim, page_stride, token_stride, head_stride});
    if (st != QMV_OK) return st;
    const int64_t width = int64_t(heads) * head_dim, most = int64_t(1) << 38;
    if (!std::isfinite(scale) || ld_q < width || ld_q % 8 != 0 || ld_q > most || ld_out < width || ld_out % 8 != 0 || ld_out > most)
        return QMV_ERR_SHAPE;
    if (flags) return QMV_ERR_FLAGS;
    for (const void *ptr : {(const void *)q, (const void *)k_cache, (const void *)v_cache, (const void *)out, (const void *)workspace})
        if (!aligned(ptr, 16)) return QMV_ERR_ALIGN;
    for (const void *ptr : {(const void *)page_table, (const void *)q_start, (const void *)kv_len, (const void *)lse})
        if (!aligned(ptr, 4)) return QMV_ERR_ALIGN;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != QMV_OK) return st;
    void *ws = nullptr;
    st = scratch(dev, qmv_attend_workspace_size(B, T, max_new, heads, kv_heads, head_dim, page_size, max_pages, window, sinks),
                 workspace, workspace_bytes, &ws);
    if (st != QMV_OK) return st;

    AttendParams p{};
    p.q = q; p.k = k_cache; p.v = v_cache; p.table = page_table; p.q_start = q_start; p.kv_len = kv_len;
    p.out = out; p.lse = lse;
    p.B = B; p.T = T; p.max_new = max_new; p.heads = heads; p.group = heads / kv_heads;
    p.page_size = page_size; p.pages = pages; p.max_pages = max_pages;
    p.scale = scale; p.window = window; p.sinks = sinks;
    p.ld_q = ld_q; p.ld_out = ld_out;
    p.page_stride = page_stride; p.token_stride = token_stride; p.head_stride = head_stride;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = head_dim == 64 ? launch_attend<64>(p, s) : head_dim == 128 ? launch_attend<128>(p, s) : launch_attend<256>(p, s);
    return e == cudaSuccess ? QMV_OK : record_cuda_failure("attention kernel launch", e);
}
