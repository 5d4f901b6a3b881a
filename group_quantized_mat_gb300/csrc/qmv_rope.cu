// qmv_rope_run: norms of each head's query and key, rotation by position, and the
// new keys and values put into a paged cache, in one pass.
//
// The mathematics: x' = x / sqrt(mean(x^2) + eps) * w over a head, then each pair
// (a, b) of its first elements turns by an angle position * frequency. Only the
// fraction of a turn matters, so a frequency is kept as a 64-bit fraction of a turn
// and the product with the position wraps around by itself: far positions lose
// nothing, and no 64-bit floating point is in the loop (152 SMs do it at two
// operations a cycle).
//
// A row (one head of one token) belongs to head_dim / 8 lanes of a warp, 16 bytes of
// bf16 each; its sum of squares joins by shuffles, and a pair's other element comes
// from the lane that holds it. A block takes tokens in turn: it computes the
// token's sines and cosines once, for all of its heads, while the rows' loads are in
// flight. It is bound by memory from a few hundred tokens on; below that by the
// latency of a launch, two loads and a store.
//
// A thread has four rows of a token in flight, or one where the tokens alone do not
// fill the SMs (see rope_rows_in_flight).
#include <cuda_bf16.h>

#include <cstdint>

#include "qmv.h"
#include "qmv_cache.h"
#include "qmv_launch.cuh"

namespace qmv {
namespace {

constexpr int kRopeThreads = 256;

struct RopeParams {
    const void *qkv;
    const uint16_t *q_norm, *k_norm;
    const int32_t *positions;
    const float *inv_freq;
    const uint8_t *axis;
    const int64_t *slots;
    uint16_t *q, *k_cache, *v_cache;
    int T, heads, kv_heads, rot, axes;
    int page_size;
    int64_t places;  // pages * page_size
    int64_t ld_qkv, page_stride, token_stride, head_stride;
    float eps, one;  // one: what is added to a norm's weights
    int neighbours;
};

__device__ __forceinline__ void widen(const uint4 &v, float (&x)[8])
{
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(in[i] << 16);
        x[2 * i + 1] = __uint_as_float(in[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 narrow(const float (&x)[8])
{
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        r[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// Eight elements as they lie in memory.
template <bool F32>
struct Octet {
    uint4 v[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *base, int64_t element)
    {
        const uint8_t *at = static_cast<const uint8_t *>(base) + element * (F32 ? 4 : 2);
        // (read once: not kept in L1)
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) v[i] = __ldcs(reinterpret_cast<const uint4 *>(at) + i);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const
    {
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[4 * i] = __uint_as_float(v[i].x);
                x[4 * i + 1] = __uint_as_float(v[i].y);
                x[4 * i + 2] = __uint_as_float(v[i].z);
                x[4 * i + 3] = __uint_as_float(v[i].w);
            }
        } else {
            widen(v[0], x);
        }
    }
};

template <int D, bool F32, int ROWS>
__global__ void __launch_bounds__(kRopeThreads) rope_rows(const RopeParams p)
{
    constexpr int kLanes = D / 8, kPass = kRopeThreads / kLanes;
    __shared__ uint64_t s_turn[D / 2];          // a pair's fraction of a turn for each position, times 2^64
    __shared__ uint8_t s_axis[D / 2];
    __shared__ float s_cos[2][D / 2], s_sin[2][D / 2];  // two tokens': one block-wide meeting for each is enough
    const int tid = threadIdx.x, li = tid % kLanes, half = p.rot / 2;
    const int rows = p.heads + 2 * p.kv_heads, row0 = int(blockIdx.y) * ROWS * kPass + tid / kLanes;
    grid_dependency_wait();
    for (int i = tid; i < half; i += kRopeThreads) {
        double f = double(__ldg(p.inv_freq + i)) * 0.15915494309189533577;  // 1 / (2 pi)
        f -= floor(f);
        s_turn[i] = __double2ull_rn(f * 18446744073709551616.0);
        s_axis[i] = uint8_t(p.axis ? min(int(__ldg(p.axis + i)), p.axes - 1) : 0);
    }
    __syncthreads();
    uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
    if (p.q_norm) wq = __ldg(reinterpret_cast<const uint4 *>(p.q_norm) + li);
    if (p.k_norm) wk = __ldg(reinterpret_cast<const uint4 *>(p.k_norm) + li);
    // halves: elements 8 li .. are all first or all second of their pairs, the others
    // of which lie rot / 16 lanes further or before
    const int lane = tid & 31, hl = p.rot / 16;
    const bool turns = li < 2 * hl, second = li >= hl;
    const int partner = p.neighbours || !turns ? lane : second ? lane - hl : lane + hl;

    for (int t = blockIdx.x, n = 0; t < p.T; t += gridDim.x, ++n) {
        Octet<F32> in[ROWS];
#pragma unroll
        for (int k = 0; k < ROWS; ++k)
            if (row0 + k * kPass < rows) in[k].load(p.qkv, t * p.ld_qkv + (int64_t)(row0 + k * kPass) * D + 8 * li);
        const int64_t slot = p.slots ? __ldg(p.slots + t) : -1;
        float *cs = s_cos[n & 1], *sn = s_sin[n & 1];
        for (int i = tid; i < half; i += kRopeThreads) {
            const int64_t pos = __ldg(p.positions + (int64_t)s_axis[i] * p.T + t);
            const int turn = int(uint32_t((uint64_t(pos) * s_turn[i]) >> 32));  // in 2^-32 of a turn, from -1/2 on
            sincospif(__fmul_rn(__int2float_rn(turn), 0x1p-31f), sn + i, cs + i);
        }
        __syncthreads();
        float c[8], s[8];
        if (turns) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = p.neighbours ? 4 * li + j / 2 : 8 * (second ? li - hl : li) + j;
                const bool b = p.neighbours ? j & 1 : second;
                c[j] = cs[i];
                s[j] = b ? sn[i] : -sn[i];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = 1.0f, s[j] = 0.0f;
        }
        const bool stored = slot >= 0 && slot < p.places;
        const int64_t place = stored ? slot / p.page_size * p.page_stride + slot % p.page_size * p.token_stride : 0;
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const int r = row0 + k * kPass, g = r - p.heads;
            // (every lane of a warp takes part in the shuffles)
            float x[8];
            if (r < rows)
                in[k].get(x);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = 0.0f;
            const bool value = g >= p.kv_heads;
            const uint16_t *norm = g < 0 ? p.q_norm : p.k_norm;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = __fmaf_rn(x[j], x[j], sum);
#pragma unroll
            for (int d = 1; d < kLanes; d *= 2) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, d));
            if (!value && norm) {
                float w[8];
                widen(g < 0 ? wq : wk, w);
                const float f = __fdiv_rn(1.0f, __fsqrt_rn(__fmaf_rn(sum, 1.0f / D, p.eps)));
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = __fmul_rn(__fmul_rn(x[j], f), __fadd_rn(w[j], p.one));
            }
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float other = p.neighbours ? x[j ^ 1] : __shfl_sync(0xffffffffu, x[j], partner);
                y[j] = value || !turns ? x[j] : __fmaf_rn(x[j], c[j], __fmul_rn(other, s[j]));
            }
            if (r >= rows) continue;
            const uint4 out = narrow(y);
            if (g < 0) {
                *reinterpret_cast<uint4 *>(p.q + ((int64_t)t * p.heads + r) * D + 8 * li) = out;
            } else if (stored) {
                uint16_t *cache = value ? p.v_cache : p.k_cache;
                *reinterpret_cast<uint4 *>(cache + place + (value ? g - p.kv_heads : g) * p.head_stride + 8 * li) = out;
            }
        }
    }
}

template <int D, bool F32, int ROWS>
cudaError_t launch_rope(const RopeParams &p, int sms, cudaStream_t stream)
{
    static std::atomic<int> configured[64] = {};
    const int rows = p.heads + 2 * p.kv_heads, block_rows = ROWS * kRopeThreads / (D / 8);
    const int y = (rows + block_rows - 1) / block_rows;
    const int fill = (4 * sms + y - 1) / y;  // four blocks for an SM
    Launch l;
    l.grid = dim3(unsigned(p.T < fill ? p.T : fill), unsigned(y));
    l.threads = kRopeThreads;
    l.smem = 0;
    l.pdl = true;
    return launch_one(rope_rows<D, F32, ROWS>, configured, l, stream, p);
}

template <int D, bool F32>
cudaError_t launch_rope_rows(const RopeParams &p, int sms, cudaStream_t stream)
{
    const int rows = p.heads + 2 * p.kv_heads, block_rows = 4 * kRopeThreads / (D / 8);
    // one row a thread while that leaves no SM with two blocks more than another's one
    if ((int64_t)p.T * ((rows + block_rows - 1) / block_rows) < sms) return launch_rope<D, F32, 1>(p, sms, stream);
    return launch_rope<D, F32, 4>(p, sms, stream);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace qmv

extern "C" qmv_status qmv_rope_run(const void *qkv, const uint16_t *q_norm, const uint16_t *k_norm,
                                   const int32_t *positions, const float *inv_freq, const uint8_t *axis,
                                   const int64_t *slots, uint16_t *q, uint16_t *k_cache, uint16_t *v_cache, int T,
                                   int heads, int kv_heads, int head_dim, int rope_dim, int page_size, int pages,
                                   int axes, float eps, int64_t ld_qkv, int64_t page_stride, int64_t token_stride,
                                   int64_t head_stride, unsigned flags, qmv_stream_t stream)
{
    using namespace qmv;
    if (!qkv || !q || (rope_dim != 0 && (!positions || !inv_freq)) || (slots && (!k_cache || !v_cache))) return QMV_ERR_NULL;
    qmv_status st = check_heads(T, heads, kv_heads, head_dim);
    if (st != QMV_OK) return st;
    if (axes < 1 || axes > QMV_MAX_AXES) return QMV_ERR_COUNT;
    if (rope_dim < 0 || rope_dim > head_dim || rope_dim % 16 != 0 || !(eps >= 0.0f) || eps > 3e38f) return QMV_ERR_SHAPE;
    const int64_t width = int64_t(heads + 2 * kv_heads) * head_dim;
    if (ld_qkv < width || ld_qkv % 8 != 0 || ld_qkv > (int64_t(1) << 38)) return QMV_ERR_SHAPE;
    if (slots) {
        st = check_cache({pages, page_size, kv_heads, head_dim, page_stride, token_stride, head_stride});
        if (st != QMV_OK) return st;
    }
    if (flags & ~(QMV_ROPE_F32_IN | QMV_ROPE_NEIGHBOURS | QMV_ROPE_NORM_PLUS_ONE)) return QMV_ERR_FLAGS;
    for (const void *ptr : {qkv, (const void *)q_norm, (const void *)k_norm, (const void *)q,
                            (const void *)(slots ? k_cache : nullptr), (const void *)(slots ? v_cache : nullptr)})
        if (!aligned(ptr, 16)) return QMV_ERR_ALIGN;
    if (!aligned(positions, 4) || !aligned(inv_freq, 4) || !aligned(slots, 8)) return QMV_ERR_ALIGN;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != QMV_OK) return st;

    RopeParams p{};
    p.qkv = qkv; p.q_norm = q_norm; p.k_norm = k_norm; p.positions = positions; p.inv_freq = inv_freq; p.axis = axis;
    p.slots = slots; p.q = q; p.k_cache = k_cache; p.v_cache = v_cache;
    p.T = T; p.heads = heads; p.kv_heads = kv_heads; p.rot = rope_dim; p.axes = axes;
    p.page_size = slots ? page_size : 1;
    p.places = slots ? int64_t(pages) * page_size : 0;
    p.ld_qkv = ld_qkv; p.page_stride = page_stride; p.token_stride = token_stride; p.head_stride = head_stride;
    p.eps = eps;
    p.one = flags & QMV_ROPE_NORM_PLUS_ONE ? 1.0f : 0.0f;
    p.neighbours = flags & QMV_ROPE_NEIGHBOURS ? 1 : 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool f32 = (flags & QMV_ROPE_F32_IN) != 0;
    cudaError_t e;
    if (head_dim == 64)
        e = f32 ? launch_rope_rows<64, true>(p, dev.sms, s) : launch_rope_rows<64, false>(p, dev.sms, s);
    else if (head_dim == 128)
        e = f32 ? launch_rope_rows<128, true>(p, dev.sms, s) : launch_rope_rows<128, false>(p, dev.sms, s);
    else
        e = f32 ? launch_rope_rows<256, true>(p, dev.sms, s) : launch_rope_rows<256, false>(p, dev.sms, s);
    return e == cudaSuccess ? QMV_OK : record_cuda_failure("rope kernel launch", e);
}
