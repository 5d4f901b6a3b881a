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
// A row (one head of one token) belongs to head_dim / 8 lanes of a warp, each with both
// elements of four pairs; its sum of squares joins by shuffles. A block takes tokens in
// turn: it computes the token's sines and cosines once, for all of its heads, while the
// next token's loads are in flight. Everything that depends on the head alone (its place, what
// is done with it, its norm's weights) stands before the loop over tokens.
//
// What bounds it: memory from a few thousand tokens on (16384 tokens of 40 + 16 heads of 128: 82
// us, 86 % of the rate of a copy, from fp32 112 us, 94 %; before rows' places left the loop the instructions did, at
// three a cycle), below that the latency of a launch, two loads and a store (one token: 2.1 us
// in a graph, 6.5 with the host's call; 1155 tokens with three axes: 8.0 us, the bytes 3.6).
//
// A thread has four rows of a token in flight (two of fp32), or one where the tokens alone do
// not fill the SMs (see launch_rope_rows).
#include <cuda_bf16.h>

#include <cstdint>

#include "qmv.h"
#include "qmv_cache.h"
#include "qmv_launch.cuh"

namespace qmv {
namespace {

constexpr int kRopeThreads = 256, kRopeBlocks = 3;  // blocks of an SM

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

__device__ __forceinline__ void widen(const uint2 &v, float *x)
{
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xffff0000u);
}

__device__ __forceinline__ uint2 narrow(const float *x)
{
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// A lane's eight elements as they lie in memory: four from `e0` on, four from `e1` on.
template <bool F32>
struct Octet {
    uint2 v[F32 ? 4 : 2];
    __device__ __forceinline__ void load(const void *base, int64_t row, int e0, int e1)
    {
        // (read once: not kept in L1)
        if constexpr (F32) {
            const float *at = static_cast<const float *>(base) + row;
            const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(at + e0)), b = __ldcs(reinterpret_cast<const uint4 *>(at + e1));
            v[0] = make_uint2(a.x, a.y);
            v[1] = make_uint2(a.z, a.w);
            v[2] = make_uint2(b.x, b.y);
            v[3] = make_uint2(b.z, b.w);
        } else {
            const uint16_t *at = static_cast<const uint16_t *>(base) + row;
            v[0] = __ldcs(reinterpret_cast<const uint2 *>(at + e0));
            v[1] = __ldcs(reinterpret_cast<const uint2 *>(at + e1));
        }
    }
    __device__ __forceinline__ void get(float (&x)[8]) const
    {
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(v[i].x);
                x[2 * i + 1] = __uint_as_float(v[i].y);
            }
        } else {
            widen(v[0], x);
            widen(v[1], x + 4);
        }
    }
};

template <int D, bool F32, bool NEIGHBOURS, int ROWS>
__global__ void __launch_bounds__(kRopeThreads, ROWS > 1 ? kRopeBlocks : 1) rope_rows(const RopeParams p)
{
    constexpr int kLanes = D / 8, kPass = kRopeThreads / kLanes;
    __shared__ uint64_t s_turn[D / 2];          // a pair's fraction of a turn for each position, times 2^64
    __shared__ uint8_t s_axis[D / 2];
    __shared__ float s_cos[2][D / 2], s_sin[2][D / 2];  // two tokens': one block-wide meeting for each is enough
    __shared__ __align__(16) float s_weight[2][D];
    __shared__ int64_t s_place[2];                      // where the cache takes them, or -1
    const int tid = threadIdx.x, li = tid % kLanes, half = p.rot / 2;
    const int rows = p.heads + 2 * p.kv_heads, row0 = int(blockIdx.y) * ROWS * kPass + tid / kLanes;
    grid_dependency_wait();
    if (tid < half) {  // (at most 128 pairs)
        double f = double(__ldg(p.inv_freq + tid)) * 0.15915494309189533577;  // 1 / (2 pi)
        f -= floor(f);
        s_turn[tid] = __double2ull_rn(f * 18446744073709551616.0);
        s_axis[tid] = uint8_t(p.axis ? min(int(__ldg(p.axis + tid)), p.axes - 1) : 0);
    }
    // norm weights as they are multiplied with, a lane's eight together
    for (int i = tid; i < D; i += kRopeThreads) {
        const int l = i / 8, j = i % 8, e = !NEIGHBOURS && l < p.rot / 8 ? (j < 4 ? 4 * l + j : half + 4 * l + j - 4) : i;
        s_weight[0][i] = p.q_norm ? __fadd_rn(bf16_bits_to_f32(__ldg(p.q_norm + e)), p.one) : 1.0f;
        s_weight[1][i] = p.k_norm ? __fadd_rn(bf16_bits_to_f32(__ldg(p.k_norm + e)), p.one) : 1.0f;
    }
    // of halves a lane has four pairs' first elements and their second ones, else eight in a row
    const bool turns = li < p.rot / 8, halves = !NEIGHBOURS && turns;
    const int e0 = halves ? 4 * li : 8 * li, e1 = halves ? half + 4 * li : 8 * li + 4;
    // a row's place beside that of its token, and what is done with it: a query, a key or a value
    int64_t to[ROWS];
    uint32_t kinds = 0;  // two bits each: 0 query, 1 key, 2 value, 3 no row
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        const int r = row0 + k * kPass, g = r - p.heads;
        const uint32_t kind = r >= rows ? 3u : g < 0 ? 0u : g < p.kv_heads ? 1u : 2u;
        kinds |= kind << 2 * k;
        to[k] = kind == 0 ? int64_t(r) * D : (kind == 2 ? g - p.kv_heads : g) * p.head_stride;
    }
    const uint8_t *from = static_cast<const uint8_t *>(p.qkv) + int64_t(row0) * D * (F32 ? 4 : 2);
    // the next token's rows, place and position are on their way while a token is worked on
    Octet<F32> ahead[ROWS];
    int64_t slot_ahead = -1;
    int pos_ahead = 0;
    const auto fetch = [&](int t) {
        if (t >= p.T) return;
#pragma unroll
        for (int k = 0; k < ROWS; ++k)
            if ((kinds >> 2 * k & 3) != 3) ahead[k].load(from + t * p.ld_qkv * (F32 ? 4 : 2), k * kPass * D, e0, e1);
        if (tid == kRopeThreads - 1) slot_ahead = p.slots ? __ldg(p.slots + t) : -1;
        if (tid < half) pos_ahead = __ldg(p.positions + (int64_t)s_axis[tid] * p.T + t);
    };
    fetch(blockIdx.x);  // (a thread reads the axis that it wrote)
    // the lanes of a row, which go one way at each branch on its kind
    const uint32_t row_lanes = (kLanes == 32 ? 0xffffffffu : (1u << kLanes) - 1u) << (tid & 31 & ~(kLanes - 1));
    const uint32_t normed = (p.q_norm ? 1u : 0u) | (p.k_norm ? 2u : 0u);
    for (int t = blockIdx.x, n = 0; t < p.T; t += gridDim.x, ++n) {
        Octet<F32> in[ROWS];
#pragma unroll
        for (int k = 0; k < ROWS; ++k) in[k] = ahead[k];
        float *cs = s_cos[n & 1], *sn = s_sin[n & 1];
        if (tid < half) {
            const int turn = int(uint32_t((uint64_t(int64_t(pos_ahead)) * s_turn[tid]) >> 32));  // in 2^-32 of a turn, from -1/2 on
            sincospif(__fmul_rn(__int2float_rn(turn), 0x1p-31f), sn + tid, cs + tid);
        }
        if (tid == kRopeThreads - 1) {
            const int64_t slot = slot_ahead;
            s_place[n & 1] = slot >= 0 && slot < p.places ? slot / p.page_size * p.page_stride + slot % p.page_size * p.token_stride : -1;
        }
        fetch(t + gridDim.x);
        __syncthreads();
        float c[4], s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            c[j] = turns ? cs[4 * li + j] : 1.0f;
            s[j] = turns ? sn[4 * li + j] : 0.0f;
        }
        const int64_t place = s_place[n & 1], token = int64_t(t) * p.heads * D;
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const uint32_t kind = kinds >> 2 * k & 3;
            float x[8];
            in[k].get(x);
            if (kind < 2) {
                // (a row without a norm is multiplied with 1 twice)
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) sum = __fmaf_rn(x[j], x[j], sum);
#pragma unroll
                for (int d = 1; d < kLanes; d *= 2) sum = __fadd_rn(sum, __shfl_xor_sync(row_lanes, sum, d));
                const float f = normed >> kind & 1 ? rsqrtf(__fmaf_rn(sum, 1.0f / D, p.eps)) : 1.0f;
                const float4 w0 = *reinterpret_cast<const float4 *>(&s_weight[kind][8 * li]), w1 = *reinterpret_cast<const float4 *>(&s_weight[kind][8 * li + 4]);
                const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = __fmul_rn(__fmul_rn(x[j], f), w[j]);
                if (turns) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float &a = x[NEIGHBOURS ? 2 * j : j], &b = x[NEIGHBOURS ? 2 * j + 1 : 4 + j];
                        const float turned = __fmaf_rn(a, c[j], -__fmul_rn(b, s[j]));
                        b = __fmaf_rn(b, c[j], __fmul_rn(a, s[j]));
                        a = turned;
                    }
                }
            }
            if (kind == 3 || (kind != 0 && place < 0)) continue;
            uint16_t *at = (kind == 0 ? p.q + token : (kind == 1 ? p.k_cache : p.v_cache) + place) + to[k];
            *reinterpret_cast<uint2 *>(at + e0) = narrow(x);
            *reinterpret_cast<uint2 *>(at + e1) = narrow(x + 4);
        }
    }
}

template <int D, bool F32, bool NEIGHBOURS, int ROWS>
cudaError_t launch_rope(const RopeParams &p, int sms, cudaStream_t stream)
{
    static std::atomic<int> configured[64] = {};
    const int rows = p.heads + 2 * p.kv_heads, block_rows = ROWS * kRopeThreads / (D / 8);
    const int y = (rows + block_rows - 1) / block_rows;
    const int fill = (kRopeBlocks * sms + y - 1) / y;
    Launch l;
    l.grid = dim3(unsigned(p.T < fill ? p.T : fill), unsigned(y));
    l.threads = kRopeThreads;
    l.smem = 0;
    l.pdl = true;
    return launch_one(rope_rows<D, F32, NEIGHBOURS, ROWS>, configured, l, stream, p);
}

template <int D, bool F32>
cudaError_t launch_rope_rows(const RopeParams &p, int sms, cudaStream_t stream)
{
    constexpr int kRows = F32 ? 2 : 4;  // 64 bytes in flight for a thread, and as many of the next token
    const int rows = p.heads + 2 * p.kv_heads, block_rows = kRows * kRopeThreads / (D / 8);
    // one row a thread while that leaves no SM with two blocks more than another's one
    const bool few = (int64_t)p.T * ((rows + block_rows - 1) / block_rows) < sms;
    if (p.neighbours) return few ? launch_rope<D, F32, true, 1>(p, sms, stream) : launch_rope<D, F32, true, kRows>(p, sms, stream);
    return few ? launch_rope<D, F32, false, 1>(p, sms, stream) : launch_rope<D, F32, false, kRows>(p, sms, stream);
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
