// qmv_moe_run: a whole mixture-of-experts layer for a few tokens,
//
//   l = router x;  ids = top-k of l;  w = softmax;  y = sum_e w_e down_e (act(gate_e x) * (up_e x)).
//
// Three kernels: moe_route, moe_hidden (gate, up and activation of every
// (token, choice)) and moe_down (down product and weighted sum).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "qmv.h"
#include "qmv_launch_decl.h"

namespace {

struct MoeParams {
    const uint16_t *x, *router;
    const uint32_t *gu_w, *dn_w;
    const uint16_t *gu_s, *gu_b, *dn_s, *dn_b;
    void *y;
    int32_t *ids;      // [M][k]
    float *weights;    // [M][k]
    float *h;          // [M][k][I]
    int32_t *ids_out;  // the caller's, or NULL
    float *weights_out;
    int M, K, I, E, k, bits, gs, f32_out, gelu, softmax_all;
};

__device__ __forceinline__ float bf(uint16_t u) { return __uint_as_float(uint32_t(u) << 16); }

__device__ __forceinline__ float warp_sum(float v)
{
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One block per token.
__global__ void moe_route(const MoeParams p)
{
    __shared__ float l[QMV_MAX_EXPERTS];
    const int m = blockIdx.x, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const uint16_t *x = p.x + size_t(m) * p.K;
    for (int e = warp; e < p.E; e += blockDim.x / 32) {
        float s = 0.0f;
        for (int i = lane; i < p.K; i += 32) s = fmaf(bf(p.router[size_t(e) * p.K + i]), bf(x[i]), s);
        s = warp_sum(s);
        if (lane == 0) l[e] = s == s ? s : -INFINITY;
    }
    __syncthreads();
    if (threadIdx.x) return;
    float top = -INFINITY, all = 0.0f, some = 0.0f;
    for (int e = 0; e < p.E; ++e) top = fmaxf(top, l[e]);
    for (int e = 0; e < p.E; ++e) all += expf(l[e] - top);
    float val[QMV_MAX_TOP_K];
    int id[QMV_MAX_TOP_K];
    for (int j = 0; j < p.k; ++j) {
        int best = -1;
        for (int e = 0; e < p.E; ++e) {
            bool used = false;
            for (int i = 0; i < j; ++i) used |= id[i] == e;
            if (!used && (best < 0 || l[e] > l[best])) best = e;
        }
        id[j] = best;
        val[j] = expf(l[best] - top);
        some += val[j];
    }
    for (int j = 0; j < p.k; ++j) {
        const float w = val[j] / (p.softmax_all ? all : some);
        p.ids[m * p.k + j] = id[j];
        p.weights[m * p.k + j] = w;
        if (p.ids_out) p.ids_out[m * p.k + j] = id[j];
        if (p.weights_out) p.weights_out[m * p.k + j] = w;
    }
}

// A warp's dot of packed row `row` of an [.., K] matrix with v(i), fp32.
template <typename V>
__device__ float packed_dot(const uint32_t *w, const uint16_t *sc, const uint16_t *bi, size_t row, int K, int bits,
                            int gs, int lane, V v)
{
    const int per = 32 / bits, words = K / per, G = K / gs;
    float y = 0.0f;
    for (int j = lane; j < words; j += 32) {
        const uint32_t word = w[row * words + j];
        float qx = 0.0f, sx = 0.0f;
        for (int f = 0; f < per; ++f) {
            const float xv = v(j * per + f);
            qx = fmaf(float((word >> (f * bits)) & ((1u << bits) - 1u)), xv, qx);
            sx += xv;
        }
        const size_t g = row * G + j * per / gs;
        y = fmaf(bf(sc[g]), qx, fmaf(bf(bi[g]), sx, y));
    }
    return warp_sum(y);
}

// One warp per (token, choice, element of h).
__global__ void moe_hidden(const MoeParams p)
{
    const int i = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32, lane = threadIdx.x % 32, pair = blockIdx.y;
    if (i >= p.I) return;
    const uint16_t *x = p.x + size_t(pair / p.k) * p.K;
    const size_t row = size_t(p.ids[pair]) * 2 * p.I + i;
    auto v = [&](int j) { return bf(x[j]); };
    const float g = packed_dot(p.gu_w, p.gu_s, p.gu_b, row, p.K, p.bits, p.gs, lane, v);
    const float u = packed_dot(p.gu_w, p.gu_s, p.gu_b, row + p.I, p.K, p.bits, p.gs, lane, v);
    const float act = p.gelu ? 0.5f * g * (1.0f + tanhf(0.7978845608028654f * (g + 0.044715f * g * g * g)))
                             : g / (1.0f + expf(-g));
    if (lane == 0) p.h[size_t(pair) * p.I + i] = act * u;
}

// One warp per (token, element of y).
__global__ void moe_down(const MoeParams p)
{
    const int n = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32, lane = threadIdx.x % 32, m = blockIdx.y;
    if (n >= p.K) return;
    float y = 0.0f;
    for (int j = 0; j < p.k; ++j) {
        const int pair = m * p.k + j;
        const float *h = p.h + size_t(pair) * p.I;
        const float d = packed_dot(p.dn_w, p.dn_s, p.dn_b, size_t(p.ids[pair]) * p.K + n, p.I, p.bits, p.gs, lane,
                                   [&](int i) { return h[i]; });
        y = fmaf(p.weights[pair], d, y);
    }
    if (lane) return;
    const size_t at = size_t(m) * p.K + n;
    if (p.f32_out) static_cast<float *>(p.y)[at] = y;
    else static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(y);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

qmv_status check_moe(int M, int K, int I, int E, int k, int bits, int gs)
{
    qmv_status st = qmv::check_weights(M, 1, K, bits, gs);
    if (st != QMV_OK) return st;
    if (I < 1 || I > (1 << 24) || I % gs) return QMV_ERR_SHAPE;
    if (E < 1 || E > QMV_MAX_EXPERTS || k < 1 || k > E || k > QMV_MAX_TOP_K) return QMV_ERR_COUNT;
    if ((long long)E * 2 * I * (K / gs) >= (1ll << 31) || (long long)E * K * (I / gs) >= (1ll << 31) ||
        (long long)E * 2 * I > (1 << 30) || (long long)E * K > (1 << 30))
        return QMV_ERR_SHAPE;
    return QMV_OK;
}

}  // namespace

extern "C" size_t qmv_moe_workspace_size(int M, int K, int inter, int experts, int top_k, int bits, int group_size)
{
    if (check_moe(M, K, inter, experts, top_k, bits, group_size) != QMV_OK) return 0;
    return size_t(M) * top_k * (size_t(inter) + 2) * 4;
}

extern "C" qmv_status qmv_moe_run(const uint16_t *x, const uint16_t *router, const uint32_t *gu_w,
                                  const uint16_t *gu_scales, const uint16_t *gu_biases, const uint32_t *dn_w,
                                  const uint16_t *dn_scales, const uint16_t *dn_biases, void *y, int32_t *topk_ids,
                                  float *topk_weights, int M, int K, int inter, int experts, int top_k, int bits,
                                  int group_size, void *workspace, size_t workspace_bytes, unsigned flags,
                                  qmv_stream_t stream)
{
    if (!x || !router || !gu_w || !gu_scales || !gu_biases || !dn_w || !dn_scales || !dn_biases || !y)
        return QMV_ERR_NULL;
    qmv_status st = check_moe(M, K, inter, experts, top_k, bits, group_size);
    if (st != QMV_OK) return st;
    if (flags & ~(QMV_F32_OUT | QMV_MOE_GELU | QMV_MOE_SOFTMAX_ALL)) return QMV_ERR_FLAGS;
    for (const void *ptr : {(const void *)x, (const void *)router, (const void *)gu_w, (const void *)gu_scales,
                            (const void *)gu_biases, (const void *)dn_w, (const void *)dn_scales,
                            (const void *)dn_biases, (const void *)workspace})
        if (!aligned(ptr, 16)) return QMV_ERR_ALIGN;
    if (!aligned(y, flags & QMV_F32_OUT ? 4 : 2) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4))
        return QMV_ERR_ALIGN;
    qmv::DeviceInfo dev;
    st = qmv::current_device(&dev);
    if (st != QMV_OK) return st;
    void *ws = nullptr;
    st = qmv::scratch(dev, qmv_moe_workspace_size(M, K, inter, experts, top_k, bits, group_size), workspace,
                      workspace_bytes, &ws);
    if (st != QMV_OK) return st;

    const size_t pairs = size_t(M) * top_k;
    MoeParams p{};
    p.x = x; p.router = router;
    p.gu_w = gu_w; p.gu_s = gu_scales; p.gu_b = gu_biases;
    p.dn_w = dn_w; p.dn_s = dn_scales; p.dn_b = dn_biases;
    p.y = y; p.ids_out = topk_ids; p.weights_out = topk_weights;
    p.h = static_cast<float *>(ws);
    p.ids = reinterpret_cast<int32_t *>(p.h + pairs * inter);
    p.weights = reinterpret_cast<float *>(p.ids + pairs);
    p.M = M; p.K = K; p.I = inter; p.E = experts; p.k = top_k; p.bits = bits; p.gs = group_size;
    p.f32_out = (flags & QMV_F32_OUT) != 0;
    p.gelu = (flags & QMV_MOE_GELU) != 0;
    p.softmax_all = (flags & QMV_MOE_SOFTMAX_ALL) != 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    moe_route<<<M, 256, 0, s>>>(p);
    moe_hidden<<<dim3((inter + 7) / 8, unsigned(pairs)), 256, 0, s>>>(p);
    moe_down<<<dim3((K + 7) / 8, M), 256, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? QMV_OK : qmv::record_cuda_failure("moe kernel launch", e);
}
