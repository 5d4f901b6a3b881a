// qmv_lora_run: a group-quantized projection shared by M vectors plus each
// vector's own low-rank adapter,
//
//   y[m] = W x[m] + c_a B_a (A_a x[m]),   a = adapter[m].
//
// Two kernels: lora_inner forms A_a x[m] (fp32) into the workspace, lora_project
// forms the projection and adds B_a times that vector.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "qmv.h"
#include "qmv_launch_decl.h"

namespace {

struct LoraParams {
    const uint32_t *w;
    const uint16_t *scales, *biases, *x, *a, *b;
    const int32_t *adapter;
    const float *c;
    float *inner;  // [M][R]
    void *y;
    int M, N, K, bits, gs, L, R, f32_out;
};

__device__ __forceinline__ float bf(uint16_t u) { return __uint_as_float(uint32_t(u) << 16); }

__device__ __forceinline__ float warp_sum(float v)
{
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One warp per (vector, row of A).
__global__ void lora_inner(const LoraParams p)
{
    const int item = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32, lane = threadIdx.x % 32;
    if (item >= p.M * p.R) return;
    const int m = item / p.R, r = item % p.R, ad = p.adapter[m];
    if (ad < 0 || ad >= p.L) return;
    const uint16_t *a = p.a + (size_t(ad) * p.R + r) * p.K, *x = p.x + size_t(m) * p.K;
    float s = 0.0f;
    for (int i = lane; i < p.K; i += 32) s = fmaf(bf(a[i]), bf(x[i]), s);
    s = warp_sum(s);
    if (lane == 0) p.inner[size_t(m) * p.R + r] = s;
}

// One warp per (row, vector); a lane takes whole words, each inside one group.
__global__ void lora_project(const LoraParams p)
{
    const int n = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32, lane = threadIdx.x % 32, m = blockIdx.y;
    if (n >= p.N) return;
    const int per = 32 / p.bits, words = p.K / per, G = p.K / p.gs;
    const uint32_t *w = p.w + size_t(n) * words;
    const uint16_t *x = p.x + size_t(m) * p.K;
    float y = 0.0f;
    for (int j = lane; j < words; j += 32) {
        const uint32_t word = w[j];
        float qx = 0.0f, sx = 0.0f;
        for (int f = 0; f < per; ++f) {
            const float xv = bf(x[j * per + f]);
            qx = fmaf(float((word >> (f * p.bits)) & ((1u << p.bits) - 1u)), xv, qx);
            sx += xv;
        }
        const size_t g = size_t(n) * G + j * per / p.gs;
        y = fmaf(bf(p.scales[g]), qx, fmaf(bf(p.biases[g]), sx, y));
    }
    y = warp_sum(y);
    if (lane) return;
    const int ad = p.adapter[m];
    if (ad >= 0 && ad < p.L) {
        const uint16_t *b = p.b + (size_t(ad) * p.N + n) * p.R;
        float d = 0.0f;
        for (int r = 0; r < p.R; ++r) d = fmaf(bf(b[r]), p.inner[size_t(m) * p.R + r], d);
        y = fmaf(p.c[ad], d, y);
    }
    const size_t at = size_t(m) * p.N + n;
    if (p.f32_out) static_cast<float *>(p.y)[at] = y;
    else static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(y);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

extern "C" size_t qmv_lora_workspace_size(int M, int N, int K, int bits, int group_size, int rank)
{
    if (qmv::check_weights(M, N, K, bits, group_size) != QMV_OK || rank < 1 || rank > QMV_MAX_RANK) return 0;
    return size_t(M) * rank * sizeof(float);
}

extern "C" qmv_status qmv_lora_run(const uint32_t *w_q, const uint16_t *scales, const uint16_t *biases,
                                   const uint16_t *x, const uint16_t *lora_a, const uint16_t *lora_b,
                                   const int32_t *adapter, const float *lora_scale, void *y, int M, int N, int K,
                                   int bits, int group_size, int adapters, int rank, void *workspace,
                                   size_t workspace_bytes, unsigned flags, qmv_stream_t stream)
{
    if (!w_q || !scales || !biases || !x || !lora_a || !lora_b || !adapter || !lora_scale || !y) return QMV_ERR_NULL;
    qmv_status st = qmv::check_weights(M, N, K, bits, group_size);
    if (st != QMV_OK) return st;
    if (adapters < 1 || adapters > QMV_MAX_ADAPTERS || rank < 1 || rank > QMV_MAX_RANK) return QMV_ERR_COUNT;
    if (flags & ~QMV_F32_OUT) return QMV_ERR_FLAGS;
    if (!aligned(w_q, 16) || !aligned(scales, 16) || !aligned(biases, 16) || !aligned(x, 16) || !aligned(lora_a, 16) ||
        !aligned(lora_b, 16) || !aligned(adapter, 4) || !aligned(lora_scale, 4) ||
        !aligned(y, flags & QMV_F32_OUT ? 4 : 2) || (workspace && !aligned(workspace, 16)))
        return QMV_ERR_ALIGN;
    qmv::DeviceInfo dev;
    st = qmv::current_device(&dev);
    if (st != QMV_OK) return st;
    void *ws = nullptr;
    st = qmv::scratch(dev, qmv_lora_workspace_size(M, N, K, bits, group_size, rank), workspace, workspace_bytes, &ws);
    if (st != QMV_OK) return st;

    LoraParams p{w_q, scales, biases, x, lora_a, lora_b, adapter, lora_scale, static_cast<float *>(ws), y,
                 M, N, K, bits, group_size, adapters, rank, (flags & QMV_F32_OUT) != 0};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    lora_inner<<<(M * rank + 7) / 8, 256, 0, s>>>(p);
    lora_project<<<dim3((N + 7) / 8, M), 256, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? QMV_OK : qmv::record_cuda_failure("lora kernel launch", e);
}
