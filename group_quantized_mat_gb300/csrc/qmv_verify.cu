// qmv_verify_run: drafted tokens against the target's probabilities, from given
// random numbers. Two kernels: verify_rows forms each row's maximum, argmax and
// sum of exponentials, verify_emit decides and samples, one block per sequence.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "qmv.h"
#include "qmv_launch_decl.h"

namespace {

struct RowStat {
    float max, sum;
    int arg, pad;
};

struct VerifyParams {
    const void *target, *draft;
    const int32_t *draft_tokens, *draft_len;
    const float *temperature, *uniform, *noise;
    int32_t *tokens, *accepted;
    float *logprob;
    RowStat *stat;  // [B][2 S + 1]: the target rows, then the draft rows
    int B, S, V, f32;
    long long ld_target, ld_draft, ld_noise;
};

// A logit as it counts: NaN as -inf, +inf as the type's largest finite value.
__device__ __forceinline__ float logit(const VerifyParams &p, const void *base, size_t at)
{
    const float l = p.f32 ? static_cast<const float *>(base)[at]
                          : __uint_as_float(uint32_t(static_cast<const uint16_t *>(base)[at]) << 16);
    const float big = p.f32 ? FLT_MAX : 3.3895313892515355e38f;
    return l > -INFINITY ? fminf(l, big) : -INFINITY;
}

__device__ __forceinline__ size_t row_at(const VerifyParams &p, int b, int r)
{
    return r <= p.S ? (size_t(b) * (p.S + 1) + r) * p.ld_target : (size_t(b) * p.S + (r - p.S - 1)) * p.ld_draft;
}

__device__ __forceinline__ float inverse_temperature(const VerifyParams &p, int b)
{
    const float t = p.temperature ? p.temperature[b] : 1.0f;
    return t > 0.0f ? 1.0f / t : 1.0f;
}

__device__ __forceinline__ bool better(float v, int i, float w, int j) { return v > w || (v == w && i < j); }

// The best (value, index) of a block of 256, in thread 0.
__device__ void block_best(float &v, int &i)
{
    __shared__ float sv[8];
    __shared__ int si[8];
    for (int o = 16; o; o >>= 1) {
        const float w = __shfl_xor_sync(0xffffffffu, v, o);
        const int j = __shfl_xor_sync(0xffffffffu, i, o);
        if (better(w, j, v, i)) { v = w; i = j; }
    }
    __syncthreads();
    if (threadIdx.x % 32 == 0) { sv[threadIdx.x / 32] = v; si[threadIdx.x / 32] = i; }
    __syncthreads();
    for (int k = 0; k < 8; ++k)
        if (better(sv[k], si[k], v, i)) { v = sv[k]; i = si[k]; }
}

__global__ void verify_rows(const VerifyParams p)
{
    __shared__ float part[8];
    const int b = blockIdx.x, r = blockIdx.y;
    const void *base = r <= p.S ? p.target : p.draft;
    const size_t at = row_at(p, b, r);
    float m = -INFINITY;
    int arg = 0x7fffffff;
    for (int v = threadIdx.x; v < p.V; v += 256) {
        const float l = logit(p, base, at + v);
        if (better(l, v, m, arg)) { m = l; arg = v; }
    }
    block_best(m, arg);
    const float inv = inverse_temperature(p, b);
    float s = 0.0f;
    if (m > -INFINITY)
        for (int v = threadIdx.x; v < p.V; v += 256) s += expf((logit(p, base, at + v) - m) * inv);
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = s;
    __syncthreads();
    if (threadIdx.x) return;
    s = 0.0f;
    for (int k = 0; k < 8; ++k) s += part[k];
    p.stat[size_t(b) * (2 * p.S + 1) + r] = {m, s, arg, 0};
}

// p or q at token v of row r, 0 where it is no token or the row has none.
__device__ __forceinline__ float prob(const VerifyParams &p, const RowStat &st, int b, int r, int v, float inv)
{
    if (v < 0 || v >= p.V || !(st.max > -INFINITY)) return 0.0f;
    return expf((logit(p, r <= p.S ? p.target : p.draft, row_at(p, b, r) + v) - st.max) * inv) / st.sum;
}

__global__ void verify_emit(const VerifyParams p)
{
    __shared__ int s_n;
    const int b = blockIdx.x;
    const RowStat *st = p.stat + size_t(b) * (2 * p.S + 1);
    const float t = p.temperature ? p.temperature[b] : 1.0f, inv = inverse_temperature(p, b);
    const bool greedy = !(t > 0.0f);
    const int len = p.draft_len ? min(max(p.draft_len[b], 0), p.S) : p.S;
    if (threadIdx.x == 0) {
        int n = 0;
        for (; n < len; ++n) {
            const int x = p.draft_tokens[size_t(b) * p.S + n];
            bool ok;
            if (greedy) ok = st[n].max > -INFINITY && x == st[n].arg;
            else {
                const float q = p.draft ? prob(p, st[p.S + 1 + n], b, p.S + 1 + n, x, inv) : 1.0f;
                ok = p.uniform[size_t(b) * p.S + n] * q < prob(p, st[n], b, n, x, inv);
            }
            if (!ok) break;
        }
        s_n = n;
    }
    __syncthreads();
    const int n = s_n;
    const RowStat row = st[n];
    float best = -1.0f;
    int arg = 0x7fffffff;
    if (greedy) arg = row.arg;
    else if (row.max > -INFINITY) {
        const int x = n < len ? p.draft_tokens[size_t(b) * p.S + n] : -1;
        const bool minus = n < len && p.draft;
        for (int pass = 0; pass < 2; ++pass) {
            best = -1.0f;
            arg = 0x7fffffff;
            for (int v = threadIdx.x; v < p.V; v += 256) {
                const float pv = prob(p, row, b, n, v, inv);
                float rest = pv;
                if (pass == 0) rest = fmaxf(pv - (minus ? prob(p, st[p.S + 1 + n], b, p.S + 1 + n, v, inv) : v == x ? 1.0f : 0.0f), 0.0f);
                const float e = fmaxf(p.noise[size_t(b) * p.ld_noise + v], FLT_MIN);
                const float ratio = rest / e;
                if (rest > 0.0f && better(ratio, v, best, arg)) { best = ratio; arg = v; }
            }
            block_best(best, arg);
            if (arg != 0x7fffffff) break;
        }
    }
    if (threadIdx.x) return;
    const bool none = !(row.max > -INFINITY);
    for (int i = 0; i <= p.S; ++i) {
        const int tok = i < n ? p.draft_tokens[size_t(b) * p.S + i] : i == n && !none ? arg : -1;
        const size_t at = size_t(b) * (p.S + 1) + i;
        p.tokens[at] = tok;
        if (p.logprob)
            p.logprob[at] = tok >= 0 ? (logit(p, p.target, row_at(p, b, i) + tok) - st[i].max) * inv - logf(st[i].sum)
                            : i == n ? -INFINITY : 0.0f;
    }
    p.accepted[b] = n;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

extern "C" size_t qmv_verify_workspace_size(int B, int S, int V)
{
    if (B < 1 || B > QMV_MAX_BATCH || S < 0 || S > QMV_MAX_DRAFT || V < 1 || V > (1 << 24)) return 0;
    return size_t(B) * (2 * S + 1) * sizeof(RowStat);
}

extern "C" qmv_status qmv_verify_run(const void *target, const void *draft, const int32_t *draft_tokens,
                                     const int32_t *draft_len, const float *temperature, const float *uniform,
                                     const float *noise, int32_t *tokens, int32_t *accepted, float *logprob, int B,
                                     int S, int V, int64_t ld_target, int64_t ld_draft, int64_t ld_noise,
                                     void *workspace, size_t workspace_bytes, unsigned flags, qmv_stream_t stream)
{
    if (!target || !noise || !tokens || !accepted) return QMV_ERR_NULL;
    if (B < 1 || B > QMV_MAX_BATCH || S < 0 || S > QMV_MAX_DRAFT) return QMV_ERR_COUNT;
    if (S > 0 && (!draft_tokens || !uniform)) return QMV_ERR_NULL;
    if (S == 0) draft = nullptr;
    const int64_t most = int64_t(1) << 40;
    if (V < 1 || V > (1 << 24) || ld_target < V || ld_target > most || (draft && (ld_draft < V || ld_draft > most)) ||
        ld_noise < V || ld_noise > most)
        return QMV_ERR_SHAPE;
    if (flags & ~QMV_VERIFY_F32_LOGITS) return QMV_ERR_FLAGS;
    const bool f32 = (flags & QMV_VERIFY_F32_LOGITS) != 0;
    if (!aligned(target, f32 ? 4 : 2) || !aligned(draft, f32 ? 4 : 2) || (workspace && !aligned(workspace, 16)))
        return QMV_ERR_ALIGN;
    for (const void *ptr : {(const void *)draft_tokens, (const void *)draft_len, (const void *)temperature,
                            (const void *)uniform, (const void *)noise, (const void *)tokens, (const void *)accepted,
                            (const void *)logprob})
        if (!aligned(ptr, 4)) return QMV_ERR_ALIGN;
    qmv::DeviceInfo dev;
    qmv_status st = qmv::current_device(&dev);
    if (st != QMV_OK) return st;
    void *ws = nullptr;
    st = qmv::scratch(dev, qmv_verify_workspace_size(B, S, V), workspace, workspace_bytes, &ws);
    if (st != QMV_OK) return st;

    VerifyParams p{target, draft, draft_tokens, draft_len, temperature, uniform, noise, tokens, accepted, logprob,
                   static_cast<RowStat *>(ws), B, S, V, f32 ? 1 : 0, ld_target, ld_draft, ld_noise};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    verify_rows<<<dim3(B, draft ? 2 * S + 1 : S + 1), 256, 0, s>>>(p);
    verify_emit<<<B, 256, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? QMV_OK : qmv::record_cuda_failure("verify kernel launch", e);
}
