// qmv_verify_run: drafted tokens against the target's probabilities, from given
// random numbers.
//
// The mathematics: a row's softmax needs its maximum m and s = sum exp((l - m) / T),
// both of which join from parts, (m, s) of two parts being
// (max, s1 exp((m1 - max) / T) + s2 exp((m2 - max) / T)). Then a token is accepted
// while u q(x) < p(x), and the token after the accepted ones wins the race
// argmax r(v) / e(v), r = max(p - q, 0) or p, which joins from parts too.
//
// Two kernels.
//  1. verify_rows reads the logits once, 16 bytes at a time, a part of a row to a
//     block: all of a part is in flight before any of it is used, and stays in
//     registers from the maximum to the sum. Rows that no outcome needs (past a
//     sequence's drafts; draft rows where the argmax decides) are not read. It is
//     bound by memory, with the integer pipe and the exponentials close behind (5
//     instructions an element).
//  2. verify_emit, several blocks to a sequence: each joins the parts of the
//     sequence's rows, decides how many tokens are accepted and runs its share of
//     the race on the one row that matters; the last of a sequence's blocks joins
//     the winners and writes the results.
#include <cuda_bf16.h>

#include <cfloat>
#include <cstdint>

#include "qmv.h"
#include "qmv_launch.cuh"

namespace qmv {
namespace {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kNone = 0x7fffffff;
constexpr int kMaxRows = 2 * QMV_MAX_DRAFT + 1;

// A part of a row: maximum, sum of exponentials relative to it, index of the
// maximum (where argmax decides).
struct Part {
    float max, sum;
    int arg, pad;
};
struct Winner {
    float ratio;
    int token;
};

struct VerifyParams {
    const void *target, *draft;
    const int32_t *draft_tokens, *draft_len;
    const float *temperature, *uniform, *noise;
    int32_t *tokens, *accepted;
    float *logprob;
    Part *parts;         // [B][rows][nparts]: the target rows, then the draft rows
    Winner *winners;     // [B][races]
    unsigned *finished;  // [B]
    int B, S, V, rows, nparts, races;
    long long ld_target, ld_draft, ld_noise;
};

__device__ __forceinline__ float big(bool f32) { return f32 ? FLT_MAX : 3.3895313892515355e38f; }

// A logit as it counts: NaN as -inf, +inf as the type's largest finite value.
template <bool F32>
__device__ __forceinline__ float logit(const void *row, long long v)
{
    const float l = F32 ? __ldg(static_cast<const float *>(row) + v)
                        : __uint_as_float(uint32_t(__ldg(static_cast<const uint16_t *>(row) + v)) << 16);
    return l > -INFINITY ? fminf(l, big(F32)) : -INFINITY;
}

template <bool F32>
__device__ __forceinline__ const void *row_of(const VerifyParams &p, int b, int r)
{
    const long long at = r <= p.S ? ((long long)b * (p.S + 1) + r) * p.ld_target : ((long long)b * p.S + (r - p.S - 1)) * p.ld_draft;
    return static_cast<const uint8_t *>(r <= p.S ? p.target : p.draft) + at * (F32 ? 4 : 2);
}

struct Mode {
    float inv;    // 1 / temperature, 1 where argmax decides
    bool greedy;  // argmax decides
    int len;
};

__device__ __forceinline__ Mode mode_of(const VerifyParams &p, int b)
{
    Mode m;
    const float t = p.temperature ? __ldg(p.temperature + b) : 1.0f;
    m.greedy = !(t > 0.0f);
    m.inv = m.greedy ? 1.0f : fmaxf(__fdiv_rn(1.0f, t), FLT_MIN);
    m.len = p.draft_len ? min(max(__ldg(p.draft_len + b), 0), p.S) : p.S;
    return m;
}

__device__ __forceinline__ bool better(float v, int i, float w, int j) { return v > w || (v == w && i < j); }

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint64_t pair_of(float lo, float hi)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void unpair(uint64_t v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// NaN as -inf and +inf as the largest finite value, two bf16 or one fp32.
template <bool F32>
__device__ __forceinline__ uint32_t clean(uint32_t w)
{
    if (F32) return __float_as_uint(fminf(fmaxf(__uint_as_float(w), -INFINITY), FLT_MAX));
    uint32_t d;
    asm("{\n\t.reg .b32 t;\n\tmax.bf16x2 t, %1, %2;\n\tmin.bf16x2 %0, t, %3;\n\t}" : "=r"(d) : "r"(w), "r"(0xff80ff80u), "r"(0x7f7f7f7fu));
    return d;
}
template <bool F32>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b)
{
    if (F32) return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The block's value of a max (over floats) or sum, in all threads.
__device__ __forceinline__ float block_max(float v, float *scratch)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    __syncthreads();
    if (threadIdx.x % 32 == 0) scratch[threadIdx.x / 32] = v;
    __syncthreads();
    v = scratch[0];
#pragma unroll
    for (int w = 1; w < kVerifyWarps; ++w) v = fmaxf(v, scratch[w]);
    return v;
}

// 16 bytes that start `bytes` (a multiple of 2) into two aligned 16.
__device__ __forceinline__ uint4 shifted(uint4 a, uint4 b, int bytes)
{
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (bytes & 8)
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    if (bytes & 4)
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    if (bytes & 2)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The 16 bytes of a row from element v0 on, elements past V as -inf. Inside the
// row one aligned load, or two that are shifted; at the ends of a row that lies
// off a 16-byte boundary (nothing beside the row is read) element by element.
template <bool F32>
__device__ __forceinline__ uint4 load16(const uint8_t *base, long long v0, int V, int off)
{
    constexpr int EV = F32 ? 4 : 8, SIZE = F32 ? 4 : 2;
    const uint32_t none = F32 ? 0xff800000u : 0xff80ff80u;
    uint4 x = make_uint4(none, none, none, none);
    if (v0 >= V) return x;
    const uint8_t *at = base + v0 * SIZE;
    if (off == 0 && v0 + EV <= V) return __ldcs(reinterpret_cast<const uint4 *>(at));
    if (off != 0 && v0 > 0 && v0 + 2 * EV <= V) {
        const uint4 *q = reinterpret_cast<const uint4 *>(at - off);
        return shifted(__ldg(q), __ldg(q + 1), off);
    }
    uint32_t w[4] = {none, none, none, none};
#pragma unroll
    for (int i = 0; i < EV; ++i) {
        if (v0 + i >= V) break;
        if (F32) w[i & 3] = __ldg(reinterpret_cast<const uint32_t *>(at) + i);
        else {
            const uint32_t h = __ldg(reinterpret_cast<const uint16_t *>(at) + i);
            w[i / 2 & 3] = i & 1 ? (w[i / 2 & 3] & 0xffffu) | h << 16 : (w[i / 2 & 3] & 0xffff0000u) | h;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One part of one row: NV vectors of 16 bytes to a thread, by the elements'
// indexes alone, so that equal rows have equal sums wherever they lie.
template <bool F32, int NV>
__global__ void __launch_bounds__(kVerifyThreads, 4) verify_rows(const VerifyParams p)
{
    constexpr int EV = F32 ? 4 : 8;
    __shared__ float scratch[kVerifyWarps];
    __shared__ int s_arg;
    const int tid = threadIdx.x;
    const int part = blockIdx.x % p.nparts, row = blockIdx.x / p.nparts, b = row / p.rows, r = row - b * p.rows;
    grid_dependency_wait();
    grid_launch_dependents();
    if (r == 0 && part == 0 && tid == 0) p.finished[b] = 0u;
    const Mode m = mode_of(p, b);
    if (r <= p.S ? r > m.len : m.greedy || r - p.S - 1 >= m.len) return;
    const uint8_t *base = static_cast<const uint8_t *>(row_of<F32>(p, b, r));
    const int off = int(reinterpret_cast<uintptr_t>(base) & 15);
    const uint32_t none = F32 ? 0xff800000u : 0xff80ff80u;
    const int v0 = part * kVerifyThreads * NV + tid;
    uint4 x[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) x[k] = load16<F32>(base, (long long)(v0 + k * kVerifyThreads) * EV, p.V, off);
    uint32_t top2 = none;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        x[k] = make_uint4(clean<F32>(x[k].x), clean<F32>(x[k].y), clean<F32>(x[k].z), clean<F32>(x[k].w));
        top2 = larger<F32>(top2, larger<F32>(larger<F32>(x[k].x, x[k].y), larger<F32>(x[k].z, x[k].w)));
    }
    float top = F32 ? __uint_as_float(top2) : fmaxf(__uint_as_float(top2 << 16), __uint_as_float(top2 & 0xffff0000u));
    top = block_max(top, scratch);
    float sum = 0.0f;
    int arg = kNone;
    if (top > -INFINITY) {
        const float c = __fmul_rn(m.inv, 1.4426950408889634f);
        const uint64_t neg = pair_of(-top, -top), cc = pair_of(c, c);
        uint64_t s2 = 0ull;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
            for (int i = 0; i < (F32 ? 2 : 4); ++i) {
                const uint64_t l = F32 ? pair_of(__uint_as_float(w[2 * i & 3]), __uint_as_float(w[(2 * i + 1) & 3]))
                                       : pair_of(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
                float lo, hi;
                unpair(mul2(add2(l, neg), cc), lo, hi);
                s2 = add2(s2, pair_of(ex2(lo), ex2(hi)));
            }
        }
        float lo, hi;
        unpair(s2, lo, hi);
        sum = __fadd_rn(lo, hi);
        if (m.greedy) {
            // the first place of the maximum
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
                const int at = (v0 + k * kVerifyThreads) * EV;
#pragma unroll
                for (int i = 0; i < EV; ++i) {
                    const float l = F32 ? __uint_as_float(w[i & 3]) : __uint_as_float(i & 1 ? w[i / 2 & 3] & 0xffff0000u : w[i / 2 & 3] << 16);
                    if (l == top && at + i < arg) arg = at + i;
                }
            }
        }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, d));
    if (tid == 0) s_arg = kNone;
    __syncthreads();
    if (tid % 32 == 0) scratch[tid / 32] = sum;
    if (arg != kNone) atomicMin(&s_arg, arg);
    __syncthreads();
    if (tid) return;
    sum = scratch[0];
#pragma unroll
    for (int w = 1; w < kVerifyWarps; ++w) sum = __fadd_rn(sum, scratch[w]);
    p.parts[(size_t)row * p.nparts + part] = {top, sum, s_arg, 0};
}

// p or q of token v in a row, 0 where it is no token or the row has none.
template <bool F32>
__device__ __forceinline__ float prob(const VerifyParams &p, const void *row, float top, float sum, int v, float inv)
{
    if (v < 0 || v >= p.V || !(top > -INFINITY)) return 0.0f;
    return __fdiv_rn(expf(__fmul_rn(__fsub_rn(logit<F32>(row, v), top), inv)), sum);
}

// The block's best (ratio, token), in all threads.
__device__ __forceinline__ void block_best(float &v, int &i, float *sv, int *si)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const float w = __shfl_xor_sync(0xffffffffu, v, d);
        const int j = __shfl_xor_sync(0xffffffffu, i, d);
        if (better(w, j, v, i)) {
            v = w;
            i = j;
        }
    }
    __syncthreads();
    if (threadIdx.x % 32 == 0) {
        sv[threadIdx.x / 32] = v;
        si[threadIdx.x / 32] = i;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kVerifyWarps; ++k)
        if (better(sv[k], si[k], v, i)) {
            v = sv[k];
            i = si[k];
        }
}

template <bool F32>
__global__ void __launch_bounds__(kVerifyThreads) verify_emit(const VerifyParams p)
{
    __shared__ float s_max[kMaxRows], s_sum[kMaxRows], sv[kVerifyWarps];
    __shared__ int s_arg[kMaxRows], s_ok[QMV_MAX_DRAFT + 1], si[kVerifyWarps], s_last;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, b = blockIdx.x / p.races, race = blockIdx.x - b * p.races;
    // (none of these is written by the first kernel)
    const Mode m = mode_of(p, b);
    int drafted = -1;
    float u = 0.0f;
    if (tid < m.len) {
        drafted = __ldg(p.draft_tokens + size_t(b) * p.S + tid);
        u = __ldg(p.uniform + size_t(b) * p.S + tid);
    }
    grid_dependency_wait();
    grid_launch_dependents();
    const Part *parts = p.parts + (size_t)b * p.rows * p.nparts;
    for (int r = warp; r < p.rows; r += kVerifyWarps) {
        if (r <= p.S ? r > m.len : m.greedy || r - p.S - 1 >= m.len) continue;
        float top = -INFINITY, sum = 0.0f;
        int arg = kNone;
        for (int k = lane; k < p.nparts; k += 32) top = fmaxf(top, __ldcg(&parts[(size_t)r * p.nparts + k].max));
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        for (int k = lane; k < p.nparts; k += 32) {
            const int4 raw = __ldcg(reinterpret_cast<const int4 *>(parts + (size_t)r * p.nparts + k));
            const float pm = __int_as_float(raw.x);
            if (pm > -INFINITY) sum = __fmaf_rn(__int_as_float(raw.y), expf(__fmul_rn(__fsub_rn(pm, top), m.inv)), sum);
            if (pm == top) arg = min(arg, raw.z);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, d));
            arg = min(arg, __shfl_xor_sync(0xffffffffu, arg, d));
        }
        if (lane == 0) {
            s_max[r] = top;
            s_sum[r] = sum;
            s_arg[r] = arg;
        }
    }
    __syncthreads();
    if (tid <= m.len) {
        bool ok = false;
        if (tid < m.len) {
            if (m.greedy) ok = s_max[tid] > -INFINITY && drafted == s_arg[tid];
            else {
                const int d = p.S + 1 + tid;
                const float q = p.draft ? prob<F32>(p, row_of<F32>(p, b, d), s_max[d], s_sum[d], drafted, m.inv) : 1.0f;
                ok = __fmul_rn(u, q) < prob<F32>(p, row_of<F32>(p, b, tid), s_max[tid], s_sum[tid], drafted, m.inv);
            }
        }
        s_ok[tid] = ok;
    }
    __syncthreads();
    int n = 0;
    while (s_ok[n]) ++n;  // s_ok[len] is false
    const float top = s_max[n], total = s_sum[n];
    const bool none = !(top > -INFINITY);
    float best = -1.0f;
    int token = kNone;
    if (m.greedy) {
        token = s_arg[n];
    } else if (!none) {
        const void *row = row_of<F32>(p, b, n), *drow = n < m.len && p.draft ? row_of<F32>(p, b, p.S + 1 + n) : nullptr;
        const float dtop = drow ? s_max[p.S + 1 + n] : -INFINITY, dsum = drow ? s_sum[p.S + 1 + n] : 1.0f;
        const int cut = n < m.len && !p.draft ? __ldg(p.draft_tokens + size_t(b) * p.S + n) : -1;
        const float *noise = p.noise + (size_t)b * p.ld_noise;
        // the share of this block, then (in a sequence's last block, where nothing
        // had a positive remainder) all of p
        const int lo = int((long long)p.V * race / p.races), hi = int((long long)p.V * (race + 1) / p.races);
        // A token enters the race by its exact ratio, two divisions and two
        // exponentials; whether it can beat the thread's best so far is seen
        // without them, from approximations good to 1e-5 of p.
        constexpr int U = 8;
        const float c = __fmul_rn(m.inv, 1.4426950408889634f), itotal = __fdiv_rn(1.0f, total), idsum = dtop > -INFINITY ? __fdiv_rn(1.0f, dsum) : 0.0f;
        const auto run = [&](int from, int to, bool rest) {
            best = -1.0f;
            token = kNone;
            for (int v0 = from + tid; v0 < to; v0 += U * kVerifyThreads) {
                float l[U], d[U], e[U];
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int v = v0 + k * kVerifyThreads;
                    const bool in = v < to;
                    l[k] = in ? logit<F32>(row, v) : -INFINITY;
                    d[k] = in && rest && dtop > -INFINITY ? logit<F32>(drow, v) : -INFINITY;
                    e[k] = in ? __ldcs(noise + v) : 1.0f;
                }
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int v = v0 + k * kVerifyThreads;
                    const float pa = __fmul_rn(ex2(__fmul_rn(__fsub_rn(l[k], top), c)), itotal);
                    const float qa = d[k] > -INFINITY ? __fmul_rn(ex2(__fmul_rn(__fsub_rn(d[k], dtop), c)), idsum) : 0.0f;
                    const float hope = __fmaf_rn(1e-5f, pa, __fsub_rn(pa, qa));
                    if (!(hope > 0.0f) || hope < __fmul_rn(0.9999f, __fmul_rn(best, e[k])) || v >= to) continue;
                    float w = __fdiv_rn(expf(__fmul_rn(__fsub_rn(l[k], top), m.inv)), total);
                    if (d[k] > -INFINITY) w = __fsub_rn(w, __fdiv_rn(expf(__fmul_rn(__fsub_rn(d[k], dtop), m.inv)), dsum));
                    if (rest && v == cut) w = 0.0f;
                    if (w > 0.0f) {
                        const float ratio = __fdiv_rn(w, fmaxf(e[k], FLT_MIN));
                        if (better(ratio, v, best, token)) {
                            best = ratio;
                            token = v;
                        }
                    }
                }
            }
            block_best(best, token, sv, si);
        };
        run(lo, hi, true);
        if (p.races > 1) {
            if (tid == 0) {
                __stcg(reinterpret_cast<float2 *>(p.winners + (size_t)b * p.races + race), make_float2(best, __int_as_float(token)));
                __threadfence();
                s_last = atomicAdd(p.finished + b, 1u) == unsigned(p.races - 1);
            }
            __syncthreads();
            if (!s_last) return;
            __threadfence();
            best = -1.0f;
            token = kNone;
            for (int k = tid; k < p.races; k += kVerifyThreads) {
                const float2 w = __ldcg(reinterpret_cast<const float2 *>(p.winners + (size_t)b * p.races + k));
                if (better(w.x, __float_as_int(w.y), best, token)) {
                    best = w.x;
                    token = __float_as_int(w.y);
                }
            }
            block_best(best, token, sv, si);
        }
        if (token == kNone) run(0, p.V, false);
    }
    if ((m.greedy || none) && race != 0) return;
    for (int i = tid; i <= p.S; i += kVerifyThreads) {
        int tok = i < n ? __ldg(p.draft_tokens + size_t(b) * p.S + i) : i == n && !none ? token : -1;
        if (tok >= p.V) tok = -1;  // (no winner: cannot be)
        const size_t at = size_t(b) * (p.S + 1) + i;
        p.tokens[at] = tok;
        if (p.logprob)
            p.logprob[at] = tok >= 0 ? __fsub_rn(__fmul_rn(__fsub_rn(logit<F32>(row_of<F32>(p, b, i), tok), s_max[i]), m.inv), logf(s_sum[i]))
                            : i == n ? -INFINITY : 0.0f;
    }
    if (tid == 0) p.accepted[b] = n;
}

// Vectors of 16 bytes to a thread of verify_rows, and parts of a row, as large as
// still gives the SMs several blocks each: 2 for small calls (3 x 32000: 14 blocks
// would be one part each), 8 otherwise.
struct Split {
    int nv, nparts, races;
};

Split split(int B, int S, int V)
{
    Split s;
    const long long all = (long long)B * (2 * S + 1) * V;
    s.nv = all < (4ll << 20) ? 2 : 8;
    // for the narrower type's vectors; the wider type takes twice as many
    s.nparts = ((V + 3) / 4 + kVerifyThreads * s.nv - 1) / (kVerifyThreads * s.nv);
    // blocks of the race: about 4096 tokens each, fewer where sequences fill the GPU
    s.races = (V + 4095) / 4096;
    const int most = B >= 304 ? 1 : (1216 + B - 1) / B;
    if (s.races > most) s.races = most;
    return s;
}

size_t up256(size_t b) { return (b + 255) & ~size_t(255); }

template <bool F32>
cudaError_t launch_verify(const VerifyParams &p, int nv, cudaStream_t stream)
{
    static std::atomic<int> configured[3][64] = {};
    Launch l;
    l.grid = dim3(unsigned((long long)p.B * p.rows * p.nparts));
    l.threads = kVerifyThreads;
    l.smem = 0;
    l.pdl = true;
    const cudaError_t e = nv == 2 ? launch_one(verify_rows<F32, 2>, configured[0], l, stream, p)
                                  : launch_one(verify_rows<F32, 8>, configured[1], l, stream, p);
    if (e != cudaSuccess) return e;
    l.grid = dim3(unsigned(p.B * p.races));
    return launch_one(verify_emit<F32>, configured[2], l, stream, p);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace qmv

extern "C" size_t qmv_verify_workspace_size(int B, int S, int V)
{
    if (B < 1 || B > QMV_MAX_BATCH || S < 0 || S > QMV_MAX_DRAFT || V < 1 || V > (1 << 24)) return 0;
    const qmv::Split s = qmv::split(B, S, V);
    return qmv::up256(size_t(B) * (2 * S + 1) * s.nparts * sizeof(qmv::Part)) +
           qmv::up256(size_t(B) * s.races * sizeof(qmv::Winner)) + qmv::up256(size_t(B) * 4);
}

extern "C" qmv_status qmv_verify_run(const void *target, const void *draft, const int32_t *draft_tokens,
                                     const int32_t *draft_len, const float *temperature, const float *uniform,
                                     const float *noise, int32_t *tokens, int32_t *accepted, float *logprob, int B,
                                     int S, int V, int64_t ld_target, int64_t ld_draft, int64_t ld_noise,
                                     void *workspace, size_t workspace_bytes, unsigned flags, qmv_stream_t stream)
{
    using namespace qmv;
    if (!target || !noise || !tokens || !accepted) return QMV_ERR_NULL;
    if (B < 1 || B > QMV_MAX_BATCH || S < 0 || S > QMV_MAX_DRAFT) return QMV_ERR_COUNT;
    if (S > 0 && (!draft_tokens || !uniform)) return QMV_ERR_NULL;
    if (S == 0) draft = nullptr;
    const int64_t most = int64_t(1) << 40;
    if (V < 1 || V > (1 << 24) || ld_target < V || ld_target > most || (draft && (ld_draft < V || ld_draft > most)) ||
        ld_noise < V || ld_noise > most)
        return QMV_ERR_SHAPE;
    // blocks of the first kernel
    if ((long long)B * (2 * S + 1) * split(B, S, V).nparts > 0x7fffffffll) return QMV_ERR_SHAPE;
    if (flags & ~QMV_VERIFY_F32_LOGITS) return QMV_ERR_FLAGS;
    const bool f32 = (flags & QMV_VERIFY_F32_LOGITS) != 0;
    if (!aligned(target, f32 ? 4 : 2) || !aligned(draft, f32 ? 4 : 2) || (workspace && !aligned(workspace, 16)))
        return QMV_ERR_ALIGN;
    for (const void *ptr : {(const void *)draft_tokens, (const void *)draft_len, (const void *)temperature,
                            (const void *)uniform, (const void *)noise, (const void *)tokens, (const void *)accepted,
                            (const void *)logprob})
        if (!aligned(ptr, 4)) return QMV_ERR_ALIGN;
    DeviceInfo dev;
    qmv_status st = current_device(&dev);
    if (st != QMV_OK) return st;
    void *ws = nullptr;
    st = scratch(dev, qmv_verify_workspace_size(B, S, V), workspace, workspace_bytes, &ws);
    if (st != QMV_OK) return st;

    const Split sp = split(B, S, V);
    VerifyParams p{};
    p.target = target; p.draft = draft; p.draft_tokens = draft_tokens; p.draft_len = draft_len;
    p.temperature = temperature; p.uniform = uniform; p.noise = noise;
    p.tokens = tokens; p.accepted = accepted; p.logprob = logprob;
    p.B = B; p.S = S; p.V = V;
    p.rows = draft ? 2 * S + 1 : S + 1;
    // a part is kVerifyThreads * nv vectors of 16 bytes, the last of a row short
    const int ev = f32 ? 4 : 8;
    p.nparts = ((V + ev - 1) / ev + kVerifyThreads * sp.nv - 1) / (kVerifyThreads * sp.nv);
    p.races = sp.races;
    p.ld_target = ld_target; p.ld_draft = ld_draft; p.ld_noise = ld_noise;
    uint8_t *at = static_cast<uint8_t *>(ws);
    p.parts = reinterpret_cast<Part *>(at); at += up256(size_t(B) * (2 * S + 1) * sp.nparts * sizeof(Part));
    p.winners = reinterpret_cast<Winner *>(at); at += up256(size_t(B) * sp.races * sizeof(Winner));
    p.finished = reinterpret_cast<unsigned *>(at);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = f32 ? launch_verify<true>(p, sp.nv, s) : launch_verify<false>(p, sp.nv, s);
    return e == cudaSuccess ? QMV_OK : record_cuda_failure("verify kernel launch", e);
}
