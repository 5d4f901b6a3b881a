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
//  1. verify_rows reads the logits once, 16 bytes at a time. A warp takes parts of
//     rows in turn and goes through each in pieces of 4 KB: a piece stays in
//     registers from its maximum to its sum while the next one's loads, of the
//     same part or of the next, are in flight; warps never wait for one another.
//     Rows that no outcome needs (past a sequence's drafts; draft rows where the
//     argmax decides) are not read. It is bound by memory, with the integer pipe
//     and the exponentials close behind (5 instructions an element).
//  2. verify_emit, several blocks to a sequence: each joins the parts of the
//     sequence's rows, decides how many tokens are accepted and runs its share of
//     the race on the one row that matters; the last of a sequence's blocks joins
//     the winners and writes the results.
//
// Measured (us; bytes of the rows that are needed, at 6.7 TB/s): 14.2 for one sequence
// of 3 drafts and 32000 tokens (0.1: the two kernels' chain), 18 for 8 x 4 x 50257 fp32
// from unaligned rows (1.5), 31 for 24 x 12 looked-up drafts of 101001 (7), 60 for
// 64 x 7 x 131072 (31: 41 us of rows, then 18 of race).
#include <cuda_bf16.h>

#include <cfloat>
#include <cstdint>

#include "qmv.h"
#include "qmv_launch.cuh"

namespace qmv {
namespace {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kRowThreads = 128, kRowBlocks = 4;  // of verify_rows, and blocks on an SM
constexpr int kMaxParts = 16;                     // of a row at most
constexpr int kNone = 0x7fffffff;
constexpr int kRace = 8 * kVerifyThreads;  // tokens of a block of verify_emit
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
    // (a number, and times log2 e still one: 0 at the maximum stays 0)
    m.inv = m.greedy ? 1.0f : fminf(fmaxf(__fdiv_rn(1.0f, t), FLT_MIN), 2e38f);
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
// The larger, NaN where one is NaN.
template <bool F32>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b)
{
    uint32_t d;
    if (F32) asm("max.NaN.f32 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ float larger(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
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

// The 16 bytes of a row from element v0 on, element by element, those past V as
// -inf (nothing beside the row is read).
template <bool F32>
__device__ __noinline__ uint4 load16_apart(const uint8_t *base, long long v0, int V)
{
    constexpr int EV = F32 ? 4 : 8;
    const uint32_t none = F32 ? 0xff800000u : 0xff80ff80u;
    uint32_t w[4] = {none, none, none, none};
#pragma unroll
    for (int i = 0; i < EV; ++i) {
        if (v0 + i >= V) break;
        if (F32) w[i & 3] = __ldg(reinterpret_cast<const uint32_t *>(base) + v0 + i);
        else {
            const uint32_t h = __ldg(reinterpret_cast<const uint16_t *>(base) + v0 + i);
            w[i / 2 & 3] = i & 1 ? (w[i / 2 & 3] & 0xffffu) | h << 16 : (w[i / 2 & 3] & 0xffff0000u) | h;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// N vectors of 16 bytes of a row, from element v0 on and `step` elements apart.
// Inside the row one aligned load each, or where the row lies off a 16-byte
// boundary (`off` bytes) two that are shifted; at its ends apart.
template <bool F32, int N>
__device__ __forceinline__ void load16(uint4 (&x)[N], const uint8_t *base, long long v0, int step, int V, int off)
{
    constexpr int EV = F32 ? 4 : 8, SIZE = F32 ? 4 : 2;
    const uint8_t *at = base + v0 * SIZE;
    if (off == 0 && v0 + (N - 1) * step + EV <= V) {
#pragma unroll
        for (int k = 0; k < N; ++k) x[k] = __ldcs(reinterpret_cast<const uint4 *>(at + k * step * SIZE));
    } else if (off != 0 && v0 > 0 && v0 + (N - 1) * step + 2 * EV <= V) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const uint4 *q = reinterpret_cast<const uint4 *>(at + k * step * SIZE - off);
            x[k] = shifted(__ldg(q), __ldg(q + 1), off);
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) x[k] = load16_apart<F32>(base, v0 + k * step, V);
    }
}

// Maximum, sum and first argmax of the pieces that a warp has seen.
template <bool F32>
struct Seen {
    static constexpr int EV = F32 ? 4 : 8, kVecs = 8, kElems = kVecs * 32 * EV;
    float top = -INFINITY, sum = 0.0f;  // the sum is the lane's own
    int arg = kNone;

    static __device__ __forceinline__ void load(uint4 (&x)[kVecs], const uint8_t *base, int piece, int V, int off, int lane)
    {
        load16<F32, kVecs>(x, base, (long long)piece * kElems + lane * EV, 32 * EV, V, off);
    }

    // By elements' indexes alone, so that equal rows have equal sums wherever they lie.
    __device__ __forceinline__ void add(uint4 (&x)[kVecs], int piece, float c, bool greedy, int lane)
    {
        float here;
        for (int pass = 0; pass < 2; ++pass) {
            uint32_t top2 = F32 ? 0xff800000u : 0xff80ff80u;
#pragma unroll
            for (int k = 0; k < kVecs; ++k) top2 = larger<F32>(top2, larger<F32>(larger<F32>(x[k].x, x[k].y), larger<F32>(x[k].z, x[k].w)));
            here = F32 ? __uint_as_float(top2) : larger(__uint_as_float(top2 << 16), __uint_as_float(top2 & 0xffff0000u));
#pragma unroll
            for (int d = 16; d; d >>= 1) here = larger(here, __shfl_xor_sync(0xffffffffu, here, d));
            if (here < INFINITY) break;
            // a NaN or +inf among them, seldom: what they count as
#pragma unroll
            for (int k = 0; k < kVecs; ++k) x[k] = make_uint4(clean<F32>(x[k].x), clean<F32>(x[k].y), clean<F32>(x[k].z), clean<F32>(x[k].w));
        }
        if (!(here > -INFINITY)) return;
        if (greedy && here > top) {
            // the first place of a new maximum
            arg = kNone;
#pragma unroll
            for (int k = 0; k < kVecs; ++k) {
                const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
                for (int i = 0; i < EV; ++i) {
                    const float l = F32 ? __uint_as_float(w[i & 3])
                                        : __uint_as_float(i & 1 ? w[i / 2 & 3] & 0xffff0000u : w[i / 2 & 3] << 16);
                    if (l == here) arg = min(arg, piece * kElems + (k * 32 + lane) * EV + i);
                }
            }
            arg = __reduce_min_sync(0xffffffffu, arg);
        }
        if (here > top) {
            sum = top > -INFINITY ? __fmul_rn(sum, ex2(__fmul_rn(__fsub_rn(top, here), c))) : 0.0f;
            top = here;
        }
        const uint64_t neg = pair_of(-top, -top), cc = pair_of(c, c);
        uint64_t s2 = pair_of(sum, 0.0f);
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
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
    }
};

// Where a warp is in its parts of rows.
template <bool F32>
struct Place {
    int item, piece, end;  // row of all rows * nparts + part, -1: none left
    const uint8_t *base;
    float c;
    bool greedy;

    // The first part from `from` on, in steps of `step`, that an outcome needs.
    __device__ __forceinline__ void find(const VerifyParams &p, long long from, int step, int items, int pieces)
    {
        for (; from < items; from += step) {
            item = int(from);
            const int row = item / p.nparts, part = item - row * p.nparts, b = row / p.rows, r = row - b * p.rows;
            const Mode m = mode_of(p, b);
            if (r <= p.S ? r > m.len : m.greedy || r - p.S - 1 >= m.len) continue;
            base = static_cast<const uint8_t *>(row_of<F32>(p, b, r));
            piece = int((long long)pieces * part / p.nparts);
            end = int((long long)pieces * (part + 1) / p.nparts);
            c = __fmul_rn(m.inv, 1.4426950408889634f);
            greedy = m.greedy;
            return;
        }
        item = -1;
    }
    __device__ __forceinline__ void advance(const VerifyParams &p, int step, int items, int pieces)
    {
        if (++piece >= end) find(p, (long long)item + step, step, items, pieces);
    }
};

template <bool F32>
__global__ void __launch_bounds__(kRowThreads, kRowBlocks) verify_rows(const VerifyParams p)
{
    using See = Seen<F32>;
    const int lane = threadIdx.x % 32, step = gridDim.x * (kRowThreads / 32), items = p.B * p.rows * p.nparts;
    const int pieces = (p.V + See::kElems - 1) / See::kElems;
    grid_dependency_wait();
    grid_launch_dependents();
    for (int i = blockIdx.x * kRowThreads + threadIdx.x; i < p.B; i += gridDim.x * kRowThreads) p.finished[i] = 0u;
    auto load = [&](uint4(&x)[See::kVecs], const Place<F32> &at) {
        See::load(x, at.base, at.piece, p.V, int(reinterpret_cast<uintptr_t>(at.base) & 15), lane);
    };
    See seen;
    // adds the piece at `at`; where `next` is of another part, the part is done
    auto take = [&](uint4(&x)[See::kVecs], const Place<F32> &at, const Place<F32> &next) {
        seen.add(x, at.piece, at.c, at.greedy, lane);
        if (next.item == at.item) return;
        float sum = seen.sum;
#pragma unroll
        for (int d = 16; d; d >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, d));
        if (lane == 0) p.parts[at.item] = {seen.top, sum, seen.arg, 0};
        seen = See();
    };
    // two sets of registers take turns
    Place<F32> a, b;
    uint4 x[See::kVecs], y[See::kVecs];
    a.find(p, (long long)blockIdx.x * (kRowThreads / 32) + threadIdx.x / 32, step, items, pieces);
    if (a.item >= 0) load(x, a);
    while (a.item >= 0) {
        b = a;
        b.advance(p, step, items, pieces);
        if (b.item >= 0) load(y, b);
        take(x, a, b);
        if (b.item < 0) break;
        a = b;
        a.advance(p, step, items, pieces);
        if (a.item >= 0) load(x, a);
        take(y, b, a);
    }
}

// p or q of a logit (-inf: no token) in a row, 0 where the row has none.
__device__ __forceinline__ float prob(float l, float top, float sum, float inv)
{
    if (!(l > -INFINITY)) return 0.0f;
    return __fdiv_rn(expf(__fmul_rn(__fsub_rn(l, top), inv)), sum);
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
__global__ void __launch_bounds__(kVerifyThreads, 3) verify_emit(const VerifyParams p)
{
    __shared__ float s_max[kMaxRows], s_sum[kMaxRows], sv[kVerifyWarps];
    __shared__ int s_arg[kMaxRows], s_ok[QMV_MAX_DRAFT + 1], si[kVerifyWarps], s_last, s_bound;
    if (threadIdx.x == 0) s_bound = 0;
    const int tid = threadIdx.x, b = blockIdx.x / p.races, race = blockIdx.x - b * p.races;
    // (none of these is written by the first kernel)
    const Mode m = mode_of(p, b);
    int drafted = -1;
    float u = 0.0f, lt = -INFINITY, ld = -INFINITY;
    if (tid < m.len) {
        drafted = __ldg(p.draft_tokens + size_t(b) * p.S + tid);
        u = __ldg(p.uniform + size_t(b) * p.S + tid);
        if (drafted >= 0 && drafted < p.V) {
            lt = logit<F32>(row_of<F32>(p, b, tid), drafted);
            if (p.draft) ld = logit<F32>(row_of<F32>(p, b, p.S + 1 + tid), drafted);
        }
    }
    grid_dependency_wait();
    grid_launch_dependents();
    const Part *parts = p.parts + (size_t)b * p.rows * p.nparts;
    if (tid < p.rows && !(tid <= p.S ? tid > m.len : m.greedy || tid - p.S - 1 >= m.len)) {
        // a row to a thread, its few parts in order
        float top = -INFINITY, sum = 0.0f;
        int arg = kNone;
        const Part *q = parts + (size_t)tid * p.nparts;
#pragma unroll
        for (int k = 0; k < kMaxParts; ++k)
            if (k < p.nparts) top = fmaxf(top, __ldcg(&q[k].max));
#pragma unroll 4
        for (int k = 0; k < p.nparts; ++k) {
            const int4 raw = __ldcg(reinterpret_cast<const int4 *>(q + k));
            const float pm = __int_as_float(raw.x);
            if (pm > -INFINITY) sum = __fmaf_rn(__int_as_float(raw.y), expf(__fmul_rn(__fsub_rn(pm, top), m.inv)), sum);
            if (pm == top) arg = min(arg, raw.z);
        }
        s_max[tid] = top;
        s_sum[tid] = sum;
        s_arg[tid] = arg;
    }
    __syncthreads();
    if (tid <= m.len) {
        bool ok = false;
        if (tid < m.len) {
            if (m.greedy) ok = s_max[tid] > -INFINITY && drafted == s_arg[tid];
            else {
                const int d = p.S + 1 + tid;
                const float q = p.draft ? prob(ld, s_max[d], s_sum[d], m.inv) : 1.0f;
                ok = __fmul_rn(u, q) < prob(lt, s_max[tid], s_sum[tid], m.inv);
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
        // A token enters the race by its exact ratio: two exponentials and two
        // divisions. Most are ruled out before: at first by p alone against the
        // noise and the block's best lower bound of a ratio so far (one exponential,
        // no division; 2e-4 off the bound for the approximations' errors), the rest
        // by the token's upper bound. Eight tokens to a lane at a time. (Bounds of
        // both kinds for every token: 46 instructions each and 48 of 80 us at
        // 64 x 131072.)
        const float c = __fmul_rn(m.inv, 1.4426950408889634f), itotal = __fdiv_rn(1.0f, total);
        const float idsum = dtop > -INFINITY ? __fdiv_rn(1.0f, dsum) : 0.0f, dref = dtop > -INFINITY ? dtop : 0.0f;
        const uint8_t *rowb = static_cast<const uint8_t *>(row), *drowb = static_cast<const uint8_t *>(drow);
        const uint8_t *noiseb = reinterpret_cast<const uint8_t *>(noise);
        const int roff = int(reinterpret_cast<uintptr_t>(rowb) & 15), doff = int(reinterpret_cast<uintptr_t>(drowb) & 15);
        const int noff = int(reinterpret_cast<uintptr_t>(noiseb) & 15), lane = tid % 32;
        float bound = 0.0f;
        constexpr int LW = F32 ? 2 : 1;
        struct Eight {
            uint4 l[LW], d[LW], e[2];
        };
        const auto fetch = [&](Eight &t, int share, bool rest) {
            const long long v0 = (long long)share * 256 + lane * 8;
            load16<F32, LW>(t.l, rowb, v0, F32 ? 4 : 8, p.V, roff);
            load16<true, 2>(t.e, noiseb, v0, 4, p.V, noff);
            if (rest && dtop > -INFINITY) load16<F32, LW>(t.d, drowb, v0, F32 ? 4 : 8, p.V, doff);
            else
#pragma unroll
                for (int k = 0; k < LW; ++k) t.d[k] = F32 ? make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u) : make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
        };
        const auto word = [](const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; };
        const auto value = [&](const uint4 (&v)[LW], int k, bool as_it_counts) {
            uint32_t w = F32 ? word(v[k / 4 * (LW - 1)], k & 3) : word(v[0], k / 2);
            if (as_it_counts) w = clean<F32>(w);
            return F32 ? __uint_as_float(w) : __uint_as_float(k & 1 ? w & 0xffff0000u : w << 16);
        };
        const auto race8 = [&](Eight &t, int share, bool rest) {
            const int v0 = share * 256 + lane * 8;
            bound = fmaxf(bound, __int_as_float(*const_cast<volatile int *>(&s_bound)));
            const float sure = __fmul_rn(bound, 0.9998f);
            uint32_t left = 0;  // tokens that are not ruled out (nor is what is NaN)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float pa = __fmul_rn(ex2(__fmul_rn(__fsub_rn(value(t.l, k, false), top), c)), itotal);
                if (!(pa < __fmul_rn(sure, __uint_as_float(word(t.e[k / 4], k & 3))))) left |= 1u << k;
            }
            if (!__any_sync(0xffffffffu, left)) return;
            if (rest && (cut & ~7) == v0 && cut >= 0) left &= ~(1u << (cut & 7));  // the refused token, its draft being certain, has nothing left
            float upper[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                upper[k] = 0.0f;
                if (!(left >> k & 1)) continue;
                const float pa = __fmul_rn(ex2(__fmul_rn(__fsub_rn(value(t.l, k, true), top), c)), itotal);
                const float qa = __fmul_rn(ex2(__fmul_rn(__fsub_rn(value(t.d, k, true), dref), c)), idsum);
                const float w = __fsub_rn(pa, qa);
                const float e = fmaxf(__uint_as_float(clean<true>(word(t.e[k / 4], k & 3))), FLT_MIN);
                // (a reciprocal of more than 2^126 comes out as 0)
                const float ea = fminf(e, 8e37f);
                float r;
                asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ea));
                upper[k] = __fmul_rn(__fmaf_rn(1e-5f, pa, w), __fmul_rn(r, 1.0001f));
                const float lower = __fmul_rn(__fmaf_rn(-1e-5f, pa, w), __fmul_rn(r, 0.9999f));
                if (e == ea) bound = fmaxf(bound, lower);
            }
#pragma unroll
            for (int d = 16; d; d >>= 1) bound = fmaxf(bound, __shfl_xor_sync(0xffffffffu, bound, d));
            if (lane == 0) atomicMax(&s_bound, __float_as_int(bound));  // (not below 0, so ordered as integers)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (!(upper[k] > 0.0f) || upper[k] < bound) continue;
                const float l = value(t.l, k, true), d = value(t.d, k, true);
                const float e = fmaxf(__uint_as_float(clean<true>(word(t.e[k / 4], k & 3))), FLT_MIN);
                float w = __fdiv_rn(expf(__fmul_rn(__fsub_rn(l, top), m.inv)), total);
                if (d > -INFINITY) w = __fsub_rn(w, __fdiv_rn(expf(__fmul_rn(__fsub_rn(d, dtop), m.inv)), dsum));
                if (w > 0.0f) {
                    const float ratio = __fdiv_rn(w, e);
                    if (better(ratio, v0 + k, best, token)) {
                        best = ratio;
                        token = v0 + k;
                    }
                }
            }
        };
        const int shares = (p.V + 255) / 256;
        const auto run = [&](int from, int step, bool rest) {
            // two sets of registers take turns
            Eight t, u;
            if (from < shares) fetch(t, from, rest);
            for (int share = from; share < shares; share += 2 * step) {
                if (share + step < shares) fetch(u, share + step, rest);
                race8(t, share, rest);
                if (share + step >= shares) break;
                if (share + 2 * step < shares) fetch(t, share + 2 * step, rest);
                race8(u, share + step, rest);
            }
        };
        run(race * kVerifyWarps + tid / 32, p.races * kVerifyWarps, true);
        block_best(best, token, sv, si);
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
        if (token == kNone) {
            // p has nothing that q has not: p itself
            bound = 0.0f;
            best = -1.0f;
            if (tid == 0) s_bound = 0;
            __syncthreads();
            run(tid / 32, kVerifyWarps, false);
            block_best(best, token, sv, si);
        }
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

// Parts of a row: at least a piece each. Blocks of the race: at most three for each
// of 152 SMs (one wave), each at least kRace tokens (every block joins the parts of
// its sequence's rows for itself, and its warps start without a bound: for 64 x 131072
// the whole call took 69 us with at most 304 blocks, 64.5 with 456, 73 with 912; and
// 60 with 456 whose warps share their bound).
struct Split {
    int nparts, races;
};

Split split(int B, int V, bool f32)
{
    Split s;
    const int elems = f32 ? Seen<true>::kElems : Seen<false>::kElems;
    s.nparts = (V + elems - 1) / elems;
    if (s.nparts > kMaxParts) s.nparts = kMaxParts;
    s.races = (V + kRace - 1) / kRace;
    const int blocks = B < 456 ? 456 / B : 1;
    if (s.races > blocks) s.races = blocks;
    return s;
}

size_t up256(size_t b) { return (b + 255) & ~size_t(255); }

template <bool F32>
cudaError_t launch_verify(const VerifyParams &p, int sms, cudaStream_t stream)
{
    static std::atomic<int> configured[2][64] = {};
    Launch l;
    const int blocks = (p.B * p.rows * p.nparts + kRowThreads / 32 - 1) / (kRowThreads / 32);
    l.grid = dim3(blocks < kRowBlocks * sms ? blocks : kRowBlocks * sms);
    l.threads = kRowThreads;
    l.smem = 0;
    l.pdl = true;
    const cudaError_t e = launch_one(verify_rows<F32>, configured[0], l, stream, p);
    if (e != cudaSuccess) return e;
    l.grid = dim3(unsigned(p.B * p.races));
    l.threads = kVerifyThreads;
    return launch_one(verify_emit<F32>, configured[1], l, stream, p);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace qmv

extern "C" size_t qmv_verify_workspace_size(int B, int S, int V)
{
    if (B < 1 || B > QMV_MAX_BATCH || S < 0 || S > QMV_MAX_DRAFT || V < 1 || V > (1 << 24)) return 0;
    const qmv::Split s = qmv::split(B, V, true);  // the wider type has more parts
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

    const Split sp = split(B, V, f32);
    VerifyParams p{};
    p.target = target; p.draft = draft; p.draft_tokens = draft_tokens; p.draft_len = draft_len;
    p.temperature = temperature; p.uniform = uniform; p.noise = noise;
    p.tokens = tokens; p.accepted = accepted; p.logprob = logprob;
    p.B = B; p.S = S; p.V = V;
    p.rows = draft ? 2 * S + 1 : S + 1;
    p.nparts = sp.nparts;
    p.races = sp.races;
    p.ld_target = ld_target; p.ld_draft = ld_draft; p.ld_noise = ld_noise;
    uint8_t *at = static_cast<uint8_t *>(ws);
    p.parts = reinterpret_cast<Part *>(at); at += up256(size_t(B) * (2 * S + 1) * sp.nparts * sizeof(Part));
    p.winners = reinterpret_cast<Winner *>(at); at += up256(size_t(B) * sp.races * sizeof(Winner));
    p.finished = reinterpret_cast<unsigned *>(at);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = f32 ? launch_verify<true>(p, dev.sms, s) : launch_verify<false>(p, dev.sms, s);
    return e == cudaSuccess ? QMV_OK : record_cuda_failure("verify kernel launch", e);
}
