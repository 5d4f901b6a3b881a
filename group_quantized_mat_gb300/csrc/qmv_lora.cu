// qmv_lora_run: a group-quantized projection shared by M vectors plus each
// vector's own low-rank adapter,
//
//   y[m] = W x[m] + c_a B_a (A_a x[m]),   a = adapter[m].
//
// Two kernels.
//  1. lora_prepare stages x as operand cells (qmv_tile.cuh) and forms the inner
//     vectors A_a x[m] in fp32, both into the workspace.
//  2. lora_project streams W once per 16 vectors. It starts under the first
//     kernel (programmatic launch): its weights are on their way while x is
//     staged, and the inner vectors are needed only by its epilogue, so the
//     adapters' first half costs no time of its own.
//
// lora_project, one CTA per SM: a producer warp brings weights through a ring of
// shared-memory slots (boxes of 8 rows x cs subgroups by tensor map, scales and
// biases by 4-byte copies), eight consumer warps run the tiles, four epilogue
// warps join the consumers' sums, add the adapters' second half and store.
//  - Rows go to CTAs in eights (1920 of them for 15360 rows: 13 at most to an
//    SM where 12.6 would be even; in sixteens it would be 7 for 6.3).
//  - A block is up to 32 rows; consumer w takes the subgroups l with l % 8 = w
//    of the CTA's range of K, so an operand read of x serves two 16-row tiles
//    and all warps finish a block together.
//  - cs is odd: rows then start 32 (or 96) bytes apart modulo 128, and the eight
//    rows x four words of a tile's read cover all banks.
//  - K goes to CTAs in ranges of at most 64 subgroups (4096), whose cells of 16
//    vectors are 128 KB. Several ranges meet in the workspace: the CTA that
//    finishes a block last adds them in their order.
// The order of every sum depends on K alone, so a vector's result does not
// depend on the batch it is in.
#include <cuda_bf16.h>

#include <cstdint>
#include <cstdio>
#include <mutex>

#include "qmv.h"
#include "qmv_launch.cuh"
#include "qmv_tile.cuh"

namespace qmv {
namespace {

constexpr int kConsumers = 8, kEpilogue = 4;
constexpr int kThreads = 32 * (kConsumers + 1 + kEpilogue);
constexpr int kBlock = 32;        // rows of a block
constexpr int kPrepareThreads = 256;
constexpr int kMaxSlotsLora = 16;
constexpr int kSmem = 227 * 1024 - 1024;
constexpr int kMaxK = 1 << 18;

struct LoraParams {
    const uint16_t *scales, *biases, *x, *a, *b;
    const int32_t *adapter;
    const float *c;
    void *y;
    uint8_t *cells;      // [pass][S][tp][128]
    uint8_t *meta;       // [pass][S][nt][64]
    float *inner;        // [M][R]
    float *partials;     // [pass][nseg][N][8 nt], with nseg > 1
    unsigned *counters;  // [pass][NO], with nseg > 1
    unsigned *err;
    int M, N, K, G, L, R, f32_out;
    int S, cs, chunks, nseg, tp, nt, NO, grid_rows, slots, nsub_max, sbw, sbp, wbytes, ksplit, stage_blocks;
};

// Vectors of pass z.
__device__ __forceinline__ int pass_vectors(const LoraParams &p, int z) { return min(p.tp, p.M - z * p.tp); }

template <int BITS>
__global__ void __launch_bounds__(kPrepareThreads) lora_prepare(const LoraParams p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x;
    if (p.counters)
        for (int i = blockIdx.x * kPrepareThreads + tid; i < p.NO * ((p.M + p.tp - 1) / p.tp);
             i += gridDim.x * kPrepareThreads)
            p.counters[i] = 0u;
    if (int(blockIdx.x) < p.stage_blocks) {
        // eight threads for each (vector, subgroup), the subgroups of a vector in a row
        const long long at = (long long)blockIdx.x * kPrepareThreads + tid;
        const int o = int(at & 7);
        long long cell = at >> 3;
        const bool live = cell < (long long)p.M * p.S;
        if (!live) cell = (long long)p.M * p.S - 1;
        const int m = int(cell / p.S), sub = int(cell - (long long)m * p.S), z = m / p.tp, tok = m - z * p.tp;
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p.x + size_t(m) * p.K + sub * 64 + o * 8));
        uint8_t *c = p.cells + (size_t(z) * p.tp * p.S + size_t(sub) * pass_vectors(p, z) + tok) * tile::kCell;
        float *meta = reinterpret_cast<float *>(p.meta + ((size_t(z) * p.S + sub) * p.nt + tok / 8) * tile::kMeta);
        // threads past the end repeat the last cell's values (the warp's exchanges need them)
        tile::stage_octet<BITS>(v, o, tok, c, meta);
        return;
    }
    // inner vectors: ksplit warps for each (vector, row of A), each an even share of K
    __shared__ float part[kPrepareThreads / 32];
    const int warp = tid / 32, lane = tid % 32, per = kPrepareThreads / 32 / p.ksplit;
    const long long item = (long long)(int(blockIdx.x) - p.stage_blocks) * per + warp / p.ksplit;
    float s = 0.0f;
    int m = 0, r = 0, ad = -1;
    if (item < (long long)p.M * p.R) {
        m = int(item / p.R);
        r = int(item - (long long)m * p.R);
        ad = __ldg(p.adapter + m);
        if (ad >= 0 && ad < p.L) {
            const uint4 *a = reinterpret_cast<const uint4 *>(p.a + (size_t(ad) * p.R + r) * p.K);
            const uint4 *x = reinterpret_cast<const uint4 *>(p.x + size_t(m) * p.K);
            const int n8 = p.K / 8, kw = warp % p.ksplit;
            const int lo = int((long long)n8 * kw / p.ksplit), hi = int((long long)n8 * (kw + 1) / p.ksplit);
#pragma unroll 4
            for (int i = lo + lane; i < hi; i += 32) {
                const uint4 av = __ldg(a + i), xv = __ldg(x + i);
                const uint32_t aw[4] = {av.x, av.y, av.z, av.w}, xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s = __fmaf_rn(__uint_as_float(aw[j] << 16), __uint_as_float(xw[j] << 16), s);
                    s = __fmaf_rn(__uint_as_float(aw[j] & 0xffff0000u), __uint_as_float(xw[j] & 0xffff0000u), s);
                }
            }
        }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, d));
    if (lane == 0) part[warp] = s;
    __syncthreads();
    if (lane == 0 && warp % p.ksplit == 0 && ad >= 0 && ad < p.L) {
        for (int j = 1; j < p.ksplit; ++j) s = __fadd_rn(s, part[warp + j]);
        p.inner[size_t(m) * p.R + r] = s;
    }
}

struct Layout {
    int x, meta, slots, slot, sb, partial, bars, total;
};

__host__ __device__ inline Layout layout(const LoraParams &p, int nt)
{
    Layout l;
    l.x = 0;
    l.meta = l.x + p.nsub_max * p.tp * tile::kCell;
    l.slots = (l.meta + p.nsub_max * nt * tile::kMeta + 127) & ~127;
    l.sb = (p.wbytes + 127) & ~127;  // scales and biases of a slot, after its weights
    l.slot = (l.sb + 2 * kBlock * p.sbp * 4 + 127) & ~127;
    l.partial = l.slots + p.slots * l.slot;
    l.bars = l.partial + 2 * kConsumers * nt * kBlock * 8 * 4;
    l.total = l.bars + (2 * p.slots + 5) * 8 + 16;
    return l;
}

// c * (B v) of one output: row n of the adapter's B with the vector's inner.
__device__ __forceinline__ float adapter_term(const LoraParams &p, int ad, int m, int n)
{
    const uint16_t *b = p.b + (size_t(ad) * p.N + n) * p.R;
    const float *v = p.inner + size_t(m) * p.R;
    float d = 0.0f;
    if (p.R % 8 == 0) {
#pragma unroll 2
        for (int r = 0; r < p.R; r += 8) {
            const uint4 bw = __ldg(reinterpret_cast<const uint4 *>(b + r));
            const float4 v0 = *reinterpret_cast<const float4 *>(v + r), v1 = *reinterpret_cast<const float4 *>(v + r + 4);
            d = __fmaf_rn(__uint_as_float(bw.x << 16), v0.x, d);
            d = __fmaf_rn(__uint_as_float(bw.x & 0xffff0000u), v0.y, d);
            d = __fmaf_rn(__uint_as_float(bw.y << 16), v0.z, d);
            d = __fmaf_rn(__uint_as_float(bw.y & 0xffff0000u), v0.w, d);
            d = __fmaf_rn(__uint_as_float(bw.z << 16), v1.x, d);
            d = __fmaf_rn(__uint_as_float(bw.z & 0xffff0000u), v1.y, d);
            d = __fmaf_rn(__uint_as_float(bw.w << 16), v1.z, d);
            d = __fmaf_rn(__uint_as_float(bw.w & 0xffff0000u), v1.w, d);
        }
    } else {
#pragma unroll 4
        for (int r = 0; r < p.R; ++r) d = __fmaf_rn(__uint_as_float(uint32_t(__ldg(b + r)) << 16), v[r], d);
    }
    return __fmul_rn(__ldg(p.c + ad), d);
}

template <int BITS, int NT>
__global__ void __launch_bounds__(kThreads, 1) lora_project(const __grid_constant__ CUtensorMap map, const LoraParams p)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_abort, s_last;
    const Layout L = layout(p, NT);
    const uint32_t base = smem_u32(smem), full0 = base + L.bars, empty0 = full0 + 8 * p.slots;
    const uint32_t xbar = empty0 + 8 * p.slots, pfull0 = xbar + 8, pempty0 = pfull0 + 16;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int cta = blockIdx.x, seg = blockIdx.y, z = blockIdx.z;
    if (tid == 0) {
        for (int i = 0; i < p.slots; ++i) {
            mbar_init(full0 + 8 * i, 1 + 32);
            mbar_init(empty0 + 8 * i, kConsumers);
        }
        mbar_init(xbar, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(pfull0 + 8 * i, kConsumers);
            mbar_init(pempty0 + 8 * i, kEpilogue);
        }
        fence_mbar_init();
        s_abort = 0;
    }
    __syncthreads();

    const int oct_lo = int((long long)p.NO * cta / p.grid_rows), oct_hi = int((long long)p.NO * (cta + 1) / p.grid_rows);
    const int ch_lo = int((long long)p.chunks * seg / p.nseg), ch_hi = int((long long)p.chunks * (seg + 1) / p.nseg);
    const int sub_lo = ch_lo * p.cs, sub_hi = min(ch_hi * p.cs, p.S), nsub = sub_hi - sub_lo;
    const int nblocks = (oct_hi - oct_lo + kBlock / 8 - 1) / (kBlock / 8);
    const int nv = pass_vectors(p, z);
    const int gs_subs = p.S / p.G;  // subgroups in a group: 1 or 2
    const uint32_t pitch = uint32_t(p.cs) * (8 * BITS);
    // A wait that ran out: the error word is set and every warp stops.
    auto give_up = [&]() {
        atomicOr(p.err, 1u);
        *reinterpret_cast<volatile int *>(&s_abort) = 1;
    };
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (mbar_wait_bounded(bar, parity)) return *reinterpret_cast<volatile int *>(&s_abort) == 0;
        give_up();
        return false;
    };

    if (warp == kConsumers) {
        // ---------------------------------------------------------- producer
        int it = 0;
        bool ok = true;
        for (int bl = 0; bl < nblocks && ok; ++bl) {
            const int oct = oct_lo + bl * (kBlock / 8), nbox = min(kBlock / 8, oct_hi - oct), row0 = oct * 8;
            for (int c = ch_lo; c < ch_hi && ok; ++c, ++it) {
                const int slot = it % p.slots, lap = it / p.slots;
                const uint32_t full = full0 + 8 * slot, dst = base + L.slots + slot * L.slot;
                if (lap > 0) ok = wait(empty0 + 8 * slot, (lap - 1) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(full, uint32_t(nbox) * 8u * pitch);
                __syncwarp();
                if (lane < nbox) tma_load_2d(dst + lane * 8 * pitch, &map, c * p.cs * BITS, row0 + lane * 8, full);
                // scales and biases: the words that hold groups g0 .. of each row
                const int g0 = c * p.cs / gs_subs;
                const long long all = (long long)p.N * p.G;
                for (int i = lane; i < nbox * 8 * 16; i += 32) {
                    const int r = i >> 4, wd = i & 15;
                    if (wd >= p.sbw) continue;
                    const int n = row0 + r;
                    long long e = ((long long)n * p.G + g0) / 2 * 2 + 2 * wd;
                    uint32_t bytes = 0;
                    if (n < p.N && e < all) bytes = e + 1 < all ? 4 : 2;
                    if (!bytes) e = 0;
                    const uint32_t d = dst + L.sb + (r * p.sbp + wd) * 4;
                    tile::copy_word(d, p.scales + e, bytes);
                    tile::copy_word(d + kBlock * p.sbp * 4, p.biases + e, bytes);
                }
                tile::copy_arrive(full);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (!ok)  // copies in flight end before the CTA does
            for (int j = max(0, it - p.slots); j < it; ++j) (void)mbar_wait_bounded(full0 + 8 * (j % p.slots), (j / p.slots) & 1);
        return;
    }

    grid_launch_dependents();
    grid_dependency_wait();  // x cells and inner vectors
    if (warp < kConsumers) {
        // --------------------------------------------------------- consumers
        if (tid == 0) {
            asm volatile("fence.proxy.async;" ::: "memory");
            const uint32_t cb = uint32_t(nsub) * nv * tile::kCell, mb = uint32_t(nsub) * NT * tile::kMeta;
            mbar_arrive_expect_tx(xbar, cb + mb);
            bulk_load_plain(base + L.x, p.cells + (size_t(z) * p.tp * p.S + size_t(sub_lo) * nv) * tile::kCell, cb, xbar);
            bulk_load_plain(base + L.meta, p.meta + (size_t(z) * p.S + sub_lo) * NT * tile::kMeta, mb, xbar);
        }
        bool ok = __all_sync(0xffffffffu, wait(xbar, 0));
        const int g = lane / 4, t = lane % 4;
        uint32_t xcol[NT], odd[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int tok = min(n * 8 + g, nv - 1);
            xcol[n] = base + L.x + tok * tile::kCell + t * 32;
            odd[n] = (tok & 1) * 16;
        }
        int it = 0;
        for (int bl = 0; bl < nblocks && ok; ++bl) {
            const int oct = oct_lo + bl * (kBlock / 8);
            const bool two = oct_hi - oct > 2;
            const long long rowg = (long long)(oct * 8 + g) * p.G;
            uint64_t y[2][NT][2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n) y[i][n][0] = y[i][n][1] = 0ull;
            for (int c = ch_lo; c < ch_hi && ok; ++c, ++it) {
                const int slot = it % p.slots, lap = it / p.slots;
                ok = wait(full0 + 8 * slot, lap & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint32_t src = base + L.slots + slot * L.slot;
                const int l0 = c * p.cs - sub_lo, l1 = min(l0 + p.cs, nsub), g0 = c * p.cs / gs_subs;
                const uint32_t sb = src + L.sb + g * p.sbp * 4 + uint32_t((rowg + g0) & 1) * 2;
#pragma unroll 2
                for (int l = l0 + ((warp - l0) & (kConsumers - 1)); l < l1; l += kConsumers) {
                    const uint32_t w = src + g * pitch + (l - l0) * (8 * BITS) + t * (2 * BITS);
                    const uint32_t s = sb + ((sub_lo + l) / gs_subs - g0) * 2;
                    uint32_t x[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) x[n] = xcol[n] + l * nv * tile::kCell;
                    const uint32_t meta = base + L.meta + l * NT * tile::kMeta + t * 16;
                    if (two)
                        tile::add_subgroup<BITS, 2, NT>(y, w, pitch, s, s + kBlock * p.sbp * 4, p.sbp * 4, x, odd, meta);
                    else
                        tile::add_subgroup<BITS, 1, NT>(y, w, pitch, s, s + kBlock * p.sbp * 4, p.sbp * 4, x, odd, meta);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty0 + 8 * slot);
            }
            if (!ok) break;
            if (bl >= 2) ok = __all_sync(0xffffffffu, wait(pempty0 + 8 * (bl & 1), (bl / 2 - 1) & 1));
            if (!ok) break;
            uint64_t *out = reinterpret_cast<uint64_t *>(smem + L.partial) + ((bl & 1) * kConsumers + warp) * NT * kBlock * 4;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) out[(n * kBlock + 16 * i + 8 * h + g) * 4 + t] = y[i][n][h];
            __syncwarp();
            if (lane == 0) mbar_arrive(pfull0 + 8 * (bl & 1));
        }
        if (!ok && tid == 0) (void)mbar_wait_bounded(xbar, 0);
        return;
    }

    // ------------------------------------------------------------- epilogue
    const int et = tid - 32 * (kConsumers + 1);
    constexpr int kVals = NT * kBlock * 8;  // sums of a block
    for (int bl = 0; bl < nblocks; ++bl) {
        const int oct = oct_lo + bl * (kBlock / 8), row0 = oct * 8, rows = min(kBlock, (oct_hi - oct) * 8);
        if (!__all_sync(0xffffffffu, wait(pfull0 + 8 * (bl & 1), (bl / 2) & 1))) break;
        const float *in = reinterpret_cast<const float *>(smem + L.partial) + (bl & 1) * kConsumers * kVals;
        float v[kVals / (32 * kEpilogue)];
#pragma unroll
        for (int j = 0; j < kVals / (32 * kEpilogue); ++j) {
            float s = in[j * 32 * kEpilogue + et];
#pragma unroll
            for (int w = 1; w < kConsumers; ++w) s = __fadd_rn(s, in[w * kVals + j * 32 * kEpilogue + et]);
            v[j] = s;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(pempty0 + 8 * (bl & 1));
        bool mine = true;
        if (p.nseg > 1) {
            float *part = p.partials + (size_t(z) * p.nseg + seg) * p.N * (8 * NT);
#pragma unroll
            for (int j = 0; j < kVals / (32 * kEpilogue); ++j) {
                const int e = j * 32 * kEpilogue + et, r = e / 8 % kBlock, col = e / (8 * kBlock) * 8 + e % 8;
                if (r < rows && row0 + r < p.N) __stcg(part + size_t(row0 + r) * (8 * NT) + col, v[j]);
            }
            __threadfence();
            tile::named_sync(1, 32 * kEpilogue);
            if (et == 0) s_last = atomicAdd(p.counters + size_t(z) * p.NO + oct, 1u) == unsigned(p.nseg - 1);
            tile::named_sync(1, 32 * kEpilogue);
            mine = s_last != 0;
            if (mine) {
                __threadfence();
                part = p.partials + size_t(z) * p.nseg * p.N * (8 * NT);
#pragma unroll
                for (int j = 0; j < kVals / (32 * kEpilogue); ++j) {
                    const int e = j * 32 * kEpilogue + et, r = e / 8 % kBlock, col = e / (8 * kBlock) * 8 + e % 8;
                    if (r >= rows || row0 + r >= p.N) continue;
                    const float *q = part + size_t(row0 + r) * (8 * NT) + col;
                    float s = __ldcg(q);
                    for (int k = 1; k < p.nseg; ++k) s = __fadd_rn(s, __ldcg(q + size_t(k) * p.N * (8 * NT)));
                    v[j] = s;
                }
            }
        }
        if (!mine) continue;
#pragma unroll
        for (int j = 0; j < kVals / (32 * kEpilogue); ++j) {
            const int e = j * 32 * kEpilogue + et, n = row0 + e / 8 % kBlock, col = e / (8 * kBlock) * 8 + e % 8;
            if (e / 8 % kBlock >= rows || n >= p.N || col >= nv) continue;
            const int m = z * p.tp + col, ad = __ldg(p.adapter + m);
            float s = v[j];
            if (ad >= 0 && ad < p.L) s = __fadd_rn(s, adapter_term(p, ad, m, n));
            const size_t at = size_t(m) * p.N + n;
            if (p.f32_out) static_cast<float *>(p.y)[at] = s;
            else static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(s);
        }
    }
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Chunks (cs subgroups, odd) and ranges of K: at least ceil(S / 64) ranges (at
// most 8), and of the chunk sizes the one that leaves the longest range the
// shortest, the larger among equals. A function of S and bits alone.
void split_k(int S, int bits, int &cs, int &chunks, int &nseg)
{
    const int most = bits == 4 ? 15 : 31;
    nseg = (S + 63) / 64;
    if (nseg > 8) nseg = 8;
    int best = 1 << 30;
    cs = 1;
    for (int c = most; c >= 1; c -= 2) {
        if (c < 9 && S >= 9) break;
        const int n = (S + c - 1) / c, longest = (n + nseg - 1) / nseg * c;
        if (longest < best) {
            best = longest;
            cs = c;
        }
    }
    chunks = (S + cs - 1) / cs;
    if (nseg > chunks) nseg = chunks;
}

struct Sizes {
    size_t cells, meta, inner, counters, partials, total;
};

size_t up256(size_t b) { return (b + 255) & ~size_t(255); }

LoraParams plan(int M, int N, int K, int bits, int gs, int R, Sizes &sz)
{
    LoraParams p{};
    p.M = M; p.N = N; p.K = K; p.G = K / gs; p.R = R;
    p.S = K / 64;
    split_k(p.S, bits, p.cs, p.chunks, p.nseg);
    p.nsub_max = (p.chunks + p.nseg - 1) / p.nseg * p.cs;
    p.tp = 16;
    while (p.tp > 1 && p.tp * p.nsub_max > 1024) p.tp /= 2;
    p.nt = M > 8 && p.tp > 8 ? 2 : 1;
    if (p.nt == 1 && p.tp > 8) p.tp = 8;
    p.NO = (N + 7) / 8;
    const int groups = gs == 64 ? p.cs : p.cs / 2 + 1;  // groups that a chunk can touch
    p.sbw = (groups + 2) / 2;                           // words that hold them, from an even element on
    p.sbp = p.sbw | 1;
    p.wbytes = kBlock * p.cs * 8 * bits;
    p.ksplit = K <= 4096 ? 1 : K <= 8192 ? 2 : K <= 16384 ? 4 : 8;
    const size_t passes = (M + p.tp - 1) / p.tp;
    sz.cells = up256(size_t(M) * p.S * tile::kCell);
    sz.meta = up256(passes * p.S * p.nt * tile::kMeta);
    sz.inner = up256(size_t(M) * R * 4);
    sz.counters = p.nseg > 1 ? up256(passes * p.NO * 4) : 0;
    sz.partials = p.nseg > 1 ? up256(passes * p.nseg * size_t(N) * 8 * p.nt * 4) : 0;
    sz.total = sz.cells + sz.meta + sz.inner + sz.counters + sz.partials;
    return p;
}

template <int BITS, int NT>
cudaError_t launch_project(const CUtensorMap &map, const LoraParams &p, int passes, cudaStream_t stream)
{
    static std::atomic<int> configured[64] = {};
    Launch l;
    l.grid = dim3(p.grid_rows, p.nseg, passes);
    l.threads = kThreads;
    l.smem = size_t(layout(p, NT).total);
    l.pdl = true;
    return launch_one(lora_project<BITS, NT>, configured, l, stream, map, p);
}

template <int BITS>
cudaError_t launch_lora(const CUtensorMap &map, const LoraParams &p, int passes, cudaStream_t stream)
{
    static std::atomic<int> configured[64] = {};
    Launch l;
    const int per = kPrepareThreads / 32 / p.ksplit;
    l.grid = dim3(p.stage_blocks + (p.M * p.R + per - 1) / per);
    l.threads = kPrepareThreads;
    l.smem = 0;
    l.pdl = true;
    const cudaError_t e = launch_one(lora_prepare<BITS>, configured, l, stream, p);
    if (e != cudaSuccess) return e;
    return p.nt == 2 ? launch_project<BITS, 2>(map, p, passes, stream) : launch_project<BITS, 1>(map, p, passes, stream);
}

}  // namespace
}  // namespace qmv

extern "C" size_t qmv_lora_workspace_size(int M, int N, int K, int bits, int group_size, int rank)
{
    if (qmv::check_weights(M, N, K, bits, group_size) != QMV_OK || K > qmv::kMaxK || rank < 1 || rank > QMV_MAX_RANK)
        return 0;
    qmv::Sizes sz;
    qmv::plan(M, N, K, bits, group_size, rank, sz);
    return sz.total;
}

extern "C" qmv_status qmv_lora_run(const uint32_t *w_q, const uint16_t *scales, const uint16_t *biases,
                                   const uint16_t *x, const uint16_t *lora_a, const uint16_t *lora_b,
                                   const int32_t *adapter, const float *lora_scale, void *y, int M, int N, int K,
                                   int bits, int group_size, int adapters, int rank, void *workspace,
                                   size_t workspace_bytes, unsigned flags, qmv_stream_t stream)
{
    using namespace qmv;
    if (!w_q || !scales || !biases || !x || !lora_a || !lora_b || !adapter || !lora_scale || !y) return QMV_ERR_NULL;
    qmv_status st = check_weights(M, N, K, bits, group_size);
    if (st != QMV_OK) return st;
    if (K > kMaxK) return QMV_ERR_SHAPE;
    if (adapters < 1 || adapters > QMV_MAX_ADAPTERS || rank < 1 || rank > QMV_MAX_RANK) return QMV_ERR_COUNT;
    if (flags & ~QMV_F32_OUT) return QMV_ERR_FLAGS;
    if (!aligned(w_q, 16) || !aligned(scales, 16) || !aligned(biases, 16) || !aligned(x, 16) || !aligned(lora_a, 16) ||
        !aligned(lora_b, 16) || !aligned(adapter, 4) || !aligned(lora_scale, 4) ||
        !aligned(y, flags & QMV_F32_OUT ? 4 : 2) || (workspace && !aligned(workspace, 16)))
        return QMV_ERR_ALIGN;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != QMV_OK) return st;
    Sizes sz;
    LoraParams p = plan(M, N, K, bits, group_size, rank, sz);
    void *ws = nullptr;
    st = scratch(dev, sz.total, workspace, workspace_bytes, &ws);
    if (st != QMV_OK) return st;

    p.scales = scales; p.biases = biases; p.x = x; p.a = lora_a; p.b = lora_b;
    p.adapter = adapter; p.c = lora_scale; p.y = y; p.err = dev.err;
    p.L = adapters;
    p.f32_out = (flags & QMV_F32_OUT) != 0;
    uint8_t *at = static_cast<uint8_t *>(ws);
    p.cells = at; at += sz.cells;
    p.meta = at; at += sz.meta;
    p.inner = reinterpret_cast<float *>(at); at += sz.inner;
    p.counters = p.nseg > 1 ? reinterpret_cast<unsigned *>(at) : nullptr; at += sz.counters;
    p.partials = p.nseg > 1 ? reinterpret_cast<float *>(at) : nullptr;
    p.stage_blocks = int(((long long)M * p.S * 8 + kPrepareThreads - 1) / kPrepareThreads);
    p.grid_rows = dev.sms / p.nseg;
    if (p.grid_rows < 1) p.grid_rows = 1;
    if (p.grid_rows > p.NO) p.grid_rows = p.NO;
    const int passes = (M + p.tp - 1) / p.tp;
    // as many slots as fit
    p.slots = 2;
    while (p.slots < kMaxSlotsLora) {
        ++p.slots;
        if (layout(p, p.nt).total > kSmem) {
            --p.slots;
            break;
        }
    }
    if (layout(p, p.nt).total > kSmem) return record_cuda_failure("lora launch plan", cudaErrorInvalidConfiguration);

    CUtensorMap map;
    st = encode_rows(&map, w_q, (long long)K * bits / 8, N, p.cs * bits, 8);
    if (st != QMV_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = bits == 4 ? launch_lora<4>(map, p, passes, s) : launch_lora<2>(map, p, passes, s);
    return e == cudaSuccess ? QMV_OK : record_cuda_failure("lora kernel launch", e);
}
