// qmv_lora_run: a group-quantized projection shared by M vectors plus each
// vector's own low-rank adapter,
//
//   y[m] = W x[m] + c_a B_a (A_a x[m]),   a = adapter[m].
//
// Two kernels.
//  1. lora_prepare stages x as operand cells (qmv_tile.cuh) and forms the inner
//     vectors A_a x[m] in fp32, both into the workspace. (Every CTA of the second
//     kernel staging x for itself took 3 us for 4 vectors, where the first kernel
//     and a copy take 1.7.)
//  2. lora_project streams W once per 16 vectors. It starts under the first
//     kernel (programmatic launch) and asks for its first weights meanwhile; the
//     rest, which fills the memory system for microseconds, it asks for after the
//     staged x.
//
// lora_project, one CTA per SM: a producer warp brings 128 bytes of each row of
// a tile, with their scales and biases, to a ring of shared-memory slots (one
// tensor-map box, 128-byte swizzle), three groups of worker warps run the tiles,
// three tensor warps multiply. A worker thread owns a row. The rows of the pass's
// adapters follow a tile's weights through the ring, each adapter once however
// many vectors have it, and each thread adds their products with the inner
// vectors to the sums it holds. (Threads reading their rows from global memory,
// 16 bytes at a time, took 16 of a tile's 47 thousand cycles at 16 vectors of
// rank 64: 168 us for 64 vectors. A third of every product in each group, before
// the groups' sums meet: 123 us, and 25.1 for 16 vectors where this takes 23.7.)
//  - Rows go to CTAs in tiles of equal height (a multiple of 8, at most 128): 104
//    for 15360 rows on 152 SMs.
//  - K goes to CTAs in ranges of at most 64 subgroups (4096), whose cells of 16
//    vectors are 128 KB (48 at ranks above 64). Several ranges meet in the workspace: the CTA that
//    finishes a tile last adds them in their order.
//  - Passes of 16 vectors follow one another in a CTA, the next one's x on its way
//    while the last tile's adapters are added; partial sums of ranges are joined a
//    tile later, so that nobody waits for a ticket. (A CTA for each pass: 135 us for
//    64 vectors, 32.9 for 24 of 5120 x 5120.)
// What bounds it: for few vectors the chain of the two kernels' starts, x, first
// weights and the join; for 16 the workers' instructions (qmv_tile.cuh) and the
// adapters' code, which runs from a cold instruction cache; above 16 every further 16
// pay for the unpacking again. Measured (us; bytes it cannot do without, at 6.7 TB/s):
// 10.7 for one vector of 1024 x 5120 (0.5), 14.8 for 4 of 15360 x 3840 (5.2), 23.2 for
// 13 of 3840 x 15360 (6.0), 117 for 64 of 17408 x 5120 in 2 bits at rank 64 (9.7); of
// 15360 x 3840 at rank 16, 24.9 for 16 vectors, 40.7 for 32 (5.9) and 73 for 64 (6.1).
// The order of an output's sums depends on N, K, the rank, its row and its adapter's number
// (which says with which range of K the adapter is added), so a vector's result depends
// neither on the batch it is in nor on the card.
#include <cuda_bf16.h>

#include <cstdint>
#include <mutex>

#include "qmv.h"
#include "qmv_launch.cuh"
#include "qmv_lora_plan.h"
#include "qmv_tile.cuh"

namespace qmv {
namespace {

using namespace lora;

constexpr int kPrepareThreads = 256;
constexpr int kBefore = 3;      // slots of weights asked for before staged x (no more than a ring has)

struct LoraParams : LoraShape {
    const uint16_t *scales, *biases, *x, *a, *b;
    const int32_t *adapter;
    const float *c;
    void *y;
    uint8_t *cells;      // [pass][subs][cell_bytes]
    uint8_t *meta;       // [pass][subs][meta_bytes]
    float *inner;        // [M][inner_pitch(R)]
    float *partials;     // [pass][nseg][nc][N], with nseg > 1
    unsigned *counters;  // [pass][tiles], with nseg > 1
    unsigned *err;
    int L, f32_out, stage_blocks;
};

template <int BITS, int NC>
__global__ void __launch_bounds__(kPrepareThreads) lora_prepare(const LoraParams p)
{
    grid_dependency_wait();
    const int tid = threadIdx.x, passes = (p.M + kPass - 1) / kPass;
    if (p.counters)
        for (int i = blockIdx.x * kPrepareThreads + tid; i < p.tiles * passes; i += gridDim.x * kPrepareThreads)
            p.counters[i] = 0u;
    if (int(blockIdx.x) < p.stage_blocks) {
        // eight threads for each (vector, subgroup), the subgroups of a vector in a row
        const long long at = (long long)blockIdx.x * kPrepareThreads + tid;
        const int o = int(at & 7);
        long long cell = at >> 3;
        // threads past the end repeat the last cell's values (the warp's exchanges need them)
        if (cell >= (long long)p.M * p.subs) cell = (long long)p.M * p.subs - 1;
        const int m = int(cell / p.subs), sub = int(cell - (long long)m * p.subs), z = m / kPass;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (sub < p.S) v = __ldg(reinterpret_cast<const uint4 *>(p.x + size_t(m) * p.K + sub * 64 + o * 8));
        grid_launch_dependents();
        float x[8];
        tile::widen8(v, x);
        const size_t s = size_t(z) * p.subs + sub;
        const int tok = m - z * kPass;
        tile::stage_octet<BITS>(
            x, o,
            [&](int h) { return p.cells + s * tile::cell_bytes(NC) + tile::operand_offset(tile::operand_index(tok, h), o >> 1); },
            [&](float sum, float f) {
                float *q = reinterpret_cast<float *>(p.meta + s * tile::meta_bytes(NC) + (tok >> 1) * 16) + (tok & 1);
                q[0] = sum;
                q[2] = f;
            });
        return;
    }
    // inner vectors: a block for each (vector, row of A), its warps sharing K
    __shared__ float part[kPrepareThreads / 32];
    const int item = int(blockIdx.x) - p.stage_blocks, m = item / p.R, r = item - m * p.R;
    const int ad = __ldg(p.adapter + m);
    if (ad < 0 || ad >= p.L) return;  // which also lets the next kernel start
    const uint4 *a = reinterpret_cast<const uint4 *>(p.a + (size_t(ad) * p.R + r) * p.K);
    const uint4 *x = reinterpret_cast<const uint4 *>(p.x + size_t(m) * p.K);
    float s = 0.0f;
    grid_launch_dependents();
    // (eight at a time against the memory's latency: 23.1 us for 13 vectors of 15360,
    // 25.9 with four; two or four rows to a block gave 25.3 and 26.6)
#pragma unroll 8
    for (int i = tid; i < p.K / 8; i += kPrepareThreads) {
        float av[8], xv[8];
        tile::widen8(__ldg(a + i), av);
        tile::widen8(__ldg(x + i), xv);
#pragma unroll
        for (int j = 0; j < 8; ++j) s = __fmaf_rn(av[j], xv[j], s);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, d));
    if (tid % 32 == 0) part[tid / 32] = s;
    __syncthreads();
    if (tid == 0) {
        for (int j = 1; j < kPrepareThreads / 32; ++j) s = __fadd_rn(s, part[j]);
        p.inner[size_t(m) * inner_pitch(p.R) + r] = s;
    }
}

// The product of a row of an adapter's B (R elements at shared address `addr`)
// with an inner vector v (padded to a multiple of eight floats), from 16-byte
// piece piece0 on where rows are whole pieces.
__device__ __forceinline__ float adapter_dot(uint32_t addr, const float *v, int R, int piece0)
{
    float d0 = 0.0f, d1 = 0.0f;
    if (R % 8 == 0) {
        const int C = R / 8;
        int c = piece0;
#pragma unroll 4
        for (int i = 0; i < C; ++i) {
            float x[8];
            tile::widen8(tile::lds_128(addr + c * 16), x);
            const float4 v0 = *reinterpret_cast<const float4 *>(v + c * 8), v1 = *reinterpret_cast<const float4 *>(v + c * 8 + 4);
            d0 = __fmaf_rn(x[0], v0.x, d0);
            d1 = __fmaf_rn(x[1], v0.y, d1);
            d0 = __fmaf_rn(x[2], v0.z, d0);
            d1 = __fmaf_rn(x[3], v0.w, d1);
            d0 = __fmaf_rn(x[4], v1.x, d0);
            d1 = __fmaf_rn(x[5], v1.y, d1);
            d0 = __fmaf_rn(x[6], v1.z, d0);
            d1 = __fmaf_rn(x[7], v1.w, d1);
            c = c + 1 == C ? 0 : c + 1;
        }
    } else {
        // words, shifted by an element where the row starts inside one
        const bool odd = addr & 2;
        const uint32_t word = addr & ~3u;
        uint32_t next = 0;
        auto lds_32 = [](uint32_t a) {
            uint32_t w;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(a));
            return w;
        };
        if (odd) next = lds_32(word);
        int r = 0;
#pragma unroll 2
        for (; r + 4 <= R; r += 4) {
            uint32_t a, b;
            if (odd) {
                const uint32_t w1 = lds_32(word + 2 * r + 4), w2 = lds_32(word + 2 * r + 8);
                a = __byte_perm(next, w1, 0x5432);
                b = __byte_perm(w1, w2, 0x5432);
                next = w2;
            } else {
                a = lds_32(word + 2 * r);
                b = lds_32(word + 2 * r + 4);
            }
            const float4 w = *reinterpret_cast<const float4 *>(v + r);
            d0 = __fmaf_rn(__uint_as_float(a << 16), w.x, d0);
            d1 = __fmaf_rn(__uint_as_float(a & 0xffff0000u), w.y, d1);
            d0 = __fmaf_rn(__uint_as_float(b << 16), w.z, d0);
            d1 = __fmaf_rn(__uint_as_float(b & 0xffff0000u), w.w, d1);
        }
        for (; r < R; ++r) {
            uint16_t e;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(e) : "r"(addr + 2 * r));
            d0 = __fmaf_rn(__uint_as_float(uint32_t(e) << 16), v[r], d0);
        }
    }
    return __fadd_rn(d0, d1);
}

template <int BITS, int GS, int NC>
__global__ void __launch_bounds__(tile::kThreads, 1) lora_project(const __grid_constant__ CUtensorMap map,
                                                                  const __grid_constant__ CUtensorMap smap,
                                                                  const __grid_constant__ CUtensorMap bmap,
                                                                  const LoraParams p)
{
    using namespace tile;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint16_t s_ad[kPasses][kPass], s_of[kPasses][kPass];
    __shared__ float s_c[kPasses][kPass];
    constexpr int SUBS = slot_subs(BITS);
    const Layout L = layout(p, BITS, NC);
    int &s_abort = *reinterpret_cast<int *>(smem + L.misc), &s_last = (&s_abort)[1], *s_ads = &s_abort + 4;
    uint32_t &s_tmem = *reinterpret_cast<uint32_t *>(smem + L.misc + 8);
    const uint32_t base = smem_u32(smem), full0 = base + L.bars, empty0 = full0 + 8 * p.slots;
    const uint32_t stored0 = empty0 + 8 * p.slots, ready0 = stored0 + 16 * kGroups, xbar = ready0 + 16 * kGroups;
    const uint32_t xfree = xbar + 8, sfull0 = xfree + 8, sempty0 = sfull0 + 16;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int seg = blockIdx.y, passes = (p.M + kPass - 1) / kPass;
    const int lo = int((long long)p.NS * seg / p.nseg), ns = int((long long)p.NS * (seg + 1) / p.nseg) - lo;
    const int g0 = lo * SUBS * 64 / GS, groups = min(ns * SUBS * 64 / GS, p.G - g0);
    static_assert(kPasses <= kThreads / 32, "a warp for each pass");
    const int lists = (warp + kPasses - 2) % kPasses;  // the pass whose lists this warp makes (warp 0 has the barriers to make)
    if (lists < passes) {
        // This range's adapters among those of a pass's vectors, each once, in their
        // order, with the vectors that have it. An adapter belongs to the range of
        // its number modulo the ranges.
        const int t = lists * kPass + lane;
        int ad = lane < kPass && t < p.M ? __ldg(p.adapter + t) : -1;
        if (ad < 0 || ad >= p.L || ad % p.nseg != seg) ad = -1;
        const uint32_t same = __match_any_sync(0xffffffffu, ad);
        const bool first = ad >= 0 && __ffs(same) - 1 == lane;
        const uint32_t firsts = __ballot_sync(0xffffffffu, first);
        if (first) {
            const int at = __popc(firsts & ((1u << lane) - 1u));
            s_ad[lists][at] = uint16_t(ad);
            s_of[lists][at] = uint16_t(same);
        }
        if (lane == 0) s_ads[lists] = __popc(firsts);
    }
    if (tid == 0) {
        for (int i = 0; i < p.slots; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, kWorkers);
        }
        for (int i = 0; i < 2 * kGroups; ++i) {
            mbar_init(stored0 + 8 * i, 4);
            mbar_init(ready0 + 8 * i, 1);
        }
        mbar_init(xbar, 1);
        mbar_init(xfree, kWorkers);
        for (int i = 0; i < 2; ++i) {
            mbar_init(sfull0 + 8 * i, 32);
            mbar_init(sempty0 + 8 * i, kWorkers);
        }
        fence_mbar_init();
        s_abort = 0;
    }
    if (warp == kWorkers) tmem_alloc(smem_u32(&s_tmem), kTmemColumns);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tm = s_tmem;
    const Waits wait{&s_abort, p.err};
    const int pieces = (p.rows + p.piece - 1) / p.piece;

    // staged x and inner vectors of a pass by bulk copies, once the first kernel has
    // ended and the pass before (`before` passes in all) needs its own no more
    auto fetch_x = [&](int z, int before) {
        if (before == 0) {
            grid_dependency_wait();
            asm volatile("fence.proxy.async;" ::: "memory");
        } else {
            wait(xfree, (before - 1) & 1);
        }
        const int nv = min(kPass, p.M - z * kPass);
        const uint32_t cb = uint32_t(ns) * SUBS * cell_bytes(NC), mb = uint32_t(ns) * SUBS * meta_bytes(NC);
        const uint32_t ib = uint32_t(nv) * inner_pitch(p.R) * 4;
        mbar_arrive_expect_tx(xbar, cb + mb + ib);
        const size_t sub = size_t(z) * p.subs + size_t(lo) * SUBS;
        bulk_load_plain(base + L.x, p.cells + sub * cell_bytes(NC), cb, xbar);
        bulk_load_plain(base + L.meta, p.meta + sub * meta_bytes(NC), mb, xbar);
        // (of vectors without an adapter: whatever is there)
        bulk_load_plain(base + inner_at(p, L, before), p.inner + size_t(z) * kPass * inner_pitch(p.R), ib, xbar);
    };

    if (warp == kThreads / 32 - 1) {
        // ---------------------------------------------------------- producer
        int it = 0, tiles = 0, fetched = 0;
        bool ok = true;
        const uint32_t bytes = uint32_t(p.rows) * kSlotBytes;
        for (int z = blockIdx.z; z < passes && ok; z += gridDim.z) {
            const int ads = s_ads[z], it0 = it, before = fetched, early = min(fetched == 0 ? kBefore : p.slots, ns);
            for (int tl = blockIdx.x; tl < p.tiles && ok; tl += p.grid_rows, ++tiles) {
                const int buf = tiles % p.sb_buffers, turn = tiles / p.sb_buffers;
                ok = __all_sync(0xffffffffu, turn == 0 || wait(sempty0 + 8 * buf, (turn - 1) & 1));
                if (!ok) break;
                p.sb.fetch(base + L.sb + buf * 2 * p.sb.block, smem + L.sb + buf * 2 * p.sb.block, p.scales, p.biases, &smap, &bmap,
                           (long long)tl * p.rows, p.rows, p.N, p.G, g0, groups, sfull0 + 8 * buf, lane);
                if (lane == 0)
                    for (int i = 0; i < ns; ++i, ++it) {
                        if (fetched == before && it - it0 == early) fetch_x(z, fetched++);
                        const int s = it % p.slots, lap = it / p.slots;
                        ok = lap == 0 || wait(empty0 + 8 * s, (lap - 1) & 1);
                        if (!ok) break;
                        mbar_arrive_expect_tx(full0 + 8 * s, bytes);
                        tma_load_2d(base + s * L.slot, &map, (lo + i) * (kSlotBytes / 8), tl * p.rows, full0 + 8 * s);
                    }
                if (lane == 0 && ok && fetched == before) fetch_x(z, fetched++);
                // the adapters' rows of the tile, from the 16-byte boundary before them
                if (lane == 0)
                    for (int j = 0; j < ads * pieces && ok; ++j, ++it) {
                        const int d = ads == 0 ? 0 : j / pieces, r0 = (j - d * pieces) * p.piece;
                        const int s = it % p.slots, lap = it / p.slots;
                        ok = lap == 0 || wait(empty0 + 8 * s, (lap - 1) & 1);
                        if (!ok) break;
                        const long long n0 = (long long)tl * p.rows + r0, n1 = min(n0 + min(p.piece, p.rows - r0), (long long)p.N);
                        const long long first = ((long long)s_ad[z][d] * p.N + n0) * p.R * 2, to = first + max(n1 - n0, 0ll) * p.R * 2;
                        const long long from = first & ~15ll, whole = min((to + 15) & ~15ll, (long long)p.L * p.N * p.R * 2 & ~15ll);
                        const uint32_t bytes = n1 > n0 && whole > from ? uint32_t(whole - from) : 0u;
                        // the array's last bytes, where they fill no 16
                        if (whole < to && n1 > n0) {
                            for (long long e = max(whole, from); e < to; e += 2)
                                *reinterpret_cast<uint16_t *>(smem + s * L.slot + (e - from)) = __ldg(p.b + e / 2);
                            fence_proxy_async_smem();
                        }
                        mbar_arrive_expect_tx(full0 + 8 * s, bytes);
                        if (bytes) bulk_load_plain(base + s * L.slot, reinterpret_cast<const uint8_t *>(p.b) + from, bytes, full0 + 8 * s);
                    }
                ok = __all_sync(0xffffffffu, ok);
            }
            fetched = __shfl_sync(0xffffffffu, fetched, 0);
        }
        if (lane == 0) {
            if (!ok) {  // copies in flight end before the CTA does
                for (int j = max(0, it - p.slots); j < it; ++j)
                    (void)mbar_wait_bounded(full0 + 8 * (j % p.slots), (j / p.slots) & 1);
                for (int j = max(0, tiles - p.sb_buffers); j < tiles; ++j)
                    (void)mbar_wait_bounded(sfull0 + 8 * (j % p.sb_buffers), (j / p.sb_buffers) & 1);
                if (fetched) (void)mbar_wait_bounded(xbar, (fetched - 1) & 1);
            }
        }
    } else if (warp >= kWorkers) {
        // ------------------------------------------------------ tensor warps
        const int group = warp - kWorkers;
        if (lane == 0) {
            Pipe pipe = Pipe::make<NC>(tm, 0, stored0, ready0, group);
            int it = 0, before = 0;
            for (int z = blockIdx.z; z < passes; z += gridDim.z, ++before) {
                const int step = ns + s_ads[z] * pieces;
                bool landed = false;
                for (int tl = blockIdx.x; tl < p.tiles; tl += p.grid_rows, it += step) {
                    const int i0 = first_slot(group, it);
                    // A pass waits for this warp only where its group has slots: without
                    // any it must not wait by a parity that may be two passes old. (Nor
                    // is the parity enough after such a pass; the workers' arrivals are,
                    // which have waited for x.)
                    if (i0 < ns && !landed) {
                        wait(xbar, before & 1);
                        landed = true;
                    }
                    for (int i = i0; i < ns; i += kGroups)
                        multiply_slot<BITS, NC>(wait, pipe, base + L.x + i * SUBS * cell_bytes(NC));
                }
            }
        }
    } else {
        // ----------------------------------------------------------- workers
        const int group = warp / 4, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
        Pipe pipe = Pipe::make<NC>(tm, lanes, stored0, ready0, group);
        const uint32_t wrow = base + row * kSlotBytes + ((row & 7) << 4);
        grid_launch_dependents();
        if (tid < kPasses * kPass && tid / kPass < passes && tid % kPass < s_ads[tid / kPass])  // (the next barrier publishes them)
            s_c[tid / kPass][tid % kPass] = __ldg(p.c + s_ad[tid / kPass][tid % kPass]);
        int it = 0, tiles = 0, before = 0;
        const int align = p.sb.alignment(p.G), pitch = inner_pitch(p.R);
        // With several ranges: the tile whose partial sums were left last and, in one
        // thread, how many ranges had left theirs before. It is looked at after the
        // next tile, so that nobody waits for the answer.
        int left_z = 0, left_tl = -1;
        unsigned others = 0;
        auto put = [&](int z, int t, int n, float v) {
            const size_t at = size_t(z * kPass + t) * p.N + n;
            if (p.f32_out) static_cast<float *>(p.y)[at] = v;
            else static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(v);
        };
        // before and after a barrier of all workers
        auto ask = [&]() {
            if (row != 0 || left_tl < 0 || group != (tiles + kGroups - 1) % kGroups) return;
            s_last = others == unsigned(p.nseg - 1);
            if (s_last) __threadfence();
        };
        auto join_ranges = [&]() {
            if (left_tl < 0 || !s_last) return;
            const int n = left_tl * p.rows + row, nv = min(kPass, p.M - left_z * kPass);
            if (row >= p.rows || n >= p.N) return;
            const float *part = p.partials + size_t(left_z) * p.nseg * NC * p.N + n;
            float s[Row<BITS, GS, NC>::kOwn];
            for (int k = 0; k < p.nseg; ++k, part += size_t(NC) * p.N) {
                float v[Row<BITS, GS, NC>::kOwn];
#pragma unroll
                for (int i = 0; i < Row<BITS, GS, NC>::kOwn; ++i) v[i] = group + kGroups * i < nv ? __ldcg(part + size_t(group + kGroups * i) * p.N) : 0.0f;
#pragma unroll
                for (int i = 0; i < Row<BITS, GS, NC>::kOwn; ++i) s[i] = k ? __fadd_rn(s[i], v[i]) : v[i];
            }
#pragma unroll
            for (int i = 0; i < Row<BITS, GS, NC>::kOwn; ++i)
                if (group + kGroups * i < nv) put(left_z, group + kGroups * i, n, s[i]);
        };
        for (int z = blockIdx.z; z < passes; z += gridDim.z, ++before) {
            const int ads = s_ads[z], nv = min(kPass, p.M - z * kPass);
            const float *inner = reinterpret_cast<const float *>(smem + inner_at(p, L, before));
            bool landed = false;  // staged x
            for (int tl = blockIdx.x; tl < p.tiles; tl += p.grid_rows, it += ns + ads * pieces, ++tiles) {
                const bool over = tl + p.grid_rows >= p.tiles;  // the pass's last tile here
                const int n = tl * p.rows + row;
                const bool live = row < p.rows && n < p.N;
                // Adapters' rows lie R/8 pieces of 16 bytes apart: each starts at another
                // piece, so that neighbours' reads fall on different banks. (By the row's
                // place in the matrix: its place in a tile depends on the card.)
                const int piece0 = p.R % 8 ? 0 : (p.R >= 64 ? n & 127 : (n & 127) * (p.R / 8) >> 3) % (p.R / 8);
                Row<BITS, GS, NC> acc;
                acc.start();
                uint32_t last = 0;
                const int buf = tiles % p.sb_buffers;
                wait(sfull0 + 8 * buf, (tiles / p.sb_buffers) & 1);
                const uint32_t sb = base + L.sb + buf * 2 * p.sb.block + min(row, p.rows - 1) * p.sb.pitch + p.sb.offset(n, p.G, g0);
#pragma unroll 1
                for (int i = first_slot(group, it); i < ns; i += kGroups) {
                    const int s = (it + i) % p.slots, lap = (it + i) / p.slots;
                    wait(full0 + 8 * s, lap & 1);
                    const uint32_t meta = base + L.meta + i * SUBS * meta_bytes(NC);
                    Affine<BITS, GS> aff;
                    aff.read(sb + i * Affine<BITS, GS>::kGroupsPerSlot * 2, p.sb.block, align,
                             groups - i * Affine<BITS, GS>::kGroupsPerSlot);
                    if (!landed) {
                        wait(xbar, before & 1);
                        landed = true;
                    }
                    acc.slot(wait, pipe, wrow + s * L.slot, aff, meta, last, lane);
                    last = meta + (SUBS - 2 * step_subs(NC)) * meta_bytes(NC);
                    __syncwarp();
                    if (lane == 0) mbar_arrive_many(empty0 + 8 * s, kGroups);
                }
                if (lane == 0) mbar_arrive(sempty0 + 8 * buf);
                acc.finish(wait, pipe, last);
                if (!landed) {  // (a group without slots needs the inner vectors)
                    wait(xbar, before & 1);
                    landed = true;
                }
                __syncwarp();
                if (over && p.inner_buffers == 2 && lane == 0) mbar_arrive(xfree);
                float sums[Row<BITS, GS, NC>::kOwn];
                acc.join(tm + lanes, group, it % kGroups, sums);
                Turn at;
                at.slot = (it + ns) % p.slots;
                at.lap = (it + ns) / p.slots;
                for (int d = 0; d < ads; ++d)
                    for (int r0 = 0; r0 < p.rows; r0 += p.piece, at.step(1, p.slots)) {
                        wait(full0 + 8 * at.slot, at.lap & 1);
                        if (live && row >= r0 && row < r0 + p.piece) {
                            // (32 bits are enough for the start's place within 16 bytes)
                            const uint32_t first = (uint32_t(s_ad[z][d]) * uint32_t(p.N) + uint32_t(tl * p.rows + r0)) * uint32_t(p.R) * 2u;
                            const uint32_t addr = base + at.slot * L.slot + (first & 15u) + (row - r0) * p.R * 2;
                            // the group's vectors: every third
#pragma unroll 1
                            for (uint32_t of = s_of[z][d] & 0x9249u << group; of; of &= of - 1) {
                                const int t = __ffs(of) - 1;
                                const float v = __fmul_rn(s_c[z][d], adapter_dot(addr, inner + t * pitch, p.R, piece0));
#pragma unroll
                                for (int k = 0; k < Row<BITS, GS, NC>::kOwn; ++k)
                                    if (t == group + kGroups * k) sums[k] = __fadd_rn(sums[k], v);
                            }
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(empty0 + 8 * at.slot);
                    }
                if (over && p.inner_buffers == 1 && lane == 0) mbar_arrive(xfree);
                if (p.nseg == 1) {
#pragma unroll
                    for (int i = 0; i < Row<BITS, GS, NC>::kOwn; ++i)
                        if (live && group + kGroups * i < nv) put(z, group + kGroups * i, n, sums[i]);
                    continue;
                }
                float *part = p.partials + (size_t(z) * p.nseg + seg) * NC * p.N + n;
#pragma unroll
                for (int i = 0; i < Row<BITS, GS, NC>::kOwn; ++i)
                    if (live && group + kGroups * i < nv) __stcg(part + size_t(group + kGroups * i) * p.N, sums[i]);
                ask();
                named_sync(1, 32 * kWorkers);
                unsigned had = 0;
                if (row == 0 && group == tiles % kGroups) {
                    __threadfence();  // (of what the barrier ordered before it, too)
                    had = atomicAdd(p.counters + size_t(z) * p.tiles + tl, 1u);
                }
                join_ranges();
                others = had;
                left_z = z;
                left_tl = tl;
            }
        }
        if (left_tl >= 0) {
            ask();
            named_sync(1, 32 * kWorkers);
            join_ranges();
        }
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == kWorkers) tmem_free(tm, kTmemColumns);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <int BITS, int NC>
cudaError_t launch_lora(const RingMaps &maps, LoraParams &p, cudaStream_t stream)
{
    static std::atomic<int> configured[3][64] = {};
    Launch l;
    l.grid = dim3(p.stage_blocks + p.M * p.R);
    l.threads = kPrepareThreads;
    l.smem = 0;
    l.pdl = true;
    const cudaError_t e = launch_one(lora_prepare<BITS, NC>, configured[0], l, stream, p);
    if (e != cudaSuccess) return e;
    l.grid = dim3(p.grid_rows, p.nseg, p.grid_passes);
    l.threads = tile::kThreads;
    l.smem = size_t(layout(p, BITS, NC).total);
    if (p.gs == 64) return launch_one(lora_project<BITS, 64, NC>, configured[1], l, stream, maps.w, maps.s, maps.b, p);
    return launch_one(lora_project<BITS, 128, NC>, configured[2], l, stream, maps.w, maps.s, maps.b, p);
}

template <int BITS>
cudaError_t launch_lora(const RingMaps &maps, LoraParams &p, cudaStream_t stream)
{
    if (!fit(p, BITS)) return cudaErrorInvalidConfiguration;
    switch (p.nc) {
        case 2: return launch_lora<BITS, 2>(maps, p, stream);
        case 4: return launch_lora<BITS, 4>(maps, p, stream);
        case 8: return launch_lora<BITS, 8>(maps, p, stream);
        default: return launch_lora<BITS, 16>(maps, p, stream);
    }
}

}  // namespace
}  // namespace qmv

extern "C" size_t qmv_lora_workspace_size(int M, int N, int K, int bits, int group_size, int rank)
{
    if (qmv::check_weights(M, N, K, bits, group_size) != QMV_OK || K > qmv::lora::kMaxK || rank < 1 || rank > QMV_MAX_RANK)
        return 0;
    qmv::lora::Sizes sz;
    qmv::lora::plan(M, N, K, bits, group_size, rank, 1, sz);
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
    LoraParams p{};
    static_cast<LoraShape &>(p) = plan(M, N, K, bits, group_size, rank, dev.sms, sz);
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
    p.stage_blocks = int(((long long)M * p.subs * 8 + kPrepareThreads - 1) / kPrepareThreads);
    RingMaps maps{};
    st = encode_rows(&maps.w, w_q, (long long)K * bits / 8, N, tile::kSlotBytes / 8, p.rows, true);
    if (st == QMV_OK && p.sb.mode == tile::kSbBoxes) st = encode_rows(&maps.s, scales, p.G * 2ll, N, p.sb.pitch / 8, p.rows, false);
    if (st == QMV_OK && p.sb.mode == tile::kSbBoxes) st = encode_rows(&maps.b, biases, p.G * 2ll, N, p.sb.pitch / 8, p.rows, false);
    if (st != QMV_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = bits == 4 ? launch_lora<4>(maps, p, s) : launch_lora<2>(maps, p, s);
    return e == cudaSuccess ? QMV_OK : record_cuda_failure("lora kernel launch", e);
}
