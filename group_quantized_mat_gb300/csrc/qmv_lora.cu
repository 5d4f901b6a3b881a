// qmv_lora_run: a group-quantized projection shared by M vectors plus each
// vector's own low-rank adapter,
//
//   y[m] = W x[m] + c_a B_a (A_a x[m]),   a = adapter[m].
//
// Two kernels.
//  1. lora_prepare forms the inner vectors A_a x[m] in fp32, and for more than
//     kStageHere vectors stages x as operand cells (qmv_tile.cuh), into the
//     workspace.
//  2. lora_project streams W once per 16 vectors. It starts under the first
//     kernel (programmatic launch): its weights are on their way meanwhile, and
//     the inner vectors are needed only at the end of a tile. Up to kStageHere
//     vectors every CTA stages x itself, which takes less time than the first
//     kernel takes to end and be seen to have ended.
//
// lora_project, one CTA per SM: a producer thread brings 128 bytes of each row of
// a tile to a ring of shared-memory slots (one tensor-map box, 128-byte swizzle),
// four groups of worker warps run the tiles, four tensor warps multiply. A
// worker thread owns a row: it reads the row's scales and biases into registers a
// slot ahead, and in the end adds the adapters' second half to the sums it holds.
//  - Rows go to CTAs in tiles of equal height (a multiple of 8, at most 128): 104
//    for 15360 rows on 152 SMs.
//  - K goes to CTAs in ranges of at most 64 subgroups (4096), whose cells of 16
//    vectors are 128 KB. Several ranges meet in the workspace: the CTA that
//    finishes a tile last adds them in their order.
// The order of every sum depends on N and K alone, so a vector's result does not
// depend on the batch it is in.
#include <cuda_bf16.h>

#include <cstdint>
#include <mutex>

#include "qmv.h"
#include "qmv_launch.cuh"
#include "qmv_tile.cuh"

namespace qmv {
namespace {

constexpr int kPrepareThreads = 256;
constexpr int kMaxSlotsLora = 12;
constexpr int kSmem = 227 * 1024 - 1024;
constexpr int kMaxK = 1 << 16;
constexpr int kRangeSubs = 64;  // subgroups of a range of K at most
constexpr int kPass = 16;       // vectors that one read of the weights serves
constexpr int kStageHere = 4;   // vectors that lora_project stages itself

struct LoraParams {
    const uint16_t *scales, *biases, *x, *a, *b;
    const int32_t *adapter;
    const float *c;
    void *y;
    uint8_t *cells;      // [pass][subs][cell_bytes]
    uint8_t *meta;       // [pass][subs][meta_bytes]
    float *inner;        // [M][R]
    float *partials;     // [pass][nseg][nc][N], with nseg > 1
    unsigned *counters;  // [pass][tiles], with nseg > 1
    unsigned *err;
    int M, N, K, G, gs, L, R, f32_out;
    int S;       // subgroups of a row
    int NS;      // slots of a row
    int subs;    // NS slots' subgroups (those past S are staged as zeros)
    int nseg;    // ranges of K
    int range;   // slots of the longest range
    int rows, tiles, grid_rows;
    int nc, slots, stage_blocks;
};

template <int BITS, int NC>
__global__ void __launch_bounds__(kPrepareThreads) lora_prepare(const LoraParams p)
{
    grid_dependency_wait();
    grid_launch_dependents();
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
        float x[8];
        tile::widen8(v, x);
        const size_t s = size_t(z) * p.subs + sub;
        tile::stage_octet<BITS>(x, o, m - z * kPass, p.cells + s * tile::cell_bytes(NC), p.meta + s * tile::meta_bytes(NC));
        return;
    }
    // inner vectors: a block for each (vector, row of A), its warps sharing K
    __shared__ float part[kPrepareThreads / 32];
    const int item = int(blockIdx.x) - p.stage_blocks, m = item / p.R, r = item - m * p.R;
    const int ad = __ldg(p.adapter + m);
    if (ad < 0 || ad >= p.L) return;
    const uint4 *a = reinterpret_cast<const uint4 *>(p.a + (size_t(ad) * p.R + r) * p.K);
    const uint4 *x = reinterpret_cast<const uint4 *>(p.x + size_t(m) * p.K);
    float s = 0.0f;
#pragma unroll 4
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
        p.inner[size_t(m) * p.R + r] = s;
    }
}

struct Layout {
    int slots, slot, x, meta, bars, total;
};

__host__ __device__ inline Layout layout(const LoraParams &p, int bits, int nc)
{
    const int subs = p.range * tile::slot_subs(bits);
    Layout l;
    l.slots = 0;
    l.slot = p.rows * tile::kSlotBytes;
    // a tile of fewer than 128 rows reads on past its slot's end
    l.x = p.slots * l.slot;
    if (l.x < (p.slots - 1) * l.slot + tile::kTileRows * tile::kSlotBytes)
        l.x = (p.slots - 1) * l.slot + tile::kTileRows * tile::kSlotBytes;
    l.x = (l.x + 1023) & ~1023;
    l.meta = l.x + subs * tile::cell_bytes(nc);
    l.bars = l.meta + subs * tile::meta_bytes(nc);
    l.total = l.bars + (2 * p.slots + 4 * tile::kGroups + 1) * 8;
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

template <int BITS, int NC>
__global__ void __launch_bounds__(tile::kThreads, 1) lora_project(const __grid_constant__ CUtensorMap map,
                                                                  const LoraParams p)
{
    using namespace tile;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int s_abort, s_last;
    __shared__ uint32_t s_tmem;
    constexpr int SUBS = slot_subs(BITS);
    const Layout L = layout(p, BITS, NC);
    const uint32_t base = smem_u32(smem), full0 = base + L.bars, empty0 = full0 + 8 * p.slots;
    const uint32_t stored0 = empty0 + 8 * p.slots, ready0 = stored0 + 16 * kGroups, xbar = ready0 + 16 * kGroups;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int seg = blockIdx.y, z = blockIdx.z;
    if (tid == 0) {
        for (int i = 0; i < p.slots; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, 4);
        }
        for (int i = 0; i < 2 * kGroups; ++i) {
            mbar_init(stored0 + 8 * i, 4);
            mbar_init(ready0 + 8 * i, 1);
        }
        mbar_init(xbar, p.cells ? 1 : kWorkers);
        fence_mbar_init();
        s_abort = 0;
    }
    if (warp == kWorkers) tmem_alloc(smem_u32(&s_tmem), kTmemColumns);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tm = s_tmem;
    const Waits wait{&s_abort, p.err};
    const int lo = int((long long)p.NS * seg / p.nseg), ns = int((long long)p.NS * (seg + 1) / p.nseg) - lo;

    if (warp == kThreads / 32 - 1) {
        // ---------------------------------------------------------- producer
        if (lane == 0) {
            int it = 0;
            const uint32_t bytes = uint32_t(p.rows) * kSlotBytes;
            for (int tl = blockIdx.x; tl < p.tiles && !*wait.abort; tl += p.grid_rows)
                for (int i = 0; i < ns; ++i, ++it) {
                    const int s = it % p.slots, lap = it / p.slots;
                    if (lap > 0 && !wait(empty0 + 8 * s, (lap - 1) & 1)) break;
                    mbar_arrive_expect_tx(full0 + 8 * s, bytes);
                    tma_load_2d(base + s * L.slot, &map, (lo + i) * (kSlotBytes / 8), tl * p.rows, full0 + 8 * s);
                }
            if (*wait.abort)  // copies in flight end before the CTA does
                for (int j = max(0, it - p.slots); j < it; ++j)
                    (void)mbar_wait_bounded(full0 + 8 * (j % p.slots), (j / p.slots) & 1);
        }
    } else if (warp >= kWorkers) {
        // ------------------------------------------------------ tensor warps
        const int group = warp - kWorkers;
        if (lane == 0) {
            wait(xbar, 0);
            Pipe pipe = Pipe::make<NC>(tm, 0, stored0, ready0, group);
            for (int tl = blockIdx.x; tl < p.tiles; tl += p.grid_rows)
                for (int i = group; i < ns; i += kGroups)
                    multiply_slot<BITS, NC>(wait, pipe, base + L.x + i * SUBS * cell_bytes(NC));
        }
    } else {
        // ----------------------------------------------------------- workers
        const int group = warp / 4, row = (warp & 3) * 32 + lane, nv = min(kPass, p.M - z * kPass);
        const bool vec = p.G % (SUBS * 64 / p.gs) == 0;
        const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
        Pipe pipe = Pipe::make<NC>(tm, lanes, stored0, ready0, group);
        const uint32_t wrow = base + row * kSlotBytes + ((row & 7) << 4);
        Affine<BITS> next;
        {
            const int n = blockIdx.x * p.rows + row;
            next.clear();
            if (row < p.rows && n < p.N && group < ns) next.load(p.scales, p.biases, n, p.G, p.gs, lo + group, vec);
        }
        grid_launch_dependents();
        if (p.cells) {
            grid_dependency_wait();
            if (tid == 0) {
                asm volatile("fence.proxy.async;" ::: "memory");
                const uint32_t cb = uint32_t(ns) * SUBS * cell_bytes(NC), mb = uint32_t(ns) * SUBS * meta_bytes(NC);
                mbar_arrive_expect_tx(xbar, cb + mb);
                const size_t sub = size_t(z) * p.subs + size_t(lo) * SUBS;
                bulk_load_plain(base + L.x, p.cells + sub * cell_bytes(NC), cb, xbar);
                bulk_load_plain(base + L.meta, p.meta + sub * meta_bytes(NC), mb, xbar);
            }
        } else {
            // eight threads for each (subgroup, vector), the vectors of a
            // subgroup in a row; whole warps take part (their exchanges need it)
            const int items = ns * SUBS * nv * 8;
            for (int i0 = warp * 32; i0 < items; i0 += 32 * kWorkers) {
                const int i = min(i0 + lane, items - 8 + (lane & 7)), cell = i >> 3, sub = cell / nv, tok = cell - sub * nv;
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (lo * SUBS + sub < p.S)
                    v = __ldg(reinterpret_cast<const uint4 *>(p.x + size_t(tok) * p.K + (lo * SUBS + sub) * 64 + (i & 7) * 8));
                float x[8];
                widen8(v, x);
                stage_octet<BITS>(x, i & 7, tok, smem + L.x + sub * cell_bytes(NC), smem + L.meta + sub * meta_bytes(NC));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(xbar);
        }
        wait(xbar, 0);
        int it = 0;
        for (int tl = blockIdx.x; tl < p.tiles; tl += p.grid_rows, it += ns) {
            const int n = tl * p.rows + row;
            const bool live = row < p.rows && n < p.N;
            Row<BITS, NC> acc;
            acc.start();
            uint32_t last = 0;
            // the adapters' rows of this tile are on their way to L2 meanwhile
            for (int t = group; live && t < nv; t += kGroups) {
                const int ad = __ldg(p.adapter + z * kPass + t);
                if (ad < 0 || ad >= p.L) continue;
                const uint16_t *b = p.b + (size_t(ad) * p.N + n) * p.R;
                for (int r = 0; r < p.R; r += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(b + r));
            }
            for (int i = group; i < ns; i += kGroups) {
                const int s = (it + i) % p.slots, lap = (it + i) / p.slots;
                const Affine<BITS> now = next;
                // the next slot's, of this tile or of the next
                const int ni = i + kGroups < ns ? i + kGroups : group, nn = i + kGroups < ns ? n : n + p.grid_rows * p.rows;
                next.clear();
                if (row < p.rows && nn < p.N) next.load(p.scales, p.biases, nn, p.G, p.gs, lo + ni, vec);
                wait(full0 + 8 * s, lap & 1);
                const uint32_t meta = base + L.meta + i * SUBS * meta_bytes(NC);
                acc.slot(wait, pipe, wrow + s * L.slot, now, meta, last, lane);
                last = meta + (SUBS - 2 * step_subs(NC)) * meta_bytes(NC);
                __syncwarp();
                if (lane == 0) mbar_arrive(empty0 + 8 * s);
            }
            acc.finish(wait, pipe, last);
            float sums[Row<BITS, NC>::kOwn];
            acc.join(tm + lanes, group, sums);
            grid_dependency_wait();  // inner vectors, cleared tickets
            bool mine = true;
            if (p.nseg > 1) {
                const size_t plane = size_t(p.N), seg_stride = plane * NC;
                float *part = p.partials + size_t(z) * p.nseg * seg_stride + n;
#pragma unroll
                for (int i = 0; i < Row<BITS, NC>::kOwn; ++i) {
                    const int t = group + kGroups * i;
                    if (live && t < nv) __stcg(part + seg * seg_stride + t * plane, sums[i]);
                }
                __threadfence();
                named_sync(1, 32 * kWorkers);
                if (tid == 0) s_last = atomicAdd(p.counters + size_t(z) * p.tiles + tl, 1u) == unsigned(p.nseg - 1);
                named_sync(1, 32 * kWorkers);
                mine = s_last != 0;
                if (mine) {
                    __threadfence();
#pragma unroll
                    for (int i = 0; i < Row<BITS, NC>::kOwn; ++i) {
                        const int t = group + kGroups * i;
                        if (!live || t >= nv) continue;
                        float s = __ldcg(part + t * plane);
                        for (int k = 1; k < p.nseg; ++k) s = __fadd_rn(s, __ldcg(part + k * seg_stride + t * plane));
                        sums[i] = s;
                    }
                }
            }
            if (!mine || !live) continue;
#pragma unroll
            for (int i = 0; i < Row<BITS, NC>::kOwn; ++i) {
                const int t = group + kGroups * i;
                if (t >= nv) continue;
                const int m = z * kPass + t, ad = __ldg(p.adapter + m);
                float s = sums[i];
                if (ad >= 0 && ad < p.L) s = __fadd_rn(s, adapter_term(p, ad, m, n));
                const size_t at = size_t(m) * p.N + n;
                if (p.f32_out) static_cast<float *>(p.y)[at] = s;
                else static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(s);
            }
        }
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == kWorkers) tmem_free(tm, kTmemColumns);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Sizes {
    size_t cells, meta, inner, counters, partials, total;
};

size_t up256(size_t b) { return (b + 255) & ~size_t(255); }

// What a call needs; `sms` only shapes the grid (tiles), never an order of sums
// or a size.
LoraParams plan(int M, int N, int K, int bits, int gs, int R, int sms, Sizes &sz)
{
    const int slot_subs = tile::slot_subs(bits);
    LoraParams p{};
    p.M = M; p.N = N; p.K = K; p.G = K / gs; p.gs = gs; p.R = R;
    p.S = K / 64;
    p.NS = (p.S + slot_subs - 1) / slot_subs;
    p.subs = p.NS * slot_subs;
    p.nseg = (p.NS * slot_subs + kRangeSubs - 1) / kRangeSubs;
    p.range = (p.NS + p.nseg - 1) / p.nseg;
    p.nc = M <= 2 ? 2 : M <= 4 ? 4 : M <= 8 ? 8 : 16;
    // tiles of equal height: as many rounds of the grid as 128 rows need
    p.grid_rows = sms / p.nseg > 0 ? sms / p.nseg : 1;
    const int rounds = (N + tile::kTileRows * p.grid_rows - 1) / (tile::kTileRows * p.grid_rows);
    p.rows = ((N + p.grid_rows * rounds - 1) / (p.grid_rows * rounds) + 7) / 8 * 8;
    p.tiles = (N + p.rows - 1) / p.rows;
    if (p.grid_rows > p.tiles) p.grid_rows = p.tiles;
    const size_t passes = (M + kPass - 1) / kPass;
    sz.cells = M > kStageHere ? up256(passes * p.subs * tile::cell_bytes(p.nc)) : 0;
    sz.meta = M > kStageHere ? up256(passes * p.subs * tile::meta_bytes(p.nc)) : 0;
    sz.inner = up256(size_t(M) * R * 4);
    sz.counters = p.nseg > 1 ? up256(passes * ((N + 7) / 8) * 4) : 0;
    sz.partials = p.nseg > 1 ? up256(passes * p.nseg * size_t(N) * p.nc * 4) : 0;
    sz.total = sz.cells + sz.meta + sz.inner + sz.counters + sz.partials;
    return p;
}

template <int BITS, int NC>
cudaError_t launch_lora(const CUtensorMap &map, LoraParams &p, cudaStream_t stream)
{
    static std::atomic<int> configured[2][64] = {};
    Launch l;
    l.grid = dim3(p.stage_blocks + p.M * p.R);
    l.threads = kPrepareThreads;
    l.smem = 0;
    l.pdl = true;
    const cudaError_t e = launch_one(lora_prepare<BITS, NC>, configured[0], l, stream, p);
    if (e != cudaSuccess) return e;
    l.grid = dim3(p.grid_rows, p.nseg, (p.M + kPass - 1) / kPass);
    l.threads = tile::kThreads;
    l.smem = size_t(layout(p, BITS, NC).total);
    return launch_one(lora_project<BITS, NC>, configured[1], l, stream, map, p);
}

template <int BITS>
cudaError_t launch_lora(const CUtensorMap &map, LoraParams &p, cudaStream_t stream)
{
    // as many slots as fit
    p.slots = kMaxSlotsLora;
    while (p.slots > 2 && layout(p, BITS, p.nc).total > kSmem) --p.slots;
    if (layout(p, BITS, p.nc).total > kSmem) return cudaErrorInvalidConfiguration;
    switch (p.nc) {
        case 2: return launch_lora<BITS, 2>(map, p, stream);
        case 4: return launch_lora<BITS, 4>(map, p, stream);
        case 8: return launch_lora<BITS, 8>(map, p, stream);
        default: return launch_lora<BITS, 16>(map, p, stream);
    }
}

}  // namespace
}  // namespace qmv

extern "C" size_t qmv_lora_workspace_size(int M, int N, int K, int bits, int group_size, int rank)
{
    if (qmv::check_weights(M, N, K, bits, group_size) != QMV_OK || K > qmv::kMaxK || rank < 1 || rank > QMV_MAX_RANK)
        return 0;
    qmv::Sizes sz;
    qmv::plan(M, N, K, bits, group_size, rank, 1, sz);
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
    LoraParams p = plan(M, N, K, bits, group_size, rank, dev.sms, sz);
    void *ws = nullptr;
    st = scratch(dev, sz.total, workspace, workspace_bytes, &ws);
    if (st != QMV_OK) return st;

    p.scales = scales; p.biases = biases; p.x = x; p.a = lora_a; p.b = lora_b;
    p.adapter = adapter; p.c = lora_scale; p.y = y; p.err = dev.err;
    p.L = adapters;
    p.f32_out = (flags & QMV_F32_OUT) != 0;
    uint8_t *at = static_cast<uint8_t *>(ws);
    p.cells = sz.cells ? at : nullptr; at += sz.cells;
    p.meta = at; at += sz.meta;
    p.inner = reinterpret_cast<float *>(at); at += sz.inner;
    p.counters = p.nseg > 1 ? reinterpret_cast<unsigned *>(at) : nullptr; at += sz.counters;
    p.partials = p.nseg > 1 ? reinterpret_cast<float *>(at) : nullptr;
    p.stage_blocks = !p.cells ? 0 : int(((long long)M * p.subs * 8 + kPrepareThreads - 1) / kPrepareThreads);
    CUtensorMap map;
    st = encode_rows(&map, w_q, (long long)K * bits / 8, N, tile::kSlotBytes / 8, p.rows);
    if (st != QMV_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = bits == 4 ? launch_lora<4>(map, p, s) : launch_lora<2>(map, p, s);
    return e == cudaSuccess ? QMV_OK : record_cuda_failure("lora kernel launch", e);
}
