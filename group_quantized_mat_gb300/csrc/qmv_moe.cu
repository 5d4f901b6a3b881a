// qmv_moe_run: a whole mixture-of-experts layer for a few tokens,
//
//   l = router x;  ids = top-k of l;  w = softmax;  y = sum_e w_e down_e (act(gate_e x) * (up_e x)),
//
// in two kernels.
//  1. moe_logits forms the router's logits and stages x (qmv_tile.cuh): rows of
//     operand bytes for each token, which the second kernel gathers.
//  2. moe_experts, one CTA per SM, all resident (a cooperative launch). Every CTA
//     picks the experts from the logits for itself (a few thousand numbers) and
//     lists the tokens of each; then it takes its share of two kinds of items:
//       A. 64 rows of an expert's gate and the 64 of its up product, for up to NC
//          of its tokens: activation, and h as operand bytes to the workspace;
//       B. 128 rows of an expert's down product, sums to the workspace.
//     An entry (an expert and up to NC of its tokens) has a count of its items of
//     A that are done; B takes it when all are, its weights already on their way.
//     After B all CTAs meet and share the sums over each token's choices, in their
//     order. (A ticket for each tile of rows, the last CTA adding its sums, cost
//     2 us an item; a meeting of all CTAs between A and B 163 us for 48 tokens
//     where this takes 157.)
//
// An expert with no token costs nothing, one with several reads its weights once
// for up to NC of them. What bounds it: for few tokens the chain logits - choice -
// A - counts - B - meeting - sums, whose code runs from cold caches; for many the
// ring: 6 slots (9 with 4 tokens to an entry) are all that fits beside the cells,
// and a slot is taken from its request to the end of its step, 6 to 8 thousand
// cycles under load.
// Measured (us; bytes a call cannot do without, at 6.7 TB/s): 22.5 for one token
// and 8 of 64 experts of 2048 x 768 (3.2), 35 to 41 from card to card for 5 and 2 of
// 8 of 3840 x 1920 in 2 bits (5.7), 80 for 16 and 8 of 128 of 2048 x 768 (33; A runs at
// 5.8 TB/s with scales and biases), 157 for 48 and 4 of 32 of 5120 x 1280 (50).
//
// The inner pipeline is qmv_tile.cuh's. A ring slot holds 128 bytes of 128 rows
// and the slot's subgroups of the item's tokens. x enters with two e4m3 terms, which
// hold its 8 bits. h, an fp32 number, enters the down product with four, which hold 19:
// the first has 4 significant bits, each further one 5 more. Five would hold all 24
// and cost a quarter more in cells, accumulators and reads; with four the results' error
// against 64 bits is that of an fp32 computation (1.5e-7 to 1e-6 of their norm over 20
// shapes, 2.7e-7 to 1.4e-6 where everything is fp32).
//
// Orders: a token's logits, its sums over K and inter, and the sum over its
// choices do not depend on the other tokens of the call.
#include <cuda_bf16.h>

#include <cstdint>
#include <mutex>

#include "qmv.h"
#include "qmv_launch.cuh"
#include "qmv_tile.cuh"

namespace qmv {
namespace {

constexpr int kLogitThreads = 256;
constexpr int kSmemMoe = 227 * 1024 - 1024;
constexpr int kMaxSlotsMoe = 12;
// Slots come in threes (see qmv_tile.cuh). Their subgroups' sums are in a ring of
// their own that is three longer: a group needs those of a slot's last steps until
// it is done with its next.
constexpr int kMinSlotsMoe = tile::kGroups;
constexpr int kHalf = 64;        // rows of a box: an item is two
constexpr int kTermsH = 4;
constexpr int kSets = 5;         // items whose sums may be on their way
// Warps: the workers; a tensor warp for each group and one that brings weights;
// four that gather what is multiplied with them; four that take the items' sums.
// (One warp for weights and gathering: a slot in 1250 cycles at 6 tokens to an
// entry. Workers that form h themselves: 83 and 165 us for 16 and 48 tokens;
// gatherers that do: 79 and 163, as with takers, but these can also afford to count
// each item, a release of thousands of cycles under the stream of weights.)
// Registers move to the workers: 768 x 80 = 384 x 112 + 128 x (40 + 40 + 64).
constexpr int kGatherers = 4, kTakers = 4;
constexpr int kGather0 = tile::kWorkers + tile::kGroups + 1, kTake0 = kGather0 + kGatherers;
constexpr int kMoeThreads = 32 * (kTake0 + kTakers);
constexpr int kWorkerRegs = 112, kOtherRegs = 40, kTakerRegs = 64;
static_assert(384 * kWorkerRegs + 256 * kOtherRegs + 128 * kTakerRegs <= kMoeThreads * 80, "registers");
// Columns of tensor memory for items' sums on their way to the warps that take them.
constexpr int kExchange = tile::kGroups * tile::kGroupColumns, kExchangeSet = tile::kGroups * 8;

struct MoeParams {
    const uint16_t *x, *router, *gu_s, *gu_b, *dn_s, *dn_b;
    void *y;
    int32_t *ids_out;
    float *weights_out;
    float *logits;      // [M][E]
    uint8_t *rows;      // staged x: [M][subs_a][hi 64, lo 64]
    float2 *xmeta;      // [M][subs_a] (sum, f)
    uint8_t *h;         // [entry][slot of B][subgroups' cells, subgroups' meta]
    float *partials;    // [pair][K]
    unsigned *counters; // CTAs done with B, then for each entry its items of A that are done
    unsigned *err;
    int M, K, I, E, k, gs, nc, f32_out, gelu, softmax_all;
    int Sa, NSa, Ga, Sb, NSb, Gb;  // subgroups, slots and groups of a row of A and of B
    int tiles_a, tiles_b, max_entries, slots, stage_blocks;
    tile::Affines sba, sbb;
    int chunk;     // groups of scales and biases that are fetched at a time
    int cha, chb;  // slots whose scales and biases are fetched at a time
    int sb_block;
};

template <int BITS>
__global__ void __launch_bounds__(kLogitThreads) moe_logits(const MoeParams p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (blockIdx.x == 0)
        for (int i = tid; i < 1 + p.max_entries; i += kLogitThreads) p.counters[i] = 0u;
    if (int(blockIdx.x) < p.stage_blocks) {
        // eight threads for each (token, subgroup)
        const int subs = p.NSa * tile::slot_subs(BITS);
        const long long at = (long long)blockIdx.x * kLogitThreads + tid;
        const int o = int(at & 7);
        long long cell = at >> 3;
        // threads past the end repeat the last cell's values (the warp's exchanges need them)
        if (cell >= (long long)p.M * subs) cell = (long long)p.M * subs - 1;
        const int m = int(cell / subs), sub = int(cell - (long long)m * subs);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (sub < p.Sa) v = __ldg(reinterpret_cast<const uint4 *>(p.x + size_t(m) * p.K + sub * 64 + o * 8));
        float x[8];
        tile::widen8(v, x);
        tile::stage_octet<BITS>(
            x, o, [&](int h) { return p.rows + cell * 128 + h * 64 + (o >> 1) * 16; },
            [&](float sum, float f) { p.xmeta[cell] = make_float2(sum, f); });
        return;
    }
    // logits: a block for each expert, its warps sharing K, for all tokens
    __shared__ float part[kLogitThreads / 32][32];
    const int e = int(blockIdx.x) - p.stage_blocks, n8 = p.K / 8;
    const int lo = n8 * warp / (kLogitThreads / 32), hi = n8 * (warp + 1) / (kLogitThreads / 32);
    const uint4 *r = reinterpret_cast<const uint4 *>(p.router + size_t(e) * p.K);
    for (int m0 = 0; m0 < p.M; m0 += 32) {
        const int tokens = min(32, p.M - m0);
        for (int t = 0; t < tokens; ++t) {
            const uint4 *x = reinterpret_cast<const uint4 *>(p.x + size_t(m0 + t) * p.K);
            float s = 0.0f;
#pragma unroll 4
            for (int i = lo + lane; i < hi; i += 32) {
                float rv[8], xv[8];
                tile::widen8(__ldg(r + i), rv);
                tile::widen8(__ldg(x + i), xv);
#pragma unroll
                for (int j = 0; j < 8; ++j) s = __fmaf_rn(rv[j], xv[j], s);
            }
#pragma unroll
            for (int d = 16; d; d >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, d));
            if (lane == 0) part[warp][t] = s;
        }
        __syncthreads();
        if (tid < tokens) {
            float s = part[0][tid];
            for (int w = 1; w < kLogitThreads / 32; ++w) s = __fadd_rn(s, part[w][tid]);
            p.logits[size_t(m0 + tid) * p.E + e] = s == s ? s : -INFINITY;
        }
        __syncthreads();
    }
}

struct MoeLayout {
    int slot, cells, meta, sb, cell, red, lists, total;
    // within lists
    int w, ids, pos, tok, base, entry, bars;
};

__host__ __device__ inline MoeLayout moe_layout(const MoeParams &p, int bits, int nc)
{
    const int SUBS = tile::slot_subs(bits), CB = tile::cell_bytes(nc, kTermsH);
    const int pairs = p.M * p.k;
    MoeLayout l;
    l.cells = tile::kTileRows * tile::kSlotBytes;
    l.slot = (l.cells + SUBS * CB + 1023) & ~1023;
    l.meta = p.slots * l.slot;
    l.sb = (l.meta + (p.slots + tile::kGroups) * SUBS * tile::meta_bytes(nc) + 127) & ~127;
    l.cell = (l.sb + 2 * 2 * p.sb_block + 15) & ~15;
    l.red = l.cell + CB + tile::meta_bytes(nc);
    l.lists = l.red + 4 * nc * 8;
    l.w = l.lists;
    l.ids = l.w + pairs * 4;
    l.pos = l.ids + ((pairs * 2 + 3) & ~3);
    l.tok = l.pos + ((pairs * 2 + 3) & ~3);
    l.base = l.tok + ((pairs * 2 + 3) & ~3);
    l.entry = l.base + (p.E + 1) * 4;
    l.bars = (l.entry + p.max_entries * 4 + 7) & ~7;
    l.total = l.bars + (2 * p.slots + 4 * tile::kGroups + 4 + 2 * kSets) * 8;
    return l;
}

// A logit as a number that orders as it does (-0 as +0, nothing chosen as 0).
__device__ __forceinline__ uint32_t order_of(float v)
{
    const uint32_t u = __float_as_uint(__fadd_rn(v, 0.0f));
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float logit_of(uint32_t key) { return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key); }

constexpr int kFew = 4;  // 32 times as many experts are chosen from in registers

// The expert choice of token t by one warp, whose lane holds every 32nd logit in
// registers, or for MANY (more than 32 kFew experts) in shared memory (l). Lane j
// ends with choice j. (Two instances and no exponential in the loop: the code runs
// once, from a cold cache, and its length is what takes the time.)
template <bool MANY>
__device__ __forceinline__ void choose(const MoeParams &p, int t, uint32_t *l, float *w, uint16_t *ids, int lane)
{
    uint32_t key[kFew], first = 0, mine = 0, id = 0;
    const float *logits = p.logits + size_t(t) * p.E;
    if (MANY) {
        for (int e = lane; e < p.E; e += 32) l[e] = order_of(__ldcg(logits + e));
    } else {
#pragma unroll
        for (int i = 0; i < kFew; ++i) key[i] = i * 32 + lane < p.E ? order_of(__ldcg(logits + i * 32 + lane)) : 0u;
    }
#pragma unroll 1
    for (int j = 0; j < p.k; ++j) {
        uint32_t best = 0, arg = 0xffffffffu;
        if (MANY) {
            for (int e = lane; e < p.E; e += 32) best = max(best, l[e]);
        } else {
#pragma unroll
            for (int i = 0; i < kFew; ++i) best = max(best, key[i]);
        }
        best = __reduce_max_sync(0xffffffffu, best);
        if (MANY) {
            for (int e = lane; e < p.E && arg == 0xffffffffu; e += 32)
                if (l[e] == best) arg = e;
        } else {
#pragma unroll
            for (int i = kFew - 1; i >= 0; --i)
                if (key[i] == best) arg = i * 32 + lane;
        }
        arg = __reduce_min_sync(0xffffffffu, arg);
        if (MANY) {
            if (lane == int(arg % 32)) l[arg] = 0u;
        } else {
#pragma unroll
            for (int i = 0; i < kFew; ++i)
                if (arg == uint32_t(i * 32 + lane)) key[i] = 0u;
        }
        if (j == 0) first = best;
        if (lane == j) {
            mine = best;
            id = arg;
        }
    }
    // (all logits -inf: equal weights)
    const float top = logit_of(first);
    auto mass = [&](float v) { return top > -INFINITY ? expf(__fsub_rn(v, top)) : 1.0f; };
    const float m = lane < p.k ? mass(logit_of(mine)) : 0.0f;
    float sum = m;
    if (p.softmax_all) {
        // over all experts, each lane's in order, then across the lanes
        sum = 0.0f;
        for (int e = lane; e < p.E; e += 32) sum = __fadd_rn(sum, mass(__ldcg(logits + e)));
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, d));
    if (lane < p.k) {
        ids[t * p.k + lane] = uint16_t(id);
        w[t * p.k + lane] = __fdiv_rn(m, sum);
    }
}

__device__ __forceinline__ float activation(float g, bool gelu)
{
    if (gelu) {
        const float c = __fmul_rn(0.7978845608028654f, __fmaf_rn(__fmul_rn(__fmul_rn(0.044715f, g), g), g, g));
        return __fmul_rn(__fmul_rn(0.5f, g), __fadd_rn(1.0f, tanhf(c)));
    }
    return __fdiv_rn(g, __fadd_rn(1.0f, expf(-g)));
}

template <int BITS, int GS, int NC>
__global__ void __launch_bounds__(kMoeThreads, 1)
    moe_experts(const __grid_constant__ CUtensorMap wa, const __grid_constant__ CUtensorMap sa,
                const __grid_constant__ CUtensorMap ba, const __grid_constant__ CUtensorMap wb,
                const __grid_constant__ CUtensorMap sbm, const __grid_constant__ CUtensorMap bb, const MoeParams p)
{
    using namespace tile;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int s_abort, s_entries;
    __shared__ uint32_t s_tmem;
    constexpr int SUBS = slot_subs(BITS), CA = cell_bytes(NC, 2), CB = cell_bytes(NC, kTermsH), MB = meta_bytes(NC);
    const MoeLayout L = moe_layout(p, BITS, NC);
    const uint32_t base = smem_u32(smem), full0 = base + L.bars, empty0 = full0 + 8 * p.slots;
    const uint32_t stored0 = empty0 + 8 * p.slots, ready0 = stored0 + 16 * kGroups, sfull0 = ready0 + 16 * kGroups;
    const uint32_t sempty0 = sfull0 + 16, joined0 = sempty0 + 16, freed0 = joined0 + 8 * kSets;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, grid = gridDim.x;
    float *s_w = reinterpret_cast<float *>(smem + L.w);
    uint16_t *s_ids = reinterpret_cast<uint16_t *>(smem + L.ids), *s_pos = reinterpret_cast<uint16_t *>(smem + L.pos);
    uint16_t *s_tok = reinterpret_cast<uint16_t *>(smem + L.tok);
    int *s_base = reinterpret_cast<int *>(smem + L.base);
    uint32_t *s_entry = reinterpret_cast<uint32_t *>(smem + L.entry);

    if (tid == 0) {
        for (int i = 0; i < p.slots; ++i) {
            mbar_init(full0 + 8 * i, 1 + 32 * kGatherers);
            mbar_init(empty0 + 8 * i, 4 + 1);  // the group's warps, and its cells read
        }
        for (int i = 0; i < 2 * kGroups; ++i) {
            mbar_init(stored0 + 8 * i, 4);
            mbar_init(ready0 + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(sfull0 + 8 * i, 2 * 32);
            mbar_init(sempty0 + 8 * i, kWorkers);
        }
        for (int i = 0; i < kSets; ++i) {
            mbar_init(joined0 + 8 * i, kWorkers);
            mbar_init(freed0 + 8 * i, 4);
        }
        fence_mbar_init();
        s_abort = 0;
    }
    if (warp == kWorkers) tmem_alloc(smem_u32(&s_tmem), kTmemColumns);
    for (int i = tid; i < p.E; i += kMoeThreads) s_base[i] = 0;
    grid_dependency_wait();
    __syncthreads();

    // ------------------------------------------------------------- routing
    // (a row of logits for each warp in the ring)
    if (p.E > 32 * kFew)
        for (int t = warp; t < p.M; t += kMoeThreads / 32) choose<true>(p, t, reinterpret_cast<uint32_t *>(smem) + warp * p.E, s_w, s_ids, lane);
    else
        for (int t = warp; t < p.M; t += kMoeThreads / 32) choose<false>(p, t, nullptr, s_w, s_ids, lane);
    __syncthreads();
    if (warp == 0) {
        // each choice's place among its expert's, in the order of the tokens
        const int pairs = p.M * p.k;
        for (int i0 = 0; i0 < pairs; i0 += 32) {
            const int i = i0 + lane, e = i < pairs ? s_ids[i] : -1 - lane;
            const uint32_t same = __match_any_sync(0xffffffffu, e), before = same & ((1u << lane) - 1u);
            const int n = e >= 0 ? s_base[e] : 0;
            __syncwarp();
            if (e >= 0) {
                s_pos[i] = uint16_t(n + __popc(before));
                if (!before) s_base[e] = n + __popc(same);
            }
            __syncwarp();
        }
        // each lane a run of experts: choices and entries before it
        const int run = (p.E + 31) / 32, e0 = min(lane * run, p.E), e1 = min(e0 + run, p.E);
        int choices = 0, entries = 0;
        for (int e = e0; e < e1; ++e) {
            choices += s_base[e];
            entries += (s_base[e] + NC - 1) / NC;
        }
        int pb = choices, eb = entries;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int a = __shfl_up_sync(0xffffffffu, pb, d), b = __shfl_up_sync(0xffffffffu, eb, d);
            if (lane >= d) {
                pb += a;
                eb += b;
            }
        }
        if (lane == 31) {
            s_entries = eb;
            s_base[p.E] = pb;
        }
        pb -= choices;
        eb -= entries;
        for (int e = e0; e < e1; ++e) {
            const int n = s_base[e];
            s_base[e] = pb;
            for (int f = 0; f < n; f += NC) s_entry[eb++] = uint32_t(e) | uint32_t(f) << 16;
            pb += n;
        }
    }
    __syncthreads();
    for (int i = tid; i < p.M * p.k; i += kMoeThreads) {
        const int e = s_ids[i], at = s_base[e] + s_pos[i];
        s_pos[i] = uint16_t(at);
        s_tok[at] = uint16_t(i / p.k);
        if (blockIdx.x == 0 && p.ids_out) p.ids_out[i] = e;
        if (blockIdx.x == 0 && p.weights_out) p.weights_out[i] = s_w[i];
    }
    fence_proxy_async_smem();  // the ring was scratch until here
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tm = s_tmem;
    const Waits wait{&s_abort, p.err};
    // entry, its expert, first pair, tokens; the item's tile
    struct Item {
        int entry, e, pair, count, tl;
    };
    // this CTA's items of `tiles` to an entry: from blockIdx.x on in steps of the grid
    struct Items {
        int entry, tl, entries, tiles, dentry, dtl;
    };
    // (`before`: items of the part before, whose round the first ones fill up)
    auto items_of = [&](int tiles, int before = 0) {
        Items s;
        s.entries = s_entries;
        s.tiles = tiles;
        int at = int(blockIdx.x) - before % grid;
        if (at < 0) at += grid;
        s.entry = at / tiles;
        s.tl = at - s.entry * tiles;
        s.dentry = grid / tiles;
        s.dtl = grid - s.dentry * tiles;
        return s;
    };
    auto advance = [](Items &s) {
        s.entry += s.dentry;
        s.tl += s.dtl;
        if (s.tl >= s.tiles) {
            s.tl -= s.tiles;
            ++s.entry;
        }
    };
    auto item_of = [&](const Items &s) {
        Item it;
        it.entry = s.entry;
        it.tl = s.tl;
        const uint32_t v = s_entry[it.entry];
        it.e = int(v & 0xffffu);
        it.pair = s_base[it.e] + int(v >> 16);
        it.count = min(NC, s_base[it.e + 1] - it.pair);
        return it;
    };

    // Waits for a count that other CTAs raise: bounded like every wait.
    auto meet = [&](const unsigned *counter, int count) {
        for (int i = 0; i < (1 << 21); ++i) {
            unsigned v;
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
            if (v >= unsigned(count)) return true;
            if ((i & 63) == 63 && *wait.abort) return false;
        }
        atomicOr(p.err, 1u);
        *wait.abort = 1;
        return false;
    };

    // after a wait that ran out: copies in flight end before the CTA does; none is
    // longer on its way than this
    auto drain = [&]() {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) {}
    };

    if (warp >= kWorkers && warp < kTake0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kWorkers + kGroups) {
            // -------------------------------------- the weights' side of the slots
            int chunk = 0;
            Turn turn;
            bool ok = true;
            // scales and biases of an item's rows from slot i on: of A the rows r0 of
            // gate and up, of B 128 rows from r0 (`rows` of them the expert's)
            auto fetch = [&](bool part_a, const Affines &a, const uint16_t *sc, const uint16_t *bi, const CUtensorMap *sm,
                             const CUtensorMap *bm, int e, int row, int rows, int G, int i) {
                const int buf = chunk & 1, round = chunk >> 1;
                ok = __all_sync(0xffffffffu, round == 0 || wait(sempty0 + 8 * buf, (round - 1) & 1));
                if (!ok) return;
                const int g0 = i * SUBS * 64 / GS, groups = min(p.chunk, G - g0);  // (of kSbRows)
                const int off = L.sb + buf * 2 * p.sb_block;
                const uint32_t bar = sfull0 + 8 * buf;
                ++chunk;
                if (a.mode == kSbBoxes) {
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar, uint32_t(2 * kTileRows * a.pitch));
                        if (part_a) {
                            tma_load_3d(base + off, sm, g0 / 8 * 2, row, 2 * e, bar);
                            tma_load_3d(base + off + p.sb_block, bm, g0 / 8 * 2, row, 2 * e, bar);
                        } else {
                            tma_load_2d(base + off, sm, g0 / 8 * 2, e * p.K + row, bar);
                            tma_load_2d(base + off + p.sb_block, bm, g0 / 8 * 2, e * p.K + row, bar);
                        }
                    } else {
                        mbar_arrive(bar);
                    }
                    mbar_arrive(bar);
                    return;
                }
                Affines b = a;
                b.block = p.sb_block;
                const long long r0 = part_a ? (long long)e * 2 * p.I + row : (long long)e * p.K + row, r1 = r0 + (part_a ? p.I : kHalf);
                const long long all = part_a ? (long long)p.E * 2 * p.I : (long long)p.E * p.K;
                b.fetch(base + off, smem + off, sc, bi, sm, bm, r0, kHalf, all, G, g0, groups, bar, lane);
                if (rows > kHalf) b.fetch(base + off + kHalf * a.pitch, smem + off + kHalf * a.pitch, sc, bi, sm, bm, r1, kHalf, all, G, g0, groups, bar, lane);
                else mbar_arrive(bar);
            };
            for (Items is = items_of(p.tiles_a); is.entry < is.entries && ok; advance(is)) {
                const Item im = item_of(is);
                int left = 0;  // slots until the next scales and biases
                for (int i = 0; i < p.NSa && ok; ++i, --left, turn.step(1, p.slots)) {
                    if (left == 0) {
                        left = p.cha;
                        fetch(true, p.sba, p.gu_s, p.gu_b, &sa, &ba, im.e, im.tl * kHalf, kTileRows, p.Ga, i);
                    }
                    if (ok && lane == 0) {
                        ok = turn.lap == 0 || wait(empty0 + 8 * turn.slot, (turn.lap - 1) & 1);
                        const uint32_t full = full0 + 8 * turn.slot;
                        if (ok) {
                            mbar_arrive_expect_tx(full, kTileRows * kSlotBytes);
                            tma_load_3d(base + turn.slot * L.slot, &wa, i * (kSlotBytes / 8), im.tl * kHalf, 2 * im.e, full);
                        }
                    }
                    ok = __all_sync(0xffffffffu, ok);
                }
            }
            for (Items is = items_of(p.tiles_b, s_entries * p.tiles_a); is.entry < is.entries && ok; advance(is)) {
                const Item im = item_of(is);
                const int row = im.tl * kTileRows;
                int left = 0;
                for (int i = 0; i < p.NSb && ok; ++i, --left, turn.step(1, p.slots)) {
                    if (left == 0) {
                        left = p.chb;
                        fetch(false, p.sbb, p.dn_s, p.dn_b, &sbm, &bb, im.e, row, min(p.K - row, kTileRows), p.Gb, i);
                    }
                    if (ok && lane == 0) {
                        ok = turn.lap == 0 || wait(empty0 + 8 * turn.slot, (turn.lap - 1) & 1);
                        const uint32_t full = full0 + 8 * turn.slot;
                        if (ok) {
                            mbar_arrive_expect_tx(full, kTileRows * kSlotBytes);
                            tma_load_2d(base + turn.slot * L.slot, &wb, i * (kSlotBytes / 8), im.e * p.K + row, full);
                        }
                    }
                    ok = __all_sync(0xffffffffu, ok);
                }
            }
            if (!ok && lane == 0) drain();
        } else if (warp >= kGather0) {
            // ------------------------------------------------- the vectors' side of the slots
            Turn turn, mturn;
            bool ok = true;
            const int which = warp - kGather0;
            constexpr int MINE = (NC + kGatherers - 1) / kGatherers;
            // the lane's 16 bytes of each token's: subgroup, term and piece
            const int gsub = lane >> 3, gh = lane >> 2 & 1, gpc = lane & 3;
            // and the token, subgroup and half of its sums
            const int msub = lane / 2 % SUBS, mf = lane & 1, mtok = which * (16 / SUBS) + lane / (2 * SUBS);
            for (Items is = items_of(p.tiles_a); is.entry < is.entries && ok; advance(is)) {
                const Item im = item_of(is);
                // where each token's bytes come from, slot by slot
                const uint8_t *from[MINE];
                const float *mfrom;
#pragma unroll
                for (int j = 0; j < MINE; ++j)
                    from[j] = p.rows + size_t(s_tok[im.pair + min(which + j * kGatherers, im.count - 1)]) * p.NSa * (SUBS * 128) + lane * 16;
                mfrom = reinterpret_cast<const float *>(p.xmeta + size_t(s_tok[im.pair + min(mtok, im.count - 1)]) * p.NSa * SUBS + msub) + mf;
                for (int i = 0; i < p.NSa; ++i, turn.step(1, p.slots), mturn.step(1, p.slots + kGroups)) {
                    ok = ok && (turn.lap == 0 || wait(empty0 + 8 * turn.slot, (turn.lap - 1) & 1));
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const uint32_t full = full0 + 8 * turn.slot, dst = base + turn.slot * L.slot;
                    const uint32_t sums = base + L.meta + mturn.slot * (SUBS * MB);
                    // the tokens' operand bytes, 512 a time, and their sums
#pragma unroll
                    for (int j = 0; j < MINE; ++j) {
                        const int tk = which + j * kGatherers;
                        if (tk >= im.count) break;
                        const uint32_t d = dst + L.cells + gsub * CA + operand_offset(operand_index(tk, gh), gpc);
#pragma unroll
                        for (int s = 0; s < SUBS / 4; ++s)
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + s * 4 * CA), "l"(from[j] + s * 512) : "memory");
                        from[j] += SUBS * 128;
                    }
                    if (mtok < im.count)
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(sums + msub * MB + (mtok >> 1) * 16 + (mtok & 1) * 4 + mf * 8),
                                     "l"(mfrom)
                                     : "memory");
                    mfrom += SUBS * 2;
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full) : "memory");
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            if (ok && which == 0 && lane == 0) {
                int ready = -1;
                for (Items is = items_of(p.tiles_b, s_entries * p.tiles_a); is.entry < is.entries && ok; advance(is)) {
                    const uint8_t *h = p.h + size_t(is.entry) * p.NSb * (SUBS * (CB + MB));
                    if (ready != is.entry) {
                        ready = is.entry;
                        ok = meet(p.counters + 1 + ready, p.tiles_a);
                        asm volatile("fence.proxy.async;" ::: "memory");
                    }
                    for (int i = 0; i < p.NSb && ok; ++i, h += SUBS * (CB + MB), turn.step(1, p.slots), mturn.step(1, p.slots + kGroups)) {
                        ok = turn.lap == 0 || wait(empty0 + 8 * turn.slot, (turn.lap - 1) & 1);
                        const uint32_t full = full0 + 8 * turn.slot;
                        if (!ok) break;
                        // (one of the lanes' arrivals, and for the others, which arrive of their own in A)
                        mbar_arrive_expect_tx(full, SUBS * (CB + MB));
                        mbar_arrive_many(full, 32 * kGatherers - 1);
                        bulk_load_plain(base + turn.slot * L.slot + L.cells, h, SUBS * CB, full);
                        bulk_load_plain(base + L.meta + mturn.slot * (SUBS * MB), h + SUBS * CB, SUBS * MB, full);
                    }
                }
            }
            if (!ok && lane == 0) drain();
        } else if (warp >= kWorkers && warp < kWorkers + kGroups) {
            // ------------------------------------------------------ tensor warps
            const int group = warp - kWorkers;
            if (lane == 0) {
                // turn: of the item's first slot
                Turn turn;
                Pipe pipe = Pipe::make<NC, 2>(tm, 0, stored0, ready0, group);
                for (Items is = items_of(p.tiles_a); is.entry < is.entries; advance(is), turn.step(p.NSa, p.slots)) {
                    Turn at = turn;
                    const int i0 = first_slot(group, turn.slot);
                    at.step(i0, p.slots);
                    for (int i = i0; i < p.NSa; i += kGroups, at.step(kGroups, p.slots))
                        multiply_slot<BITS, NC, 2, true>(wait, pipe, base + at.slot * L.slot + L.cells, empty0 + 8 * at.slot);
                }
                Pipe pb = Pipe::make<NC, kTermsH>(tm, 0, stored0, ready0, group);
                pb.steps = pipe.steps;
                for (Items is = items_of(p.tiles_b, s_entries * p.tiles_a); is.entry < is.entries; advance(is), turn.step(p.NSb, p.slots)) {
                    Turn at = turn;
                    const int i0 = first_slot(group, turn.slot);
                    at.step(i0, p.slots);
                    for (int i = i0; i < p.NSb; i += kGroups, at.step(kGroups, p.slots))
                        multiply_slot<BITS, NC, kTermsH>(wait, pb, base + at.slot * L.slot + L.cells, empty0 + 8 * at.slot);
                }
            }
        }
    } else if (warp >= kTake0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTakerRegs));
        // ------------------------------------------- what comes of the items' sums
        // (The four warps meet in every item, also after a wait has run out.)
        Turn set;
        const int row = (warp - kTake0) * 32 + lane;
        const uint32_t ex0 = tm + (uint32_t((warp - kTake0) * 32) << 16) + kExchange;
        uint8_t *own = smem + L.cell;  // an item's cell of h and its sums
        float2 *red = reinterpret_cast<float2 *>(smem + L.red);
        const int half = lane >> 4, r = (warp - kTake0) * 16 + (lane & 15);  // as in the workers
        // B may start on an entry when all its items are counted. (A release takes
        // thousands of cycles under the stream of weights; by the workers, or by
        // warps that gather as well, it cost more than it gave.)
        int written = -1;  // entry of the last item
        auto publish = [&]() {
            if (row == 0 && written >= 0) {
                asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
                asm volatile("fence.proxy.async;" ::: "memory");
                asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p.counters + 1 + written) : "memory");
            }
            written = -1;
        };
        for (Items is = items_of(p.tiles_a); is.entry < is.entries; advance(is)) {
            const Item im = item_of(is);
            float sums[NC];
            Row<BITS, GS, NC, 2>::take(wait, ex0 + set.slot * kExchangeSet, joined0 + 8 * set.slot, freed0 + 8 * set.slot, set.lap, lane, sums);
            set.step(1, kSets);
            publish();  // the last item's h, which has long been written
            // lanes of gate rows form h of the even tokens, those of up rows of the odd
            float h[NC / 2];
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) {
                const float mine = half ? sums[2 * i + 1] : sums[2 * i];
                const float other = __shfl_xor_sync(0xffffffffu, half ? sums[2 * i] : sums[2 * i + 1], 16);
                h[i] = __fmul_rn(activation(half ? other : mine, p.gelu), half ? mine : other);
            }
            // sum and largest exponent of the 64
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) {
                const uint32_t E = __reduce_max_sync(0xffffu << (lane & 16), max(kLeastExponent, (__float_as_uint(h[i]) >> 23) & 0xffu));
                float sum = __fmul_rn(h[i], kSumScale);
#pragma unroll
                for (int d = 8; d; d >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, d));
                if ((lane & 15) == 0) red[(half * (NC / 2) + i) * 4 + (warp & 3)] = make_float2(sum, __uint_as_float(E));
            }
            named_sync(2, 32 * kTakers);
            // the element's byte of its row, in the order of the masks
            const int pc = r >> 4, e = r & 15;
            const int at = BITS == 4 ? (e >> 3) * 8 + (e & 1) * 4 + ((e & 7) >> 1) : (e & 3) * 4 + (e >> 2);
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) {
                const int j = 2 * i + half;
                const float4 r0 = reinterpret_cast<const float4 *>(red)[(half * (NC / 2) + i) * 2];
                const float4 r1 = reinterpret_cast<const float4 *>(red)[(half * (NC / 2) + i) * 2 + 1];
                const uint32_t E = max(max(__float_as_uint(r0.y), __float_as_uint(r0.w)), max(__float_as_uint(r1.y), __float_as_uint(r1.w)));
                const int pw = scale_power(E);
                float v = __fmul_rn(__fmul_rn(h[i], exp2i(pw / 2)), exp2i(pw - pw / 2));
                if (BITS == 2 && (e & 1)) v = __fmul_rn(v, 0.25f);
#pragma unroll
                for (int t = 0; t < kTermsH; ++t) {
                    const uint32_t b = to_e4m3x2(v, 0.0f);
                    float back, none;
                    from_e4m3x2(b, back, none);
                    v = __fmul_rn(__fsub_rn(v, back), 32.0f);
                    own[operand_offset(operand_index(j, t, kTermsH), pc) + at] = uint8_t(b);
                }
                if (r == 0) {
                    float *m = reinterpret_cast<float *>(own + CB + i * 16) + half;
                    m[0] = __fadd_rn(__fadd_rn(r0.x, r0.z), __fadd_rn(r1.x, r1.z));
                    m[2] = unscale(E);
                }
            }
            uint8_t *slot_h = p.h + (size_t(im.entry) * p.NSb + im.tl / SUBS) * (SUBS * (CB + MB));
            // subgroups that fill the last slot
            if (im.tl == p.tiles_a - 1 && p.Sb % SUBS) {
                for (int sub = p.Sb % SUBS; sub < SUBS; ++sub) {
                    uint32_t *c = reinterpret_cast<uint32_t *>(slot_h + sub * CB), *m = reinterpret_cast<uint32_t *>(slot_h + SUBS * CB + sub * MB);
                    for (int i = row; i < CB / 4; i += 32 * kTakers) c[i] = 0u;
                    for (int i = row; i < MB / 4; i += 32 * kTakers) m[i] = 0u;
                }
                asm volatile("fence.proxy.async;" ::: "memory");
                __threadfence();
            }
            fence_proxy_async_smem();
            named_sync(2, 32 * kTakers);
            if (row == 0) {
                const uint32_t from = smem_u32(own);
                bulk_store(slot_h + im.tl % SUBS * CB, from, CB);
                bulk_store(slot_h + SUBS * CB + im.tl % SUBS * MB, from + CB, MB);
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
            written = im.entry;
        }
        publish();
        for (Items is = items_of(p.tiles_b, s_entries * p.tiles_a); is.entry < is.entries; advance(is)) {
            const Item im = item_of(is);
            const int n = im.tl * kTileRows + row;
            float sums[NC];
            Row<BITS, GS, NC, kTermsH>::take(wait, ex0 + set.slot * kExchangeSet, joined0 + 8 * set.slot, freed0 + 8 * set.slot, set.lap, lane, sums);
            set.step(1, kSets);
#pragma unroll
            for (int j = 0; j < NC; ++j)
                if (j < im.count && n < p.K) __stcg(p.partials + size_t(im.pair + j) * p.K + n, sums[j]);
        }
        named_sync(2, 32 * kTakers);
        if (row == 0) {
            __threadfence();  // (of what the barrier ordered before it, too)
            asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p.counters) : "memory");
        }
    } else {
        // ----------------------------------------------------------- workers
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWorkerRegs));
        const int group = warp / 4, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
        Turn turn, mturn;  // of the item's first slot
        int chunk = 0;
        // all slots of an item's rows into acc
        auto run = [&](auto &acc, Pipe &pipe, const Affines &a, int ch, int NS, int G, int row, long long grow) {
            const uint32_t wrow = base + row * kSlotBytes + ((row & 7) << 4);
            const int align = a.alignment(G);
            constexpr int STEP = std::remove_reference_t<decltype(acc)>::kStep;
            uint32_t last = 0;
            acc.start();
            Turn at = turn, mat = mturn;
            const int i0 = first_slot(group, turn.slot);
            at.step(i0, p.slots);
            mat.step(i0, p.slots + kGroups);
            for (int c0 = 0; c0 < NS; c0 += ch, ++chunk) {
                const int buf = chunk & 1, c1 = min(c0 + ch, NS), g0 = c0 * SUBS * 64 / GS;
                wait(sfull0 + 8 * buf, (chunk >> 1) & 1);
                const uint32_t sb = base + L.sb + buf * 2 * p.sb_block + row * a.pitch + a.offset(grow, G, g0);
#pragma unroll 1
                for (int i = c0 + (i0 + kGroups - c0 % kGroups) % kGroups; i < c1;
                     i += kGroups, at.step(kGroups, p.slots), mat.step(kGroups, p.slots + kGroups)) {
                    const int s = at.slot;
                    wait(full0 + 8 * s, at.lap & 1);
                    Affine<BITS, GS> aff;
                    constexpr int GP = Affine<BITS, GS>::kGroupsPerSlot;
                    aff.read(sb + (i - c0) * GP * 2, p.sb_block, align, G - i * GP);
                    const uint32_t meta = base + L.meta + mat.slot * (SUBS * MB);
                    acc.slot(wait, pipe, wrow + s * L.slot, aff, meta, last, lane);
                    last = meta + (SUBS - 2 * STEP) * MB;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(empty0 + 8 * s);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(sempty0 + 8 * buf);
            }
            acc.finish(wait, pipe, last);
            __syncwarp();
            turn.step(NS, p.slots);
            mturn.step(NS, p.slots + kGroups);
        };

        // the sums' set and how many items had it before
        Turn set;
        auto give = [&](auto &acc, int c) {
            acc.give(wait, tm + lanes + kExchange + set.slot * kExchangeSet, c, joined0 + 8 * set.slot, freed0 + 8 * set.slot, set.lap, lane);
            set.step(1, kSets);
        };
        Pipe pipe = Pipe::make<NC, 2>(tm, lanes, stored0, ready0, group);
        // A warp holds 16 gate rows and the same 16 up rows.
        const int half = lane >> 4, r = (warp & 3) * 16 + (lane & 15), arow = half * kHalf + r;
        for (Items is = items_of(p.tiles_a); is.entry < is.entries; advance(is)) {
            const Item im = item_of(is);
            const int c = first_slot(group, turn.slot);
            Row<BITS, GS, NC, 2> acc;
            run(acc, pipe, p.sba, p.cha, p.NSa, p.Ga, arow, (long long)im.e * 2 * p.I + half * p.I + im.tl * kHalf + r);
            give(acc, c);
        }
        Pipe pb = Pipe::make<NC, kTermsH>(tm, lanes, stored0, ready0, group);
        pb.steps = pipe.steps;
        for (Items is = items_of(p.tiles_b, s_entries * p.tiles_a); is.entry < is.entries; advance(is)) {
            const Item im = item_of(is);
            const int c = first_slot(group, turn.slot);
            Row<BITS, GS, NC, kTermsH> acc;
            run(acc, pb, p.sbb, p.chb, p.NSb, p.Gb, row, (long long)im.e * p.K + im.tl * kTileRows + row);
            give(acc, c);
        }
        if (tid == 0) {
            (void)meet(p.counters, grid);
            __threadfence();
        }
        named_sync(1, 32 * kWorkers);
        // y, four elements at a time (K is a multiple of 64)
        const int quads = p.M * p.K / 4;
        for (int i = blockIdx.x * 32 * kWorkers + tid; i < quads; i += grid * 32 * kWorkers) {
            const int t = i / (p.K / 4), n = (i - t * (p.K / 4)) * 4;
            float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int j0 = 0; j0 < p.k; j0 += 4) {
                float4 v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j0 + j < p.k) v[j] = __ldcg(reinterpret_cast<const float4 *>(p.partials + size_t(s_pos[t * p.k + j0 + j]) * p.K + n));
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j0 + j < p.k) {
                        const float w = s_w[t * p.k + j0 + j];
                        s.x = __fmaf_rn(w, v[j].x, s.x);
                        s.y = __fmaf_rn(w, v[j].y, s.y);
                        s.z = __fmaf_rn(w, v[j].z, s.z);
                        s.w = __fmaf_rn(w, v[j].w, s.w);
                    }
            }
            const size_t at = size_t(t) * p.K + n;
            const float o[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (p.f32_out) static_cast<float *>(p.y)[at + j] = o[j];
                else static_cast<__nv_bfloat16 *>(p.y)[at + j] = __float2bfloat16_rn(o[j]);
        }
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == kWorkers) tmem_free(tm, kTmemColumns);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

qmv_status check_moe(int M, int K, int I, int E, int k, int bits, int gs)
{
    qmv_status st = check_weights(M, 1, K, bits, gs);
    if (st != QMV_OK) return st;
    if (K > (1 << 16) || I < 1 || I > (1 << 16) || I % gs) return QMV_ERR_SHAPE;
    if (E < 1 || E > QMV_MAX_EXPERTS || k < 1 || k > E || k > QMV_MAX_TOP_K || M * k > QMV_MAX_CHOICES) return QMV_ERR_COUNT;
    if ((long long)E * 2 * I * (K / gs) >= (1ll << 31) || (long long)E * K * (I / gs) >= (1ll << 31) ||
        (long long)E * 2 * I > (1 << 30) || (long long)E * K > (1 << 30))
        return QMV_ERR_SHAPE;
    return QMV_OK;
}

size_t up256(size_t b) { return (b + 255) & ~size_t(255); }

struct MoeSizes {
    size_t logits, rows, xmeta, h, partials, counters, total;
};

// Tokens of an expert that one read of its weights serves: 2, 4 or 8, so that
// the mean number and some spread fit.
int columns(int M, int E, int k)
{
    const double mean = double(M) * k / E;
    if (M <= 2 || mean <= 0.3) return 2;
    return M <= 4 || mean <= 1.5 ? 4 : 8;
}

// The plan with p.nc tokens to an entry and p.chunk groups to a fetch, if its
// shared memory fits.
bool fit(MoeParams &p, int bits)
{
    const int subs = tile::slot_subs(bits), pairs = p.M * p.k;
    p.max_entries = pairs < p.E + pairs / p.nc ? pairs : p.E + pairs / p.nc;
    p.sba = tile::Affines::plan(p.Ga, p.Ga < p.chunk ? p.Ga : p.chunk, tile::kTileRows, 2 * p.chunk);
    p.sbb = tile::Affines::plan(p.Gb, p.Gb < p.chunk ? p.Gb : p.chunk, tile::kTileRows, 2 * p.chunk);
    p.cha = p.sba.mode == tile::kSbWhole ? p.NSa : p.chunk * p.gs / 64 / subs;
    p.chb = p.sbb.mode == tile::kSbWhole ? p.NSb : p.chunk * p.gs / 64 / subs;
    p.sb_block = p.sba.block > p.sbb.block ? p.sba.block : p.sbb.block;
    p.slots = kMaxSlotsMoe;
    while (p.slots > kMinSlotsMoe && moe_layout(p, bits, p.nc).total > kSmemMoe) p.slots -= tile::kGroups;
    // (the routing's rows of logits lie before the lists)
    const MoeLayout l = moe_layout(p, bits, p.nc);
    return l.total <= kSmemMoe && l.lists >= kMoeThreads / 32 * p.E * 4;
}

MoeParams plan_moe(int M, int K, int I, int E, int k, int bits, int gs, MoeSizes &z)
{
    const int subs = tile::slot_subs(bits);
    MoeParams p{};
    p.M = M; p.K = K; p.I = I; p.E = E; p.k = k; p.gs = gs;
    p.Sa = K / 64; p.NSa = (p.Sa + subs - 1) / subs; p.Ga = K / gs;
    p.Sb = I / 64; p.NSb = (p.Sb + subs - 1) / subs; p.Gb = I / gs;
    p.tiles_a = I / kHalf;
    p.tiles_b = (K + tile::kTileRows - 1) / tile::kTileRows;
    // scales and biases 32 groups at a time, or 16 where there is no room; fewer
    // tokens to an entry where there is none still (2-bit weights with 8)
    const int pairs = M * k;
    for (p.nc = columns(M, E, k);; p.nc /= 2) {
        p.chunk = 32;
        if (fit(p, bits)) break;
        p.chunk = 16;
        if (fit(p, bits) || p.nc == 2) break;
    }
    const size_t hs = size_t(p.max_entries) * p.NSb * subs;
    z.logits = up256(size_t(M) * E * 4);
    z.rows = up256(size_t(M) * p.NSa * subs * 128);
    z.xmeta = up256(size_t(M) * p.NSa * subs * 8);
    z.h = up256(hs * (tile::cell_bytes(p.nc, kTermsH) + tile::meta_bytes(p.nc)));
    z.partials = up256(size_t(pairs) * K * 4);
    z.counters = up256((1 + size_t(p.max_entries)) * 4);
    z.total = z.logits + z.rows + z.xmeta + z.h + z.partials + z.counters;
    return p;
}

struct MoeMaps {
    CUtensorMap wa, sa, ba, wb, sb, bb;
};

template <int BITS, int GS, int NC>
cudaError_t launch_experts(const MoeMaps &m, MoeParams &p, int sms, cudaStream_t stream)
{
    static std::atomic<int> configured[64] = {};
    const int smem = moe_layout(p, BITS, NC).total;
    if (smem > kSmemMoe) return cudaErrorInvalidConfiguration;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::mutex lock;
    if (configured[dev].load() < smem) {
        std::lock_guard<std::mutex> hold(lock);
        if (configured[dev].load() < smem) {
            e = cudaFuncSetAttribute(moe_experts<BITS, GS, NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            configured[dev].store(smem);
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sms);
    cfg.blockDim = dim3(kMoeThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, moe_experts<BITS, GS, NC>, m.wa, m.sa, m.ba, m.wb, m.sb, m.bb, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int BITS, int GS>
cudaError_t launch_experts_nc(const MoeMaps &m, MoeParams &p, int sms, cudaStream_t stream)
{
    if (p.nc == 2) return launch_experts<BITS, GS, 2>(m, p, sms, stream);
    if (p.nc == 4) return launch_experts<BITS, GS, 4>(m, p, sms, stream);
    return launch_experts<BITS, GS, 8>(m, p, sms, stream);
}

template <int BITS>
cudaError_t launch_moe(const MoeMaps &m, MoeParams &p, int sms, cudaStream_t stream)
{
    static std::atomic<int> configured[64] = {};
    Launch l;
    l.grid = dim3(p.stage_blocks + p.E);
    l.threads = kLogitThreads;
    l.smem = 0;
    l.pdl = true;
    const cudaError_t e = launch_one(moe_logits<BITS>, configured, l, stream, p);
    if (e != cudaSuccess) return e;
    return p.gs == 64 ? launch_experts_nc<BITS, 64>(m, p, sms, stream) : launch_experts_nc<BITS, 128>(m, p, sms, stream);
}

}  // namespace
}  // namespace qmv

extern "C" size_t qmv_moe_workspace_size(int M, int K, int inter, int experts, int top_k, int bits, int group_size)
{
    if (qmv::check_moe(M, K, inter, experts, top_k, bits, group_size) != QMV_OK) return 0;
    qmv::MoeSizes z;
    qmv::plan_moe(M, K, inter, experts, top_k, bits, group_size, z);
    return z.total;
}

extern "C" qmv_status qmv_moe_run(const uint16_t *x, const uint16_t *router, const uint32_t *gu_w,
                                  const uint16_t *gu_scales, const uint16_t *gu_biases, const uint32_t *dn_w,
                                  const uint16_t *dn_scales, const uint16_t *dn_biases, void *y, int32_t *topk_ids,
                                  float *topk_weights, int M, int K, int inter, int experts, int top_k, int bits,
                                  int group_size, void *workspace, size_t workspace_bytes, unsigned flags,
                                  qmv_stream_t stream)
{
    using namespace qmv;
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
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != QMV_OK) return st;
    MoeSizes z;
    MoeParams p = plan_moe(M, K, inter, experts, top_k, bits, group_size, z);
    void *ws = nullptr;
    st = scratch(dev, z.total, workspace, workspace_bytes, &ws);
    if (st != QMV_OK) return st;

    p.x = x; p.router = router;
    p.gu_s = gu_scales; p.gu_b = gu_biases; p.dn_s = dn_scales; p.dn_b = dn_biases;
    p.y = y; p.ids_out = topk_ids; p.weights_out = topk_weights;
    p.err = dev.err;
    p.f32_out = (flags & QMV_F32_OUT) != 0;
    p.gelu = (flags & QMV_MOE_GELU) != 0;
    p.softmax_all = (flags & QMV_MOE_SOFTMAX_ALL) != 0;
    uint8_t *at = static_cast<uint8_t *>(ws);
    p.logits = reinterpret_cast<float *>(at); at += z.logits;
    p.rows = at; at += z.rows;
    p.xmeta = reinterpret_cast<float2 *>(at); at += z.xmeta;
    p.h = at; at += z.h;
    p.partials = reinterpret_cast<float *>(at); at += z.partials;
    p.counters = reinterpret_cast<unsigned *>(at);
    p.stage_blocks = int(((long long)M * p.NSa * tile::slot_subs(bits) * 8 + kLogitThreads - 1) / kLogitThreads);

    MoeMaps m{};
    const long long rb = (long long)experts * K;
    const long long two_e = 2ll * experts;
    st = encode_rows(&m.wa, gu_w, (long long)K * bits / 8, inter, tile::kSlotBytes / 8, kHalf, true, two_e, 2);
    if (st == QMV_OK) st = encode_rows(&m.wb, dn_w, (long long)inter * bits / 8, rb, tile::kSlotBytes / 8, tile::kTileRows, true);
    if (p.sba.mode == tile::kSbBoxes) {
        if (st == QMV_OK) st = encode_rows(&m.sa, gu_scales, p.Ga * 2ll, inter, p.sba.pitch / 8, kHalf, false, two_e, 2);
        if (st == QMV_OK) st = encode_rows(&m.ba, gu_biases, p.Ga * 2ll, inter, p.sba.pitch / 8, kHalf, false, two_e, 2);
    }
    if (p.sbb.mode == tile::kSbBoxes) {
        if (st == QMV_OK) st = encode_rows(&m.sb, dn_scales, p.Gb * 2ll, rb, p.sbb.pitch / 8, tile::kTileRows, false);
        if (st == QMV_OK) st = encode_rows(&m.bb, dn_biases, p.Gb * 2ll, rb, p.sbb.pitch / 8, tile::kTileRows, false);
    }
    if (st != QMV_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = bits == 4 ? launch_moe<4>(m, p, dev.sms, s) : launch_moe<2>(m, p, dev.sms, s);
    return e == cudaSuccess ? QMV_OK : record_cuda_failure("moe kernel launch", e);
}
