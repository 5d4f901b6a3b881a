// qmv_attend_run: attention of new tokens over a paged cache.
//
// Two kinds of sequences: those of a few new tokens, whose keys and values are read
// once for all of them (attend_few, attend_join), and prompts, which are bound by their
// products (attend_prompt, attend_join_pieces). A call that may hold both launches both; each
// takes its own.
#include <cuda.h>
#include <cuda_bf16.h>

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "qmv.h"
#include "qmv_attend_plan.h"
#include "qmv_cache.h"
#include "qmv_launch.cuh"
#include "qmv_tile.cuh"

namespace qmv {
namespace {

using namespace attend;
using tile::named_sync;
using tile::settle;
using tile::tmem_commit;
using tile::tmem_fence_after;
using tile::tmem_fence_before;
using tile::tmem_ld;
using tile::tmem_wait_ld;
using tile::tmem_wait_st;
using tile::Waits;

struct AttendParams {
    const int32_t *table, *q_start, *kv_len;
    uint16_t *out;
    float *lse;
    int B, T, max_new, heads, kv_heads, group;
    int page_size, pages, max_pages;
    uint64_t magic;       // of page_size: see page_of
    int map_code;         // of the largest boxes in use
    float scale;
    int window, sinks;
    int64_t ld_out;
    unsigned *err;
    // the plan, and the workspace's parts
    int items;  // at most
    bool by_row;
    int kept;   // rows whose sums have a place
    int tokens, rows, units, unit_shift, pieces, slots, key_slots, q_sets;
    int p_off, q_off, misc_off;
    int32_t *prefix;
    float2 *meta;
    float *parts;
};

// First row, new tokens (and those of them that are computed), keys and the first new
// token's position of a sequence.
struct Sequence {
    int row, n, done, keys, pos;
    __device__ __forceinline__ Sequence(const AttendParams &p, const int4 &kept) : row(kept.x), n(kept.y), done(min(n, p.max_new)), keys(kept.z), pos(keys - n) {}
    __device__ __forceinline__ Sequence(const AttendParams &p, int b)
    {
        row = p.q_start ? min(max(__ldg(p.q_start + b), 0), p.T) : b * p.max_new;
        n = p.q_start ? min(max(__ldg(p.q_start + b + 1), row), p.T) - row : p.max_new;
        done = min(n, p.max_new);
        keys = min(max(__ldg(p.kv_len + b), 0), p.max_pages * p.page_size);
        pos = keys - n;
    }
};

// Keys that some of a sequence's queries at positions first .. last see: below `end`, and
// from `low` on or below `first` (of which none where there is no window).
struct Seen {
    int end, low, sinks;
    __device__ __forceinline__ Seen(const AttendParams &p, int first, int last)
    {
        end = max(last + 1, 0);
        low = p.window ? max(first - p.window + 1, 0) : 0;
        sinks = p.window ? min(p.sinks, low) : 0;
    }
    __device__ __forceinline__ bool operator()(int key) const { return key < end && (key >= low || key < sinks); }
    // Does it hold for a key of key .. key + n - 1?
    __device__ __forceinline__ bool any(int key, int n) const { return key < end && (key + n > low || key < sinks); }
};

// Bits 0 .. n - 1.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// One lane of a converged warp, for the instructions that a single thread issues. (With a
// plain lane == 0 the compiler does not know that one thread is left, and a step of four
// products took some 800 cycles.)
__device__ __forceinline__ bool one_lane()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// Has the phase of that parity ended? (Asked ahead of a wait, whose answer takes some 300 cycles
// while products read shared memory.)
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^e for a whole number e <= 0, exactly (0 below 2^-126).
__device__ __forceinline__ float power_of_two(float e) { return e < -126.0f ? 0.0f : tile::exp2i(int(e)); }

// The largest of a warp's values, of those that are numbers, for each of 16: lanes 2 i
// and 2 i + 1 end with that of value i. Each step halves what a lane keeps.
template <int N>
__device__ __forceinline__ void max_step(float (&v)[16], int lane)
{
    const bool upper = (lane & 2 * N) != 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float keep = upper ? v[N + i] : v[i], send = upper ? v[i] : v[N + i];
        v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 2 * N));
    }
}
__device__ __forceinline__ float max_scatter(float (&v)[16], int lane)
{
    max_step<8>(v, lane);
    max_step<4>(v, lane);
    max_step<2>(v, lane);
    max_step<1>(v, lane);
    return fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// Tensor maps of keys and of values, with boxes of 8, 16, 32 and 64 keys.
struct CacheMaps {
    CUtensorMap k[4], v[4];
};

// A lane's eight keys of 128 or 256 from a multiple of 128 on (lanes past them have none).
// Keys that lie together, in one page and in one block of 64, come by as few boxes as the
// binary digits of their number. (A box takes some 100 cycles of the warp that issues it,
// whatever its size.)
struct Boxes {
    int page, place;  // outside the map where there is none (zeros); in the page
    int code;         // of the box's size
    bool start;       // does a box start with the lane's keys?
    uint32_t there;   // bits of the lanes whose keys' page is there

    __device__ __forceinline__ void find(const AttendParams &p, const Seen &seen, const int32_t *table, int first, int lane, int lanes)
    {
        const int key = first + 8 * lane, row = page_of(p.magic, key), at = key - row * p.page_size;
        const int before = min(lane & 7, at / 8), all = before + min(8 - (lane & 7), (p.page_size - at) / 8);
        code = -1;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if ((all >> c & 1) && before == (all >> (c + 1)) << (c + 1)) code = c;
        start = code >= 0 && lane < lanes;
        page = start && seen.any(key, 8 << code) ? __ldg(table + row) : -1;
        const bool found = unsigned(page) < unsigned(p.pages);
        if (!found) page = p.pages;
        place = at;
        there = __reduce_or_sync(0xffffffffu, found ? ((1u << (1 << (code & 3))) - 1u) << lane : 0u);
    }

    // The boxes of the keys of lanes from .. from + n - 1, to `dst` on: BLOCKS times 64 elements,
    // `apart` bytes apart. (The lanes where they start issue them; one lane that goes through
    // them with shuffles took half as long again.)
    template <int BLOCKS>
    __device__ __forceinline__ void bring(const CUtensorMap *maps, uint32_t dst, int lane, int from, int n, int column, int apart, int g, uint32_t bar) const
    {
        if (!start || lane < from || lane >= from + n) return;
#pragma unroll
        for (int c = 0; c < BLOCKS; ++c) tma_load_4d(dst + (lane - from) * 1024 + c * apart, maps + code, column + 64 * c, place, g, page, bar);
    }
};

// Descriptor of an operand in shared memory: `leading` and `stride` bytes as the layout
// has them, layout 2 for the 128-byte swizzle and 4 for the 64-byte one.
__device__ __forceinline__ uint64_t descriptor(uint32_t addr, uint32_t leading, uint32_t stride, uint32_t layout)
{
    return uint64_t((addr >> 4) & 0x3fffu) | uint64_t((leading >> 4) & 0x3fffu) << 16 | uint64_t((stride >> 4) & 0x3fffu) << 32 |
           uint64_t(1) << 46 | uint64_t(layout) << 61;
}

// Kind of a product of bf16 operands with fp32 sums, 128 x N; a operand whose rows
// are contiguous instead of its products' index is `rows` major.
__host__ __device__ constexpr uint32_t mma_kind(int N, bool a_rows, bool b_rows)
{
    return 1u << 4 | 1u << 7 | 1u << 10 | uint32_t(a_rows) << 15 | uint32_t(b_rows) << 16 | uint32_t(N >> 3) << 17 | (128u >> 4) << 24;
}

// D (128 x N fp32, tensor memory) (+)= A (128 x 16) B^T (N x 16), both from shared memory.
__device__ __forceinline__ void mma_ss(uint32_t kind, uint32_t d, uint64_t a, uint64_t b, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(kind), "r"(uint32_t(add))
        : "memory");
}

template <int N>
__device__ __forceinline__ void tmem_st(uint32_t a, const float (&v)[N])
{
    static_assert(N == 16, "columns");
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
    tile::tmem_st(a, r);
}

// ------------------------------------------------------------ few new tokens --
//
// Sequences of up to 16 new tokens. The query rows of one kv head (tokens x group of
// them) are columns, keys are rows:
//
//   S^T (keys x columns)          = K Q^T         K from shared memory as it lies in the cache
//   P^T = exp2(S^T scale log2(e) - m)             a thread has a key, in registers
//   O^T (head_dim x columns)     += V^T P^T       V from shared memory as it lies in the cache
//
// both by tcgen05, keys and values brought by TMA through a ring of 16 KB slots. Keys as
// rows, because a product's time hardly depends on how few columns there are (128 rows and 16
// columns 52 cycles, 128 columns 66), and K and V go into it as they lie. P is kept in two bf16
// terms (16 bits of it), as 2 x columns columns of one product, so that the weights' rounding
// is below that of fp32 sums' order.
//
// What bounds it: with 16 columns the bytes of K and V (64 sequences of 8192 keys, 8 kv heads of
// 128: 247 us, 97 % of the rate of a copy; the tensor cores are busy for 7 %), of a few thousand
// keys the chain of two launches, the first loads and the join (4100 keys: 11.3 us, of which the
// bytes are 2.5), with 64 columns mostly shared memory (13 tokens of 8 heads over 131000 keys: 95 us,
// the bytes 40: of a leaf products read 224 KB there, 128 arrive and weights are 64, 3300 of its
// 5000 cycles at 128 bytes each; what the others go to is not known). What the chain of a leaf costs was mostly waits and meetings:
// every warp forms the references for itself (one meeting a leaf instead of two), barriers are
// asked ahead of their waits (104 us to 95; one token 13.9 to 11.7 with the masks below).
//
// Order. A work item is a unit of 256, 512 or 1024 keys (see few_plan), from a multiple of
// that on, in leaves of 256, whose products are added in the order of keys. A column's reference
// m is a whole number, 8 above the largest score when it is set, and moves only when a score
// passes it: a change of m scales by powers of two without a rounding, and weights are at most
// 1. Units are joined by attend_join in an order given by their places. So a row's result
// depends on its query and the keys that it sees alone: not on the other tokens of the call, nor
// on how many SMs there are.

struct Item {
    int b, g, block, unit;
    uint32_t part;                 // of its first row's sums
    int row, tokens, rows;         // first row of q, its tokens and columns
    int pos;                       // position of the first token; of the last: pos + tokens - 1
    int leaf, leaves;
    bool whole;                    // the sequence has one unit
};

// Units of a sequence: those of its first tokens, then those from its window on.
struct Units {
    int sinks, low, count;
    __device__ __forceinline__ Units(const AttendParams &p, const Sequence &s)
    {
        const Seen seen(p, s.pos, s.pos + s.done - 1);
        low = seen.low >> p.unit_shift;
        sinks = min((seen.sinks + (1 << p.unit_shift) - 1) >> p.unit_shift, low);
        count = seen.end > 0 ? sinks + ((seen.end - 1) >> p.unit_shift) - low + 1 : 1;
        count = s.done > 0 && s.done <= kFew ? min(count, p.units) : 0;
    }
    __device__ __forceinline__ int place(int u) const { return u < sinks ? u : low + u - sinks; }
};

// The sequences in shared memory: each one's first work item, then row, n and keys.
struct Sequences {
    const int32_t *first;  // [B + 1]
    const int4 *kept;      // [B]
};

// Where the sums of token i of sequence b, at the given row of q, lie in the workspace, in groups of
// heads: units, then kv heads, then rows, so that an item's columns lie together. (By rows of q
// there are T places; where 16 for each sequence are fewer, those. Fewer than 2^32 in all, as
// a workspace of at most 2^40 bytes has 264 or more for each.)
__device__ __forceinline__ uint32_t part_of(const AttendParams &p, int b, int row, int i, int u, int g)
{
    return uint32_t(u * p.kv_heads + g) * uint32_t(p.kept) + uint32_t(p.by_row ? row : b * min(p.max_new, kFew) + i);
}

// Counts first[1 .. B] become running sums from first[0] = 0 on, at most `most` (more are there
// only if rows belong to several sequences; of prompts that many have a place); by one warp.
__device__ __forceinline__ void sum_firsts(int32_t *first, int B, int most, int lane)
{
    int64_t sum = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < B; b0 += 32) {
        int64_t v = b0 + lane < B ? first[b0 + lane + 1] : 0;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int64_t u = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += u;
        }
        if (b0 + lane < B) first[b0 + lane + 1] = int32_t(sum + v < most ? sum + v : most);
        sum += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) first[0] = 0;
}

__device__ __forceinline__ Item item_at(const AttendParams &p, const Sequences &all, int index)
{
    int lo = 0, hi = p.B;
#pragma unroll 1
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        (all.first[mid] <= index ? lo : hi) = mid;
    }
    const int4 kept = all.kept[lo];
    const Sequence s(p, kept);
    const Units units(p, s);
    const unsigned blocks = unsigned(kept.w);
    Item it;
    it.b = lo;
    index -= all.first[lo];
    it.block = 0;
    if (blocks > 1) {
        it.block = int(unsigned(index) % blocks);
        index = int(unsigned(index) / blocks);
    }
    const int u = int(unsigned(index) / unsigned(p.kv_heads));
    it.g = index - u * p.kv_heads;
    it.unit = units.place(u);
    it.row = s.row + it.block * p.tokens;
    it.part = part_of(p, lo, it.row, it.block * p.tokens, u, it.g);
    it.tokens = min(p.tokens, s.done - it.block * p.tokens);
    it.rows = it.tokens * p.group;
    it.pos = s.pos + it.block * p.tokens;
    it.whole = units.count == 1;
    const Seen seen(p, it.pos, it.pos + it.tokens - 1);
    int from = it.unit << p.unit_shift;
    int to = min(from + (1 << p.unit_shift), seen.end);
    if (to <= seen.low) to = min(to, seen.sinks);
    if (from >= seen.sinks) from = max(from, seen.low);  // (sinks <= low)
    it.leaf = from / kLeaf;
    it.leaves = from < to ? (to - 1) / kLeaf - it.leaf + 1 : 0;
    return it;
}

// What lies behind the ring, the weights and the queries.
template <int NC>
struct FewShared {
    uint64_t full[16], empty[16], q_full[2], q_empty[2], s_ready[2], p_ready[4], o_done, finished;
    int abort;
    uint32_t tmem;
    float4 top[2][NC];  // a column's largest score in each of four warps, of a leaf and the next
    float sum[4][NC], total[NC];
    int64_t out[NC];        // where its sums go
    uint32_t there[8];      // of the last leaves: which eights of keys have a page
    int4 seqs[1];           // [B], then the sequences' first items [B + 1]
};

// A place in a ring of slots [first, end) and the parity of its lap. A ring has one
// consumer, which takes its slots in order: a wait for a lap's parity is right only when the
// lap before has landed.
struct Place {
    int first, end, slot;
    uint32_t lap = 0;
    int issued = 0;  // (by the producer)
    __device__ __forceinline__ Place(int first, int end) : first(first), end(end), slot(first) {}
    __device__ __forceinline__ void step()
    {
        if (++slot == end) {
            slot = first;
            lap ^= 1;
        }
    }
    __device__ __forceinline__ bool full() const { return issued >= end - first; }
};

static_assert(offsetof(FewShared<16>, seqs) <= few_misc(16) && offsetof(FewShared<32>, seqs) <= few_misc(32) && offsetof(FewShared<64>, seqs) <= few_misc(64), "the plan's room for it");

__host__ __device__ constexpr int few_threads(int NC) { return NC / 16 * 128 + 128; }

// What the first loads need, on its way into the caches while the sequences' lengths are.
__device__ __forceinline__ void prefetch_maps(const CUtensorMap &qmap, const CacheMaps &maps, const AttendParams &p)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&qmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(maps.k + p.map_code)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(maps.v + p.map_code)) : "memory");
}
__device__ __forceinline__ void prefetch_table(const AttendParams &p, int tid)
{
    // 32 entries a line; a small table, by the blocks together
    const int64_t lines = (int64_t(p.B) * p.max_pages + 31) / 32;
    const int64_t line = int64_t(tid) * gridDim.x + blockIdx.x;
    if (lines <= 2048 && line < lines) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.table + 32 * line) : "memory");
}

template <int D, int NC>
__global__ void __launch_bounds__(few_threads(NC), D < 256 && NC == 16 ? 2 : 1)
    attend_few(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CacheMaps maps, const AttendParams p)
{
    constexpr int DB = D / 64, HALVES = D < 128 ? 1 : D / 128;  // blocks of 64 elements; tiles of 128 in V^T's rows
    constexpr int kChunks = 2 * DB;                              // of a leaf's keys, and of its values
    constexpr int kScores = 2 * NC;  // columns of a leaf's scores, of which there are two
    constexpr int kColumns = 2 * kScores + 2 * NC * HALVES, kAlloc = kColumns <= 128 ? 128 : kColumns <= 256 ? 256 : 512;
    constexpr int kKeyBytes = NC == 16 ? 64 : 128;  // of a key's weights in a block of P
    constexpr int kThreads = few_threads(NC), kProducer = kThreads / 32 - 4, kTensor = kProducer + 2;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    FewShared<NC> &sh = *reinterpret_cast<FewShared<NC> *>(smem + p.misc_off);
    int32_t *first = reinterpret_cast<int32_t *>(sh.seqs + p.B);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
    const uint32_t base = smem_u32(smem), full0 = smem_u32(sh.full), empty0 = smem_u32(sh.empty);
    const uint32_t q_full = smem_u32(sh.q_full), q_empty = smem_u32(sh.q_empty), s_ready = smem_u32(sh.s_ready);
    const uint32_t p_ready = smem_u32(sh.p_ready), o_done = smem_u32(&sh.o_done), finished = smem_u32(&sh.finished);
    const uint32_t P = base + p.p_off, Q = base + p.q_off;
    if (tid == 0) {
#pragma unroll 1
        for (int i = 0; i < p.slots; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + 8 * i, 1);
            mbar_init(q_empty + 8 * i, 1);
            mbar_init(s_ready + 8 * i, 2);  // the scores, and the warp that has seen the keys land
            mbar_init(p_ready + 16 * i, NC / 4);  // a warp's arrival
            mbar_init(p_ready + 16 * i + 8, NC / 4);
        }
        mbar_init(o_done, 1);
        mbar_init(finished, 2);
        fence_mbar_init();
        sh.abort = 0;
    }
    if (warp == kTensor) tile::tmem_alloc(smem_u32(&sh.tmem), kAlloc);
    if (tid == 0) prefetch_maps(qmap, maps, p);
    grid_dependency_wait();
    prefetch_table(p, tid);
#pragma unroll 1
    for (int b = tid; b < p.B; b += kThreads) {
        const Sequence s(p, b);
        const int blocks = (s.done + p.tokens - 1) / p.tokens;
        sh.seqs[b] = make_int4(s.row, s.n, s.keys, blocks);
        first[b + 1] = Units(p, s).count * blocks * p.kv_heads;
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    // What comes next may read what was there before this kernel. (And not before the block has
    // its tensor memory: a block of the next kernel that took it would wait for this one.)
    grid_launch_dependents();
    if (warp == 0) sum_firsts(first, p.B, p.items, lane);
    __syncthreads();
    const uint32_t tm = sh.tmem, S = tm, O = tm + 2 * kScores;
    const Sequences all{first, sh.seqs};
    const int items = first[p.B];
    const Waits wait{&sh.abort, p.err};

    if (warp >= kProducer && warp < kTensor) {
        // ------------------------------------------------------------ producers
        // One brings keys (and queries), one values: neither ring waits for the other.
        const bool values = warp > kProducer;
        const CUtensorMap *map = values ? maps.v : maps.k;
        Place at(values ? p.key_slots : 0, values ? p.slots : p.key_slots);
        int n = 0, brought = 0;  // items' queries, leaves
        bool ok = true;
#pragma unroll 1
        for (int index = blockIdx.x; index < items && ok; index += gridDim.x) {
            const Item it = item_at(p, all, index);
            if (it.leaves == 0) continue;  // (no queries are brought for an item without keys)
            const Seen seen(p, it.pos, it.pos + it.tokens - 1);
            const int32_t *table = p.table + int64_t(it.b) * p.max_pages;
            const int leaves = it.leaf + it.leaves, g = it.g;
            for (int leaf = it.leaf; leaf < leaves && ok; ++leaf) {
                Boxes boxes;
                boxes.find(p, seen, table, leaf * kLeaf, lane, 32);
                if (!values && lane == 0) sh.there[brought & 7] = boxes.there;
                ++brought;
#pragma unroll 1
                for (int i = 0; i < kChunks; ++i, ++at.issued, at.step()) {
                    if (ok && at.full()) ok = wait(empty0 + 8 * at.slot, at.lap ^ 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const uint32_t full = full0 + 8 * at.slot, dst = base + at.slot * kChunk;
                    if (lane == 0) mbar_arrive_expect_tx(full, kChunk);
                    __syncwarp();
                    // keys: 128, 64 elements; values: 64, twice 64 elements (128, 64 elements of head_dim 64)
                    if (D > 64 && values)
                        boxes.bring<2>(map, dst, lane, i / HALVES * 8, 8, i % HALVES * 128, 8192, g, full);
                    else
                        boxes.bring<1>(map, dst, lane, i / DB * 16, 16, i % DB * 64, 0, g, full);
                    // (an item's queries behind its first keys, which have further to come)
                    if (!values && leaf == it.leaf && i == 0) {
                        const int set = n % p.q_sets;
                        ok = __all_sync(0xffffffffu, n < p.q_sets || wait(q_empty + 8 * set, (n / p.q_sets - 1) & 1));
                        if (ok && lane == 0) {
                            mbar_arrive_expect_tx(q_full + 8 * set, uint32_t(p.rows) * D * 2);
                            for (int c = 0; c < DB; ++c)
                                tile::tma_load_3d(Q + (set * DB + c) * NC * 128, &qmap, 64 * c, g * p.group, it.row, q_full + 8 * set);
                        }
                        n += ok;
                    }
                }
            }
        }
        if (!ok) {
            // copies in flight have to land before the block ends
            const int slots = at.end - at.first;
#pragma unroll 1
            for (int i = max(at.issued - slots, 0); i < at.issued; ++i) mbar_wait_bounded(full0 + 8 * (at.first + i % slots), (i / slots) & 1);
#pragma unroll 1
            for (int i = max(n - p.q_sets, 0); i < n; ++i) mbar_wait_bounded(q_full + 8 * (i % p.q_sets), (i / p.q_sets) & 1);
        }
    } else if (warp >= kTensor) {
        // --------------------------------------------------------- tensor warps
        // One for the scores, which run a leaf ahead, one for the sums: a wait for a
        // barrier takes some 300 cycles while products keep shared memory busy, and the tensor
        // cores' queue is short, so that one warp's waits leave them idle.
        const bool first_warp = warp == kTensor;
        constexpr uint32_t kScoreKind = mma_kind(NC, false, false), kValueKind = mma_kind(2 * NC, true, true);
        // (head_dim 64: the tile's second 64 rows repeat the first, and are not read)
        const uint64_t keys0 = descriptor(base, 16, 1024, 2), queries = descriptor(Q, 16, 1024, 2);
        const uint64_t values0 = descriptor(base, D == 64 ? 0 : 8192, 1024, 2);
        const uint64_t weights = NC == 16 ? descriptor(P, 16, 512, 4) : descriptor(P, kLeaf * 128, 1024, 2);
        Place at(first_warp ? 0 : p.key_slots, first_warp ? p.key_slots : p.slots);
        int n = 0, leaf = 0;
        const auto sums = [&](int leaf, bool fresh) {
#pragma unroll 1
            for (int i = 0; i < kChunks; ++i, at.step()) {
                if (i % DB == 0) {
                    // (a tile's values first: they come before its weights)
                    Place next = at;
#pragma unroll 1
                    for (int c = 0; c < DB; ++c, next.step()) wait(full0 + 8 * next.slot, next.lap);
                    wait(p_ready + 16 * (leaf & 1) + 8 * (i / DB), (leaf / 2) & 1);
                    tmem_fence_after();
                }
                constexpr int kKeys = D == 64 ? 128 : 64;
                const int c = i % HALVES, key = i / HALVES * kKeys;
                if (one_lane()) {
                    const uint64_t a = values0 + uint32_t(at.slot * (kChunk >> 4)), b = weights + uint32_t(key * (kKeyBytes >> 4));
#pragma unroll
                    for (int k = 0; k < kKeys / 16; ++k)
                        mma_ss(kValueKind, O + c * 2 * NC, a + k * (2048 >> 4), b + k * (16 * kKeyBytes >> 4), !fresh || key + k > 0);
                    tmem_commit(empty0 + 8 * at.slot);
                    if (i == kChunks - 1) tmem_commit(o_done);
                }
                __syncwarp();
            }
        };
#pragma unroll 1
        for (int index = blockIdx.x; index < items; index += gridDim.x) {
            const Item it = item_at(p, all, index);
            if (it.leaves == 0) continue;
            const int set = n % p.q_sets, leaves = it.leaves;
            if (first_warp) wait(q_full + 8 * set, (n / p.q_sets) & 1);
#pragma unroll 1
            for (int l = 0; l < leaves; ++l, ++leaf) {
                if (first_warp) {
                    if (leaf >= 2) {
                        wait(p_ready + 16 * (leaf & 1) + 8, (leaf / 2 - 1) & 1);  // (its scores of before have been read)
                        tmem_fence_after();
                    }
#pragma unroll 1
                    for (int i = 0; i < kChunks; ++i, at.step()) {
                        wait(full0 + 8 * at.slot, at.lap);
                        const int c = i % DB;
                        if (one_lane()) {
                            const uint32_t d = S + (leaf & 1) * kScores + i / DB * NC;
                            const uint64_t a = keys0 + uint32_t(at.slot * (kChunk >> 4)), b = queries + uint32_t((set * DB + c) * NC * (128 >> 4));
#pragma unroll
                            for (int k = 0; k < 4; ++k) mma_ss(kScoreKind, d, a + 2 * k, b + 2 * k, c + k > 0);
                            tmem_commit(empty0 + 8 * at.slot);
                            if (i == kChunks - 1) {
                                tmem_commit(s_ready + 8 * (leaf & 1));
                                mbar_arrive(s_ready + 8 * (leaf & 1));
                                if (l == leaves - 1) tmem_commit(q_empty + 8 * set);
                            }
                        }
                        __syncwarp();
                    }
                } else {
                    sums(leaf, l == 0);
                }
            }
            ++n;
        }
        if (one_lane()) tmem_commit(finished);
        __syncwarp();
        mbar_wait_bounded(finished, 0);
    } else {
        // ---------------------------------------------------------------- weights
        // Four warps have 16 columns. A thread has the key `mine` of each of the leaf's
        // two tiles, then the element `mine` of the sums (and mine + 128 of head_dim
        // 256). Its lanes of tensor memory are its warp's. (One body of code for 16 columns, and
        // masks as bits that a short loop makes: with all columns in a thread the code did
        // not stay in the instruction cache, and a leaf of 64 columns took 20 us.)
        const int group = warp / 4, c0 = 16 * group, quarter = warp & 3, mine = tid & 127, meet = 1 + group;
        const uint32_t lanes = uint32_t(quarter * 32) << 16;
        const float c2 = __fmul_rn(p.scale, 1.4426950408889634f);
        const int column = c0 + (mine & 15), token = column / p.group, head = column - token * p.group;  // of the first 16 threads
        int leaf = 0;
#pragma unroll 1
        for (int index = blockIdx.x; index < items; index += gridDim.x) {
            const Item it = item_at(p, all, index);
            const Seen seen(p, it.pos, it.pos + it.tokens - 1);
            if (mine < 16) {
                const int r = column;
                sh.out[r] = (it.row + token) * p.ld_out + (it.g * p.group + head) * D;
            }
            float sum[16], ref = -INFINITY;  // ref: of column c0 + lane % 16, in each warp
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[i] = 0.0f;
            named_sync(meet, 128);
            bool scored = false;  // are the next leaf's scores there already?
#pragma unroll 1
            for (int l = 0; l < it.leaves; ++l, ++leaf) {
                const int key0 = (it.leaf + l) * kLeaf + mine;
                const uint32_t scores = S + (leaf & 1) * kScores + lanes + c0;
                if (!scored) wait(s_ready + 8 * (leaf & 1), (leaf / 2) & 1);
                tmem_fence_after();
                uint32_t see[2] = {0xffffu, 0xffffu};  // which columns see the key
                // (keys whose page is there, as the producer found it)
                const uint32_t there = sh.there[leaf & 7];
                const bool there0 = seen(key0) && (there >> (mine / 8) & 1), there1 = seen(key0 + 128) && (there >> (16 + mine / 8) & 1);
                if (!(there0 && there1 && key0 + 128 <= it.pos && (!p.window || key0 >= it.pos + it.tokens - p.window))) {
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        // of tokens from `from` to below `to`, whose columns lie side by side
                        const int key = key0 + 128 * h, from = min(max(key - it.pos, 0), it.tokens);
                        const int to = p.window && key >= p.sinks ? max(min(key - it.pos + p.window, it.tokens), 0) : it.tokens;
                        (h ? see[1] : see[0]) = (h ? there1 : there0) ? below(to * p.group - c0) & ~below(from * p.group - c0) : 0u;
                    }
                }
                float s0[16], s1[16], top[16];
                tmem_ld<16>(scores, s0);
                tmem_ld<16>(scores + NC, s1);
                tmem_wait_ld();
                settle(s0);
                settle(s1);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    s0[i] = see[0] >> i & 1 ? __fmul_rn(s0[i], c2) : -INFINITY;
                    s1[i] = see[1] >> i & 1 ? __fmul_rn(s1[i], c2) : -INFINITY;
                    top[i] = fmaxf(s0[i], s1[i]);
                }
                // (lanes 2 i and 2 i + 1 have the largest of column i)
                const float most = max_scatter(top, lane);
                if (!(lane & 1)) (&sh.top[leaf & 1][c0 + lane / 2].x)[quarter] = most;
                const bool summed = leaf == 0 || mbar_test(o_done, (leaf - 1) & 1);
                named_sync(meet, 128);
                const float4 four = sh.top[leaf & 1][c0 + (lane & 15)];
                // (a column without a query has none)
                const float m = c0 + (lane & 15) < it.rows ? fmaxf(fmaxf(four.x, four.y), fmaxf(four.z, four.w)) : -INFINITY;
                // above the largest score, and kept while it is
                const float now = m > ref ? __fadd_rn(ceilf(m), 8.0f) : ref;
                const bool moved = now != ref && ref != -INFINITY;
                const float shift = moved ? power_of_two(__fsub_rn(ref, now)) : 1.0f;
                ref = now;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float use = __shfl_sync(0xffffffffu, now == -INFINITY ? 0.0f : now, i);
                    s0[i] = __fsub_rn(s0[i], use);
                    s1[i] = __fsub_rn(s1[i], use);
                }
                // the last leaf's products are done: P is free, O stands still
                if (!summed) wait(o_done, (leaf - 1) & 1);
                if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) sum[i] = __fmul_rn(sum[i], __shfl_sync(0xffffffffu, shift, i));
                    tmem_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 2 * HALVES; ++c) {
                        float o[16];
                        tmem_ld<16>(O + lanes + c * NC + c0, o);
                        tmem_wait_ld();
                        settle(o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __fmul_rn(o[i], __shfl_sync(0xffffffffu, shift, i));
                        tmem_st<16>(O + lanes + c * NC + c0, o);
                    }
                    tmem_wait_st();
                }
                scored = l + 1 < it.leaves && mbar_test(s_ready + 8 * ((leaf + 1) & 1), ((leaf + 1) / 2) & 1);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float(&w)[16] = h ? s1 : s0;
                    const int k = h * 128 + mine;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        w[i] = exp2_fast(w[i]);
                        sum[i] = __fadd_rn(sum[i], w[i]);
                    }
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        hi[i] = pack_bf16(w[2 * i], w[2 * i + 1]);
                        lo[i] = pack_bf16(__fsub_rn(w[2 * i], __uint_as_float(hi[i] << 16)),
                                          __fsub_rn(w[2 * i + 1], __uint_as_float(hi[i] & 0xffff0000u)));
                    }
                    const uint32_t row = P + k * kKeyBytes, swizzle = NC == 16 ? (k >> 1) & 3 : k & 7;
                    const int low_at = NC == 16 ? 2 : NC == 32 ? 4 : 0;  // of 64 columns the second terms are a block of their own
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t piece = 2 * group + i;
                        sts_v4_u32(row + ((piece ^ swizzle) << 4), make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]));
                        sts_v4_u32(row + (NC == 64 ? kLeaf * 128 : 0) + (((piece + low_at) ^ swizzle) << 4),
                                   make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]));
                    }
                    // Values of keys that no column sees may be anything, and 0 x NaN is NaN: zeros
                    // in their place, once the tile's values have landed. (A wait for a slot's lap is
                    // right only when the lap before has landed and while the lap itself is not
                    // consumed: the leaf before's values have been used, the second tile's
                    // come after the first's. A tile's values fit in the ring at once.)
                    const uint32_t unseen = __ballot_sync(0xffffffffu, !(h ? there1 : there0));  // of the warp's keys
                    if (group == 0 && !__all_sync(0xffffffffu, there0 && there1)) {
                        const int from = leaf * kChunks + h * DB, slots = p.slots - p.key_slots;
#pragma unroll 1
                        for (int c = 0; c < DB; ++c) {
                            const int slot = p.key_slots + (from + c) % slots;
                            wait(full0 + 8 * slot, ((from + c) / slots) & 1);
                            // does the chunk hold 64 elements (of head_dim 64) or 128 of the warp's keys?
                            if (unseen == 0 || (D > 64 && c / HALVES != mine / 64)) continue;
                            // (the warp's 32 rows, four at a time: a row by each lane has bank conflicts, and a
                            // window's first leaf took 5500 cycles)
                            const uint32_t at = base + slot * kChunk + (quarter & (D == 64 ? 3 : 1)) * 4096 + lane * 16;
#pragma unroll 1
                            for (int i = 0; i < 8; ++i)
                                if (unseen >> (4 * i + lane / 8) & 1)
                                    for (int d = 0; d < (D == 64 ? 1 : 2); ++d) sts_v4_u32(at + i * 512 + d * 8192, make_uint4(0, 0, 0, 0));
                        }
                    }
                    tmem_fence_before();
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_ready + 16 * (leaf & 1) + 8 * h);
                }
            }
            // ------------------------------------------------ what the item gives
            const float part = tree_reduce_scatter<16>(sum, lane);
            if (!(lane & 1)) sh.sum[quarter][c0 + lane / 2] = part;
            named_sync(meet, 128);
            if (mine < 16 && c0 + mine < it.rows) {
                const int r = c0 + mine;
                const float t = __fadd_rn(__fadd_rn(sh.sum[0][r], sh.sum[1][r]), __fadd_rn(sh.sum[2][r], sh.sum[3][r]));
                if (it.whole) {
                    const bool none = t == 0.0f;  // (not one whose scores are NaN, which stay it)
                    sh.total[r] = none ? 0.0f : __fdiv_rn(1.0f, t);
                    if (p.lse)
                        p.lse[int64_t(it.row + token) * p.heads + it.g * p.group + head] = none ? -INFINITY : __fmul_rn(0.6931471805599453f, __fadd_rn(ref, log2f(t)));
                } else {
                    p.meta[int64_t(it.part) * p.group + r] = make_float2(ref, t);
                }
            }
            if (it.leaves > 0) wait(o_done, (leaf - 1) & 1);
            named_sync(meet, 128);
            tmem_fence_after();
#pragma unroll 1
            for (int half = 0; half < HALVES; ++half) {
                const int d = half * 128 + mine;
                float a[16], b[16];
                tmem_ld<16>(O + lanes + half * 2 * NC + c0, a);
                tmem_ld<16>(O + lanes + half * 2 * NC + NC + c0, b);
                tmem_wait_ld();
                settle(a);
                settle(b);
                if (d >= D) continue;
                if (it.leaves == 0) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) a[i] = b[i] = 0.0f;
                }
                const int left = it.rows - c0;
                if (!it.whole) {
                    float *to = p.parts + (int64_t(it.part) * p.group + c0) * D + d;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (i < left) to[i * D] = __fadd_rn(a[i], b[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (i < left) {
                            const float f = sh.total[c0 + i];
                            reinterpret_cast<__nv_bfloat16 *>(p.out)[sh.out[c0 + i] + d] = __float2bfloat16_rn(f == 0.0f ? 0.0f : __fmul_rn(__fadd_rn(a[i], b[i]), f));
                        }
                }
            }
            tmem_fence_before();
            named_sync(meet, 128);  // (the columns' lists are for the next item now)
        }
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == kTensor) tile::tmem_free(tm, kAlloc);
}

// Joins a row's units: their sums times powers of two that bring them to one reference,
// those of places u = w, w + 8, .. by warp w in order, then the warps' in order. A block
// has a row. (It starts under attend_few, and reads what that left in L2.)
constexpr int kJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) attend_join(const AttendParams p)
{
    constexpr int E = D / 32;
    __shared__ float s_sum[kJoinWarps][D], s_total[kJoinWarps], s_top[kJoinWarps];
    grid_launch_dependents();  // (what comes next waits for this kernel's end, and so for attend_few's)
    // (what is read here was there before attend_few began)
    const int few = min(p.max_new, kFew), b = int(blockIdx.x) / few, i = int(blockIdx.x) - b * few, h = blockIdx.y;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const Sequence s(p, b);
    const Units units(p, s);
    const int g = h / p.group, head = h - g * p.group;
    grid_dependency_wait();
    if (i >= s.done || units.count <= 1) return;
    // units whose places are the warp's, of the first tokens and of the others
    float top = -INFINITY, total = 0.0f, sum[E];
#pragma unroll
    for (int e = 0; e < E; ++e) sum[e] = 0.0f;
#pragma unroll 1
    for (int from = 0; from < units.count; from = from < units.sinks ? units.sinks : units.count) {
        const int to = from < units.sinks ? units.sinks : units.count;
        int u = from + ((warp - units.place(from)) & (kJoinWarps - 1));
#pragma unroll 4
        for (; u < to; u += kJoinWarps) {
            const int64_t at = int64_t(part_of(p, b, s.row + i, i, u, g)) * p.group + head;
            const float2 m = __ldcg(p.meta + at);
            float v[E];
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = __ldcg(p.parts + at * D + lane + 32 * e);
            // (powers of two: a reference that moves rounds nothing)
            const float now = fmaxf(top, m.x), keep = top == -INFINITY ? 0.0f : power_of_two(__fsub_rn(top, now));
            const float w = m.x == -INFINITY ? 0.0f : power_of_two(__fsub_rn(m.x, now));
            top = now;
            total = __fmaf_rn(m.y, w, __fmul_rn(total, keep));
#pragma unroll
            for (int e = 0; e < E; ++e) sum[e] = __fmaf_rn(v[e], w, __fmul_rn(sum[e], keep));
        }
    }
    if (lane == 0) s_top[warp] = top;
#pragma unroll
    for (int e = 0; e < E; ++e) s_sum[warp][lane + 32 * e] = sum[e];
    if (lane == 0) s_total[warp] = total;
    __syncthreads();
    float all = -INFINITY, o = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) all = fmaxf(all, s_top[w]);
    total = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        const float f = s_top[w] == -INFINITY ? 0.0f : power_of_two(__fsub_rn(s_top[w], all));
        total = __fmaf_rn(s_total[w], f, total);
        if (threadIdx.x < D) o = __fmaf_rn(s_sum[w][threadIdx.x], f, o);
    }
    const bool none = total == 0.0f;
    const int64_t row = s.row + i;
    // (times the reciprocal, as attend_few does where a row has one unit: a token that has one alone
    // has two with drafts behind it, and its bits are to be the same)
    if (threadIdx.x < D)
        reinterpret_cast<__nv_bfloat16 *>(p.out)[row * p.ld_out + h * D + threadIdx.x] = __float2bfloat16_rn(none ? 0.0f : __fmul_rn(o, __fdiv_rn(1.0f, total)));
    if (p.lse && threadIdx.x == 0)
        p.lse[row * p.heads + h] = none ? -INFINITY : __fmul_rn(0.6931471805599453f, __fadd_rn(all, log2f(total)));
}

// ----------------------------------------------------------------- prompts --
//
// Sequences of more new tokens than that. Query rows (tokens x heads of one kv head) are rows,
// 128 to a tile, two threads each:
//
//   S (rows x keys)      = Q K^T      from shared memory
//   P = exp2(S |scale| log2(e) - m)   in registers, then bf16 in tensor memory in S's place
//   O (rows x head_dim) += P V        V from shared memory as it lies in the cache
//
// Two tiles of rows take turns (of head_dim 256, whose sums fill half of tensor
// memory, two tiles of keys): the tensor cores work on one while the weights of the
// other are formed. What bounds it is the products, 4 x head_dim operations for each pair of
// row and key, and the loads of scores from tensor memory, which wait for them (64 columns: 650
// to 880 cycles while products run). Six prompts of up to 8192 tokens, 40 heads of 128: 1883 us, 65 % of
// the measured rate of bf16 products, counting the pairs that are seen alone; 8000 tokens of 16
// heads of 256 with a window of 1024: 159 us; six prompts of 32 heads of 64: 1362 us, 36 %, as a
// pair of row and key has as many exponentials and half the products. (One thread for a row took 2 to 7 % longer. Some
// of the exponentials by polynomials: slower, the exponentials' unit is busy for 28 %.)
//
// m is 8 above the largest score when it is set and moves when one passes it, so that sums are
// rarely scaled. The weights are rounded to bf16 (2^-8 of each, as an operand next to bf16 values
// has to be); their total is not. So m is not a whole number as above: the largest weight
// of the tile that sets it is 2^-8, which bf16 has, and a key that a row sees nearly alone (a first
// token that all look at, a row's only key) has no rounding: the error against 64 bits is then
// that of the result's rounding, as in fp32 (0.0016 to 0.0017 of the norm; 0.0023 with a whole number).
//
// Items go from a sequence's last rows, which see the most keys, to its first. Where there are
// too few of them the keys are divided into pieces, which attend_join_pieces joins in
// order; the pieces depend on the call's sizes, and a row's last bits with them.

struct PromptItem {
    int b, g, index;
    int row, tok, tokens;  // first row of q, first token of the sequence, tokens
    int pos;               // of the first token
    int end;               // behind the last key that the sequence's computed queries see
    int sinks, low;        // tiles of the first tokens; first tile of the others
    int low_all;           // the first key that the sequence's queries see behind the first tokens
    int from, to;          // of the list of tiles
    int pieces;
    __device__ __forceinline__ int tile(int i) const { return i < sinks ? i : low + i - sinks; }
};

// Tiles of keys that the rows of tokens [tok, tok + tokens) see.
struct Tiles {
    int sinks, low, count;
    __device__ __forceinline__ Tiles(const AttendParams &p, int first, int last)
    {
        const Seen seen(p, first, last);
        low = seen.low / 128;
        sinks = min((seen.sinks + 127) / 128, low);
        count = seen.end > 0 ? sinks + (seen.end - 1) / 128 - low + 1 : 0;
    }
};

// Parts of a sequence's items: of eight tiles at least, by its last rows.
__device__ __forceinline__ int pieces_of(const AttendParams &p, const Sequence &s, int each)
{
    const int last = (s.done - 1) / each * each;
    return max(1, min(p.pieces, Tiles(p, s.pos + last, s.pos + s.done - 1).count / 8));
}

template <int STREAMS>
__device__ __forceinline__ PromptItem prompt_at(const AttendParams &p, const Sequences &all, int index)
{
    int lo = 0, hi = p.B;
#pragma unroll 1
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        (all.first[mid] <= index ? lo : hi) = mid;
    }
    const Sequence s(p, all.kept[lo]);
    const int each = STREAMS * p.tokens;
    PromptItem it;
    it.b = lo;
    it.index = index;
    it.pieces = pieces_of(p, s, each);
    index -= all.first[lo];
    const int piece = index % it.pieces;
    index /= it.pieces;
    it.g = index % p.kv_heads;
    it.tok = ((s.done - 1) / each - index / p.kv_heads) * each;
    it.tokens = min(each, s.done - it.tok);
    it.row = s.row + it.tok;
    it.pos = s.pos + it.tok;
    it.end = s.pos + s.done;
    const Tiles tiles(p, it.pos, it.pos + it.tokens - 1);
    it.sinks = tiles.sinks;
    it.low = tiles.low;
    it.low_all = Seen(p, s.pos, s.pos).low;
    it.from = int(int64_t(tiles.count) * piece / it.pieces);
    it.to = int(int64_t(tiles.count) * (piece + 1) / it.pieces);
    return it;
}

// The keys that a stream's rows see.
template <int STREAMS>
__device__ __forceinline__ Seen stream_sees(const AttendParams &p, const PromptItem &it, int x, int &tokens)
{
    tokens = STREAMS == 1 ? it.tokens : max(min(it.tokens - x * p.tokens, p.tokens), 0);
    const int first = it.pos + x * p.tokens;
    Seen seen(p, first, first + tokens - 1);
    if (tokens == 0) seen.end = 0;
    return seen;
}

__device__ __forceinline__ void hide(float (&s)[32], uint32_t see)
{
#pragma unroll
    for (int k = 0; k < 32; ++k)
        if (!(see >> k & 1)) s[k] = -INFINITY;
}

__device__ __forceinline__ void tmem_ld32(uint32_t a, float (&v)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]),
          "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]),
          "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(a));
}

// Columns of 16 keys' weights in a tile's scores: 32 for its first 64 keys, where theirs
// were, and 32 for the others.
__device__ __forceinline__ int weights_at(int k) { return 8 * k + (k >= 4 ? 32 : 0); }

__device__ __forceinline__ float tmem_ld1(uint32_t a)
{
    float v[1] = {tile::tmem_ld1(a)};
    tmem_wait_ld();
    settle(v);
    return v[0];
}

struct PromptShared {
    uint64_t full[12], empty[12], q_full, q_empty, edge, s_ready[2], o_done[2], finished;
    int abort;
    uint32_t tmem, there[8];  // (of the last tiles: which eights of keys have a page)
    int4 seqs[1];             // [B], then the sequences' first items [B + 1]
};
static_assert(offsetof(PromptShared, seqs) <= kPromptMisc, "the plan's room for it");

// Hardware barriers: at 1 and 2 the 256 threads of a stream (of one stream: of the even and of
// the odd tiles) arrive, whose weights are there, and the tensor warp that issues waits for them;
// at 3 that warp and the one that watches the ring meet; at 4 and 5 the two threads of a row
// exchange its maximum. (Each barrier has one number of threads for good: one whose number
// changed from tile to tile would take a warp that is a tile ahead for one of the tile before.)
constexpr int kMeetWeights = 288, kMeetRing = 64, kMeetRows = 256;
__device__ __forceinline__ void named_arrive(int id, int threads) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

__host__ __device__ constexpr int prompt_threads(int D) { return (D == 256 ? 256 : 512) + 128; }

// D (128 x N fp32) (+)= A (128 x 16, tensor memory) B^T (N x 16, shared memory).
template <uint32_t KIND>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(KIND), "r"(uint32_t(add))
        : "memory");
}

template <int D>
__global__ void __launch_bounds__(prompt_threads(D), 1)
    attend_prompt(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CacheMaps maps, const AttendParams p)
{
    // A chunk of keys is 128 of them, KW elements; one of values VK keys, all elements. (Of
    // 32 KB each where they can be: with 16 KB of head_dim 256 the tensor warps wait twice as
    // often, and a prompt with a window took 199 us instead of 163.)
    constexpr int STREAMS = D == 256 ? 1 : 2, KW = D == 64 ? 64 : 128, VK = D == 256 ? 64 : 128;
    constexpr int DB = D / 64, kBytes = 128 * KW * 2, KC = D / KW, VC = 128 / VK;  // chunks of a tile
    static_assert(kBytes == VK * D * 2, "a ring slot holds either");
    constexpr int kThreads = prompt_threads(D), kProducer = kThreads / 32 - 4, kTensor = kProducer + 2;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    PromptShared &sh = *reinterpret_cast<PromptShared *>(smem + p.misc_off);
    int32_t *first = reinterpret_cast<int32_t *>(sh.seqs + p.B);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
    const uint32_t base = smem_u32(smem), full0 = smem_u32(sh.full), empty0 = smem_u32(sh.empty), Q = base + p.q_off;
    const uint32_t q_full = smem_u32(&sh.q_full), q_empty = smem_u32(&sh.q_empty), edge = smem_u32(&sh.edge), finished = smem_u32(&sh.finished);
    const uint32_t s_ready = smem_u32(sh.s_ready), o_done = smem_u32(sh.o_done);
    if (tid == 0) {
#pragma unroll 1
        for (int i = 0; i < p.slots; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(edge, 1);
        mbar_init(finished, 2);
        for (int x = 0; x < 2; ++x) {
            mbar_init(s_ready + 8 * x, 2);  // the scores, and the warp that has seen the keys land
            mbar_init(o_done + 8 * x, 1);
        }
        fence_mbar_init();
        sh.abort = 0;
    }
    if (warp == kTensor) tile::tmem_alloc(smem_u32(&sh.tmem), 512);
    if (tid == 0) prefetch_maps(qmap, maps, p);
    grid_dependency_wait();
    prefetch_table(p, tid);
#pragma unroll 1
    for (int b = tid; b < p.B; b += kThreads) {
        const Sequence s(p, b);
        sh.seqs[b] = make_int4(s.row, s.n, s.keys, 0);
        const int each = STREAMS * p.tokens;
        const int64_t count = s.done > kFew ? int64_t((s.done + each - 1) / each) * p.kv_heads * pieces_of(p, s, each) : 0;
        first[b + 1] = int32_t(count < p.items ? count : p.items);
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    grid_launch_dependents();  // (behind the allocation, as in attend_few)
    if (warp == 0) sum_firsts(first, p.B, p.items, lane);
    __syncthreads();
    if (blockIdx.x == 0 && p.pieces > 1)
#pragma unroll 1
        for (int b = tid; b <= p.B; b += kThreads) p.prefix[b] = first[b];
    const uint32_t tm = sh.tmem, S = tm, O = tm + 256;
    const Sequences all{first, sh.seqs};
    const int items = first[p.B];
    const Waits wait{&sh.abort, p.err};
    // Items get smaller, so that every other round goes the other way (six prompts: the
    // longest block has 2 % more than the mean, instead of 6).
    const auto item_of = [](int round) { return round * int(gridDim.x) + int(round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x); };

    if (warp >= kProducer && warp < kTensor) {
        // ------------------------------------------------------------ producers
        // One brings keys (and queries), one values.
        const bool values = warp > kProducer;
        const CUtensorMap *map = values ? maps.v : maps.k;
        Place at(values ? p.key_slots : 0, values ? p.slots : p.key_slots);
        int n = 0, edges = 0, brought = 0;
        bool ok = true;
#pragma unroll 1
        for (int round = 0, index; ok && (index = item_of(round)) < items; ++round) {
            const PromptItem it = prompt_at<STREAMS>(p, all, index);
            const int from = it.from, to = it.to, g = it.g;
            if (from == to) continue;
            const Seen seen(p, it.pos, it.pos + it.tokens - 1);
            const int32_t *table = p.table + int64_t(it.b) * p.max_pages;
#pragma unroll 1
            for (int i = from; i < to && ok; ++i, ++brought) {
                Boxes boxes;
                boxes.find(p, seen, table, it.tile(i) * 128, lane, 16);
                if (!values && lane == 0) sh.there[brought & 7] = boxes.there;
                // Values that no query of the sequence sees may be anything, and 0 x NaN is NaN:
                // zeros in their place, behind the last one seen, before its window and behind its first tokens.
                const int chunks = values ? VC : KC;
#pragma unroll 1
                for (int c = 0; c < chunks; ++c, ++at.issued, at.step()) {
                    const int key0 = it.tile(i) * 128 + c * VK;
                    const bool zeros = values && (key0 + VK > it.end || (key0 < it.low_all && key0 + VK > min(p.sinks, it.low_all)));
                    if (ok && at.full()) ok = wait(empty0 + 8 * at.slot, at.lap ^ 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const uint32_t full = full0 + 8 * at.slot, bar = zeros ? edge : full, dst = base + at.slot * kBytes;
                    if (lane == 0) mbar_arrive_expect_tx(bar, kBytes);
                    __syncwarp();
                    if (values)
                        boxes.bring<DB>(map, dst, lane, c * (VK / 8), VK / 8, 0, VK * 128, g, bar);
                    else
                        boxes.bring<KW / 64>(map, dst, lane, 0, 16, c * KW, 16384, g, bar);
                    // (an item's queries behind its first keys, which have further to come)
                    if (!values && i == from && c == 0) {
                        ok = __all_sync(0xffffffffu, n == 0 || wait(q_empty, (n - 1) & 1));
                        if (ok && lane == 0) {
                            const int sets = STREAMS == 2 && it.tokens > p.tokens ? 2 : 1;
                            mbar_arrive_expect_tx(q_full, uint32_t(sets * p.tokens * p.group) * D * 2);
                            for (int q = 0; q < sets * DB; ++q)
                                tile::tma_load_3d(Q + q * 16384, &qmap, q % DB * 64, g * p.group, it.row + q / DB * p.tokens, q_full);
                        }
                        n += ok;
                    }
                    if (zeros) {
                        __syncwarp();
                        ok = __all_sync(0xffffffffu, wait(edge, edges & 1));
                        ++edges;
#pragma unroll 1
                        for (int e = lane; e < VK * 8; e += 32) {
                            const int key = key0 + e / 8;
                            if (key < it.end && (key >= it.low_all || key < p.sinks)) continue;
                            for (int d = 0; d < DB; ++d) sts_v4_u32(dst + d * VK * 128 + e * 16, make_uint4(0, 0, 0, 0));
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(full);
                    }
                }
            }
        }
        if (!ok) {
            // copies in flight have to land before the block ends (those of an edge have been waited for)
            const int slots = at.end - at.first;
#pragma unroll 1
            for (int i = max(at.issued - slots, 0); i < at.issued; ++i) mbar_wait_bounded(full0 + 8 * (at.first + i % slots), (i / slots) & 1);
            if (n > 0) mbar_wait_bounded(q_full, (n - 1) & 1);
        }
    } else if (warp >= kTensor) {
        // --------------------------------------------------------- tensor warps
        // A wait for a barrier in shared memory takes some 300 cycles while products read
        // their operands there, and the tensor cores' queue is short: a warp that waits leaves
        // them idle. So the first warp issues products and waits at hardware barriers alone,
        // where the second comes when what the rings bring is there. (With a warp for
        // each of two streams their products slow one another down: 2339 us instead of 2003 for six
        // prompts; of one stream a warp for the scores and one for the sums took 163 us for one
        // with a window.)
        const int x = warp - kTensor;
        Place keys(0, p.key_slots), values(p.key_slots, p.slots);
        constexpr uint32_t kValueKind = mma_kind(D, false, true);
        const uint32_t score_kind = mma_kind(128, false, false) | (p.scale < 0.0f ? 1u << 13 : 0u);  // (of the scale's sign: - Q)
        const uint64_t keys0 = descriptor(base, 16, 1024, 2), queries = descriptor(Q, 16, 1024, 2);
        const uint64_t values0 = descriptor(base, VK * 128, 1024, 2);
        int n = 0, tiles = 0;
        const auto landed = [&](Place &at, int chunks) {
#pragma unroll 1
            for (int c = 0; c < chunks; ++c, at.step()) wait(full0 + 8 * at.slot, at.lap);
        };
#pragma unroll 1
        for (int round = 0, index; (index = item_of(round)) < items; ++round) {
            const PromptItem it = prompt_at<STREAMS>(p, all, index);
            const int from = it.from, to = it.to;
            if (from == to) continue;
            if (STREAMS == 1) {
                // S(0), then S(i + 1), O(i)
#pragma unroll 1
                for (int i = from; i <= to; ++i) {
                    if (x) {
                        if (i == from) wait(q_full, n & 1);
                        if (i < to) {
                            landed(keys, KC);
                            named_sync(3, kMeetRing);
                        }
                        if (i > from) {
                            landed(values, VC);
                            named_sync(3, kMeetRing);
                        }
                        continue;
                    }
                    if (i < to) {
                        const int buffer = tiles & 1;
                        named_sync(3, kMeetRing);
#pragma unroll 1
                        for (int c = 0; c < KC; ++c, keys.step()) {
                            if (one_lane()) {
                                const uint64_t k0 = keys0 + uint32_t(keys.slot * (kBytes >> 4)), q0 = queries + uint32_t(c * (KW / 64) * (16384 >> 4));
#pragma unroll
                                for (int k = 0; k < KW / 16; ++k)
                                    mma_ss(score_kind, S + buffer * 128, q0 + (k / 4) * (16384 >> 4) + 2 * (k & 3), k0 + (k / 4) * (16384 >> 4) + 2 * (k & 3), c + k > 0);
                                tmem_commit(empty0 + 8 * keys.slot);
                                if (c == KC - 1) {
                                    tmem_commit(s_ready + 8 * buffer);
                                    mbar_arrive(s_ready + 8 * buffer);
                                    if (i == to - 1) tmem_commit(q_empty);
                                }
                            }
                            __syncwarp();
                        }
                        ++tiles;
                    }
                    if (i > from) {
                        const int buffer = (tiles - (i < to ? 2 : 1)) & 1;
                        named_sync(1 + buffer, kMeetWeights);
                        named_sync(3, kMeetRing);
                        tmem_fence_after();
#pragma unroll 1
                        for (int c = 0; c < VC; ++c, values.step()) {
                            if (one_lane()) {
                                const uint64_t v0 = values0 + uint32_t(values.slot * (kBytes >> 4));
#pragma unroll
                                for (int k = 0; k < VK / 16; ++k)
                                    mma_ts<kValueKind>(O, S + buffer * 128 + weights_at(c * (VK / 16) + k), v0 + k * (2048 >> 4), i > from + 1 || c + k > 0);
                                tmem_commit(empty0 + 8 * values.slot);
                                if (c == VC - 1) tmem_commit(o_done + 8 * buffer);
                            }
                            __syncwarp();
                        }
                    }
                }
            } else {
                // S0(0), S1(0), then O0(i), S0(i + 1), O1(i), S1(i + 1); streams that see nothing
                // of a tile leave it out
                int tokens;
                const Seen see0 = stream_sees<STREAMS>(p, it, 0, tokens), see1 = stream_sees<STREAMS>(p, it, 1, tokens);
                uint32_t active = 0, started = 0;  // streams at work on tile i - 1; with sums of this item
#pragma unroll 1
                for (int i = from; i <= to; ++i) {
                    const int key = it.tile(i) * 128;
                    const uint32_t next = i < to ? uint32_t(see0.any(key, 128)) | uint32_t(see1.any(key, 128)) << 1 : 0u;
                    if (x) {
                        // the values of tile i - 1 and the keys of tile i (the queries)
                        if (i == from) {
                            wait(q_full, n & 1);
                        } else {
                            wait(full0 + 8 * values.slot, values.lap);
                            values.step();
                        }
                        if (i < to) {
                            wait(full0 + 8 * keys.slot, keys.lap);
                            keys.step();
                        }
                    }
                    named_sync(3, kMeetRing);
                    if (!x) {
                        const uint32_t vslot = values.slot, kslot = keys.slot;
                        if (i > from) values.step();
                        if (i < to) keys.step();
#pragma unroll 1
                        for (int s = 0; s < 2; ++s) {
                            const bool last = s == 1;
                            if (active >> s & 1) {
                                named_sync(1 + s, kMeetWeights);
                                tmem_fence_after();
                            }
                            if (one_lane()) {
                                if (active >> s & 1) {
                                    const uint64_t v0 = values0 + vslot * (kBytes >> 4);
#pragma unroll
                                    for (int k = 0; k < 8; ++k)
                                        mma_ts<kValueKind>(O + s * D, S + s * 128 + weights_at(k), v0 + k * (2048 >> 4), k > 0 || (started >> s & 1));
                                    tmem_commit(o_done + 8 * s);
                                }
                                if (last && i > from) tmem_commit(empty0 + 8 * vslot);
                                if (next >> s & 1) {
                                    const uint64_t k0 = keys0 + kslot * (kBytes >> 4), q0 = queries + uint32_t(s * DB * (16384 >> 4));
#pragma unroll
                                    for (int k = 0; k < KW / 16; ++k)
                                        mma_ss(score_kind, S + s * 128, q0 + (k / 4) * (16384 >> 4) + 2 * (k & 3), k0 + (k / 4) * (16384 >> 4) + 2 * (k & 3), k > 0);
                                    tmem_commit(s_ready + 8 * s);
                                    mbar_arrive(s_ready + 8 * s);
                                }
                                if (last && i < to) tmem_commit(empty0 + 8 * kslot);
                                if (last && i == to - 1) tmem_commit(q_empty);
                            }
                            __syncwarp();
                        }
                        started |= active;
                    }
                    active = next;
                }
            }
            ++n;
        }
        if (one_lane()) tmem_commit(finished);
        __syncwarp();
        mbar_wait_bounded(finished, 0);
    } else {
        // ---------------------------------------------------------------- weights
        // Two threads have a row, each 64 keys of a tile and then half of the sums.
        const int x = warp / 8, half = warp / 4 & 1, r = tid & 127, quarter = warp & 3;
        const uint32_t lanes = uint32_t(quarter * 32) << 16, mine = O + lanes + x * D + half * (D / 2);
        // (the products have the scale's sign already; above 0, so that a hidden score's weight is 0)
        const float c2 = fmaxf(__fmul_rn(fabsf(p.scale), 1.4426950408889634f), 1.2e-38f);
        const uint64_t scale2 = tile::pack2(c2, c2);
        int tiles = 0, ring_tiles = 0;  // of the stream so far, and of the block's items before this one
        // The last tile's sums are in. (One stream's scores run ahead of the sums of the tile
        // before, so that its tiles have a barrier each in turn: with one for all, the wait for
        // an item's last tile could see the parity of the tile before the one before it.)
        const auto sums_in = [&]() {
            if (STREAMS == 1)
                wait(o_done + 8 * ((tiles - 1) & 1), ((tiles - 1) / 2) & 1);
            else
                wait(o_done + 8 * x, (tiles - 1) & 1);
        };
#pragma unroll 1
        for (int round = 0, index; (index = item_of(round)) < items; ++round) {
            const PromptItem it = prompt_at<STREAMS>(p, all, index);
            int tokens;
            const Seen sees = stream_sees<STREAMS>(p, it, x, tokens);
            const int start = it.pos + x * p.tokens;  // position of the stream's first token
            const bool real = r < tokens * p.group;
            const int last = real ? start + r / p.group : -1, low = p.window ? last - p.window + 1 : 0;
            float ref = -INFINITY, use = 0.0f;
            uint64_t total[2] = {0ull, 0ull};
            int worked = 0;
#pragma unroll 1
            for (int i = it.from; i < it.to; ++i) {
                const int key0 = it.tile(i) * 128;
                if (!sees.any(key0, 128)) continue;
                const int buffer = STREAMS == 1 ? tiles & 1 : x;
                wait(s_ready + 8 * buffer, (STREAMS == 1 ? tiles / 2 : tiles) & 1);
                tmem_fence_after();
                const uint32_t at = S + buffer * 128 + half * 64 + lanes, other = S + buffer * 128 + (1 - half) * 64 + lanes;
                const uint32_t there = sh.there[(ring_tiles + i - it.from) & 7];  // eights of keys whose page is there, as the producer found them
                const bool plain = there == 0xffffu && key0 + 127 <= start && (!p.window || key0 >= start + tokens - p.window);
                float s[2][32];
#pragma unroll
                for (int h = 0; h < 2; ++h) tmem_ld32(at + 32 * h, s[h]);
                tmem_wait_ld();
#pragma unroll
                for (int h = 0; h < 2; ++h) settle(s[h]);
                if (!plain) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        // which of the 32 keys from `key` on the row sees
                        const int from = half * 64 + 32 * h, key = key0 + from;
                        uint32_t see = (below(p.sinks - key) | ~below(low - key)) & below(last + 1 - key), eights = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) eights |= (there >> (from / 8 + e) & 1u) * (0xffu << 8 * e);
                        hide(s[h], see & eights);
                    }
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < 64; k += 2) top[(k / 2) & 3] = fmaxf(top[(k / 2) & 3], fmaxf(s[k / 32][k & 31], s[k / 32][(k & 31) + 1]));
                float m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                // the row's other half, by the last column of either half's scores
                tile::tmem_st1(at + 63, m);
                tmem_wait_st();
                tmem_fence_before();
                named_sync(4 + x, kMeetRows);
                tmem_fence_after();
                m = fmaxf(m, tmem_ld1(other + 63));
                m = __fmul_rn(m, c2);
                // 8 above the largest score, and kept while it is above
                const bool moves = m > ref;
                const float now = moves ? __fadd_rn(m, 8.0f) : ref;
                use = now == -INFINITY ? 0.0f : now;
                // A row whose scores reach 2^29 rounds them as its maximum is rounded: the exact products may
                // lie further from it than an exponential can hold. (Each row by itself: what a row
                // without a query has here is left over from before.)
                const bool huge = real && fabsf(m) >= 0x1p29f && m != -INFINITY, rescale = moves && ref != -INFINITY;
                if (__any_sync(0xffffffffu, rescale || huge)) {
                    if (huge) {
#pragma unroll
                        for (int k = 0; k < 64; ++k) s[k / 32][k & 31] = __fmul_rn(__fsub_rn(__fmul_rn(s[k / 32][k & 31], c2), use), __frcp_rn(c2));
                        use = 0.0f;
                    }
                    __syncwarp();
                    if (__any_sync(0xffffffffu, rescale)) {
                        const float f = rescale ? exp2_fast(__fsub_rn(ref, now)) : 1.0f;
                        sums_in();
                        tmem_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 2; c += 16) {
                            float o[16];
                            tmem_ld<16>(mine + c, o);
                            tmem_wait_ld();
                            settle(o);
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = __fmul_rn(o[k], f);
                            tmem_st<16>(mine + c, o);
                        }
                        tmem_wait_st();
                        const uint64_t ff = tile::pack2(f, f);
                        total[0] = tile::mul2(total[0], ff);
                        total[1] = tile::mul2(total[1], ff);
                    }
                }
                ref = now;
                const uint64_t minus = tile::pack2(-use, -use);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        float a, b;
                        tile::unpack2(tile::fma2(tile::pack2(s[h][2 * k], s[h][2 * k + 1]), scale2, minus), a, b);
                        a = exp2_fast(a);
                        b = exp2_fast(b);
                        total[k & 1] = tile::add2(total[k & 1], tile::pack2(a, b));
                        w[k] = pack_bf16(a, b);
                    }
                    tile::tmem_st(at + 16 * h, w);  // (in the place of the half's own scores)
                }
                tmem_wait_st();
                tmem_fence_before();
                named_arrive(1 + buffer, kMeetWeights);
                ++tiles;
                ++worked;
            }
            ring_tiles += it.to - it.from;
            // ------------------------------------------------ what the item gives
            float t0, t1, t2, t3;
            tile::unpack2(total[0], t0, t1);
            tile::unpack2(total[1], t2, t3);
            float sum = __fadd_rn(__fadd_rn(t0, t1), __fadd_rn(t2, t3));
            if (worked) sums_in();
            tmem_fence_after();
            // The other half's total, by the first column of either half's sums, which is kept
            // meanwhile. (The scores' place may have the next item's already.) Both halves have one
            // only of an item with a tile for the stream, which all of its threads agree on. A half
            // may store the next item's total only when the other has loaded this one: between
            // the two lies a meeting at a tile's maxima, so an item without a tile must not store.
            float kept = 0.0f;
            if (worked) {
                kept = tmem_ld1(mine);
                tile::tmem_st1(mine, sum);
                tmem_wait_st();
                tmem_fence_before();
                named_sync(4 + x, kMeetRows);
                tmem_fence_after();
                const float theirs = tmem_ld1(O + lanes + x * D + (1 - half) * (D / 2));
                sum = half ? __fadd_rn(theirs, sum) : __fadd_rn(sum, theirs);
            }
            const bool none = sum == 0.0f;  // (not one whose scores are NaN, which stay it)
            const int64_t row = it.row + x * p.tokens + r / p.group;
            const int head = it.g * p.group + r % p.group;
            const int64_t part = (int64_t(it.index) * STREAMS + x) * 128 + r;
            const bool whole = it.pieces == 1;
            const float f = none ? 0.0f : whole ? __fdiv_rn(1.0f, sum) : 1.0f;
            if (real && half == 0) {
                if (!whole)
                    p.meta[part] = make_float2(ref, sum);
                else if (p.lse)
                    p.lse[row * p.heads + head] = none ? -INFINITY : __fmul_rn(0.6931471805599453f, __fadd_rn(ref, log2f(sum)));
            }
#pragma unroll 1
            for (int c = 0; c < D / 2; c += 16) {
                float o[16];
                tmem_ld<16>(mine + c, o);
                tmem_wait_ld();
                settle(o);
                if (c == 0) o[0] = kept;
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = none ? 0.0f : __fmul_rn(o[k], f);
                if (!real) continue;
                if (whole) {
                    uint4 *to = reinterpret_cast<uint4 *>(p.out + row * p.ld_out + head * D + half * (D / 2) + c);
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        to[k] = make_uint4(pack_bf16(o[8 * k], o[8 * k + 1]), pack_bf16(o[8 * k + 2], o[8 * k + 3]),
                                           pack_bf16(o[8 * k + 4], o[8 * k + 5]), pack_bf16(o[8 * k + 6], o[8 * k + 7]));
                } else {
                    float4 *to = reinterpret_cast<float4 *>(p.parts + part * D + half * (D / 2) + c);
#pragma unroll
                    for (int k = 0; k < 4; ++k) to[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                }
            }
            tmem_fence_before();
        }
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == kTensor) tile::tmem_free(tm, 512);
}

// Joins a row's pieces in order; a warp has a row. (Two chunks of 512 tokens over 16500 keys,
// 40 heads and 8 kv heads, are 176 items, too few for 152 SMs to share evenly; in four pieces
// each they are not.)
template <int D>
__global__ void __launch_bounds__(256) attend_join_pieces(const AttendParams p)
{
    constexpr int E = D / 32, STREAMS = D == 256 ? 1 : 2;
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t unit = int64_t(blockIdx.x) * 8 + threadIdx.x / 32;
    const int lane = threadIdx.x & 31, t = int(unit / p.heads), h = int(unit % p.heads), each = STREAMS * p.tokens;
    if (t >= p.T) return;
#pragma unroll 1
    for (int b = 0; b < p.B; ++b) {
        const Sequence s(p, b);
        const int i = t - s.row;
        if (i < 0 || i >= s.done || s.done <= kFew) continue;
        const int pieces = pieces_of(p, s, each);
        if (pieces == 1) continue;
        const int index = ((s.done - 1) / each - i / each) * p.kv_heads + h / p.group;
        if (int64_t(p.prefix[b]) + int64_t(index + 1) * pieces > p.items) continue;
        const int64_t first = (int64_t(p.prefix[b] + index * pieces) * STREAMS + i % each / p.tokens) * 128 + i % p.tokens * p.group + h % p.group;
        float top = -INFINITY, total = 0.0f, sum[E];
#pragma unroll 1
        for (int k = 0; k < pieces; ++k) top = fmaxf(top, p.meta[first + int64_t(k) * STREAMS * 128].x);
#pragma unroll
        for (int e = 0; e < E; ++e) sum[e] = 0.0f;
#pragma unroll 2
        for (int k = 0; k < pieces; ++k) {
            const int64_t at = first + int64_t(k) * STREAMS * 128;
            const float2 m = p.meta[at];
            const float w = m.x == -INFINITY ? 0.0f : exp2_fast(__fsub_rn(m.x, top));
            total = __fmaf_rn(m.y, w, total);
#pragma unroll
            for (int e = 0; e < E; ++e) sum[e] = __fmaf_rn(p.parts[at * D + lane + 32 * e], w, sum[e]);
        }
        const bool none = total == 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            reinterpret_cast<__nv_bfloat16 *>(p.out)[t * p.ld_out + h * D + lane + 32 * e] = __float2bfloat16_rn(none ? 0.0f : __fdiv_rn(sum[e], total));
        if (p.lse && lane == 0)
            p.lse[int64_t(t) * p.heads + h] = none ? -INFINITY : __fmul_rn(0.6931471805599453f, __fadd_rn(top, log2f(total)));
    }
}

struct Maps {
    CUtensorMap q;
    CacheMaps cache;
};

template <int D, int NC>
cudaError_t launch_few(const AttendParams &p, const Maps &m, const FewPlan &f, int sms, cudaStream_t stream)
{
    static std::atomic<int> configured[2][64] = {};
    Launch l;
    const int64_t most = int64_t(f.ctas) * sms;
    l.grid = dim3(unsigned(f.items < most ? f.items : most));
    l.threads = few_threads(NC);
    l.smem = size_t(f.smem);
    l.pdl = true;
    cudaError_t e = launch_one(attend_few<D, NC>, configured[0], l, stream, m.q, m.cache, p);
    if (e != cudaSuccess || f.units == 1) return e;
    l.grid = dim3(unsigned(p.B * (p.max_new < kFew ? p.max_new : kFew)), unsigned(p.heads));
    l.threads = kJoinWarps * 32;
    l.smem = 0;
    return launch_one(attend_join<D>, configured[1], l, stream, p);
}

template <int D>
cudaError_t launch_prompt(const AttendParams &p, const Maps &m, const PromptPlan &f, int sms, cudaStream_t stream)
{
    static std::atomic<int> configured[2][64] = {};
    Launch l;
    l.grid = dim3(unsigned(f.items < sms ? f.items : sms));
    l.threads = prompt_threads(D);
    l.smem = size_t(f.smem);
    l.pdl = true;
    cudaError_t e = launch_one(attend_prompt<D>, configured[0], l, stream, m.q, m.cache, p);
    if (e != cudaSuccess || f.pieces == 1) return e;
    l.grid = dim3(unsigned((int64_t(p.T) * p.heads + 7) / 8));
    l.threads = 256;
    l.smem = 0;
    return launch_one(attend_join_pieces<D>, configured[1], l, stream, p);
}

template <int D>
cudaError_t launch_attend(const AttendParams &p, const Maps &m, const FewPlan &f, int sms, cudaStream_t stream)
{
    return f.columns == 16   ? launch_few<D, 16>(p, m, f, sms, stream)
           : f.columns == 32 ? launch_few<D, 32>(p, m, f, sms, stream)
                             : launch_few<D, 64>(p, m, f, sms, stream);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

qmv_status check_attend(int B, int T, int max_new, int heads, int kv_heads, int head_dim, int page_size, int max_pages, int window, int sinks)
{
    const qmv_status st = check_heads(T, heads, kv_heads, head_dim);
    if (st != QMV_OK) return st;
    if (B < 1 || B > QMV_MAX_SEQUENCES || max_new < 1 || max_new > T) return QMV_ERR_COUNT;
    if (page_size < 8 || page_size % 8 != 0 || page_size > 65536 || max_pages < 1 || int64_t(max_pages) * page_size > (1 << 26) ||
        window < 0 || window > (1 << 30) || sinks < 0 || sinks > (1 << 30))
        return QMV_ERR_SHAPE;
    const int64_t capacity = int64_t(max_pages) * page_size;
    const FewPlan f = few_plan(B, T, max_new, heads, kv_heads, head_dim, capacity, window, sinks);
    const PromptPlan g = prompt_plan(B, T, max_new, heads, kv_heads, head_dim, capacity, window, sinks);
    return f.workspace + g.workspace > (size_t(1) << 40) || f.items >= (int64_t(1) << 31) || g.items >= (int64_t(1) << 31) ? QMV_ERR_SHAPE : QMV_OK;
}

}  // namespace
}  // namespace qmv

extern "C" size_t qmv_attend_workspace_size(int B, int T, int max_new, int heads, int kv_heads, int head_dim, int page_size,
                                            int max_pages, int window, int sinks)
{
    if (qmv::check_attend(B, T, max_new, heads, kv_heads, head_dim, page_size, max_pages, window, sinks) != QMV_OK) return 0;
    // (the two kinds of sequences run one after the other, each with the whole of it)
    const int64_t capacity = int64_t(max_pages) * page_size;
    const size_t few = qmv::attend::few_plan(B, T, max_new, heads, kv_heads, head_dim, capacity, window, sinks).workspace;
    const size_t prompt = qmv::attend::prompt_plan(B, T, max_new, heads, kv_heads, head_dim, capacity, window, sinks).workspace;
    return few > prompt ? few : prompt;
}

extern "C" qmv_status qmv_attend_run(const uint16_t *q, const uint16_t *k_cache, const uint16_t *v_cache,
                                     const int32_t *page_table, const int32_t *q_start, const int32_t *kv_len,
                                     uint16_t *out, float *lse, int B, int T, int max_new, int heads, int kv_heads,
                                     int head_dim, int page_size, int pages, int max_pages, float scale, int window,
                                     int sinks, int64_t ld_q, int64_t ld_out, int64_t page_stride, int64_t token_stride,
                                     int64_t head_stride, void *workspace, size_t workspace_bytes, unsigned flags,
                                     qmv_stream_t stream)
{
    using namespace qmv;
    if (!q || !k_cache || !v_cache || !page_table || !kv_len || !out) return QMV_ERR_NULL;
    qmv_status st = check_attend(B, T, max_new, heads, kv_heads, head_dim, page_size, max_pages, window, sinks);
    if (st != QMV_OK) return st;
    if (!q_start && int64_t(B) * max_new != T) return QMV_ERR_COUNT;
    st = check_cache({pages, page_size, kv_heads, head_dim, page_stride, token_stride, head_stride});
    if (st != QMV_OK) return st;
    const int64_t width = int64_t(heads) * head_dim, most = int64_t(1) << 38;
    if (!std::isfinite(scale) || ld_q < width || ld_q % 8 != 0 || ld_q > most || ld_out < width || ld_out % 8 != 0 || ld_out > most)
        return QMV_ERR_SHAPE;
    if (flags) return QMV_ERR_FLAGS;
    for (const void *ptr : {(const void *)q, (const void *)k_cache, (const void *)v_cache, (const void *)out, (const void *)workspace})
        if (!aligned(ptr, 16)) return QMV_ERR_ALIGN;
    for (const void *ptr : {(const void *)page_table, (const void *)q_start, (const void *)kv_len, (const void *)lse})
        if (!aligned(ptr, 4)) return QMV_ERR_ALIGN;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != QMV_OK) return st;
    void *ws = nullptr;
    st = scratch(dev, qmv_attend_workspace_size(B, T, max_new, heads, kv_heads, head_dim, page_size, max_pages, window, sinks),
                 workspace, workspace_bytes, &ws);
    if (st != QMV_OK) return st;

    AttendParams p{};
    p.table = page_table; p.q_start = q_start; p.kv_len = kv_len;
    p.out = out; p.lse = lse;
    p.B = B; p.T = T; p.max_new = max_new; p.heads = heads; p.group = heads / kv_heads;
    p.page_size = page_size; p.pages = pages; p.max_pages = max_pages;
    p.scale = scale; p.window = window; p.sinks = sinks;
    p.ld_out = ld_out;
    p.kv_heads = kv_heads;
    p.err = dev.err;
    const FewPlan f = few_plan(B, T, max_new, heads, kv_heads, head_dim, int64_t(max_pages) * page_size, window, sinks);
    p.items = int(f.items);
    p.by_row = f.by_row;
    p.kept = f.kept;
    p.tokens = f.tokens; p.rows = f.rows; p.units = f.units;
    p.unit_shift = f.unit == kLeaf ? 8 : f.unit == 2 * kLeaf ? 9 : 10;
    p.slots = f.slots; p.key_slots = f.key_slots; p.q_sets = f.q_sets;
    p.p_off = f.p_off; p.q_off = f.q_off; p.misc_off = f.misc_off;
    uint8_t *at = static_cast<uint8_t *>(ws);
    p.meta = reinterpret_cast<float2 *>(at + f.meta_off);
    p.parts = reinterpret_cast<float *>(at + f.parts_off);
    p.magic = page_magic(page_size);
    // Keys and values by boxes of 64 elements and 64 keys at most: one size where pages are
    // a power of two or multiples of 64, else all that fit a page.
    Maps m;
    const int64_t cache_dims[4] = {head_dim, page_size, kv_heads, pages}, cache_strides[3] = {token_stride, head_stride, page_stride};
    p.map_code = page_size >= 64 ? 3 : page_size >= 32 ? 2 : page_size >= 16 ? 1 : 0;
    const bool one_size = page_size % 64 == 0 || (page_size & (page_size - 1)) == 0;
    for (int c = one_size ? p.map_code : 0; c <= p.map_code && st == QMV_OK; ++c) {
        const int box[4] = {64, 8 << c, 1, 1};
        st = encode_bf16(&m.cache.k[c], k_cache, 4, cache_dims, cache_strides, box);
        if (st == QMV_OK) st = encode_bf16(&m.cache.v[c], v_cache, 4, cache_dims, cache_strides, box);
    }
    const int64_t q_dims[3] = {head_dim, heads, T}, q_strides[2] = {head_dim, ld_q};
    const int q_box[3] = {64, p.group, f.tokens};
    if (st == QMV_OK) st = encode_bf16(&m.q, q, 3, q_dims, q_strides, q_box);
    if (st != QMV_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = head_dim == 64    ? launch_attend<64>(p, m, f, dev.sms, s)
                    : head_dim == 128 ? launch_attend<128>(p, m, f, dev.sms, s)
                                      : launch_attend<256>(p, m, f, dev.sms, s);
    const PromptPlan g = prompt_plan(B, T, max_new, heads, kv_heads, head_dim, int64_t(max_pages) * page_size, window, sinks);
    if (e == cudaSuccess && g.items > 0) {
        p.items = int(g.items);
        p.tokens = g.tokens; p.pieces = g.pieces; p.slots = g.slots; p.key_slots = g.key_slots;
        p.q_off = g.q_off; p.misc_off = g.misc_off;
        p.prefix = reinterpret_cast<int32_t *>(at + g.prefix_off);
        p.meta = reinterpret_cast<float2 *>(at + g.meta_off);
        p.parts = reinterpret_cast<float *>(at + g.parts_off);
        const int tile_box[3] = {64, p.group, g.tokens};
        st = encode_bf16(&m.q, q, 3, q_dims, q_strides, tile_box);
        if (st != QMV_OK) return st;
        e = head_dim == 64    ? launch_prompt<64>(p, m, g, dev.sms, s)
            : head_dim == 128 ? launch_prompt<128>(p, m, g, dev.sms, s)
                              : launch_prompt<256>(p, m, g, dev.sms, s);
    }
    return e == cudaSuccess ? QMV_OK : record_cuda_failure("attention kernel launch", e);
}
