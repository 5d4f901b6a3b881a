// Tensor-core tiles over packed weights, shared by the operators that take
// several vectors (qmv_lora.cu, qmv_moe.cu).
//
// The mathematics. A subgroup is 64 consecutive k of a row; it lies inside one
// quantization group with scale s and bias b, so its part of an output is
//
//   s * sum_k q_k x_k  +  b * sum_k x_k                    (fp32)
//
// and the first sum is formed by tcgen05, 128 rows and up to 16 vectors at a
// time, on 8-bit operands that are exact:
//  - A byte 0x00..0x0f read as e4m3 is exactly its value times 2^-9 (up to 7 it
//    is subnormal, from 8 on it is the first normal binade; the formula is the
//    same). So a packed word becomes operand registers by masks alone: a 4-bit
//    word's eight fields by v & 0x0f0f0f0f and (v >> 4) & 0x0f0f0f0f; a 2-bit
//    word's sixteen by four masks and a shift, two of the masks leaving 4 q.
//  - x is brought to a largest magnitude of 2^7 .. 2^8 in the subgroup by a power
//    of two, and split into two e4m3 of 4 significant bits each, x' = hi + lo/32.
//    bf16 has 8 bits, so the split is exact down to 2^-14 of the subgroup's
//    largest |x| (2^-12 for a 2-bit matrix's odd fields); below that an element
//    is rounded to 2^-22 (2^-20) of that largest. hi and lo are two rows of the B
//    operand, their sums two accumulators, joined as (hi + lo/32) * f.
// The accumulators are fp32: sums of exact products come out exact, also where terms
// lie 2^21 apart (tested with whole numbers).
//
// Sums are kept as a 2^10th of what they are until they leave the tile (the staged
// sum x and f are times 2^-10): f, which undoes x's scaling, would not
// be a number from |x| of 2^126 on, and q x of the largest x sum to up to 2^138. As
// powers of two change no rounding, results are those of sums kept as they are,
// but for results below 2^-116, which are multiples of 2^-139.
//
// The tile. A thread owns a row (a lane of tensor memory). For each subgroup it
// reads its 32 (2-bit: 16) bytes from the ring, masks them into 16 registers,
// stores those as its 16 columns of the A operand in tensor memory, and two
// steps (of two subgroups, or of one where 16 vectors need the columns) later
// reads the accumulator's columns back and adds s * (..) + b * sum x to its sums,
// which stay in registers over all of K. What bounds it is the integer pipe (one
// instruction in two cycles), of which the masks are 24 instructions for a 4-bit
// subgroup, and the latency of a step, which three warps on each scheduler cover.
// Measured with everything resident, in bytes of 4-bit weights a cycle of an SM
// (6.8 TB/s over 152 SMs are 23.5): 35 up to 4 vectors, 32 at 8, 24 at 16; with
// four worker groups, whose warps have 80 registers instead of 128, 40, 36 and 25,
// but they hold more of the ring while they work; with steps of one subgroup 31
// and 28. Before it, on the same card: bf16 operands (the masks of a low byte are
// exact there too, 40 for a subgroup) through tcgen05 25, 24 and 21; through
// mma.sync, whose instruction holds the issue slot for 8 cycles, 27 and 19.
//
// Order. Slots i, i + 3, .. of a row's range of K belong to one worker group,
// which adds their subgroups in order; the three groups' sums are added in the
// order of their first slots. Nothing depends on how many vectors there are.
//
// The ring has a multiple of three slots and slot s of it always goes to group
// s % 3. A wait for a slot's next lap by its barrier's parity alone is right only
// if the lap before has landed; here the waiting group itself has seen it land.
// (With any number of slots a group could be a lap ahead of a copy that is late.)
#pragma once

#include "qmv_kernel.cuh"
#include "qmv_tile_plan.h"

namespace qmv {
namespace tile {

__device__ __forceinline__ uint64_t pack2(float lo, float hi)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
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

__device__ __forceinline__ uint4 lds_128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// 3-D tensor-map box load (see tma_load_2d).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// The first of a tile's slots that group `group` takes, `at` being the place in
// the ring of the tile's first.
__device__ __forceinline__ int first_slot(int group, int at) { return (group + kGroups - at % kGroups) % kGroups; }

// A place in a ring of `slots`: index and parity of the lap, kept without divisions.
struct Turn {
    int slot = 0, lap = 0;
    __device__ __forceinline__ void step(int n, int slots)
    {
        slot += n;
        while (slot >= slots) {
            slot -= slots;
            ++lap;
        }
    }
};

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// Two floats as e4m3 (a in the low byte), and back.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b)
{
    uint16_t v;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ void from_e4m3x2(uint32_t v, float &a, float &b)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(v)));
    asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(a), "=f"(b)
        : "r"(h));
}

// Row of the B operand that holds term h of vector tok: pairs of vectors
// together, so that their sums are adjacent accumulator columns.
__device__ __forceinline__ int operand_index(int tok, int h, int terms = 2) { return (tok >> 1) * 2 * terms + h * 2 + (tok & 1); }
// Byte of 16-byte piece c of that row in a subgroup's cell (64-byte swizzle).
__device__ __forceinline__ int operand_offset(int r, int c) { return (r >> 3) * 512 + (r & 7) * 64 + ((c ^ (r >> 1)) & 3) * 16; }

// The scale of sums inside a tile, and back.
constexpr float kSumScale = 0x1p-10f, kSumUnscale = 0x1p10f;

// By the largest exponent field E of a subgroup: the power of two that brings its
// elements to 2^7 .. 2^8 at most, and the factor f that undoes it (and the operands'
// 2^-9) in the scale of sums. From 2^-118 down the power stays what it is there, so
// that f is a normal number; bf16 elements are exact all the same. An infinity or
// NaN makes f NaN, and with it everything that the vector gives.
constexpr uint32_t kLeastExponent = 9;
__device__ __forceinline__ int scale_power(uint32_t E) { return 134 - int(E); }
__device__ __forceinline__ float unscale(uint32_t E) { return E == 255 ? __uint_as_float(0x7fc00000u) : exp2i(int(E) - 135); }

// Stages eight elements of a vector: octet o (0..7) of a subgroup, by the eight
// consecutive threads of a warp that hold its octets. x: elements 8 o .. 8 o + 7;
// piece(h): where the 16-byte piece o / 2 of term h goes; keep(sum, f), in the scale
// of sums, is called by one of the eight.
template <int BITS, typename Piece, typename Keep>
__device__ __forceinline__ void stage_octet(const float (&x)[8], int o, Piece piece, Keep keep)
{
    float sum = 0.0f;
    uint32_t E = kLeastExponent;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        sum = __fmaf_rn(x[i], kSumScale, sum);  // (the product is exact)
        E = max(E, (__float_as_uint(x[i]) >> 23) & 0xffu);
    }
    E = __reduce_max_sync(0xffu << (threadIdx.x & 24), E);
#pragma unroll
    for (int d = 1; d < 8; d *= 2) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, d));
    const int p = scale_power(E);
    const float p1 = exp2i(p / 2), p2 = exp2i(p - p / 2);
    uint32_t hi[4], lo[4];  // elements (2i, 2i + 1) as bytes
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // a 2-bit matrix's odd fields come out of the masks as 4 q
        const float a = __fmul_rn(__fmul_rn(x[2 * i], p1), p2);
        const float b = __fmul_rn(__fmul_rn(__fmul_rn(x[2 * i + 1], p1), p2), BITS == 2 ? 0.25f : 1.0f);
        float ah, bh;
        hi[i] = to_e4m3x2(a, b);
        from_e4m3x2(hi[i], ah, bh);
        lo[i] = to_e4m3x2(__fmul_rn(__fsub_rn(a, ah), 32.0f), __fmul_rn(__fsub_rn(b, bh), 32.0f));
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t *v = h ? lo : hi;
        uint8_t *out = piece(h);
        // bytes of even elements and of odd ones, in order
        const uint32_t even = __byte_perm(__byte_perm(v[0], v[1], 0x0040), __byte_perm(v[2], v[3], 0x0040), 0x5410);
        const uint32_t odd = __byte_perm(__byte_perm(v[0], v[1], 0x0051), __byte_perm(v[2], v[3], 0x0051), 0x5410);
        if (BITS == 4) {
            // a word's fields 0 2 4 6, then 1 3 5 7
            *reinterpret_cast<uint2 *>(out + (o & 1) * 8) = make_uint2(even, odd);
        } else {
            // a word spans two octets: fields 0 4 8 12, then 1 5 9 13, 2 6 10 14, 3 7 11 15
            uint16_t *w = reinterpret_cast<uint16_t *>(out) + (o & 1);
            w[0] = uint16_t(__byte_perm(even, 0, 0x0020));
            w[2] = uint16_t(__byte_perm(odd, 0, 0x0020));
            w[4] = uint16_t(__byte_perm(even, 0, 0x0031));
            w[6] = uint16_t(__byte_perm(odd, 0, 0x0031));
        }
    }
    if (o == 0) keep(sum, unscale(E));
}

// Eight bf16 of a 16-byte load as floats.
__device__ __forceinline__ void widen8(uint4 v, float (&x)[8])
{
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(in[i] << 16);
        x[2 * i + 1] = __uint_as_float(in[i] & 0xffff0000u);
    }
}

// A row's 64 packed fields as 16 operand registers, in the order of staged x.
template <int BITS>
__device__ __forceinline__ void operand_row(const uint32_t (&w)[2 * BITS], uint32_t (&r)[16])
{
#pragma unroll
    for (int i = 0; i < 2 * BITS; ++i) {
        const uint32_t v = w[i], u = v >> 4;
        if (BITS == 4) {
            r[(2 * i) & 15] = v & 0x0f0f0f0fu;
            r[(2 * i + 1) & 15] = u & 0x0f0f0f0fu;
        } else {
            r[(4 * i) & 15] = v & 0x03030303u;
            r[(4 * i + 1) & 15] = v & 0x0c0c0c0cu;
            r[(4 * i + 2) & 15] = u & 0x03030303u;
            r[(4 * i + 3) & 15] = u & 0x0c0c0c0cu;
        }
    }
}

// ------------------------------------------------------------ tensor memory --

__device__ __forceinline__ void tmem_alloc(uint32_t out, uint32_t columns)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(out), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// N columns of the warp's 32 lanes.
__device__ __forceinline__ void tmem_st(uint32_t a, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st1(uint32_t a, float v)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(a), "f"(v) : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_st_few(uint32_t a, const float (&v)[N])
{
    static_assert(N == 2 || N == 4 || N == 8, "columns");
    if constexpr (N == 2)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1,%2};" ::"r"(a), "f"(v[0]), "f"(v[1]) : "memory");
    else if constexpr (N == 4)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3])
                     : "memory");
    else
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                     "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                     : "memory");
}
__device__ __forceinline__ float tmem_ld1(uint32_t a)
{
    float v;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=f"(v) : "r"(a));
    return v;
}
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t a, float (&v)[N])
{
    static_assert(N == 2 || N == 4 || N == 8 || N == 16 || N == 32 || N == 64, "columns");
    if constexpr (N == 2)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "r"(a));
    else if constexpr (N == 4)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                     : "r"(a));
    else if constexpr (N == 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                     : "r"(a));
    else if constexpr (N == 16)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
              "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
            : "r"(a));
    else {
#pragma unroll
        for (int k = 0; k < N / 16; ++k) {
            float part[16];
            tmem_ld<16>(a + 16 * k, part);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[16 * k + i] = part[i];
        }
    }
}

// Orders what follows after the wait that made `v` valid.
template <int N>
__device__ __forceinline__ void settle(float (&v)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i])::"memory");
}

// D (128 x ND fp32) (+)= A (128 x 32 e4m3, tensor memory) B^T (ND x 32 e4m3, shared memory).
template <int ND>
__device__ __forceinline__ void tmem_mma(uint32_t d, uint32_t a, uint64_t b, bool add)
{
    // fp32 accumulator, e4m3 operands, both K-major, N = ND, M = 128
    constexpr uint32_t kind = 1u << 4 | uint32_t(ND >> 3) << 17 | (128u >> 4) << 24;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(kind), "r"(uint32_t(add))
        : "memory");
}

// Descriptor of a B operand: rows of 64 bytes under the 64-byte swizzle, eight
// rows to an atom, `stride` bytes from atom to atom. 32 bytes further along a
// row is an address 2 units further.
__device__ __forceinline__ uint64_t b_descriptor(uint32_t addr, uint32_t stride)
{
    return uint64_t((addr >> 4) & 0x3fffu) | uint64_t(1) << 16 | uint64_t(stride >> 4) << 32 | uint64_t(1) << 46 |
           uint64_t(4) << 61;
}

__device__ __forceinline__ void mbar_arrive_many(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

// Bulk store of shared memory; the thread commits and waits for its group.
__device__ __forceinline__ void bulk_store(void *dst, uint32_t src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}

// An arrival on `bar` when the thread's earlier tensor instructions are done.
__device__ __forceinline__ void tmem_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void named_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// A bounded wait that all of a CTA's roles share: one that runs out sets the
// device error word and a flag in shared memory, from then on every wait
// returns at once and the roles run to their ends without computing anything
// useful (the output of that launch is invalid).
struct Waits {
    volatile int *abort;
    unsigned *err;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const
    {
        // bounded by attempts alone (tens of milliseconds at least): the global
        // timer takes longer to read than most waits last
#pragma unroll 1
        for (int i = 1; i < 1 << 22; ++i) {
            if (mbar_try_wait(bar, parity)) return true;
            if ((i & 63) == 0 && *abort) return false;
        }
        atomicOr(err, 1u);
        *abort = 1;
        return false;
    }
};

__device__ __forceinline__ void Affines::fetch(uint32_t dst, uint8_t *gen, const uint16_t *sc, const uint16_t *bi,
                                               const CUtensorMap *smap, const CUtensorMap *bmap, long long row0,
                                               int rows, long long all, int G, int g0, int groups, uint32_t bar,
                                               int lane) const
{
    if (mode == kSbBoxes) {
        if (lane == 0) {
            mbar_arrive_expect_tx(bar, uint32_t(2 * rows * pitch));
            tma_load_2d(dst, smap, g0 / 8 * 2, int(row0), bar);  // eight groups are two elements
            tma_load_2d(dst + block, bmap, g0 / 8 * 2, int(row0), bar);
        } else {
            mbar_arrive(bar);
        }
        return;
    }
    // from the 16-byte boundary before the first; the last bytes of the
    // arrays, where they fill no 16, go one by one
    const long long end = all * G * 2;
    const int step = mode == kSbWhole ? rows : 1;
    uint32_t total = 0;
    for (int pass = 0; pass < 2; ++pass) {
        for (int r = mode == kSbWhole ? (lane == 0 ? 0 : rows) : lane; r < rows; r += mode == kSbWhole ? rows : 32) {
            const long long n = row0 + r;
            if (n >= all) break;
            const long long first = mode == kSbWhole ? n * G * 2 : (n * G + g0) * 2, from = first & ~15ll;
            const long long to = mode == kSbWhole ? min(first + (long long)step * G * 2, end) : first + 2 * groups;
            const long long whole = min((to + 15) & ~15ll, end & ~15ll);
            const uint32_t bytes = whole > from ? uint32_t(whole - from) : 0u, d = uint32_t(r * pitch);
            if (pass == 0) {
                total += 2 * bytes;
                for (long long e = max(whole, from); e < to; e += 2) {
                    *reinterpret_cast<uint16_t *>(gen + d + (e - from)) = __ldg(sc + e / 2);
                    *reinterpret_cast<uint16_t *>(gen + d + block + (e - from)) = __ldg(bi + e / 2);
                }
                if (whole < to) fence_proxy_async_smem();  // (copies come here again)
            } else if (bytes) {
                bulk_load_plain(dst + d, reinterpret_cast<const uint8_t *>(sc) + from, bytes, bar);
                bulk_load_plain(dst + d + block, reinterpret_cast<const uint8_t *>(bi) + from, bytes, bar);
            }
        }
        if (pass == 0) mbar_arrive_expect_tx(bar, total);
    }
}

// Scales and biases of a row for the groups of one slot.
template <int BITS, int GS>
struct Affine {
    static constexpr int kSubs = slot_subs(BITS), kGroupsPerSlot = kSubs * 64 / GS, kWords = kGroupsPerSlot / 2;
    uint32_t s[kWords], b[kWords];

    // At shared address `addr`, the biases `block` bytes further; `left` groups of
    // the row from there on, those past them being zeros.
    __device__ __forceinline__ void read(uint32_t addr, uint32_t block, int align, int left)
    {
        get(addr, align, s);
        get(addr + block, align, b);
        if (left < kGroupsPerSlot) {
#pragma unroll
            for (int g = 0; g < kGroupsPerSlot; ++g)
                if (g >= left) {
                    s[g / 2] &= g & 1 ? 0x0000ffffu : 0u;
                    b[g / 2] &= g & 1 ? 0x0000ffffu : 0u;
                }
        }
    }
    // Of subgroup j of the slot.
    __device__ __forceinline__ float scale(int j) const { return half(s, j); }
    __device__ __forceinline__ float bias(int j) const { return half(b, j); }

private:
    static __device__ __forceinline__ float half(const uint32_t (&v)[kWords], int j)
    {
        const int g = j * 64 / GS;
        return __uint_as_float(g & 1 ? v[g / 2] & 0xffff0000u : v[g / 2] << 16);
    }
    static __device__ __forceinline__ void get(uint32_t addr, int align, uint32_t (&v)[kWords])
    {
        if (align == 8 && kWords > 1) {
#pragma unroll
            for (int i = 0; i + 1 < kWords; i += 2)
                asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v[i]), "=r"(v[i + 1]) : "r"(addr + 4 * i));
        } else if (align >= 4) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[i]) : "r"(addr + 4 * i));
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                uint16_t lo, hi;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(lo) : "r"(addr + 4 * i));
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(hi) : "r"(addr + 4 * i + 2));
                v[i] = uint32_t(lo) | uint32_t(hi) << 16;
            }
        }
    }
};

// A group's barriers (A stored, accumulators ready) and tensor memory; `lanes`
// is the warp's part of it for workers, 0 for the tensor warp. `steps` counts the
// group's steps from the launch's start, the same in workers and tensor warp.
struct Pipe {
    uint32_t stored, ready, a, d;
    uint32_t steps;

    template <int NC, int TERMS = 2>
    __device__ __forceinline__ static Pipe make(uint32_t tm, uint32_t lanes, uint32_t stored0, uint32_t ready0, int group)
    {
        static_assert(a_columns(NC, TERMS) <= kGroupColumns / 2 && d_columns(NC, TERMS) <= kGroupColumns / 2, "a group's columns");
        const uint32_t a = tm + lanes + group * kGroupColumns;
        return {stored0 + 16 * group, ready0 + 16 * group, a, a + kGroupColumns / 2, 0u};
    }
};

// A worker thread's row of a tile: sums of NC vectors over the slots it is given.
// Two steps are in flight: the accumulators of one are read two steps later, when
// its A columns are needed again.
template <int BITS, int GS, int NC, int TERMS = 2>
struct Row {
    static constexpr int kSubs = slot_subs(BITS), kStep = step_subs(NC, TERMS), kSteps = kSubs / kStep;
    static constexpr int kVals = TERMS * NC;
    static_assert(kSteps % 2 == 0, "a slot's steps use the two buffers alike");
    uint64_t y[NC / 2];
    float last_s[2 * kStep], last_b[2 * kStep];  // of the previous slot's last two steps
    bool primed;

    __device__ __forceinline__ void start()
    {
#pragma unroll
        for (int i = 0; i < NC / 2; ++i) y[i] = 0ull;
#pragma unroll
        for (int i = 0; i < 2 * kStep; ++i) last_s[i] = last_b[i] = 0.0f;
        primed = false;
    }

    __device__ __forceinline__ void add(const float (&v)[kVals], float s, float b, uint32_t meta)
    {
        const uint64_t ss = pack2(s, s), bb = pack2(b, b), r32 = pack2(0.03125f, 0.03125f);
#pragma unroll
        for (int c = 0; c < NC / 2; ++c) {
            const uint4 m = lds_128(meta + c * 16);
            const uint64_t sum = pack2(__uint_as_float(m.x), __uint_as_float(m.y));
            const uint64_t f = pack2(__uint_as_float(m.z), __uint_as_float(m.w));
            // terms from the last, each 1/32 of the one before
            uint64_t d = pack2(v[2 * TERMS * c + 2 * TERMS - 2], v[2 * TERMS * c + 2 * TERMS - 1]);
#pragma unroll
            for (int h = TERMS - 2; h >= 0; --h) d = fma2(d, r32, pack2(v[2 * TERMS * c + 2 * h], v[2 * TERMS * c + 2 * h + 1]));
            d = mul2(d, f);
            y[c] = fma2(ss, d, fma2(bb, sum, y[c]));
            // (keeps the loads of the next pairs from being hoisted into registers
            // that are not there)
            if (c % 4 == 3) asm volatile("" : "+l"(y[c]), "+l"(y[c - 1]), "+l"(y[c - 2]), "+l"(y[c - 3]));
        }
    }

    // One slot: `w` is the row's address in it with its swizzle bits, `meta` the
    // address of the slot's first subgroup's meta and `last_meta` that of the
    // first subgroup of the previous slot's last two steps.
    __device__ __forceinline__ void slot(const Waits &wait, Pipe &p, uint32_t w, const Affine<BITS, GS> &aff, uint32_t meta,
                                         uint32_t last_meta, int lane)
    {
        constexpr int MB = meta_bytes(NC), ND = acc_columns(NC, TERMS);
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            uint32_t words[kStep][2 * BITS];
#pragma unroll
            for (int u = 0; u < kStep; ++u)
#pragma unroll
                for (int h = 0; h < BITS / 2; ++h) {
                    const uint4 v = lds_128(w ^ uint32_t(((j * kStep + u) * (BITS / 2) + h) << 4));
                    words[u][4 * h] = v.x;
                    words[u][4 * h + 1] = v.y;
                    words[u][4 * h + 2] = v.z;
                    words[u][4 * h + 3] = v.w;
                }
            const bool take = j >= 2 || primed;
            if (take) wait(p.ready + 8 * (j & 1), ((p.steps + j) / 2 + 1) & 1);
            tmem_fence_after();
            float v[kStep][kVals];
#pragma unroll
            for (int u = 0; u < kStep; ++u) tmem_ld<kVals>(p.d + ((j & 1) * kStep + u) * ND, v[u]);
#pragma unroll
            for (int u = 0; u < kStep; ++u) {
                uint32_t r[16];
                operand_row<BITS>(words[u], r);
                tmem_st(p.a + ((j & 1) * kStep + u) * 16, r);
            }
            tmem_wait_ld();
#pragma unroll
            for (int u = 0; u < kStep; ++u) settle(v[u]);
            tmem_wait_st();
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p.stored + 8 * (j & 1));
            if (take) {
#pragma unroll
                for (int u = 0; u < kStep; ++u) {
                    const int sub = (j - 2) * kStep + u;  // below 0: of the previous slot
                    if (j < 2) add(v[u], last_s[sub + 2 * kStep], last_b[sub + 2 * kStep], last_meta + (sub + 2 * kStep) * MB);
                    else add(v[u], aff.scale(sub), aff.bias(sub), meta + sub * MB);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 2 * kStep; ++i) {
            last_s[i] = aff.scale(kSubs - 2 * kStep + i);
            last_b[i] = aff.bias(kSubs - 2 * kStep + i);
        }
        p.steps += kSteps;
        primed = true;
    }

    // The last slot's last two steps.
    __device__ __forceinline__ void finish(const Waits &wait, const Pipe &p, uint32_t last_meta)
    {
        if (!primed) return;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            wait(p.ready + 8 * j, (p.steps / 2 + 1) & 1);
            tmem_fence_after();
            float v[kStep][kVals];
#pragma unroll
            for (int u = 0; u < kStep; ++u) tmem_ld<kVals>(p.d + (j * kStep + u) * acc_columns(NC, TERMS), v[u]);
            tmem_wait_ld();
#pragma unroll
            for (int u = 0; u < kStep; ++u) {
                settle(v[u]);
                add(v[u], last_s[j * kStep + u], last_b[j * kStep + u], last_meta + (j * kStep + u) * meta_bytes(NC));
            }
        }
    }

    // How the three groups' sums of a tile's rows meet. Either (give, take) other warps
    // get them all when they have time, and the groups go on to their next tile at once:
    // these leave theirs in columns `ex` of tensor memory (three sets of 8), free when
    // `freed` says so, and arrive on `joined`. `use`: the tiles that had the columns
    // before; c: the group's place in the order of the sums.
    __device__ __forceinline__ void give(const Waits &wait, uint32_t ex, int c, uint32_t joined, uint32_t freed, int use, int lane) const
    {
        if (use > 0) wait(freed, (use - 1) & 1);
        tmem_fence_after();
        float v[NC];
#pragma unroll
        for (int i = 0; i < NC / 2; ++i) unpack2(y[i], v[2 * i], v[2 * i + 1]);
        tmem_st_few<NC>(ex + c * 8, v);
        tmem_wait_st();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(joined);
    }
    static __device__ __forceinline__ void take(const Waits &wait, uint32_t ex, uint32_t joined, uint32_t freed, int use, int lane,
                                                float (&sums)[NC])
    {
        wait(joined, use & 1);
        tmem_fence_after();
        float v[kGroups][NC];
#pragma unroll
        for (int c = 0; c < kGroups; ++c) tmem_ld<NC>(ex + c * 8, v[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < kGroups; ++c) settle(v[c]);
#pragma unroll
        for (int i = 0; i < NC; ++i) sums[i] = __fmul_rn(__fadd_rn(__fadd_rn(v[0][i], v[1][i]), v[2][i]), kSumUnscale);
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(freed);
    }

    // Or (join) the groups wait for one another and share them: through tensor memory
    // (each group its own A columns, `tm` being the first with the warp's lanes) sums[i]
    // becomes the total of vector group + 3 i, added from group `first` on, which had
    // the tile's first slot.
    static constexpr int kOwn = (NC + kGroups - 1) / kGroups;
    __device__ __forceinline__ void join(uint32_t tm, int group, int first, float (&sums)[kOwn])
    {
#pragma unroll
        for (int c = 0; c < NC / 2; ++c) {
            float lo, hi;
            unpack2(y[c], lo, hi);
            tmem_st1(tm + group * kGroupColumns + 2 * c, lo);
            tmem_st1(tm + group * kGroupColumns + 2 * c + 1, hi);
        }
        tmem_wait_st();
        tmem_fence_before();
        named_sync(1, 32 * kWorkers);
        tmem_fence_after();
        float v[kOwn][kGroups];
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
                v[i][g] = tmem_ld1(tm + (first + g) % kGroups * kGroupColumns + min(group + kGroups * i, NC - 1));
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            settle(v[i]);
            sums[i] = __fmul_rn(__fadd_rn(__fadd_rn(v[i][0], v[i][1]), v[i][2]), kSumUnscale);
        }
        tmem_fence_before();
        named_sync(1, 32 * kWorkers);
        tmem_fence_after();
    }
};

// The tensor warp's part of one slot: waits for each step's A operands and
// multiplies them with the subgroups' cells. `cell` is the slot's first.
// FENCE: the cells were written by threads, not by bulk copies. release: a barrier
// that gets an arrival when the slot's cells have been read, 0: none.
template <int BITS, int NC, int TERMS = 2, bool FENCE = false>
__device__ __forceinline__ void multiply_slot(const Waits &wait, Pipe &p, uint32_t cell, uint32_t release = 0)
{
    constexpr int ND = acc_columns(NC, TERMS), CB = cell_bytes(NC, TERMS), U = step_subs(NC, TERMS);
    constexpr int STEPS = slot_subs(BITS) / U;
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
        wait(p.stored + 8 * (j & 1), ((p.steps + j) / 2) & 1);
        if (FENCE && j == 0) fence_proxy_async_smem();
        tmem_fence_after();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint64_t b = b_descriptor(cell + (j * U + u) * CB, operand_rows(NC, TERMS) <= 8 ? 0 : 512);
            const uint32_t a = p.a + ((j & 1) * U + u) * 16, d = p.d + ((j & 1) * U + u) * ND;
            tmem_mma<ND>(d, a, b, false);
            tmem_mma<ND>(d, a + 8, b + 2, true);
        }
        tmem_commit(p.ready + 8 * (j & 1));
    }
    if (release) tmem_commit(release);
    p.steps += STEPS;
}

}  // namespace tile
}  // namespace qmv
