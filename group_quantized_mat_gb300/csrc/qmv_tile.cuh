// Tensor-core tiles over packed weights, shared by the operators that take
// several vectors (qmv_lora.cu, qmv_moe.cu).
//
// The mathematics. A subgroup is 64 consecutive k of a row; it lies inside one
// quantization group with scale s and bias b, so its part of an output is
//
//   s * sum_k q_k x_k  +  b * sum_k x_k                    (fp32)
//
// and the first sum is a product of small integers with bf16 values: one
// m16n8k16 bf16 instruction covers 16 rows, 16 of the k and 8 vectors. A row's
// 64 packed fields need no conversion to become bf16 operands: the bf16 whose
// low byte is n and whose high byte is zero is exactly n * 2^-133 (n < 128 is
// subnormal, 128 <= n < 256 is the first normal binade; the formula is the
// same), and the tensor core takes subnormal operands exactly. So one mask
// isolates two fields (one in each half word), wherever in the half word's low
// byte they lie, and a shift by 8 serves the high bytes: a 4-bit word's eight
// fields cost five instructions, a 2-bit word's sixteen cost nine. The factor
// 2^(field position) goes into x, whose staged form is
//
//   x'_k = x_k * 2^(p - position),  p = 240 - E (at least 6),
//
// E being the largest exponent field of the subgroup's x. All factors are
// powers of two and exact, so sum q x = acc * f with f = 2^(133 - p). (For x of
// 2^122 and above, infinities and NaN, the vector's own result is unspecified.)
//
// What it costs: per 16 rows x 64 k (512 bytes of 4-bit weights) and 8 vectors
// about 45 instructions and four tensor instructions (8 cycles of an SM at the
// measured 0.51 a cycle), against 22 cycles that the bytes take at 6.8 TB/s
// over 152 SMs. The fp32 cores would need 32 fused multiply-adds of a warp for
// each vector. tcgen05 would need the fields written out as bf16 to shared or
// tensor memory first (four times the weight bytes) and its accumulators read
// back for every group.
//
// Staged x. A cell is one subgroup of one vector: 64 bf16 in operand order, 128
// bytes. The thread with index t of a quad holds k = 16 t .. 16 t + 15, 32
// bytes: operand registers in the order of the masks. The two 16-byte halves of
// the 32 bytes are exchanged in odd vectors, so that a quarter warp's 16-byte
// reads of two vectors cover all banks. Beside the cells lie, for each subgroup
// and pair of vectors, (sum x, sum x, f, f).
#pragma once

#include "qmv_kernel.cuh"

namespace qmv {
namespace tile {

constexpr int kCell = 128;  // bytes of a staged cell
constexpr int kMeta = 64;   // bytes of a subgroup's (sum, f) of 8 vectors

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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds_128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 lds_64(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds_32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
// A bf16 of shared memory as fp32.
__device__ __forceinline__ float lds_bf16(uint32_t addr)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return __uint_as_float(uint32_t(v) << 16);
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// Stages eight elements of a vector: octet o (0..7) of a subgroup, by the
// eight consecutive threads of a warp that hold its octets. `v` holds the bf16
// of elements 8 o .. 8 o + 7; `tok` is the vector's index in its block, `cell`
// the subgroup's cell of it, `meta` the subgroup's meta of its eight vectors.
template <int BITS>
__device__ __forceinline__ void stage_octet(uint4 v, int o, int tok, uint8_t *cell, float *meta)
{
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
    float x[8], sum = 0.0f;
    uint32_t E = 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(in[i] << 16);
        x[2 * i + 1] = __uint_as_float(in[i] & 0xffff0000u);
        E = max(E, max((in[i] >> 7) & 0xffu, (in[i] >> 23) & 0xffu));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = __fadd_rn(sum, x[i]);
#pragma unroll
    for (int d = 1; d < 8; d *= 2) {
        sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, d));
        E = max(E, __shfl_xor_sync(0xffffffffu, E, d));
    }
    const int p = max(240 - int(E), 6);  // 6 .. 239
    // x * 2^(p - position) in two exact steps; what would come out below the
    // least normal bf16 is more than 2^200 times smaller than the largest x
    const float p1 = exp2i(p / 2), p2 = exp2i(p - p / 2);
    uint32_t y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int pos = BITS == 4 ? 4 * (i & 1) : 2 * (i & 3);
        const float s = __fmul_rn(__fmul_rn(__fmul_rn(x[i], p1), p2), exp2i(-pos));
        y[i] = __float_as_uint(fabsf(s) < 1.17549435e-38f ? 0.0f : s) >> 16;
    }
    uint4 out;
    if (BITS == 4) {
        // masks of a word: fields (0,4), (1,5), then of the word >> 8: (2,6), (3,7)
        out = make_uint4(y[0] | y[4] << 16, y[1] | y[5] << 16, y[2] | y[6] << 16, y[3] | y[7] << 16);
    } else {
        // a word spans two octets: (0,8) .. (3,11), then (4,12) .. (7,15)
        const uint32_t a = y[0] | y[1] << 16, b = y[2] | y[3] << 16, c = y[4] | y[5] << 16, d = y[6] | y[7] << 16;
        const bool odd = o & 1;
        const uint32_t r0 = __shfl_xor_sync(0xffffffffu, odd ? a : c, 1);
        const uint32_t r1 = __shfl_xor_sync(0xffffffffu, odd ? b : d, 1);
        const uint32_t lo0 = odd ? r0 : a, lo1 = odd ? r1 : b, hi0 = odd ? c : r0, hi1 = odd ? d : r1;
        out = make_uint4((lo0 & 0xffffu) | hi0 << 16, lo0 >> 16 | (hi0 & 0xffff0000u), (lo1 & 0xffffu) | hi1 << 16,
                         lo1 >> 16 | (hi1 & 0xffff0000u));
    }
    *reinterpret_cast<uint4 *>(cell + (o >> 1) * 32 + ((o ^ tok) & 1) * 16) = out;
    if (o == 0) {
        float *m = meta + ((tok & 7) >> 1) * 4 + (tok & 1);
        m[0] = sum;
        m[2] = exp2i(min(int(E) - 107, 127));
    }
}

// The operand words of one subgroup and row: two for 4 bits, one for 2.
template <int BITS>
struct Words {
    uint32_t w[BITS / 2];
    __device__ __forceinline__ void load(uint32_t addr)
    {
        if (BITS == 4) {
            const uint2 v = lds_64(addr);
            w[0] = v.x;
            w[BITS / 2 - 1] = v.y;
        } else {
            w[0] = lds_32(addr);
        }
    }
    // The two operand registers of step q = 0..3.
    __device__ __forceinline__ void fields(int q, uint32_t &lo, uint32_t &hi) const
    {
        if (BITS == 4) {
            const uint32_t v = q & 1 ? w[q >> 1] >> 8 : w[q >> 1];
            lo = v & 0x000f000fu;
            hi = v & 0x00f000f0u;
        } else {
            const uint32_t v = q & 2 ? w[0] >> 8 : w[0];
            lo = v & (q & 1 ? 0x00300030u : 0x00030003u);
            hi = v & (q & 1 ? 0x00c000c0u : 0x000c000cu);
        }
    }
};

// Adds one subgroup of MT x 16 rows and NT x 8 vectors to y (y[i][n][h]: rows
// 16 i + 8 h + lane / 4, vectors 8 n + 2 (lane % 4) and the next).
//  w      shared address of the lane's words in row lane / 4 of the block
//  pitch  bytes from row to row
//  s, b   shared addresses of that row's scale and bias; sp bytes from row to row
//  x[n]   shared address of the lane's 32 bytes in the cell of vector 8 n + lane / 4
//  odd[n] 16 where that vector's halves are exchanged
//  meta   shared address of the lane's (sum, sum, f, f) of vectors 0..7
template <int BITS, int MT, int NT>
__device__ __forceinline__ void add_subgroup(uint64_t (&y)[2][NT][2], uint32_t w, uint32_t pitch, uint32_t s,
                                             uint32_t b, uint32_t sp, const uint32_t (&x)[NT], const uint32_t (&odd)[NT],
                                             uint32_t meta)
{
    Words<BITS> wr[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) wr[i][h].load(w + (16 * i + 8 * h) * pitch);
    uint4 xa[NT], xb[NT], m[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        xa[n] = lds_128(x[n] + odd[n]);
        xb[n] = lds_128(x[n] + (odd[n] ^ 16u));
        m[n] = lds_128(meta + n * kMeta);
    }
    float sv[MT][2], bv[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            sv[i][h] = lds_bf16(s + (16 * i + 8 * h) * sp);
            bv[i][h] = lds_bf16(b + (16 * i + 8 * h) * sp);
        }
    float acc[MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][n][j] = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            uint32_t a0, a1, a2, a3;
            wr[i][0].fields(q, a0, a2);
            wr[i][1].fields(q, a1, a3);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 &v = q < 2 ? xa[n] : xb[n];
                mma_bf16(acc[i][n], a0, a1, a2, a3, q & 1 ? v.z : v.x, q & 1 ? v.w : v.y);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint64_t ss = pack2(sv[i][h], sv[i][h]), bb = pack2(bv[i][h], bv[i][h]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint64_t sum = pack2(__uint_as_float(m[n].x), __uint_as_float(m[n].y));
                const uint64_t f = pack2(__uint_as_float(m[n].z), __uint_as_float(m[n].w));
                const uint64_t d = mul2(pack2(acc[i][n][2 * h], acc[i][n][2 * h + 1]), f);
                y[i][n][h] = fma2(ss, d, fma2(bb, sum, y[i][n][h]));
            }
        }
}

// 4-byte asynchronous copy global -> shared of which `bytes` (0, 2 or 4) are
// read and the rest are zeros.
__device__ __forceinline__ void copy_word(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// An arrival on `bar` when this thread's earlier copies have landed.
__device__ __forceinline__ void copy_arrive(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void named_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

}  // namespace tile
}  // namespace qmv
