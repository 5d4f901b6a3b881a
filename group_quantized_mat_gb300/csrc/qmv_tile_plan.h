// What a launch plan has to know of the tensor-core tiles (qmv_tile.cuh): sizes in
// shared and tensor memory, and how scales and biases are brought there. Plain host
// code but for what is marked, so that plans can be checked without a GPU.
#pragma once

#include <cuda.h>

#include <cstdint>

namespace qmv {
namespace tile {

constexpr int kGroups = 3;                   // worker groups of four warps
constexpr int kWorkers = 4 * kGroups;        // worker warps; then a tensor warp for each group
constexpr int kThreads = 32 * (kWorkers + kGroups + 1);  // and the producer
constexpr int kTileRows = 128;
constexpr int kSlotBytes = 128;              // bytes of a row in a ring slot

__host__ __device__ constexpr int slot_subs(int bits) { return kSlotBytes * 8 / bits / 64; }  // 4 or 8
// nc vectors of `terms` e4m3 each are the rows of a subgroup's B operand: atoms of
// 8 rows x 64 bytes. The instruction's N is 16 at least; where there are only 8
// rows its second eight are the first again.
__host__ __device__ constexpr int operand_rows(int nc, int terms = 2) { return nc * terms; }
__host__ __device__ constexpr int cell_bytes(int nc, int terms = 2) { return operand_rows(nc, terms) <= 8 ? 512 : operand_rows(nc, terms) * 64; }
// Bytes of a subgroup's (sum, sum, f, f), for each pair of vectors.
__host__ __device__ constexpr int meta_bytes(int nc) { return nc / 2 * 16; }
// Columns of an accumulator: the instruction's N.
__host__ __device__ constexpr int acc_columns(int nc, int terms = 2) { return operand_rows(nc, terms) <= 16 ? 16 : operand_rows(nc, terms); }
// Subgroups of a step, and a group's columns of A (two steps) and of accumulators.
__host__ __device__ constexpr int step_subs(int nc, int terms = 2) { return operand_rows(nc, terms) <= 16 ? 2 : 1; }
__host__ __device__ constexpr int a_columns(int nc, int terms = 2) { return 2 * step_subs(nc, terms) * 16; }
__host__ __device__ constexpr int d_columns(int nc, int terms = 2) { return 2 * step_subs(nc, terms) * acc_columns(nc, terms); }
constexpr int kTmemColumns = 512;
// A group's, half for A and half for accumulators whatever the number of vectors
// and terms, so that groups may be at work with different ones.
constexpr int kGroupColumns = 128;

// How a tile's scales and biases come to shared memory, once for its range of K:
// by tensor map where rows start on 16 bytes (boxes an odd number of 16 bytes
// wide, so that 32 rows' reads spread over the banks), else whole rows in one
// piece where that is small, else row by row. What was tried instead: a thread
// reading its own row's from global memory, up to three slots ahead, waited for
// microseconds behind the stream of weights; copies of 8 bytes a row and slot by
// the producer warp kept it busy for twice the time of a slot.
enum { kSbBoxes, kSbWhole, kSbRows };

struct Affines {
    int mode, pitch, block;  // bytes from row to row, and of each of the two arrays

    // `whole`: most groups of a row that are fetched as whole rows.
    __host__ __device__ static Affines plan(int G, int groups, int rows, int whole)
    {
        Affines a;
        a.mode = G % 8 == 0 ? kSbBoxes : G <= whole ? kSbWhole : kSbRows;
        a.pitch = a.mode == kSbWhole ? 2 * G : (((2 * groups + 30) / 16) | 1) * 16;
        a.block = (rows * a.pitch + 127) & ~127;
        return a;
    }
    // By the whole producer warp, each lane arriving once on `bar`: rows row0 .. row0 + rows - 1 of `all`, groups g0 ..
    // g0 + groups - 1 of G, into dst (generic address `gen`). smap, bmap: tensor
    // maps for kSbBoxes.
    __device__ void fetch(uint32_t dst, uint8_t *gen, const uint16_t *sc, const uint16_t *bi, const CUtensorMap *smap,
                          const CUtensorMap *bmap, long long row0, int rows, long long all, int G, int g0, int groups,
                          uint32_t bar, int lane) const;
    // Offset of group g0 of a row in its bytes there.
    __device__ uint32_t offset(long long row, int G, int g0) const
    {
        return mode == kSbBoxes ? (g0 & 7) * 2u : mode == kSbWhole ? g0 * 2u : uint32_t((row * G + g0) * 2) & 15u;
    }
    // Bytes by which a row's groups of a slot are aligned there, at most 8.
    __device__ int alignment(int G) const
    {
        return mode == kSbRows ? 2 : mode == kSbBoxes || G % 4 == 0 ? 8 : G % 2 == 0 ? 4 : 2;
    }
};

}  // namespace tile
}  // namespace qmv
