// The launch plan of qmv_lora_run: its sizes, what lies where in shared memory and in
// the workspace. Host code without a CUDA call, so that plans can be checked without a GPU.
#pragma once

#include <cstddef>
#include <cstdint>

#include "qmv.h"
#include "qmv_tile_plan.h"

namespace qmv {
namespace lora {

constexpr int kMaxSlots = 12;
constexpr int kSmem = 225 * 1024;  // beside 2 KB of static lists
constexpr int kMaxK = 1 << 16;
// Subgroups of a range of K at most. The ring's three slots, a range's cells of 16
// vectors, its scales and biases and the inner vectors have to fit at 128 rows.
__host__ __device__ constexpr int range_subs(int rank) { return rank <= 64 ? 64 : 48; }
constexpr int kPass = 16;       // vectors that one read of the weights serves
constexpr int kPasses = QMV_MAX_M / kPass;
constexpr int kSms = 152;       // for orders of sums, which depend on no device

struct LoraShape {
    int M, N, K, G, gs, R;
    int S;       // subgroups of a row
    int NS;      // slots of a row
    int subs;    // NS slots' subgroups (those past S are staged as zeros)
    int nseg;    // ranges of K
    int range;   // slots of the longest range
    int rows, tiles, grid_rows;
    int piece;   // rows of an adapter's B that a ring slot holds
    int nc, slots, sb_buffers, inner_buffers;
    int grid_passes;  // passes that are at work at a time
    tile::Affines sb;
};

// Floats from an inner vector to the next, so that all of a pass's are one bulk copy.
__host__ __device__ constexpr int inner_pitch(int rank) { return (rank + 7) & ~7; }

struct Layout {
    int slots, slot, x, meta, sb, inner, inner_bytes, bars, misc, total;
};

__host__ __device__ inline Layout layout(const LoraShape &p, int bits, int nc)
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
    l.sb = (l.meta + subs * tile::meta_bytes(nc) + 127) & ~127;
    l.inner = l.sb + p.sb_buffers * 2 * p.sb.block;
    l.inner_bytes = nc * inner_pitch(p.R) * 4;
    l.bars = l.inner + p.inner_buffers * l.inner_bytes;
    l.misc = l.bars + (2 * p.slots + 4 * tile::kGroups + 6) * 8;
    l.total = l.misc + (4 + kPasses) * 4;
    return l;
}

// Where the inner vectors of a CTA's pass lie, `before` passes of it having gone
// before: the producer's copy and the workers' reads both ask here.
__host__ __device__ inline int inner_at(const LoraShape &p, const Layout &l, int before)
{
    return l.inner + (before & (p.inner_buffers - 1)) * l.inner_bytes;
}

struct Sizes {
    size_t cells, meta, inner, counters, partials, total;
};

inline size_t up256(size_t b) { return (b + 255) & ~size_t(255); }

// What a call needs; `sms` only shapes the grid (tiles), never an order of sums
// or a size.
inline LoraShape plan(int M, int N, int K, int bits, int gs, int R, int sms, Sizes &sz)
{
    const int slot_subs = tile::slot_subs(bits);
    LoraShape p{};
    p.M = M; p.N = N; p.K = K; p.G = K / gs; p.gs = gs; p.R = R;
    p.S = K / 64;
    p.NS = (p.S + slot_subs - 1) / slot_subs;
    p.subs = p.NS * slot_subs;
    // Ranges of K: as few as fit, and for few rows as many as give each SM of the
    // card a tile of 128, of three slots at least (one for each worker group).
    p.nseg = (p.NS * slot_subs + range_subs(R) - 1) / range_subs(R);
    int spread = kSms / ((N + tile::kTileRows - 1) / tile::kTileRows);
    if (spread > p.NS / tile::kGroups) spread = p.NS / tile::kGroups;
    if (p.nseg < spread) p.nseg = spread;
    p.range = (p.NS + p.nseg - 1) / p.nseg;
    p.nc = M <= 2 ? 2 : M <= 4 ? 4 : M <= 8 ? 8 : 16;
    // tiles of equal height: as many rounds of the grid as 128 rows need
    p.grid_rows = sms / p.nseg > 0 ? sms / p.nseg : 1;
    const int rounds = (N + tile::kTileRows * p.grid_rows - 1) / (tile::kTileRows * p.grid_rows);
    p.rows = ((N + p.grid_rows * rounds - 1) / (p.grid_rows * rounds) + 7) / 8 * 8;
    p.tiles = (N + p.rows - 1) / p.rows;
    if (p.grid_rows > p.tiles) p.grid_rows = p.tiles;
    // (with room for the bytes before the first where pieces may start off 16 bytes)
    const int slot = p.rows * tile::kSlotBytes;
    p.piece = (long long)N * R % 8 == 0 && R * 2 <= tile::kSlotBytes ? p.rows : (slot - 16) / (2 * R);
    if (p.piece > p.rows) p.piece = p.rows;
    // (whole rows of up to 96 groups where the ring's three slots still fit beside them)
    p.slots = tile::kGroups;
    p.sb_buffers = p.inner_buffers = 1;
    p.sb = tile::Affines::plan(p.G, p.range * slot_subs * 64 / gs, p.rows, 96);
    if (layout(p, bits, p.nc).total > kSmem) p.sb = tile::Affines::plan(p.G, p.range * slot_subs * 64 / gs, p.rows, 64);
    const size_t passes = (M + kPass - 1) / kPass;
    // passes side by side where one does not fill the card; the others one after the other
    p.grid_passes = sms / (p.grid_rows * p.nseg);
    if (p.grid_passes > int(passes)) p.grid_passes = int(passes);
    if (p.grid_passes < 1) p.grid_passes = 1;
    p.sb_buffers = rounds > 1 || int(passes) > p.grid_passes ? 2 : 1;
    sz.cells = up256(passes * p.subs * tile::cell_bytes(p.nc));
    sz.meta = up256(passes * p.subs * tile::meta_bytes(p.nc));
    sz.inner = up256(size_t(M) * inner_pitch(R) * 4);
    sz.counters = p.nseg > 1 ? up256(passes * ((N + 7) / 8) * 4) : 0;
    sz.partials = p.nseg > 1 ? up256(passes * p.nseg * size_t(N) * p.nc * 4) : 0;
    sz.total = sz.cells + sz.meta + sz.inner + sz.counters + sz.partials;
    return p;
}

// As many ring slots as fit, in threes (see qmv_tile.cuh); false where not even three do.
inline bool fit(LoraShape &p, int bits)
{
    p.slots = 2 * tile::kGroups;
    p.inner_buffers = p.M > kPass * p.grid_passes ? 2 : 1;
    if (layout(p, bits, p.nc).total > kSmem) p.sb_buffers = 1;
    if (layout(p, bits, p.nc).total > kSmem) p.inner_buffers = 1;
    p.slots = kMaxSlots;
    while (p.slots > tile::kGroups && layout(p, bits, p.nc).total > kSmem) p.slots -= tile::kGroups;
    // (whatever a pass brings to its inner vectors stays before the barriers)
    const Layout l = layout(p, bits, p.nc);
    return l.total <= kSmem && inner_at(p, l, 0) + l.inner_bytes <= l.bars && inner_at(p, l, 1) + l.inner_bytes <= l.bars;
}

}  // namespace lora
}  // namespace qmv
