// The launch plan of qmv_attend_run: tiles, what lies where in shared memory and in
// the workspace, and the division of keys into pages. Code without a CUDA call, so that
// it can be checked without a GPU.
#pragma once

#include <cstddef>
#include <cstdint>

#include "qmv.h"

#ifdef __CUDACC__
#define QMV_BOTH __host__ __device__ __forceinline__
#else
#define QMV_BOTH inline
#endif

namespace qmv {
namespace attend {

// The page of a key, key / page_size, for keys that are multiples of 8. Page sizes are multiples
// of 8 too, so eighths are divided: with e = page_size / 8 up to 2^13 the magic number is
// (2^37 + r) / e, r < e, and n r < 2^37 for n eighths below 2^24, so that r adds less than 1 / e to
// the quotient; the product stays below 2^62. (That of whole keys and a magic number for them
// passes 64 bits from key 2^25 on, with pages of 8.)
inline uint64_t page_magic(int page_size)
{
    const uint64_t e = uint64_t(page_size) / 8;
    return ((uint64_t(1) << 37) + e - 1) / e;
}
QMV_BOTH int page_of(uint64_t magic, int key) { return int(uint64_t(unsigned(key) >> 3) * magic >> 37); }

constexpr int kFew = QMV_TILE_M;  // new tokens of a sequence up to which they share one read of its keys
constexpr int kLeaf = 256;        // keys whose weights are formed at once: two tiles of 128
constexpr int kChunk = 16384;     // bytes of a ring slot
constexpr int kSmemSm = 228 * 1024, kSmemBlock = 227 * 1024, kSmemReserved = 1024;

// Work items of sequences of a few new tokens: query rows of one kv head are the
// columns of a tile, `tokens` of a sequence at a time.
struct FewPlan {
    int columns;  // 16, 32 or 64
    int tokens;   // new tokens of an item at most
    int blocks;   // items of one kv head and unit
    int rows;     // columns in use: tokens * group
    int slots, key_slots, ctas;  // ring slots, those of keys; blocks of an SM
    int q_sets;                  // items whose queries are held
    int p_off, q_off, misc_off, smem;
    int unit;     // keys of one item, from a multiple of it on
    int units;    // of a sequence at most
    int64_t items;
    bool by_row;  // where a token's sums lie: by its row of q, or by its sequence's place
    int kept;     // tokens whose sums the workspace has room for
    size_t meta_off, parts_off, workspace;
};

inline size_t up256(size_t b) { return (b + 255) & ~size_t(255); }

// What lies before the sequences in shared memory: barriers, columns' maxima, sums and places.
constexpr int few_misc(int columns) { return 512 + columns * 64; }
constexpr int kPromptMisc = 512;

// Fixed shared memory behind the ring: weights of a leaf (two bf16 terms), two items' queries,
// then barriers, maxima, sums and the sequences.
inline void few_smem(FewPlan &f, int D, int B, bool alone)
{
    f.q_sets = D == 256 && f.columns == 64 ? 1 : 2;
    const int p_bytes = kLeaf * f.columns * 4, q_bytes = f.q_sets * f.columns * D * 2;
    const int misc = few_misc(f.columns) + B * 16 + (B + 1) * 4;
    const int fixed = p_bytes + q_bytes + ((misc + 1023) & ~1023);
    // (a tile's values, D / 64 slots, have to be there at once: see the zeroing of unseen rows)
    const int least = D / 64 + 2 > 5 ? D / 64 + 2 : 5, two = (kSmemSm / 2 - kSmemReserved - 1024 - fixed) / kChunk;
    f.ctas = f.columns == 16 && two >= least && !alone ? 2 : 1;
    f.slots = f.ctas == 2 ? two : (kSmemBlock - 1024 - fixed) / kChunk;
    if (f.slots > 11) f.slots = 11;
    f.key_slots = f.slots / 2 < f.slots - D / 64 ? f.slots / 2 : f.slots - D / 64;
    f.p_off = f.slots * kChunk;
    f.q_off = f.p_off + p_bytes;
    f.misc_off = f.q_off + q_bytes;
    f.smem = f.slots * kChunk + fixed + 1024;  // (1024: to align the ring)
}

// Work items of longer sequences: two tiles of 128 query rows (one of head_dim 256) over
// the tiles of 128 keys that they see, or over one of `pieces` parts of them.
struct PromptPlan {
    int tokens;  // of a tile: as many as their heads of one kv head fit 128 rows
    int streams, slots, chunk;
    int key_slots;  // those of keys
    int q_off, misc_off, smem;
    int pieces;
    int64_t items;
    size_t prefix_off, meta_off, parts_off, workspace;
};

inline PromptPlan prompt_plan(int B, int T, int max_new, int heads, int kv_heads, int D, int64_t capacity, int window, int sinks)
{
    PromptPlan f{};
    if (max_new <= kFew) return f;
    f.tokens = 128 / (heads / kv_heads);
    f.streams = D == 256 ? 1 : 2;
    f.chunk = D == 64 ? 16384 : 32768;
    const int q_bytes = f.streams * 128 * D * 2, misc = (kPromptMisc + B * 16 + (B + 1) * 4 + 1023) & ~1023;
    f.slots = (kSmemBlock - 1024 - q_bytes - misc) / f.chunk;
    // (keys run four tiles ahead at most, and PromptShared knows of the last eight tiles)
    if (f.slots > (D == 64 ? 8 : 12)) f.slots = D == 64 ? 8 : 12;
    f.key_slots = (f.slots + 1) / 2;
    f.q_off = f.slots * f.chunk;
    f.misc_off = f.q_off + q_bytes;
    f.smem = f.misc_off + misc + 1024;
    // sequences of more than kFew tokens, their last items not whole
    const int each = f.streams * f.tokens, sequences = T / (kFew + 1) < B ? T / (kFew + 1) : B;
    const int64_t tiles = int64_t(T / each + sequences) * kv_heads;
    // enough parts that four rounds of items fill 152 SMs, of 1024 keys at least
    int64_t keys = capacity;
    if (window && int64_t(window) + each + sinks < keys) keys = int64_t(window) + each + sinks;
    int64_t pieces = tiles > 0 ? (4 * 152 + tiles - 1) / tiles : 1;
    if (pieces > (keys + 1023) / 1024) pieces = (keys + 1023) / 1024;
    f.pieces = int(pieces < 1 ? 1 : pieces);
    f.items = tiles * f.pieces;
    f.prefix_off = 0;
    f.meta_off = up256(size_t(B + 1) * 4);
    const size_t rows = f.pieces > 1 ? size_t(f.items) * f.streams * 128 : 0;
    f.parts_off = f.meta_off + up256(rows * 8);
    f.workspace = f.parts_off + up256(rows * D * 4);
    return f;
}

// The workspace of `rows` tokens: sums of each token, unit and head.
inline void few_sums(FewPlan &f, int64_t rows, int heads, int D)
{
    const size_t sums = size_t(rows) * f.units * heads;
    f.kept = int(rows);
    f.meta_off = 0;
    f.parts_off = up256(sums * 8);
    f.workspace = f.units > 1 ? f.parts_off + up256(sums * D * 4) : 256;  // (0 would be a refusal)
}

// (whatever T is)
inline FewPlan few_plan(int B, int max_new, int heads, int kv_heads, int D, int64_t capacity, int window, int sinks)
{
    FewPlan f{};
    const int group = heads / kv_heads, most = max_new < kFew ? max_new : kFew;
    const int rows = most * group;
    f.columns = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    f.tokens = f.columns / group < most ? f.columns / group : most;
    f.blocks = (most + f.tokens - 1) / f.tokens;
    f.rows = f.tokens * group;
    // An item is two leaves; one where that makes a sequence no more items than a card has
    // SMs (one token over 4100 keys: 12.2 us with two, 11.7 with one), four where it makes
    // it eight times as many (13 tokens over 131000 keys: 119 us with two, 95 with four). By
    // the longest sequence that the call has room for, not by how long they are nor by how
    // many there are, so that a row's sums keep their order from call to call. Of a window
    // one or two make little difference for single tokens (1024 keys of 8 kv heads, 1 and 32
    // sequences: 11.3 and 40.4 us with one, 11.4 and 40.4 with two; 4096 keys, 8 sequences: 33.8 and
    // 34.3), but 32 sequences of 5 tokens take 63.3 with one and 59.0 with two.
    const int64_t sees = window && int64_t(window) + sinks + kFew < capacity ? int64_t(window) + sinks + kFew : capacity;
    const int64_t leaves = (sees + kLeaf - 1) / kLeaf * kv_heads;
    f.unit = leaves <= 152 ? kLeaf : leaves <= 8 * 152 ? 2 * kLeaf : 4 * kLeaf;
    int64_t units = (capacity + f.unit - 1) / f.unit;
    if (window) {
        // the units of window + most - 1 keys, and those of the first tokens
        const int64_t near = (int64_t(window) + most - 1 + f.unit - 2) / f.unit + 1, first = (int64_t(sinks) + f.unit - 1) / f.unit;
        if (near + first < units) units = near + first;
    }
    f.units = int(units);
    f.items = int64_t(B) * kv_heads * f.blocks * units;
    // (a ring that holds a whole leaf where every item has an SM for itself)
    few_smem(f, D, B, f.items <= 152);
    f.by_row = false;
    few_sums(f, int64_t(B) * f.blocks * f.tokens, heads, D);
    return f;
}

// The plan of a call of T rows. Their number bounds what sequences of few tokens have, and kFew for
// each sequence does: 255 sequences of one token and a prompt of 512 rows are 767 rows and not
// 4096 (keys for 131072 of them, 40 heads of 128: 2.0 GB of sums, not 16).
inline FewPlan few_plan(int B, int T, int max_new, int heads, int kv_heads, int D, int64_t capacity, int window, int sinks)
{
    FewPlan f = few_plan(B, max_new, heads, kv_heads, D, capacity, window, sinks);
    const int64_t most = int64_t(B) * (max_new < kFew ? max_new : kFew);
    f.by_row = T <= most;
    few_sums(f, f.by_row ? T : most, heads, D);
    return f;
}

}  // namespace attend
}  // namespace qmv
