// The plan of a vocabulary call on the host, without CUDA calls: tile sizes, the
// vocabulary's cut into launches, and the workspace.
#pragma once

#include "ar.h"

#include <cstddef>
#include <cstdint>

#include "ar_context.h"

namespace tps {

constexpr int kFewTokens = 64;  // up to here a tile is vocabulary rows by all tokens
constexpr int kMaxSegs = 16;
constexpr int kVM = 256;      // rows of a tile, 128 in each CTA
constexpr int kVN = 256;      // columns of a tile (at most), half of B's rows in each CTA
constexpr int kVK = 64;       // elements of the reduction per stage: 128 bytes

// Blocks of K that storing a tile of dW takes as long as: the least a dW tile counts for.
constexpr int kVStoreBlocks = 10;

// One counted token of a gradient call, in the order of the list.
struct VocabRow {
    float lse, g;   // g: dloss / max |dloss| of the finite ones (times 2^14 for f16)
    long long y;    // global vocabulary row of the target
};

// What the list kernel leaves for the others.
struct VocabList {
    int live;      // counted tokens
    float unscale; // what undoes the scaling of VocabRow::g
};

namespace plan {

// The gradient of the logits is held for one chunk of the vocabulary at a
// time, and packed rows likewise: as many rows as fit this many bytes, at
// least one tile.  (Packed rows get more room: a launch over a few thousand
// rows would leave most SMs without a tile.)
constexpr size_t kChunkBytes = 256ull << 20;
constexpr size_t kPackBytes = 2048ull << 20;
// Partial sums of dH that a split reduction may take.
constexpr size_t kSliceBytes = 64ull << 20;

struct Carve {  // hands out 256-byte aligned parts of the workspace
    size_t at = 0;
    size_t take(size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    }
};

inline size_t total_rows(const ar_vocab *v) {
    size_t n = 0;
    for (int r = 0; r < v->n_pieces; ++r) n += v->piece_rows[r];
    return n;
}

inline size_t row_bytes(int64_t given, const ar_vocab *v) {
    return given ? static_cast<size_t>(given) : v->dim * dtype_bytes(v->dtype);
}

inline size_t weight_stride(const ar_vocab *v, int r) { return row_bytes(v->weight_row_bytes ? v->weight_row_bytes[r] : 0, v); }

inline size_t matrix_bytes(size_t rows, size_t stride, const ar_vocab *v) {
    return rows ? (rows - 1) * stride + v->dim * dtype_bytes(v->dtype) : 0;
}

inline size_t round_up(size_t n, size_t to) { return (n + to - 1) / to * to; }
inline size_t tiles_of(size_t n, size_t tile) { return (n + tile - 1) / tile; }

inline int parts_of(const ar_vocab *v) { return v->dtype == AR_F32 ? 3 : 1; }

// Parts of D: 16-bit types hold it in one, in two with few tokens.
inline int d_parts_of(const ar_vocab *v) { return v->dtype == AR_F32 ? 3 : v->rows <= kFewTokens ? 2 : 1; }

// Rows that the tiled copies can read in place: 16-bit, starts and strides on 16-byte boundaries.
inline bool in_place(const void *p, size_t stride, const ar_vocab *v) {
    return v->dtype != AR_F32 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 16 == 0;
}

inline bool hidden_in_place(const ar_vocab *v) { return in_place(v->hidden, row_bytes(v->hidden_row_bytes, v), v); }

inline bool weights_in_place(const ar_vocab *v) {
    for (int r = 0; r < v->n_pieces; ++r)
        if (v->piece_rows[r] && !in_place(v->weights[r], weight_stride(v, r), v)) return false;
    return true;
}

// Elements between packed rows (of hidden states or weights): whole blocks of K, zeros behind the row's
// end, so that no copy of them reaches outside the tensor.
inline size_t packed_ld(const ar_vocab *v) { return round_up(v->dim, kVK); }

// One launch's vocabulary: whole pieces, or rows [row0, row0 + rows) of one that is larger than a chunk.
struct Group {
    int nseg = 0;
    int piece[kMaxSegs];
    size_t row0[kMaxSegs], rows[kMaxSegs];
    size_t padded = 0;  // rows, each segment rounded up to whole tiles
    bool begins = true, ends = true;  // its pieces' first and last rows are here
};

// The next group of at most `cap` padded rows from (piece, row); false when the vocabulary is done.
inline bool next_group(const ar_vocab *v, size_t cap, int &piece, size_t &row, Group &g) {
    g = Group{};
    while (piece < v->n_pieces) {
        const size_t left = v->piece_rows[piece] - row;
        if (left == 0) {
            ++piece, row = 0;
            continue;
        }
        const size_t padded = round_up(left, kVN);
        if (row || (g.nseg == 0 && padded > cap)) {  // part of a large piece, alone
            g.piece[0] = piece;
            g.row0[0] = row;
            g.rows[0] = left < cap ? left : cap;
            g.padded = round_up(g.rows[0], kVN);
            g.nseg = 1;
            g.begins = row == 0;
            row += g.rows[0];
            g.ends = row == v->piece_rows[piece];
            return true;
        }
        if (g.padded + padded > cap) return true;
        g.piece[g.nseg] = piece;
        g.row0[g.nseg] = 0;
        g.rows[g.nseg++] = left;
        g.padded += padded;
        ++piece;
    }
    return g.nseg > 0;
}

// Vocabulary rows of a group, a multiple of the tile, when each takes `bytes_per_row`.
inline size_t group_cap(size_t bytes, size_t bytes_per_row) {
    const size_t n = bytes / (bytes_per_row ? bytes_per_row : 1) / kVN * kVN;
    return n < kVN ? static_cast<size_t>(kVN) : n;
}

inline size_t padded_vocab(const ar_vocab *v) {
    size_t n = 0;
    for (int r = 0; r < v->n_pieces; ++r) n += round_up(v->piece_rows[r], kVN);
    return n;
}

constexpr size_t kPairs = 76;  // of SMs on a GB300: what the plans are made for

// Columns of a kStats tile, a multiple of 16 and at least half a tile: the width that makes the rounds of one
// tile a pair cheapest.  With one tile row a round is bound by reading W and takes as long as its width and some
// 56 columns more (one token of 4096 elements: 22.7 us at 256 columns, 20.0 at 224, 15.7 at 176, 13.4 at 128;
// 32768 rows 50.2 us at 224, 52.6 at 256 and 61.7 at 128); with more tile rows it is bound by the products,
// and narrow tiles copy more of H for each.
inline int stats_width(const ar_vocab *v) {
    const size_t mt = tiles_of(v->rows, kVM), fixed = mt > 1 ? 24 : 56;
    size_t best = SIZE_MAX;
    int bn = kVN;
    for (int n = kVN; n >= kVN / 2; n -= 16) {
        size_t tiles = 0;
        for (int r = 0; r < v->n_pieces; ++r) tiles += tiles_of(v->piece_rows[r], static_cast<size_t>(n));
        const size_t cost = tiles_of(tiles * mt, kPairs) * (static_cast<size_t>(n) + fixed);
        if (cost < best) best = cost, bn = n;
    }
    return bn;
}

// Few tokens: vocabulary rows of a tile in each CTA, a multiple of `step`, so that the rounds of one tile a pair are
// cheapest (a round costs its rows and some 24 more).
inline int few_rows(const ar_vocab *v, int step) {
    size_t best = SIZE_MAX;
    int rows = 128;
    for (int n = 128; n >= 32; n -= step) {
        size_t tiles = 0;
        for (int r = 0; r < v->n_pieces; ++r) tiles += tiles_of(v->piece_rows[r], static_cast<size_t>(2 * n));
        const size_t cost = tiles_of(tiles, kPairs) * static_cast<size_t>(2 * n + 24);
        if (cost < best) best = cost, rows = n;
    }
    return rows;
}

// Tiles of the statistics.
struct StatsTile {
    int bn, few_rows;  // of the launch; few_rows: with few tokens, else 0
    size_t rows;       // vocabulary rows
    size_t parts;      // statistics that a tile leaves for a token: of each half of its columns, or (few tokens) of
                       // every 32 vocabulary rows of each CTA
};

inline StatsTile stats_tile(const ar_vocab *v) {
    if (v->rows > kFewTokens) {
        const int bn = stats_width(v);
        return StatsTile{bn, 0, static_cast<size_t>(bn), 2};
    }
    const int n = few_rows(v, 8);
    return StatsTile{static_cast<int>(round_up(v->rows, 16)), n, static_cast<size_t>(2 * n), 2 * tiles_of(static_cast<size_t>(n), 32)};
}

struct LossPlan {
    StatsTile tile;
    size_t cap;    // vocabulary rows of a group
    size_t parts;  // statistics of a token
    size_t part, picked, hidden, weights, bytes;
};

inline LossPlan plan_loss(const ar_vocab *v) {
    LossPlan p{};
    p.tile = stats_tile(v);
    const size_t row = packed_ld(v) * 2 * static_cast<size_t>(parts_of(v));
    const bool pack = !weights_in_place(v);
    const size_t all = padded_vocab(v);
    p.cap = pack && group_cap(kPackBytes, row) < all ? group_cap(kPackBytes, row) : all;
    // counted group by group, as the launches are: each cut of a piece may leave one more tile, because `cap` is no
    // multiple of a tile's rows
    int piece = 0;
    size_t at = 0;
    Group g;
    while (next_group(v, p.cap, piece, at, g))
        for (int s = 0; s < g.nseg; ++s) p.parts += p.tile.parts * tiles_of(g.rows[s], p.tile.rows);
    Carve c;
    p.part = c.take(p.parts * v->rows * 2 * sizeof(float));
    p.picked = c.take(v->rows * sizeof(float));
    p.hidden = c.take(hidden_in_place(v) ? 0 : v->rows * row);
    p.weights = c.take(pack ? p.cap * row : 0);
    p.bytes = c.at;
    return p;
}

struct GradPlan {
    size_t cap;         // vocabulary rows of a group
    size_t d_rows;      // tokens, whole tiles
    size_t k_rows;      // tokens, whole blocks of K
    int slices;         // of dH's reductions
    bool sums;          // dH goes through partial sums
    size_t list, row, index, place, hidden, d, weights, sum, bytes;
};

inline GradPlan plan_grad(const ar_vocab *v) {
    GradPlan p{};
    const size_t parts = static_cast<size_t>(parts_of(v)), d_parts = static_cast<size_t>(d_parts_of(v));
    const size_t row = packed_ld(v) * 2 * parts;
    p.d_rows = round_up(v->rows, kVM);
    p.k_rows = round_up(v->rows, kVK);
    const bool pack = !weights_in_place(v);
    const size_t all = padded_vocab(v);
    size_t cap = group_cap(kChunkBytes, p.d_rows * 2 * d_parts);
    if (pack && group_cap(kPackBytes, row) < cap) cap = group_cap(kPackBytes, row);
    p.cap = cap < all ? cap : all;
    // The dH tiles reduce over the vocabulary, the dW tiles over the tokens.  Where one dH tile would take
    // more than a pair's share of all blocks of K, its reduction is cut into slices of half a share (none
    // shorter than eight blocks), whose partial sums (kSliceBytes at most) a last kernel adds.
    size_t longest = 0, blocks = 0;
    int segs = 0;
    const size_t nt = tiles_of(v->dim, kVN), mt = p.d_rows / kVM, kw = tiles_of(v->rows, kVK);
    for (int r = 0; r < v->n_pieces; ++r) {
        const size_t n = v->piece_rows[r];
        longest = n > longest ? n : longest;
        segs += n != 0;
        blocks += nt * (mt * tiles_of(n, kVK) + tiles_of(n, kVM) * (kw < kVStoreBlocks ? kVStoreBlocks : kw));
    }
    const bool split = round_up(longest, kVN) > p.cap;
    if (split) blocks = blocks / (longest / p.cap + 1), longest = p.cap;
    const size_t share = blocks / kPairs + 1, tile = tiles_of(longest, kVK);
    const size_t slice = p.d_rows * round_up(v->dim, 8) * sizeof(float) * static_cast<size_t>(segs ? segs : 1);
    size_t s = 1;
    if (tile > share) s = tiles_of(tile, share / 2 < 8 ? 8 : share / 2);
    if (s > kSliceBytes / (slice + 1)) s = kSliceBytes / (slice + 1);
    p.slices = s < 2 ? 1 : static_cast<int>(s);
    p.sums = split || p.slices > 1;
    Carve c;
    p.list = c.take(sizeof(VocabList));
    p.row = c.take(v->rows * sizeof(VocabRow));
    p.index = c.take(v->rows * sizeof(int));
    p.place = c.take(v->rows * sizeof(int));
    p.hidden = c.take(p.k_rows * row);
    p.d = c.take(p.d_rows * p.cap * 2 * d_parts);
    p.weights = c.take(pack ? p.cap * row : 0);
    p.sum = c.take(p.sums ? static_cast<size_t>(p.slices) * slice : 0);
    p.bytes = c.at;
    return p;
}

}  // namespace plan
}  // namespace tps
