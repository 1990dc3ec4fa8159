// The plans of ar_reduce_norm, ar_reduce_norm_grad and the checkpoint calls: which form a call takes and how it lies over
// blocks and threads.  Host code that reads no device memory, apart from the launches so that tests can walk it.
#pragma once

#include <cstddef>
#include <cstdint>

namespace tps {

constexpr int kRowBlocks = 8;      // most blocks of a cluster along a row
constexpr int kRowThreads = 512;   // of the backward pass, at most
constexpr int kNormThreads = 128;  // of the forward pass

namespace plan {

// How a row lies over threads: `bx` lanes of a warp (warp), or the threads of `cluster` blocks, each with U units of
// eight columns; `vecs` vectors of a unit and row in the ring, `stages` rows deep.
struct RowShape {
    bool warp;
    int U, bx, cluster, stages, vecs;  // U = 0: too long
    unsigned threads;
    int resident;  // blocks on an SM
    size_t smem;
};

// Dynamic shared memory of each of n blocks on an SM, next to 2 KB of their own and 1 KB of the system's.
constexpr size_t ring_bytes(size_t n) { return 227 * 1024 / n - 3 * 1024; }
constexpr size_t kSMs = 152;

// `cols`: columns of a unit; vecs: its 16-byte vectors in a row of the ring; `most_u`: the most units of a thread.
inline RowShape row_shape(size_t ne0, size_t ne1, size_t cols, int vecs, int most_u) {
    const size_t units = (ne0 + cols - 1) / cols;
    RowShape s{};
    s.cluster = 1;
    s.vecs = vecs;
    if (units <= 32 * static_cast<size_t>(most_u)) {
        s.warp = true;
        s.threads = 256;
        s.U = units <= 32 ? 1 : 2;
        s.bx = 32;
        while (s.bx > 4 && static_cast<size_t>(s.bx) / 2 >= units) s.bx /= 2;
    } else {
        auto share = [&] { return (units + s.cluster - 1) / s.cluster; };
        auto bytes = [&] { return share() * 16 * static_cast<size_t>(vecs); };
        auto fits = [&](size_t rows) {
            return share() <= static_cast<size_t>(kRowThreads) * most_u && bytes() * rows <= ring_bytes(1);
        };
        while (s.cluster < kRowBlocks && !fits(2)) s.cluster *= 2;
        if (!fits(1)) return s;
        // few rows: the blocks that would be idle share them
        while (s.cluster < kRowBlocks && ne1 * s.cluster * 2 <= kSMs && share() >= 128) s.cluster *= 2;
        s.U = share() <= 128 ? 1 : most_u;
        s.threads = static_cast<unsigned>(((share() + s.U - 1) / s.U + 31) / 32 * 32);
        s.bx = static_cast<int>(s.threads);
    }
    // two rows in the ring at least, if blocks have to go for it; four at most
    const size_t row = static_cast<size_t>(s.threads) * s.U * 16 * vecs;
    s.resident = static_cast<int>(kRowThreads / s.threads);
    while (s.resident > 1 && row * 2 > ring_bytes(s.resident)) --s.resident;
    const size_t rows = ring_bytes(s.resident) / row;
    s.stages = static_cast<int>(rows < 1 ? 1 : rows > 4 ? 4 : rows);
    s.smem = row * s.stages;
    if (s.smem > ring_bytes(1)) s.U = 0;
    return s;
}

// The same for rows that the copy engine brings: 16 columns a thread, `bytes` of a column in a row of the ring.  U = 0:
// too short or too long.
inline RowShape copied_shape(size_t ne0, size_t ne1, size_t es, size_t bytes) {
    RowShape s{};
    // few rows gain nothing from copies ahead, and a copy takes longer to start (one row of 4096 floats: 4.2 us, by
    // copies 6.7)
    if (ne0 <= 512 || ne1 < kSMs) return s;
    s.cluster = 1;
    const size_t vectors = (ne0 * es + 15) / 16, units = 16 * es / 16;  // a thread's vectors
    auto share = [&] { return (vectors + s.cluster - 1) / s.cluster; };
    auto threads = [&] { return ((share() + units - 1) / units + 31) / 32 * 32; };
    auto fits = [&](size_t rows) { return threads() <= kRowThreads && threads() * 16 * bytes * rows <= ring_bytes(1); };
    while (s.cluster < kRowBlocks && !fits(2)) s.cluster *= 2;
    if (!fits(2)) return s;
    s.threads = static_cast<unsigned>(threads());
    s.U = static_cast<int>(units);
    s.bx = static_cast<int>(s.threads);
    const size_t row = s.threads * 16 * bytes;
    s.resident = static_cast<int>(kRowThreads / s.threads);
    if (s.resident > 8) s.resident = 8;
    while (s.resident > 1 && row * 2 > ring_bytes(s.resident)) --s.resident;
    const size_t rows = ring_bytes(s.resident) / row;
    s.stages = static_cast<int>(rows > 4 ? 4 : rows);
    s.smem = row * s.stages;
    return s;
}

// Blocks of a launch over ne1 rows, whole clusters.
inline size_t row_grid(const RowShape &s, size_t ne1) {
    const size_t turn = s.warp ? s.threads / s.bx : 1;
    const size_t most = kSMs * s.resident / s.cluster;
    const size_t groups = (ne1 + turn - 1) / turn;
    return (groups < most ? groups : most) * s.cluster;
}

// Rows of partial column sums: of the element-wise form (64 rows or more each) and at most of the other.
inline size_t any_rows(size_t ne1) {
    const size_t rows = (ne1 + 303) / 304;
    return rows < 64 ? 64 : rows;
}
inline size_t any_blocks(size_t ne1) { return (ne1 + any_rows(ne1) - 1) / any_rows(ne1); }
inline size_t ring_blocks(size_t ne0, size_t ne1) {
    // 512 threads of at most 16 columns on an SM
    const size_t most = kSMs * (ne0 <= 512 ? 2 : (8192 + ne0 - 1) / ne0);
    return ne1 < most ? ne1 : most;
}
inline size_t part_ld(size_t n) { return (n + 15) / 16 * 16; }  // whole units of 16 columns

// How the forward pass lays a row over threads; U = 0: too long.
inline RowShape forward_shape(size_t ne0, size_t ne1, size_t es, bool aligned) {
    const size_t cols = aligned ? 32 / es : 8, units = (ne0 + cols - 1) / cols;
    RowShape s{};
    s.cluster = 1;
    s.threads = kNormThreads;
    auto share = [&] { return (units + s.cluster - 1) / s.cluster; };
    if (units <= 128) {
        s.warp = true;
        s.threads = 128;
        s.bx = 32;
        while (s.bx > 4 && static_cast<size_t>(s.bx) / 2 >= units) s.bx /= 2;
    } else {
        // few rows: the blocks that would be idle share them
        while (s.cluster < kRowBlocks && ne1 * s.cluster * 2 <= kSMs && share() >= 128) s.cluster *= 2;
        while (s.cluster < kRowBlocks && share() * cols * es > 16 * 1024) s.cluster *= 2;
        s.bx = static_cast<int>(s.threads);
    }
    s.U = static_cast<int>((share() + s.bx - 1) / s.bx);
    s.smem = static_cast<size_t>(s.threads) * s.U * cols * es;
    if (s.smem > ring_bytes(1)) s.U = 0;
    return s;
}

// Its blocks: every block takes one turn of rows.
inline size_t forward_grid(const RowShape &s, size_t ne1) {
    const size_t turn = s.warp ? s.threads / s.bx : 1;
    return (ne1 + turn - 1) / turn * s.cluster;
}

// What the row starts of a call's buffers have in common.
struct Alignment {
    uintptr_t bits = 0;
    bool narrow = true;  // strides of 32 bits, and row numbers that stay below them a grid further on
    void add(const void *p, long long stride, size_t rows) {
        if (p && rows > 1 && (stride > 0xFFFFFFFFll || rows > 0x3FFFFFFFull)) narrow = false;
        bits |= reinterpret_cast<uintptr_t>(p) | (rows > 1 ? static_cast<uintptr_t>(stride) : 0);
    }
};

// The checkpoint calls' vectors: columns of a thread's unit, units of a row (whole blocks of 32 columns), and blocks of 256
// threads; element by element where rows, strides or the grid pass 32 bits.
struct PackShape {
    bool vectors, aligned;
    size_t per_row, blocks;
};
inline PackShape pack_shape(size_t ne0, size_t ne1, size_t es, const Alignment &al) {
    PackShape s{};
    s.aligned = al.bits % 32 == 0;
    const size_t cols = s.aligned ? 32 / es : 8, lanes = 32 / cols;
    s.per_row = ((ne0 + cols - 1) / cols + lanes - 1) / lanes * lanes;
    s.blocks = (s.per_row * ne1 + 255) / 256;
    s.vectors = al.narrow && ne0 <= 0x7FFFFFFF && s.blocks <= 0x7FFFFFFF;
    return s;
}

}  // namespace plan
}  // namespace tps
