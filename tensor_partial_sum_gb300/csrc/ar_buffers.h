// Overlap checks of calls with many buffers.
#pragma once

#include "ar_context.h"

namespace tps {

// The byte spans of a call's buffers: outputs may overlap neither each other nor an input.
class Buffers {
public:
    void input(const void *p, size_t n) { add(p, n, false); }
    void output(const void *p, size_t n) { add(p, n, true); }
    bool clash() const {
        for (int i = 0; i < n_; ++i)
            for (int j = 0; j < i; ++j)
                if ((b_[i].out || b_[j].out) && spans_overlap(b_[i].p, b_[i].n, b_[j].p, b_[j].n)) return true;
        return false;
    }
    // Whether a span of this set overlaps one of the other's.
    bool meets(const Buffers &other) const {
        for (int i = 0; i < n_; ++i)
            for (int j = 0; j < other.n_; ++j)
                if (spans_overlap(b_[i].p, b_[i].n, other.b_[j].p, other.b_[j].n)) return true;
        return false;
    }

private:
    struct Span {
        const void *p;
        size_t n;
        bool out;
    };
    Span b_[64];
    int n_ = 0;
    void add(const void *p, size_t n, bool out) {
        if (p && n && n_ < 64) b_[n_++] = Span{p, n, out};
    }
};

// Bytes from the first element of `rows` rows to the end of the last.
inline size_t rows_bytes(size_t rows, size_t stride, size_t row) { return rows ? (rows - 1) * stride + row : 0; }

// Whether rows of `row` bytes at `stride` from p on stay apart and inside the address space.
inline bool rows_fit(const void *p, size_t rows, int64_t stride, size_t row) {
    if (rows <= 1) return row <= UINTPTR_MAX - reinterpret_cast<uintptr_t>(p);
    if (stride < 0 || static_cast<uint64_t>(stride) < row) return false;
    const unsigned __int128 n = static_cast<unsigned __int128>(rows - 1) * static_cast<uint64_t>(stride) + row;
    return n <= UINTPTR_MAX - reinterpret_cast<uintptr_t>(p);
}

}  // namespace tps
