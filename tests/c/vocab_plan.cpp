// Walks the plan of ar_vocab_loss and ar_vocab_loss_grad as their launches do.
// Reads calls, one a line (tokens, dim, dtype, row stride in bytes of hidden states and weights, pieces,
// rows of each piece), and prints for each what the launches write and the room there is:
//   bytes of statistics, bytes of their area; most rows packed at once, rows of room in the loss's plan;
//   the same of the gradient's plan; columns of D at most, columns of room; groups; 1 if the groups hold
//   every vocabulary row once and in order.
#include <cstdio>
#include <vector>

#include "ar_vocab_plan.h"

using namespace tps;
using namespace tps::plan;

namespace {

struct Walk {
    size_t tiles = 0, packed = 0, padded = 0, groups = 0;
    bool whole = true;
};

Walk walk(const ar_vocab *v, size_t cap, size_t tile) {
    Walk w;
    int piece = 0, at_piece = 0;
    size_t row = 0, at_row = 0;
    Group g;
    while (next_group(v, cap, piece, row, g)) {
        size_t rows = 0, padded = 0;
        ++w.groups;
        if (g.nseg < 1 || g.nseg > kMaxSegs) w.whole = false;
        for (int s = 0; s < g.nseg; ++s) {
            while (at_piece < v->n_pieces && at_row == v->piece_rows[at_piece]) ++at_piece, at_row = 0;
            if (g.piece[s] != at_piece || g.row0[s] != at_row || g.rows[s] == 0) w.whole = false;
            at_row += g.rows[s];
            rows += g.rows[s];
            padded += (g.rows[s] + kVN - 1) / kVN * kVN;
            w.tiles += (g.rows[s] + tile - 1) / tile;
        }
        if (padded != g.padded) w.whole = false;
        if (rows > w.packed) w.packed = rows;
        if (padded > w.padded) w.padded = padded;
    }
    while (at_piece < v->n_pieces && at_row == v->piece_rows[at_piece]) ++at_piece, at_row = 0;
    if (at_piece != v->n_pieces) w.whole = false;
    return w;
}

}  // namespace

int main() {
    size_t T, D, stride;
    int dtype, n;
    while (std::scanf("%zu %zu %d %zu %d", &T, &D, &dtype, &stride, &n) == 5) {
        std::vector<size_t> rows(static_cast<size_t>(n));
        for (size_t &r : rows)
            if (std::scanf("%zu", &r) != 1) return 1;
        std::vector<const void *> weights(static_cast<size_t>(n), reinterpret_cast<const void *>(4096));
        std::vector<int64_t> strides(static_cast<size_t>(n), static_cast<int64_t>(stride));
        ar_vocab v{};
        v.rows = T, v.dim = D, v.hidden = reinterpret_cast<const void *>(4096);
        v.hidden_row_bytes = static_cast<int64_t>(stride);
        v.n_pieces = n, v.piece_rows = rows.data(), v.weights = weights.data(), v.weight_row_bytes = strides.data();
        v.targets = reinterpret_cast<const int64_t *>(4096), v.dtype = dtype;
        const LossPlan p = plan_loss(&v);
        const bool few = T <= static_cast<size_t>(kFewTokens);
        const int height = few ? few_rows(&v, 8) : 0;
        const Walk w = walk(&v, p.cap, static_cast<size_t>(few ? 2 * height : stats_width(&v)));
        // a float pair for each token, each half of a tile, or each 32 rows of a CTA's share
        const size_t needed = w.tiles * static_cast<size_t>(few ? 2 * ((height + 31) / 32) : 2) * T * 8;
        const size_t packed_row = packed_ld(&v) * 2 * static_cast<size_t>(parts_of(&v));
        const bool pack = !weights_in_place(&v);
        const GradPlan q = plan_grad(&v);
        const Walk u = walk(&v, q.cap, kVN);
        const size_t d_col = q.d_rows * 2 * static_cast<size_t>(d_parts_of(&v));
        std::printf("%zu %zu %zu %zu %zu %zu %zu %zu %zu %d\n", needed, p.picked - p.part, pack ? w.packed : 0,
                    (p.bytes - p.weights) / packed_row, pack ? u.packed : 0, (q.sum - q.weights) / packed_row, u.padded,
                    (q.weights - q.d) / d_col, w.groups, w.whole && u.whole ? 1 : 0);
    }
    return 0;
}
