// Prints the plans of the norm and checkpoint calls.  Reads calls, one a line: columns, rows, bytes of an element, whether
// rows start on 32-byte boundaries, 16-byte vectors of a unit and row in the ring (v, for the backward pass: of dy, the
// kept sum and dsum together), bytes of a column in a row of the ring, whether strides fit 32 bits.  Prints
//   forward: U bx cluster threads warp smem; ring: U bx cluster threads warp smem stages blocks;
//   copied: U cluster threads smem stages blocks; rows of partial sums; pack: vectors per_row blocks; forward: blocks.
#include <cstdio>

#include "ar_norm_plan.h"

using namespace tps::plan;

int main() {
    unsigned long long ne0, ne1, es, bytes;
    int aligned, vecs, narrow;
    while (scanf("%llu %llu %llu %d %d %llu %d", &ne0, &ne1, &es, &aligned, &vecs, &bytes, &narrow) == 7) {
        const RowShape f = forward_shape(ne0, ne1, es, aligned);
        printf("%d %d %d %u %d %zu ", f.U, f.bx, f.cluster, f.threads, f.warp, f.smem);
        const size_t cols = aligned ? 32 / es : 8;
        const RowShape r = row_shape(ne0, ne1, cols, vecs, cols == 16 ? 1 : 2);
        printf("%d %d %d %u %d %zu %d %zu ", r.U, r.bx, r.cluster, r.threads, r.warp, r.smem, r.stages, r.U ? row_grid(r, ne1) : 0);
        const RowShape c = aligned ? copied_shape(ne0, ne1, es, bytes) : RowShape{};
        printf("%d %d %u %zu %d %zu ", c.U, c.cluster, c.threads, c.smem, c.stages, c.U ? row_grid(c, ne1) : 0);
        printf("%zu ", ring_blocks(ne0, ne1));
        Alignment al;
        al.bits = aligned ? 0 : es;
        al.narrow = narrow;
        const PackShape p = pack_shape(ne0, ne1, es, al);
        printf("%d %zu %zu %zu\n", p.vectors, p.per_row, p.blocks, f.U ? forward_grid(f, ne1) : 0);
    }
    return 0;
}
