// Host side of ar_reduce_dropout and ar_reduce_dropout_grad: checks, launch
// shapes and launches.  The operation is specified in include/ar.h.
#include "ar.h"

#include <cstring>

#include "ar_context.h"
#include "ar_kernels_dropout.cuh"

using tps::dtype_bytes;
using tps::launched;
using tps::spans_overlap;

namespace {

// Threads of a block: bx along a row (eight columns each) by `by` row groups.
struct Shape {
    int bx, by;
    unsigned gx;       // blocks along a row
    unsigned threads;
};

// Short rows share a block; long rows are cut into blocks of the width (half to all of `widest`) that
// leaves the fewest threads idle.
Shape block_shape(size_t ne0, int threads, int widest) {
    const size_t units = (ne0 + tps::kDropCols - 1) / tps::kDropCols;
    Shape s{};
    if (units <= static_cast<size_t>(widest)) {
        s.bx = static_cast<int>(units < 1 ? 1 : units);
    } else {
        size_t best = 0;
        for (int t = widest; t >= widest / 2; t -= 32) {
            const size_t cover = (units + t - 1) / t * t;
            if (best == 0 || cover < best) best = cover, s.bx = t;
        }
    }
    s.by = threads / s.bx;
    s.gx = static_cast<unsigned>((units + s.bx - 1) / s.bx);
    s.threads = static_cast<unsigned>((s.bx * s.by + 31) / 32 * 32);
    return s;
}

// Forward: eight blocks of 128 threads an SM (64 registers); 256 x 4: 28.4 us against 27.7 at f32 [2048, 4096] x
// (2 + 2), 103.6 against 101.5 at bf16 [4096, 8192] x (4 + 4); 512 x 2: 29.6, 108.5.
constexpr int kForwardThreads = 128;
// Backward: two blocks of 512 threads fill an SM, and 64 threads along a row leave eight row groups, whose
// sums meet in the block.  Measured with a bias gradient at bf16 [4096, 8192] x 4, f32 [2048, 4096] x 2 and
// f16 [1021, 4099]: 61.5, 20.9 and 10.9 us; 128 threads along a row 61.7, 20.3, 12.9; three or four blocks of
// 256 threads an SM 67.3, 22.2, 16.2 and 62.0, 21.0, 15.2.
constexpr int kGradThreads = 512;
constexpr int kGradWidest = 64;
constexpr int kGradBlocks = 304;  // two on each of 152 SMs

Shape forward_shape(size_t ne0) { return block_shape(ne0, kForwardThreads, kForwardThreads); }
Shape grad_shape(size_t ne0) { return block_shape(ne0, kGradThreads, kGradWidest); }

// Rows of a block of the backward pass.  With column sums, as many as leave just enough blocks to fill the
// GPU once, because each block leaves ne0 partial sums; without, two for each of
// its row groups.
unsigned rows_per_block(const ar_layout *L, int n_sums) {
    const Shape s = grad_shape(L->ne0);
    const size_t turn = static_cast<size_t>(s.by);
    size_t rows = 2 * turn;
    if (n_sums) {
        const size_t blocks = s.gx < kGradBlocks ? kGradBlocks / s.gx : 1;
        rows = (L->ne1 + blocks - 1) / blocks;
    }
    // the grid's second dimension has 65535 blocks
    const size_t least = L->ne1 / 65535 + 1;
    if (rows < least) rows = least;
    return static_cast<unsigned>((rows + turn - 1) / turn * turn);
}

unsigned row_blocks(const ar_layout *L, int n_sums) {
    const size_t r = rows_per_block(L, n_sums);
    return static_cast<unsigned>((L->ne1 + r - 1) / r);
}

// Bytes from the first element of a strided tensor to the end of its last row.
size_t span_bytes(const ar_layout *L, const int64_t *rows, int k, size_t es) {
    const size_t stride = rows ? static_cast<size_t>(rows[k]) : L->ne0 * es;
    return (L->ne1 > 1 ? (L->ne1 - 1) * stride : 0) + L->ne0 * es;
}

int check_drop(const ar_layout *L, const ar_dropout *drop) {
    if (!drop || !(drop->p >= 0.0f && drop->p <= 1.0f)) return AR_ERR_INVALID_ARG;
    if (L->ne1 > 0xFFFFFFFFull || L->ne0 > (1ull << 34)) return AR_ERR_TOO_LARGE;  // counter words
    return AR_OK;
}

tps::DropParams drop_params(const ar_dropout &d) {
    tps::DropParams p;
    p.keys = tps::philox_keys(d.seed);
    p.off_lo = static_cast<uint32_t>(d.offset);
    p.off_hi = static_cast<uint32_t>(d.offset >> 32);
    const double t = static_cast<double>(d.p) * 4294967296.0;
    p.any = t < 4294967296.0;
    p.threshold = p.any ? static_cast<uint32_t>(t) : 0xFFFFFFFFu;
    p.scale = p.any ? 1.0f / (1.0f - d.p) : 0.0f;
    return p;
}

using DropFn = void (*)(tps::ArDropParams);
using GradFn = void (*)(tps::ArDropGradParams);

template <int Td, bool ALIGNED>
DropFn pick_wire(int wire) {
    return wire == AR_F32   ? tps::ar_dropout_kernel<Td, tps::kF32, ALIGNED>
           : wire == AR_F16 ? tps::ar_dropout_kernel<Td, tps::kF16, ALIGNED>
                            : tps::ar_dropout_kernel<Td, tps::kBF16, ALIGNED>;
}

template <bool ALIGNED>
DropFn pick_types(int dst, int wire) {
    return dst == AR_F32   ? pick_wire<tps::kF32, ALIGNED>(wire)
           : dst == AR_F16 ? pick_wire<tps::kF16, ALIGNED>(wire)
                           : pick_wire<tps::kBF16, ALIGNED>(wire);
}

template <int Td, bool ALIGNED>
GradFn pick_sums(int sums) {
    return sums == 0   ? tps::ar_dropout_grad_kernel<Td, ALIGNED, 0>
           : sums == 1 ? tps::ar_dropout_grad_kernel<Td, ALIGNED, 1>
           : sums == 2 ? tps::ar_dropout_grad_kernel<Td, ALIGNED, 2>
                       : tps::ar_dropout_grad_kernel<Td, ALIGNED, 3>;
}

template <bool ALIGNED>
GradFn pick_grad(int dst, int sums) {
    return dst == AR_F32   ? pick_sums<tps::kF32, ALIGNED>(sums)
           : dst == AR_F16 ? pick_sums<tps::kF16, ALIGNED>(sums)
                           : pick_sums<tps::kBF16, ALIGNED>(sums);
}

// Whether every row of every buffer starts on a vector boundary (32 bytes for f32, else 16).
struct Alignment {
    uintptr_t bits = 0;
    void add(const void *p, long long stride, size_t rows) {
        bits |= reinterpret_cast<uintptr_t>(p) | (rows > 1 ? static_cast<uintptr_t>(stride) : 0);
    }
    bool holds(size_t es) const { return bits % (es == 4 ? 32 : 16) == 0; }
};

}  // namespace

extern "C" {

int ar_check_dropout(int R, const void *const *srcs, void *const *dsts, int n_dsts, const ar_layout *L,
                     const ar_dropout *drop, size_t max_elems, int dst_dtype, int wire_dtype) {
    int st = ar_check_layout(R, srcs, dsts, n_dsts, L, max_elems, dst_dtype, wire_dtype);
    if (st != AR_OK) return st;
    st = check_drop(L, drop);
    if (st != AR_OK || L->ne0 * L->ne1 == 0) return st;
    if (drop->bias) {
        const size_t es = dtype_bytes(dst_dtype);
        if (reinterpret_cast<uintptr_t>(drop->bias) % es) return AR_ERR_INVALID_ARG;
        for (int d = 0; d < n_dsts; ++d)
            if (spans_overlap(drop->bias, L->ne0 * es, dsts[d], span_bytes(L, L->dst_row_bytes, d, es)))
                return AR_ERR_OVERLAP;
    }
    return AR_OK;
}

int ar_reduce_dropout(const void *const *srcs, void *const *dsts, int n_dsts, const ar_layout *L,
                      const ar_dropout *drop, int dst_dtype, int wire_dtype, cudaStream_t stream) {
    std::lock_guard<std::mutex> lock(tps::context_mutex());
    tps::CallContext c;
    if (!tps::current_context(&c)) return AR_ERR_NOT_INITIALIZED;
    int st = ar_check_dropout(c.R, srcs, dsts, n_dsts, L, drop, c.max_elems, dst_dtype, wire_dtype);
    if (st != AR_OK || L->ne0 * L->ne1 == 0) return st;
    st = tps::check_launch_device(c);
    if (st != AR_OK) return st;

    const int64_t packed = static_cast<int64_t>(L->ne0 * dtype_bytes(dst_dtype));
    tps::ArDropParams p;
    memset(&p, 0, sizeof p);
    tps::ArExParams &x = p.ex;
    x.ne0 = L->ne0;
    x.ne1 = L->ne1;
    x.R = c.R;
    x.n_dsts = n_dsts;
    x.inactive = L->inactive_mask;
    for (int r = 0; r < c.R; ++r) {
        if ((L->inactive_mask >> r) & 1u) continue;
        x.src[r] = srcs[r];
        x.src_stride[r] = L->src_row_bytes ? L->src_row_bytes[r] : packed;
    }
    for (int d = 0; d < n_dsts; ++d) {
        x.dst[d] = dsts[d];
        x.dst_stride[d] = L->dst_row_bytes ? L->dst_row_bytes[d] : packed;
    }
    x.residual = L->residual;
    x.res_stride = L->residual_row_bytes;
    p.drop = drop_params(*drop);
    p.bias = drop->bias;
    Alignment al;
    for (int r = 0; r < c.R; ++r)
        if (x.src[r]) al.add(x.src[r], x.src_stride[r], x.ne1);
    for (int d = 0; d < n_dsts; ++d) al.add(x.dst[d], x.dst_stride[d], x.ne1);
    al.add(x.residual, x.res_stride, x.ne1);
    al.add(p.bias, 0, 1);
    p.stride = x.dst_stride[0];
    for (int r = 0; r < c.R; ++r)
        if (x.src[r] && x.src_stride[r] != x.dst_stride[0]) p.stride = -1;
    for (int d = 1; d < n_dsts; ++d)
        if (x.dst_stride[d] != x.dst_stride[0]) p.stride = -1;
    const Shape s = forward_shape(L->ne0);
    p.bx = s.bx;
    p.by = s.by;
    const size_t turn = static_cast<size_t>(s.by), gy = (L->ne1 + turn - 1) / turn;
    const dim3 grid(s.gx, static_cast<unsigned>(gy < 65535 ? gy : 65535));
    const DropFn fn = al.holds(dtype_bytes(dst_dtype)) ? pick_types<true>(dst_dtype, wire_dtype)
                                                       : pick_types<false>(dst_dtype, wire_dtype);
    return launched(tps::launch_dependent(fn, grid, s.threads, 0, stream, c.pdl, p));
}

int ar_reduce_dropout_grad_workspace(const ar_layout *L, int n_sums, size_t *bytes) {
    if (!L || !bytes || n_sums < 0 || n_sums > 2) return AR_ERR_INVALID_ARG;
    if (L->ne1 > 0xFFFFFFFFull || L->ne0 > (1ull << 34)) return AR_ERR_TOO_LARGE;
    *bytes = L->ne0 ? static_cast<size_t>(n_sums) * row_blocks(L, n_sums) * L->ne0 * sizeof(float) : 0;
    return AR_OK;
}

int ar_reduce_dropout_grad(const void *dy, void *const *dxs, int n_dxs, const ar_layout *L, const ar_dropout *drop,
                           float *dbias, float *dresidual, void *ws, size_t ws_bytes, int dst_dtype,
                           cudaStream_t stream) {
    std::lock_guard<std::mutex> lock(tps::context_mutex());
    tps::CallContext c;
    if (!tps::current_context(&c)) return AR_ERR_NOT_INITIALIZED;
    if (!L || L->residual || L->inactive_mask) return AR_ERR_INVALID_ARG;
    const void *srcs[1] = {dy};
    int st = ar_check_layout(1, srcs, dxs, n_dxs, L, c.max_elems, dst_dtype, dst_dtype);
    if (st != AR_OK) return st;
    st = check_drop(L, drop);
    if (st != AR_OK) return st;
    if (L->ne0 == 0) return AR_OK;
    const size_t es = dtype_bytes(dst_dtype), row = L->ne0 * sizeof(float);
    float *sums[2] = {dbias, dresidual};
    const int n_sums = (dbias != nullptr) + (dresidual != nullptr);
    if (L->ne1 == 0 && n_sums == 0) return AR_OK;
    size_t need = 0;
    st = ar_reduce_dropout_grad_workspace(L, n_sums, &need);
    if (st != AR_OK) return st;
    if (need && (!ws || ws_bytes < need || reinterpret_cast<uintptr_t>(ws) % 16)) return AR_ERR_INVALID_ARG;
    for (int k = 0; k < 2; ++k) {
        if (!sums[k]) continue;
        if (reinterpret_cast<uintptr_t>(sums[k]) % sizeof(float)) return AR_ERR_INVALID_ARG;
        if (spans_overlap(sums[k], row, ws, need) || (k && spans_overlap(sums[0], sums[0] ? row : 0, sums[1], row)))
            return AR_ERR_OVERLAP;
    }
    if (L->ne1 > 0) {
        const size_t in = span_bytes(L, L->src_row_bytes, 0, es);
        if (spans_overlap(ws, need, dy, in)) return AR_ERR_OVERLAP;
        for (int k = 0; k < 2; ++k)
            if (sums[k] && spans_overlap(sums[k], row, dy, in)) return AR_ERR_OVERLAP;
        for (int d = 0; d < n_dxs; ++d) {
            const size_t out = span_bytes(L, L->dst_row_bytes, d, es);
            if (spans_overlap(ws, need, dxs[d], out)) return AR_ERR_OVERLAP;
            for (int k = 0; k < 2; ++k)
                if (sums[k] && spans_overlap(sums[k], row, dxs[d], out)) return AR_ERR_OVERLAP;
        }
    }
    st = tps::check_launch_device(c);
    if (st != AR_OK) return st;

    const int64_t packed = static_cast<int64_t>(L->ne0 * es);
    const unsigned blocks = row_blocks(L, n_sums);
    float *part[2] = {nullptr, nullptr};
    int at = 0;
    for (int k = 0; k < 2; ++k)
        if (sums[k]) part[k] = static_cast<float *>(ws) + static_cast<size_t>(at++) * blocks * L->ne0;
    if (L->ne1 > 0) {
        tps::ArDropGradParams p;
        memset(&p, 0, sizeof p);
        p.dy = dy;
        p.dy_stride = L->src_row_bytes ? L->src_row_bytes[0] : packed;
        for (int d = 0; d < n_dxs; ++d) {
            p.dx[d] = dxs[d];
            p.dx_stride[d] = L->dst_row_bytes ? L->dst_row_bytes[d] : packed;
        }
        p.ne0 = L->ne0;
        p.ne1 = L->ne1;
        p.n_dxs = n_dxs;
        p.rows_per_block = rows_per_block(L, n_sums);
        p.drop = drop_params(*drop);
        p.part_bias = part[0];
        p.part_res = part[1];
        Alignment al;
        al.add(dy, p.dy_stride, L->ne1);
        for (int d = 0; d < n_dxs; ++d) al.add(p.dx[d], p.dx_stride[d], L->ne1);
        p.stride = p.dx_stride[0];
        for (int d = 1; d < n_dxs; ++d)
            if (p.dx_stride[d] != p.dx_stride[0]) p.stride = -1;
        const Shape s = grad_shape(L->ne0);
        p.bx = s.bx;
        p.by = s.by;
        const int which = (dbias ? 1 : 0) | (dresidual ? 2 : 0);
        const GradFn fn = al.holds(es) ? pick_grad<true>(dst_dtype, which) : pick_grad<false>(dst_dtype, which);
        st = launched(tps::launch_dependent(fn, dim3(s.gx, blocks), s.threads, 0, stream, c.pdl, p));
        if (st != AR_OK) return st;
    }
    if (n_sums == 0) return AR_OK;
    tps::ColumnSums s;
    memset(&s, 0, sizeof s);
    at = 0;
    for (int k = 0; k < 2; ++k)
        if (sums[k]) s.part[at] = part[k], s.out[at++] = sums[k];
    s.ne0 = L->ne0;
    s.blocks = blocks;
    return launched(tps::launch_dependent(tps::ar_column_sum_kernel,
                                          dim3(static_cast<unsigned>((L->ne0 + 31) / 32), n_sums), 256u, 0, stream,
                                          c.pdl, s));
}

}  // extern "C"
