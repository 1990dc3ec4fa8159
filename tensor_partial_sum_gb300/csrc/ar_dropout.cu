// Host side of ar_reduce_dropout and ar_reduce_dropout_grad: checks, launch
// shapes and launches.  The operation is specified in include/ar.h.
#include "ar.h"

#include <cstring>

#include "ar_context.h"
#include "ar_kernels_dropout.cuh"

using tps::dtype_bytes;

namespace {

// Row blocks of the column sums: enough to fill the GPU, few enough that the
// partial sums stay small beside the gradient (at most 128 rows of ne0).
constexpr unsigned kMaxRowBlocks = 128;

unsigned rows_per_block(size_t ne1) {
    const size_t r = (ne1 + kMaxRowBlocks - 1) / kMaxRowBlocks;
    return static_cast<unsigned>(r < 16 ? 16 : r);
}

unsigned row_blocks(size_t ne1) {
    const unsigned r = rows_per_block(ne1);
    return static_cast<unsigned>((ne1 + r - 1) / r);
}

bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
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

template <int Td>
DropFn pick_wire(int wire) {
    return wire == AR_F32   ? tps::ar_dropout_kernel<Td, tps::kF32>
           : wire == AR_F16 ? tps::ar_dropout_kernel<Td, tps::kF16>
                            : tps::ar_dropout_kernel<Td, tps::kBF16>;
}

DropFn pick(int dst, int wire) {
    return dst == AR_F32   ? pick_wire<tps::kF32>(wire)
           : dst == AR_F16 ? pick_wire<tps::kF16>(wire)
                           : pick_wire<tps::kBF16>(wire);
}

GradFn pick_grad(int dst) {
    return dst == AR_F32   ? tps::ar_dropout_grad_kernel<tps::kF32>
           : dst == AR_F16 ? tps::ar_dropout_grad_kernel<tps::kF16>
                           : tps::ar_dropout_grad_kernel<tps::kBF16>;
}

int launched(cudaError_t e) {
    if (e == cudaSuccess) return AR_OK;
    cudaGetLastError();
    return AR_ERR_CUDA;
}

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
            if (overlap(drop->bias, L->ne0 * es, dsts[d], span_bytes(L, L->dst_row_bytes, d, es)))
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
    const size_t gx = (L->ne0 + 255) / 256;
    const dim3 grid(static_cast<unsigned>(gx < 4096 ? gx : 4096), static_cast<unsigned>(L->ne1 < 65535 ? L->ne1 : 65535));
    return launched(tps::launch_dependent(pick(dst_dtype, wire_dtype), grid, 256u, 0, stream, c.pdl, p));
}

int ar_reduce_dropout_grad_workspace(const ar_layout *L, int n_sums, size_t *bytes) {
    if (!L || !bytes || n_sums < 0 || n_sums > 2) return AR_ERR_INVALID_ARG;
    if (L->ne1 > 0xFFFFFFFFull || L->ne0 > (1ull << 34)) return AR_ERR_TOO_LARGE;
    *bytes = static_cast<size_t>(n_sums) * row_blocks(L->ne1) * L->ne0 * sizeof(float);
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
        if (overlap(sums[k], row, ws, need) || (k && overlap(sums[0], sums[0] ? row : 0, sums[1], row)))
            return AR_ERR_OVERLAP;
    }
    if (L->ne1 > 0) {
        const size_t in = span_bytes(L, L->src_row_bytes, 0, es);
        if (overlap(ws, need, dy, in)) return AR_ERR_OVERLAP;
        for (int k = 0; k < 2; ++k)
            if (sums[k] && overlap(sums[k], row, dy, in)) return AR_ERR_OVERLAP;
        for (int d = 0; d < n_dxs; ++d) {
            const size_t out = span_bytes(L, L->dst_row_bytes, d, es);
            if (overlap(ws, need, dxs[d], out)) return AR_ERR_OVERLAP;
            for (int k = 0; k < 2; ++k)
                if (sums[k] && overlap(sums[k], row, dxs[d], out)) return AR_ERR_OVERLAP;
        }
    }
    st = tps::check_launch_device(c);
    if (st != AR_OK) return st;

    const int64_t packed = static_cast<int64_t>(L->ne0 * es);
    const unsigned blocks = row_blocks(L->ne1);
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
        p.rows_per_block = rows_per_block(L->ne1);
        p.drop = drop_params(*drop);
        p.part_bias = part[0];
        p.part_res = part[1];
        const size_t gx = (L->ne0 + 255) / 256;
        st = launched(tps::launch_dependent(pick_grad(dst_dtype), dim3(static_cast<unsigned>(gx < 4096 ? gx : 4096), blocks),
                                            256u, 0, stream, c.pdl, p));
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
                                          dim3(static_cast<unsigned>((L->ne0 + 255) / 256), n_sums), 256u, 0, stream,
                                          c.pdl, s));
}

}  // extern "C"
