// Host side of ar_vocab_loss and ar_vocab_loss_grad: checks, the plan of
// vocabulary chunks, workspace layout and launches.  The operation is
// specified in include/ar.h.
#include "ar.h"

#include <cstring>

#include "ar_context.h"
#include "ar_kernels_vocab.cuh"

using tps::dtype_bytes;
using tps::VocabMat;

namespace {

// The gradient of the logits is held for one chunk of the vocabulary at a
// time: as many rows of a piece as fit this many bytes, at least kMinChunk.
constexpr size_t kChunkBytes = 256ull << 20;
constexpr size_t kMinChunk = 1024;

struct Carve {  // hands out 256-byte aligned parts of the workspace
    size_t at = 0;
    size_t take(size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    }
};

size_t total_rows(const ar_vocab *v) {
    size_t n = 0;
    for (int r = 0; r < v->n_pieces; ++r) n += v->piece_rows[r];
    return n;
}

size_t row_bytes(int64_t given, const ar_vocab *v) {
    return given ? static_cast<size_t>(given) : v->dim * dtype_bytes(v->dtype);
}

size_t weight_stride(const ar_vocab *v, int r) { return row_bytes(v->weight_row_bytes ? v->weight_row_bytes[r] : 0, v); }

size_t matrix_bytes(size_t rows, size_t stride, const ar_vocab *v) {
    return rows ? (rows - 1) * stride + v->dim * dtype_bytes(v->dtype) : 0;
}

// A stride is 0 (packed) or holds a row of whole elements, and rows of it stay within the address space.
bool valid_rows(const void *p, size_t rows, int64_t stride, const ar_vocab *v) {
    const size_t es = dtype_bytes(v->dtype);
    if (rows == 0) return true;
    if (!p || reinterpret_cast<uintptr_t>(p) % es) return false;
    if (stride < 0 || (stride && (static_cast<size_t>(stride) < v->dim * es || stride % static_cast<int64_t>(es)))) return false;
    const unsigned __int128 n = static_cast<unsigned __int128>(rows) * row_bytes(stride, v);
    return n <= UINTPTR_MAX - reinterpret_cast<uintptr_t>(p);
}

struct Span {
    const void *p;
    size_t n;
};

bool overlap(const Span &a, const Span &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.n && b.n && x < y + b.n && y < x + a.n;
}

// Whether an output overlaps an input or another output.
bool any_overlap(const Span *in, int n_in, const Span *out, int n_out) {
    for (int o = 0; o < n_out; ++o) {
        for (int i = 0; i < n_in; ++i)
            if (overlap(out[o], in[i])) return true;
        for (int q = 0; q < o; ++q)
            if (overlap(out[o], out[q])) return true;
    }
    return false;
}

size_t tiles_of(size_t rows) { return (rows + tps::kVT - 1) / tps::kVT; }

struct LossPlan {
    size_t tiles, part, picked, bytes;
};

LossPlan plan_loss(const ar_vocab *v) {
    LossPlan p{};
    for (int r = 0; r < v->n_pieces; ++r) p.tiles += tiles_of(v->piece_rows[r]);
    Carve c;
    p.part = c.take(p.tiles * v->rows * sizeof(float2));
    p.picked = c.take(v->rows * sizeof(float));
    p.bytes = c.at;
    return p;
}

struct GradPlan {
    size_t chunk, d, sum, live, bytes;
};

GradPlan plan_grad(const ar_vocab *v) {
    GradPlan p{};
    size_t most = 0;
    for (int r = 0; r < v->n_pieces; ++r) most = v->piece_rows[r] > most ? v->piece_rows[r] : most;
    p.chunk = v->rows ? kChunkBytes / (v->rows * sizeof(float)) : most;
    if (p.chunk < kMinChunk) p.chunk = kMinChunk;
    if (p.chunk > most) p.chunk = most;
    Carve c;
    p.d = c.take(p.chunk * v->rows * sizeof(float));
    p.sum = c.take(v->rows * v->dim * sizeof(float));
    p.live = c.take(v->rows);
    p.bytes = c.at;
    return p;
}

int launched(cudaError_t e) {
    if (e == cudaSuccess) return AR_OK;
    cudaGetLastError();
    return AR_ERR_CUDA;
}

template <typename P>
using Fn = void (*)(P);

template <typename P>
Fn<P> by_type(int dtype, Fn<P> f32, Fn<P> f16, Fn<P> bf16) {
    return dtype == AR_F32 ? f32 : dtype == AR_F16 ? f16 : bf16;
}

dim3 tile_grid(size_t m, size_t n) {
    return dim3(static_cast<unsigned>(tiles_of(n)), static_cast<unsigned>(tiles_of(m)));
}

}  // namespace

extern "C" {

int ar_check_vocab(const ar_vocab *v, size_t max_elems) {
    if (!v || v->n_pieces < 1 || v->n_pieces > AR_MAX_RANKS || !v->piece_rows || !v->weights || v->dim == 0)
        return AR_ERR_INVALID_ARG;
    if (!dtype_bytes(v->dtype)) return AR_ERR_UNSUPPORTED;
    // matrix rows and columns are 32-bit coordinates of the copies into shared memory
    if (v->dim > 0x7FFFFFFFull || v->rows > 65535ull * 64) return AR_ERR_TOO_LARGE;
    size_t total = 0;
    for (int r = 0; r < v->n_pieces; ++r) {
        if (v->piece_rows[r] > 0x7FFFFFFFull) return AR_ERR_TOO_LARGE;
        total += v->piece_rows[r];
    }
    if (total == 0) return AR_ERR_INVALID_ARG;
    if (v->rows > max_elems / v->dim) return AR_ERR_TOO_LARGE;
    if (v->rows == 0) return AR_OK;
    if (!valid_rows(v->hidden, v->rows, v->hidden_row_bytes, v)) return AR_ERR_INVALID_ARG;
    if (!v->targets || reinterpret_cast<uintptr_t>(v->targets) % 8) return AR_ERR_INVALID_ARG;
    for (int r = 0; r < v->n_pieces; ++r)
        if (!valid_rows(v->weights[r], v->piece_rows[r], v->weight_row_bytes ? v->weight_row_bytes[r] : 0, v))
            return AR_ERR_INVALID_ARG;
    return AR_OK;
}

int ar_vocab_workspace(const ar_vocab *v, int grad, size_t *bytes) {
    if (!bytes || (grad != 0 && grad != 1)) return AR_ERR_INVALID_ARG;
    const int st = ar_check_vocab(v, SIZE_MAX);
    if (st != AR_OK) return st;
    *bytes = v->rows == 0 ? 0 : grad ? plan_grad(v).bytes : plan_loss(v).bytes;
    return AR_OK;
}

int ar_vocab_loss(const ar_vocab *v, float *loss, float *lse, void *ws, size_t ws_bytes, cudaStream_t stream) {
    std::lock_guard<std::mutex> lock(tps::context_mutex());
    tps::CallContext c;
    if (!tps::current_context(&c)) return AR_ERR_NOT_INITIALIZED;
    int st = ar_check_vocab(v, c.max_elems);
    if (st != AR_OK || v->rows == 0) return st;
    const LossPlan plan = plan_loss(v);
    if (!loss || !lse || reinterpret_cast<uintptr_t>(loss) % 4 || reinterpret_cast<uintptr_t>(lse) % 4 || !ws ||
        reinterpret_cast<uintptr_t>(ws) % 256 || ws_bytes < plan.bytes)
        return AR_ERR_INVALID_ARG;
    Span in[AR_MAX_RANKS + 2] = {{v->hidden, matrix_bytes(v->rows, row_bytes(v->hidden_row_bytes, v), v)},
                                 {v->targets, v->rows * 8}};
    for (int r = 0; r < v->n_pieces; ++r)
        in[2 + r] = Span{v->weights[r], matrix_bytes(v->piece_rows[r], weight_stride(v, r), v)};
    const Span out[3] = {{loss, v->rows * 4}, {lse, v->rows * 4}, {ws, plan.bytes}};
    if (any_overlap(in, 2 + v->n_pieces, out, 3)) return AR_ERR_OVERLAP;
    st = tps::check_launch_device(c);
    if (st != AR_OK) return st;

    const long long es = static_cast<long long>(dtype_bytes(v->dtype));
    char *base = static_cast<char *>(ws);
    tps::VocabStatParams p;
    memset(&p, 0, sizeof p);
    p.h = VocabMat{v->hidden, static_cast<long long>(row_bytes(v->hidden_row_bytes, v)) / es, 1, nullptr};
    p.rows = v->rows;
    p.dim = v->dim;
    p.targets = reinterpret_cast<const long long *>(v->targets);
    p.part = reinterpret_cast<float2 *>(base + plan.part);
    p.picked = reinterpret_cast<float *>(base + plan.picked);
    for (int r = 0; r < v->n_pieces; ++r) {
        if (v->piece_rows[r] == 0) continue;
        p.w = VocabMat{v->weights[r], static_cast<long long>(weight_stride(v, r)) / es, 1, nullptr};
        p.vocab = v->piece_rows[r];
        st = launched(tps::launch_dependent(by_type<tps::VocabStatParams>(v->dtype, tps::ar_vocab_stat_kernel<tps::kF32>,
                                                                          tps::ar_vocab_stat_kernel<tps::kF16>,
                                                                          tps::ar_vocab_stat_kernel<tps::kBF16>),
                                            tile_grid(v->rows, p.vocab), 256u, 0, stream, c.pdl, p));
        if (st != AR_OK) return st;
        p.tile0 += static_cast<unsigned>(tiles_of(p.vocab));
        p.first += static_cast<long long>(p.vocab);
    }
    tps::VocabJoinParams j;
    memset(&j, 0, sizeof j);
    j.part = p.part;
    j.picked = p.picked;
    j.targets = p.targets;
    j.ignore = v->ignore_index;
    j.vocab = p.first;
    j.rows = v->rows;
    j.tiles = p.tile0;
    j.loss = loss;
    j.lse = lse;
    return launched(tps::launch_dependent(tps::ar_vocab_join_kernel, dim3(static_cast<unsigned>((v->rows + 255) / 256)),
                                          256u, 0, stream, c.pdl, j));
}

int ar_vocab_loss_grad(const ar_vocab *v, const float *lse, const float *dloss, void *const *dhidden,
                       const int64_t *dh_rows, void *const *dweights, const int64_t *dw_rows, void *ws, size_t ws_bytes,
                       cudaStream_t stream) {
    std::lock_guard<std::mutex> lock(tps::context_mutex());
    tps::CallContext c;
    if (!tps::current_context(&c)) return AR_ERR_NOT_INITIALIZED;
    int st = ar_check_vocab(v, c.max_elems);
    if (st != AR_OK) return st;
    if (!dhidden && !dweights) return AR_OK;
    const size_t es = dtype_bytes(v->dtype);
    Span in[AR_MAX_RANKS + 4], out[2 * AR_MAX_RANKS + 1];
    int n_in = 0, n_out = 0;
    for (int r = 0; r < v->n_pieces; ++r) {
        const int64_t hs = dh_rows ? dh_rows[r] : 0, wst = dw_rows ? dw_rows[r] : 0;
        if (dhidden) {
            if (!valid_rows(dhidden[r], v->rows, hs, v)) return AR_ERR_INVALID_ARG;
            out[n_out++] = Span{dhidden[r], matrix_bytes(v->rows, row_bytes(hs, v), v)};
        }
        if (dweights) {
            if (!valid_rows(dweights[r], v->piece_rows[r], wst, v)) return AR_ERR_INVALID_ARG;
            out[n_out++] = Span{dweights[r], matrix_bytes(v->piece_rows[r], row_bytes(wst, v), v)};
        }
        in[n_in++] = Span{v->weights[r], matrix_bytes(v->piece_rows[r], weight_stride(v, r), v)};
    }
    const GradPlan plan = plan_grad(v);
    if (v->rows) {
        if (!lse || !dloss || reinterpret_cast<uintptr_t>(lse) % 4 || reinterpret_cast<uintptr_t>(dloss) % 4 || !ws ||
            reinterpret_cast<uintptr_t>(ws) % 256 || ws_bytes < plan.bytes)
            return AR_ERR_INVALID_ARG;
        in[n_in++] = Span{v->hidden, matrix_bytes(v->rows, row_bytes(v->hidden_row_bytes, v), v)};
        in[n_in++] = Span{v->targets, v->rows * 8};
        in[n_in++] = Span{lse, v->rows * 4};
        in[n_in++] = Span{dloss, v->rows * 4};
        out[n_out++] = Span{ws, plan.bytes};
    }
    if (any_overlap(in, n_in, out, n_out)) return AR_ERR_OVERLAP;
    st = tps::check_launch_device(c);
    if (st != AR_OK) return st;

    char *base = static_cast<char *>(ws);
    const long long e = static_cast<long long>(es);
    tps::VocabGradParams p;
    memset(&p, 0, sizeof p);
    p.h = VocabMat{v->hidden, static_cast<long long>(row_bytes(v->hidden_row_bytes, v)) / e, 1, nullptr};
    p.rows = v->rows;
    p.dim = v->dim;
    p.ignore = v->ignore_index;
    p.total = static_cast<long long>(total_rows(v));
    p.targets = reinterpret_cast<const long long *>(v->targets);
    p.lse = lse;
    p.dloss = dloss;
    p.d = reinterpret_cast<float *>(base + plan.d);
    p.live = reinterpret_cast<unsigned char *>(base + plan.live);
    const auto product = by_type<tps::VocabOutParams>(v->dtype, tps::ar_vocab_product_kernel<tps::kF32>,
                                                      tps::ar_vocab_product_kernel<tps::kF16>,
                                                      tps::ar_vocab_product_kernel<tps::kBF16>);
    long long first = 0;  // global index of the piece's first row
    for (int r = 0; r < v->n_pieces; ++r) {
        const size_t n = v->piece_rows[r], ld = weight_stride(v, r);
        const size_t hs = row_bytes(dh_rows ? dh_rows[r] : 0, v), wst = row_bytes(dw_rows ? dw_rows[r] : 0, v);
        for (size_t v0 = 0; v0 == 0 || v0 < n; v0 += plan.chunk) {
            const size_t rows = n - v0 < plan.chunk ? n - v0 : plan.chunk;
            p.w = VocabMat{static_cast<const char *>(v->weights[r]) + v0 * ld, static_cast<long long>(ld) / e, 1, nullptr};
            p.vocab = rows;
            p.first = first + static_cast<long long>(v0);
            if (rows && v->rows) {
                st = launched(tps::launch_dependent(
                    by_type<tps::VocabGradParams>(v->dtype, tps::ar_vocab_dlogits_kernel<tps::kF32>,
                                                  tps::ar_vocab_dlogits_kernel<tps::kF16>,
                                                  tps::ar_vocab_dlogits_kernel<tps::kBF16>),
                    tile_grid(v->rows, rows), 256u, 0, stream, c.pdl, p));
                if (st != AR_OK) return st;
            }
            tps::VocabOutParams o;
            memset(&o, 0, sizeof o);
            if (dhidden && v->rows) {  // a piece without rows still writes its zeros
                o.a = VocabMat{p.d, static_cast<long long>(rows), 1, nullptr};
                o.b = VocabMat{p.w.base, 1, p.w.row, nullptr};
                o.m = v->rows, o.n = v->dim, o.k = rows;
                o.sum = reinterpret_cast<float *>(base + plan.sum);
                o.begin = v0 == 0;
                o.out = v0 + rows >= n ? dhidden[r] : nullptr;
                o.out_row = static_cast<long long>(hs) / e;
                st = launched(tps::launch_dependent(product, tile_grid(o.m, o.n), 256u, 0, stream, c.pdl, o));
                if (st != AR_OK) return st;
            }
            if (dweights && rows) {
                memset(&o, 0, sizeof o);
                o.a = VocabMat{p.d, 1, static_cast<long long>(rows), nullptr};
                o.b = VocabMat{v->hidden, 1, p.h.row, p.live};
                o.m = rows, o.n = v->dim, o.k = v->rows;
                o.out = static_cast<char *>(dweights[r]) + v0 * wst;
                o.out_row = static_cast<long long>(wst) / e;
                st = launched(tps::launch_dependent(product, tile_grid(o.m, o.n), 256u, 0, stream, c.pdl, o));
                if (st != AR_OK) return st;
            }
            if (n == 0) break;
        }
        first += static_cast<long long>(n);
    }
    return AR_OK;
}

}  // extern "C"
