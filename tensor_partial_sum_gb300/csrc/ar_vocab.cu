// Host side of ar_vocab_loss and ar_vocab_loss_grad: checks, the plan of
// vocabulary chunks, workspace layout and launches.  The operation is
// specified in include/ar.h.
#include "ar.h"

#include <cstring>

#include "ar_context.h"
#include "ar_kernels_vocab.cuh"

using tps::dtype_bytes;
using tps::launched;
using namespace tps::plan;

namespace {

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

bool overlap(const Span &a, const Span &b) { return tps::spans_overlap(a.p, a.n, b.p, b.n); }

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

template <typename P>
using Fn = void (*)(P);

template <typename P>
Fn<P> by_type(int dtype, Fn<P> f32, Fn<P> f16, Fn<P> bf16) {
    return dtype == AR_F32 ? f32 : dtype == AR_F16 ? f16 : bf16;
}

// cuTensorMapEncodeTiled, through the runtime so that the library loads where there is no driver.
using EncodeFn = decltype(&cuTensorMapEncodeTiled);

EncodeFn encode_fn() {
    static EncodeFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// A tensor map over [parts][rows][cols] 16-bit elements, `ld` elements between rows and `part`
// between parts, copied in boxes of 64 columns by box_rows rows, 128-byte swizzled.
bool make_map(CUtensorMap *m, bool f16, const void *base, size_t cols, size_t rows, size_t parts, size_t ld, size_t part,
              unsigned box_rows) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {cols, rows, parts};
    const cuuint64_t strides[2] = {ld * 2, (parts > 1 ? part : rows * ld) * 2};
    const cuuint32_t box[3] = {64, box_rows, 1}, step[3] = {1, 1, 1};
    return fn(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims,
              strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Few tokens: the map of the hidden states, in boxes of half the tokens (rounded up to 16), and the rows left over of
// a segment's last tile.
bool make_few_map(tps::VocabGemmParams &p, bool f16, const void *base, size_t cols, size_t rows, size_t parts, size_t ld,
                  size_t part) {
    p.a_rows = static_cast<int>(rows);
    return make_map(&p.a_map, f16, base, cols, rows, parts, ld, part, static_cast<unsigned>(p.bn / 2));
}
unsigned few_tail(size_t rows, int few) {
    const size_t left = rows % static_cast<size_t>(few);
    return static_cast<unsigned>(left ? round_up(left, 8) : 8);
}

// Rows of the boxes of a segment's last column tile: half its width.
template <int MODE>
unsigned tail_box(size_t rows, int bn) {
    const int left = static_cast<int>(rows % static_cast<size_t>(bn));
    const int width = tps::tail_width<MODE>(left ? left : bn);
    return static_cast<unsigned>((width < bn ? width : bn) / 2);
}

// The two maps of a K-major A: boxes of 128 rows, and of the rows left over (8 at least).
bool make_a_maps(tps::VocabGemmParams &p, bool f16, const void *base, size_t cols, size_t rows, size_t parts, size_t ld,
                 size_t part) {
    p.a_rows = static_cast<int>(rows);
    p.a_tail = static_cast<int>(round_up(rows % 128, 8));
    return make_map(&p.a_map, f16, base, cols, rows, parts, ld, part, 128) &&
           make_map(&p.a_tail_map, f16, base, cols, rows, parts, ld, part, p.a_tail ? static_cast<unsigned>(p.a_tail) : 8u);
}

// A call under way: what its launches share.
struct Call {
    const ar_vocab *v;
    tps::CallContext c;
    cudaStream_t stream;
    char *ws;
    size_t parts, ld;     // of packed rows
    bool f16, pack;       // the weights are packed, group by group

    template <typename P>
    int launch(Fn<P> fn, dim3 grid, unsigned threads, size_t smem, const P &p) const {
        return launched(tps::launch_dependent(fn, grid, threads, smem, stream, c.pdl, p));
    }

    // Packed rows at `dst`, `rows_max` rows apart in parts, of the matrices that add_pack names.
    tps::VocabPackParams pack_params(void *dst, size_t rows_max) const {
        tps::VocabPackParams p;
        memset(&p, 0, sizeof p);
        p.dim = static_cast<int>(v->dim);
        p.dst = static_cast<unsigned short *>(dst);
        p.dst_ld = static_cast<long long>(ld);
        p.dst_part = static_cast<long long>(rows_max * ld);
        return p;
    }
    static void add_pack(tps::VocabPackParams &p, int m, const void *src, size_t stride, size_t rows, size_t at) {
        p.src[m] = src;
        p.src_row[m] = static_cast<long long>(stride);
        p.rows[m] = static_cast<int>(rows);
        p.dst_at[m] = static_cast<long long>(at);
    }
    int launch_pack(const tps::VocabPackParams &p, int n) const {
        // a thread for each eight elements of a row, as far as 256 go: idle ones cost bytes in flight
        const size_t groups = ld / 8, threads = groups < 256 ? round_up(groups, 32) : 256;
        int rows = 64, most = c.sm_count * static_cast<int>(4096 / threads) / n;
        for (int m = 0; m < n; ++m) rows = p.rows[m] > rows ? p.rows[m] : rows;
        return launch(by_type<tps::VocabPackParams>(v->dtype, tps::ar_vocab_pack_kernel<tps::kF32>,
                                                    tps::ar_vocab_pack_kernel<tps::kF16>,
                                                    tps::ar_vocab_pack_kernel<tps::kBF16>),
                      dim3(static_cast<unsigned>(rows < most ? rows : most), static_cast<unsigned>(n)),
                      static_cast<unsigned>(threads), 0, p);
    }

    // The weights of a group: packed at `area` (room for `cap` rows) where they have to be; per segment
    // the base, columns, rows, row stride in elements and part stride of what the copies read.
    struct Matrix {
        const char *base;
        size_t cols, rows, ld, part;
    };
    int group_weights(const Group &g, size_t area, size_t cap, Matrix *out) const {
        size_t at = 0;
        tps::VocabPackParams p = pack_params(ws + area, cap);
        for (int s = 0; s < g.nseg; ++s) {
            const size_t stride = weight_stride(v, g.piece[s]);
            const char *src = static_cast<const char *>(v->weights[g.piece[s]]) + g.row0[s] * stride;
            if (!pack) {
                out[s] = Matrix{src, v->dim, g.rows[s], stride / 2, 0};
                continue;
            }
            add_pack(p, s, src, stride, g.rows[s], at);
            out[s] = Matrix{ws + area + at * ld * 2, ld, g.rows[s], ld, cap * ld};
            at += g.rows[s];
        }
        return pack ? launch_pack(p, g.nseg) : static_cast<int>(AR_OK);
    }

    // With few rows of A a stage holds less, and more stages fit: these launches are bound by the bytes
    // in flight.  (dW's A is a full tile of vocabulary rows.)
    template <int MODE>
    int launch_gemm(tps::VocabGemmParams &p, size_t tiles) const {
        if (tps::kVFew<MODE>) p.a_room = p.few_rows;
        else p.a_room = p.a_rows >= 128 || (tps::kVGrads<MODE> && p.tiles) ? 128 : p.a_tail;
        // a product reads 128 rows of A wherever the stage starts: the last stage's have to lie in the ring
        const bool f32 = parts == 3;
        const int pa = f32 ? tps::kVPartsA<MODE, tps::kF32> : tps::kVPartsA<MODE, tps::kBF16>;
        const int pb = f32 ? tps::kVPartsB<MODE, tps::kF32> : tps::kVPartsB<MODE, tps::kBF16>;
        const int blocks = f32 ? tps::kVBlocks<MODE, tps::kF32> : tps::kVBlocks<MODE, tps::kBF16>;
        // (the last part of A of the last block: 128 rows from (pa - 1) a_room rows on)
        const int block = (pa * p.a_room + pb * p.bn / 2) * tps::kVRow, stage = blocks * block;
        const int last = tps::kVRing - (blocks - 1) * block - ((pa - 1) * p.a_room + 128) * tps::kVRow;
        p.stages = tps::kVRing / stage;
        if (p.stages > last / stage + 1) p.stages = last / stage + 1;
        if (p.stages > tps::kVMaxStages) p.stages = tps::kVMaxStages;
        constexpr int kMode32 = MODE == tps::kGradsFew ? static_cast<int>(tps::kGrads) : MODE;  // float: parts enough
        const auto fn = by_type<tps::VocabGemmParams>(v->dtype, tps::ar_vocab_gemm_kernel<kMode32, tps::kF32>,
                                                      tps::ar_vocab_gemm_kernel<MODE, tps::kF16>,
                                                      tps::ar_vocab_gemm_kernel<MODE, tps::kBF16>);
        if (cudaFuncSetAttribute(reinterpret_cast<const void *>(fn), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(tps::kVSmem)) != cudaSuccess) {
            cudaGetLastError();
            return AR_ERR_CUDA;
        }
        if (v->dtype == AR_F32 ? tps::kVSplitRegs<MODE, tps::kF32> : tps::kVSplitRegs<MODE, tps::kBF16>) {
            // result warps take registers that the feeding warps give up; a launch that was given fewer
            // than the split adds up to would wait for them for ever
            cudaFuncAttributes a;
            if (cudaFuncGetAttributes(&a, reinterpret_cast<const void *>(fn)) != cudaSuccess) {
                cudaGetLastError();
                return AR_ERR_CUDA;
            }
            if (a.numRegs < tps::kVLaunchRegs) return AR_ERR_UNSUPPORTED;
        }
        const size_t most = static_cast<size_t>(c.sm_count / 2);
        const size_t pairs = tiles < 1 ? 1 : tiles < most ? tiles : most;
        return launch(fn, dim3(static_cast<unsigned>(2 * pairs)), static_cast<unsigned>(tps::kVThreads), tps::kVSmem, p);
    }
};

}  // namespace

extern "C" {

int ar_check_vocab(const ar_vocab *v, size_t max_elems) {
    if (!v || v->n_pieces < 1 || v->n_pieces > AR_MAX_RANKS || !v->piece_rows || !v->weights || v->dim == 0)
        return AR_ERR_INVALID_ARG;
    if (!dtype_bytes(v->dtype)) return AR_ERR_UNSUPPORTED;
    // rows and columns are 32-bit coordinates of the tiled copies
    if (v->dim > (1ull << 28) || v->rows > (1ull << 28)) return AR_ERR_TOO_LARGE;
    size_t total = 0;
    for (int r = 0; r < v->n_pieces; ++r) {
        if (v->piece_rows[r] > (1ull << 28)) return AR_ERR_TOO_LARGE;
        total += v->piece_rows[r];
    }
    if (total == 0) return AR_ERR_INVALID_ARG;
    // tiles of a launch are counted in 31 bits
    constexpr size_t kMostTiles = 1ull << 30;
    const size_t nt = v->dim / 128 + 1;
    if (total / tps::kVM + AR_MAX_RANKS > kMostTiles / nt || v->rows / tps::kVM + 1 > kMostTiles / AR_MAX_RANKS / nt)
        return AR_ERR_TOO_LARGE;
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

    Call call{v, c, stream, static_cast<char *>(ws), static_cast<size_t>(parts_of(v)), packed_ld(v), v->dtype == AR_F16,
              !weights_in_place(v)};
    const size_t T = v->rows, D = v->dim;
    // the hidden states as the tiled copies read them
    Call::Matrix h{static_cast<const char *>(v->hidden), D, T, row_bytes(v->hidden_row_bytes, v) / 2, 0};
    if (!hidden_in_place(v)) {
        h = Call::Matrix{call.ws + plan.hidden, call.ld, T, call.ld, T * call.ld};
        tps::VocabPackParams hp = call.pack_params(call.ws + plan.hidden, T);
        Call::add_pack(hp, 0, v->hidden, row_bytes(v->hidden_row_bytes, v), T, 0);
        st = call.launch_pack(hp, 1);
        if (st != AR_OK) return st;
    }
    tps::VocabGemmParams p;
    memset(&p, 0, sizeof p);
    p.rows = static_cast<int>(T);
    p.dim = static_cast<int>(D);
    const bool few = T <= tps::kFewTokens;
    p.bn = plan.tile.bn;
    p.few_rows = plan.tile.few_rows;
    p.targets = reinterpret_cast<const long long *>(v->targets);
    p.part = reinterpret_cast<float2 *>(call.ws + plan.part);
    p.picked = reinterpret_cast<float *>(call.ws + plan.picked);
    p.status = c.dev_status;
    if (!(few ? make_few_map(p, call.f16, h.base, h.cols, h.rows, call.parts, h.ld, h.part)
              : make_a_maps(p, call.f16, h.base, h.cols, h.rows, call.parts, h.ld, h.part)))
        return AR_ERR_CUDA;
    long long first[AR_MAX_RANKS], total = 0;
    for (int r = 0; r < v->n_pieces; ++r) first[r] = total, total += static_cast<long long>(v->piece_rows[r]);
    int piece = 0;
    size_t row = 0;
    Group g;
    while (next_group(v, plan.cap, piece, row, g)) {
        Call::Matrix w[tps::kMaxSegs];
        st = call.group_weights(g, plan.weights, plan.cap, w);
        if (st != AR_OK) return st;
        p.nseg = g.nseg;
        p.tiles = 0;
        for (int s = 0; s < g.nseg; ++s) {
            p.seg[s].first = first[g.piece[s]] + static_cast<long long>(g.row0[s]);
            p.seg[s].rows = static_cast<int>(g.rows[s]);
            p.seg[s].tile0 = p.tiles;
            p.tiles += static_cast<int>(tiles_of(g.rows[s], plan.tile.rows));
            const unsigned tail = few ? few_tail(g.rows[s], p.few_rows) : tail_box<tps::kStats>(g.rows[s], p.bn);
            if (!make_map(&p.b_map[s], call.f16, w[s].base, w[s].cols, w[s].rows, call.parts, w[s].ld, w[s].part,
                          static_cast<unsigned>(plan.tile.rows / 2)) ||
                !make_map(&p.b_tail[s], call.f16, w[s].base, w[s].cols, w[s].rows, call.parts, w[s].ld, w[s].part, tail))
                return AR_ERR_CUDA;
        }
        st = few ? call.launch_gemm<tps::kStatsFew>(p, static_cast<size_t>(p.tiles))
                 : call.launch_gemm<tps::kStats>(p, static_cast<size_t>(p.tiles) * tiles_of(T, tps::kVM));
        if (st != AR_OK) return st;
        p.part += plan.tile.parts * static_cast<size_t>(p.tiles) * T;
    }
    tps::VocabJoinParams j;
    memset(&j, 0, sizeof j);
    j.part = reinterpret_cast<float2 *>(call.ws + plan.part);
    j.picked = p.picked;
    j.targets = p.targets;
    j.ignore = v->ignore_index;
    j.vocab = total;
    j.rows = p.rows;
    j.parts = static_cast<int>(plan.parts);
    j.loss = loss;
    j.lse = lse;
    return few ? call.launch<tps::VocabJoinParams>(tps::ar_vocab_join_kernel<1>, dim3(static_cast<unsigned>(T)), 256u, 0, j)
               : call.launch<tps::VocabJoinParams>(tps::ar_vocab_join_kernel<4>, dim3(static_cast<unsigned>((T + 3) / 4)),
                                                   256u, 0, j);
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

    Call call{v, c, stream, static_cast<char *>(ws), static_cast<size_t>(parts_of(v)), packed_ld(v), v->dtype == AR_F16,
              !weights_in_place(v)};
    const size_t T = v->rows, D = v->dim;
    if (T == 0) {  // no tokens: the weights' gradients are zero
        for (int r = 0; dweights && r < v->n_pieces; ++r)
            if (v->piece_rows[r] &&
                cudaMemset2DAsync(dweights[r], row_bytes(dw_rows ? dw_rows[r] : 0, v), 0, D * es, v->piece_rows[r], stream) !=
                    cudaSuccess)
                return launched(cudaErrorUnknown);
        return AR_OK;
    }
    tps::VocabListParams l;
    memset(&l, 0, sizeof l);
    l.targets = reinterpret_cast<const long long *>(v->targets);
    l.lse = lse;
    l.dloss = dloss;
    l.ignore = v->ignore_index;
    l.vocab = static_cast<long long>(total_rows(v));
    l.rows = static_cast<int>(T);
    l.gain = call.f16 ? 16384.0f : 1.0f;
    l.list = reinterpret_cast<tps::VocabList *>(call.ws + plan.list);
    l.row = reinterpret_cast<tps::VocabRow *>(call.ws + plan.row);
    l.index = reinterpret_cast<int *>(call.ws + plan.index);
    l.place = reinterpret_cast<int *>(call.ws + plan.place);
    st = call.launch<tps::VocabListParams>(tps::ar_vocab_list_kernel, dim3(1), 1024u, 0, l);
    if (st != AR_OK) return st;
    tps::VocabPackParams hp = call.pack_params(call.ws + plan.hidden, plan.k_rows);
    Call::add_pack(hp, 0, v->hidden, row_bytes(v->hidden_row_bytes, v), T, 0);
    hp.place = l.place;
    hp.list = l.list;
    for (int r = 0; dhidden && r < v->n_pieces; ++r) {
        hp.dh[r] = static_cast<char *>(dhidden[r]);
        hp.dh_row[r] = static_cast<long long>(row_bytes(dh_rows ? dh_rows[r] : 0, v));
        hp.n_dh = r + 1;
        // a piece without rows has no product that would write its zeros
        if (v->piece_rows[r] == 0 &&
            cudaMemset2DAsync(dhidden[r], static_cast<size_t>(hp.dh_row[r]), 0, D * es, T, stream) != cudaSuccess)
            return launched(cudaErrorUnknown);
    }
    st = call.launch_pack(hp, 1);
    if (st != AR_OK) return st;

    tps::VocabGemmParams p;
    memset(&p, 0, sizeof p);
    p.rows = l.rows;
    p.dim = static_cast<int>(D);
    p.list = l.list;
    p.row = l.row;
    p.index = l.index;
    p.d = reinterpret_cast<unsigned short *>(call.ws + plan.d);
    p.status = c.dev_status;
    const size_t mt = plan.d_rows / tps::kVM;
    const bool few = T <= tps::kFewTokens;
    if (!make_map(&p.ht_map, call.f16, call.ws + plan.hidden, call.ld, plan.k_rows, call.parts, call.ld, plan.k_rows * call.ld, 64))
        return AR_ERR_CUDA;
    long long first[AR_MAX_RANKS], total = 0;
    for (int r = 0; r < v->n_pieces; ++r) first[r] = total, total += static_cast<long long>(v->piece_rows[r]);
    int piece = 0;
    size_t row = 0;
    Group g;
    while (next_group(v, plan.cap, piece, row, g)) {
        Call::Matrix w[tps::kMaxSegs];
        st = call.group_weights(g, plan.weights, plan.cap, w);
        if (st != AR_OK) return st;
        // D of this group's logits
        p.d_ld = static_cast<long long>(g.padded);
        p.d_part = p.d_ld * static_cast<long long>(plan.d_rows);
        p.nseg = g.nseg;
        p.bn = few ? static_cast<int>(round_up(T, 16)) : static_cast<int>(tps::kVN);
        p.few_rows = few ? few_rows(v, 32) : 0;  // whole blocks of K: D's columns are zeroed to there
        const int tile = few ? 2 * p.few_rows : p.bn;
        p.tiles = 0;
        if (!(few ? make_few_map(p, call.f16, call.ws + plan.hidden, call.ld, plan.k_rows, call.parts, call.ld, plan.k_rows * call.ld)
                  : make_a_maps(p, call.f16, call.ws + plan.hidden, call.ld, plan.k_rows, call.parts, call.ld, plan.k_rows * call.ld)))
            return AR_ERR_CUDA;
        long long col = 0;
        for (int s = 0; s < g.nseg; ++s) {
            p.seg[s].first = first[g.piece[s]] + static_cast<long long>(g.row0[s]);
            p.seg[s].rows = static_cast<int>(g.rows[s]);
            p.seg[s].tile0 = p.tiles;
            p.seg[s].col0 = col;
            col += static_cast<long long>(round_up(g.rows[s], tps::kVN));
            p.tiles += static_cast<int>(tiles_of(g.rows[s], static_cast<size_t>(tile)));
            const unsigned tail = few ? few_tail(g.rows[s], p.few_rows) : tail_box<tps::kDlogits>(g.rows[s], p.bn);
            if (!make_map(&p.b_map[s], call.f16, w[s].base, w[s].cols, w[s].rows, call.parts, w[s].ld, w[s].part,
                          static_cast<unsigned>(tile / 2)) ||
                !make_map(&p.b_tail[s], call.f16, w[s].base, w[s].cols, w[s].rows, call.parts, w[s].ld, w[s].part, tail))
                return AR_ERR_CUDA;
        }
        st = few ? call.launch_gemm<tps::kDlogitsFew>(p, static_cast<size_t>(p.tiles))
                 : call.launch_gemm<tps::kDlogits>(p, static_cast<size_t>(p.tiles) * mt);
        if (st != AR_OK) return st;
        // dH and dW from it
        const size_t parts = call.parts, dparts = static_cast<size_t>(d_parts_of(v)), dl = static_cast<size_t>(p.d_ld), dp = static_cast<size_t>(p.d_part);
        if (!make_a_maps(p, call.f16, p.d, dl, plan.k_rows, dparts, dl, dp) ||
            !make_map(&p.at_map, call.f16, p.d, dl, plan.k_rows, dparts, dl, dp, 64))
            return AR_ERR_CUDA;
        p.bn = D <= tps::kVN / 2 ? tps::kVN / 2 : tps::kVN;
        p.slices = plan.slices;
        p.dh_tiles = dhidden ? static_cast<int>(tiles_of(D, static_cast<size_t>(p.bn))) : 0;
        p.sum_rows = static_cast<long long>(plan.d_rows);
        p.sum_ld = static_cast<long long>(round_up(D, 8));
        const bool sums = plan.slices > 1 || !(g.begins && g.ends);
        p.sum = sums ? reinterpret_cast<float *>(call.ws + plan.sum) : nullptr;
        p.sum_begin = g.begins;
        const bool straight = plan.slices == 1 && g.ends;  // this launch finishes dH
        p.tiles = 0;
        for (int s = 0; s < g.nseg; ++s) {
            const int r = g.piece[s];
            p.seg[s].tile0 = p.tiles;
            p.seg[s].dh = dhidden && straight ? static_cast<char *>(dhidden[r]) : nullptr;
            p.seg[s].dh_row = hp.dh_row[r];
            p.seg[s].dw_row = static_cast<long long>(row_bytes(dw_rows ? dw_rows[r] : 0, v));
            p.seg[s].dw = dweights ? static_cast<char *>(dweights[r]) + g.row0[s] * static_cast<size_t>(p.seg[s].dw_row) : nullptr;
            p.tiles += static_cast<int>(tiles_of(g.rows[s], tps::kVM));
            if (!make_map(&p.b_map[s], call.f16, w[s].base, w[s].cols, w[s].rows, parts, w[s].ld, w[s].part, 64)) return AR_ERR_CUDA;
        }
        p.tiles = dweights ? p.tiles * static_cast<int>(tiles_of(D, static_cast<size_t>(p.bn))) : 0;
        const size_t tiles = static_cast<size_t>(p.tiles) + static_cast<size_t>(g.nseg * p.slices * p.dh_tiles) * mt;
        st = dparts == 2 ? call.launch_gemm<tps::kGradsFew>(p, tiles) : call.launch_gemm<tps::kGrads>(p, tiles);
        if (st != AR_OK) return st;
        if (dhidden && plan.slices > 1 && g.ends) {
            tps::VocabSumParams q;
            memset(&q, 0, sizeof q);
            q.sum = p.sum;
            q.sum_rows = p.sum_rows;
            q.sum_ld = p.sum_ld;
            q.slices = p.slices;
            q.dim = p.dim;
            q.list = l.list;
            q.index = l.index;
            for (int s = 0; s < g.nseg; ++s) {
                q.dh[s] = static_cast<char *>(dhidden[g.piece[s]]);
                q.dh_row[s] = hp.dh_row[g.piece[s]];
            }
            st = call.launch(by_type<tps::VocabSumParams>(v->dtype, tps::ar_vocab_sum_kernel<tps::kF32>,
                                                          tps::ar_vocab_sum_kernel<tps::kF16>,
                                                          tps::ar_vocab_sum_kernel<tps::kBF16>),
                             dim3(static_cast<unsigned>((D + 1023) / 1024), static_cast<unsigned>(T < 4096 ? T : 4096),
                                  static_cast<unsigned>(g.nseg)),
                             256u, 0, q);
            if (st != AR_OK) return st;
        }
    }
    return AR_OK;
}

}  // extern "C"
