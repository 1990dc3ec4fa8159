// Host side of ar_reduce_norm, ar_reduce_norm_grad and the checkpoint calls:
// checks, launch shapes and launches.  The operations are specified in
// include/ar.h.
#include "ar.h"

#include <cmath>
#include <cstring>

#include "ar_buffers.h"
#include "ar_kernels_norm.cuh"

using tps::Buffers;
using tps::dtype_bytes;
using tps::launched;
using tps::rows_bytes;
using namespace tps::plan;

namespace {

template <typename Fn>
Fn by_type(int dtype, Fn f32, Fn f16, Fn bf16) {
    return dtype == AR_F32 ? f32 : dtype == AR_F16 ? f16 : bf16;
}

// ---- checkpoints -----------------------------------------------------------------

size_t code_stride(const ar_checkpoint &c) {
    return c.code_row_bytes ? static_cast<size_t>(c.code_row_bytes) : (c.ne0 + 15) / 16 * 16;
}
size_t scale_row(const ar_checkpoint &c) { return (c.ne0 + AR_CHECKPOINT_BLOCK - 1) / AR_CHECKPOINT_BLOCK; }
size_t scale_stride(const ar_checkpoint &c) {
    return c.scale_row_bytes ? static_cast<size_t>(c.scale_row_bytes) : scale_row(c);
}

int check_codes(const ar_checkpoint *c, size_t max_elems) {
    if (!c) return AR_ERR_INVALID_ARG;
    if (c->format != AR_E4M3 && c->format != AR_INT8) return AR_ERR_UNSUPPORTED;
    if (c->ne0 && c->ne1 > SIZE_MAX / c->ne0) return AR_ERR_TOO_LARGE;
    if (c->ne0 * c->ne1 > max_elems) return AR_ERR_TOO_LARGE;
    if (c->ne0 * c->ne1 == 0) return AR_OK;
    if (!c->codes || !c->scales || reinterpret_cast<uintptr_t>(c->codes) % 16) return AR_ERR_INVALID_ARG;
    if (c->code_row_bytes < 0 || c->scale_row_bytes < 0 || c->code_row_bytes % 16) return AR_ERR_INVALID_ARG;
    if (!tps::rows_fit(c->codes, c->ne1, static_cast<int64_t>(code_stride(*c)), c->ne0) ||
        !tps::rows_fit(c->scales, c->ne1, static_cast<int64_t>(scale_stride(*c)), scale_row(*c)))
        return AR_ERR_INVALID_ARG;
    return AR_OK;
}

void add_codes(Buffers &b, const ar_checkpoint *c, bool out) {
    if (!c) return;
    const size_t codes = rows_bytes(c->ne1, code_stride(*c), c->ne0);
    const size_t scales = rows_bytes(c->ne1, scale_stride(*c), scale_row(*c));
    if (out) {
        b.output(c->codes, codes);
        b.output(c->scales, scales);
    } else {
        b.input(c->codes, codes);
        b.input(c->scales, scales);
    }
}

tps::CodeRows code_rows(const ar_checkpoint *c) {
    if (!c) return tps::CodeRows{};
    return tps::CodeRows{static_cast<uint8_t *>(c->codes), static_cast<long long>(code_stride(*c)),
                         static_cast<uint8_t *>(c->scales), static_cast<long long>(scale_stride(*c)), c->format};
}

// ---- norm ------------------------------------------------------------------------

int check_norm(const ar_norm *n, size_t es) {
    if (!n || (n->kind != AR_NORM_LAYER && n->kind != AR_NORM_RMS)) return AR_ERR_INVALID_ARG;
    if (!(n->eps >= 0.0f) || !std::isfinite(n->eps)) return AR_ERR_INVALID_ARG;
    for (const void *row : {n->weight, n->shift, n->bias})
        if (reinterpret_cast<uintptr_t>(row) % es) return AR_ERR_INVALID_ARG;
    return AR_OK;
}

size_t row_stride(const int64_t *rows, int k, size_t packed) { return rows ? static_cast<size_t>(rows[k]) : packed; }

// The type that operands of dst are really rounded through: a value of a format rounds to itself.
int wire_of(int dst, int wire) { return dst == wire ? AR_F32 : wire; }

constexpr int kAnyThreads = 512;

template <typename Fn>
int allow_ring(Fn fn, const RowShape &s) {
    if (s.smem <= 44 * 1024) return AR_OK;  // 48 KB with what the kernel declares itself
    return launched(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(ring_bytes(1))));
}

using NormFn = void (*)(tps::NormParams);

using GradFn = void (*)(tps::NormGradParams);

template <int Td, bool ALIGNED>
GradFn pick_backward(const RowShape &s) {
    if (s.U == 1) return s.warp ? tps::ar_norm_grad_kernel<Td, ALIGNED, 1, true> : tps::ar_norm_grad_kernel<Td, ALIGNED, 1, false>;
    if constexpr (ALIGNED && Td != tps::kF32)
        return nullptr;  // one unit is 16 columns
    else
        return s.warp ? tps::ar_norm_grad_kernel<Td, ALIGNED, 2, true> : tps::ar_norm_grad_kernel<Td, ALIGNED, 2, false>;
}

template <bool BIAS>
GradFn pick_copied(int dtype) {
    return by_type<GradFn>(dtype, tps::ar_norm_grad_rows_kernel<tps::kF32, BIAS>, tps::ar_norm_grad_rows_kernel<tps::kF16, BIAS>,
                           tps::ar_norm_grad_rows_kernel<tps::kBF16, BIAS>);
}

template <typename Fn, template <int, bool> class Pick>
Fn pick_rows(int dtype, bool aligned, const RowShape &s) {
    if (aligned)
        return dtype == AR_F32   ? Pick<tps::kF32, true>::of(s)
               : dtype == AR_F16 ? Pick<tps::kF16, true>::of(s)
                                 : Pick<tps::kBF16, true>::of(s);
    return dtype == AR_F32   ? Pick<tps::kF32, false>::of(s)
           : dtype == AR_F16 ? Pick<tps::kF16, false>::of(s)
                             : Pick<tps::kBF16, false>::of(s);
}

template <int Td, bool ALIGNED>
struct Forward {
    static NormFn of(const RowShape &s) {
        return s.warp ? tps::ar_norm_kernel<Td, ALIGNED, true> : tps::ar_norm_kernel<Td, ALIGNED, false>;
    }
};
template <int Td, bool ALIGNED>
struct Backward {
    static GradFn of(const RowShape &s) { return pick_backward<Td, ALIGNED>(s); }
};

// A tensor's rows and where they end; `rows` of them, one where the stride is 0.
tps::RowSource source_of(const void *p, long long stride, size_t rows, size_t row) {
    const char *base = static_cast<const char *>(p);
    return tps::RowSource{base, base ? base + (rows - 1) * static_cast<size_t>(stride) + row : nullptr, stride,
                          static_cast<unsigned>(stride), stride >= 64};
}

// ---- checkpoint calls ---------------------------------------------------------------

using PackFn = void (*)(tps::PackParams);
using PackAnyFn = void (*)(tps::PackParams, bool);

template <bool ALIGNED>
PackFn pick_pack(int dtype, bool pack) {
    return pack ? by_type<PackFn>(dtype, tps::ar_checkpoint_pack_kernel<tps::kF32, ALIGNED>,
                                  tps::ar_checkpoint_pack_kernel<tps::kF16, ALIGNED>,
                                  tps::ar_checkpoint_pack_kernel<tps::kBF16, ALIGNED>)
                : by_type<PackFn>(dtype, tps::ar_checkpoint_unpack_kernel<tps::kF32, ALIGNED>,
                                  tps::ar_checkpoint_unpack_kernel<tps::kF16, ALIGNED>,
                                  tps::ar_checkpoint_unpack_kernel<tps::kBF16, ALIGNED>);
}

int run_checkpoint(const ar_checkpoint *ck, const void *tensor, int64_t row_bytes, int dtype, cudaStream_t stream,
                   bool pack) {
    std::lock_guard<std::mutex> lock(tps::context_mutex());
    tps::CallContext c;
    if (!tps::current_context(&c)) return AR_ERR_NOT_INITIALIZED;
    int st = ar_check_checkpoint(ck, tensor, row_bytes, c.max_elems, dtype);
    if (st != AR_OK || ck->ne0 * ck->ne1 == 0) return st;
    st = tps::check_launch_device(c);
    if (st != AR_OK) return st;
    const size_t es = dtype_bytes(dtype), row = ck->ne0 * es;
    tps::PackParams p;
    memset(&p, 0, sizeof p);
    Alignment al;
    al.add(tensor, row_bytes ? row_bytes : static_cast<int64_t>(row), ck->ne1);
    p.tensor = source_of(tensor, row_bytes ? row_bytes : static_cast<int64_t>(row), ck->ne1, row);
    p.ne0 = ck->ne0;
    p.ne1 = ck->ne1;
    p.kept = code_rows(ck);
    const PackShape s = pack_shape(ck->ne0, ck->ne1, es, al);
    p.per_row = static_cast<unsigned>(s.per_row);
    if (!s.vectors) {
        const PackAnyFn any = by_type<PackAnyFn>(dtype, tps::ar_checkpoint_any_kernel<tps::kF32>, tps::ar_checkpoint_any_kernel<tps::kF16>,
                                                 tps::ar_checkpoint_any_kernel<tps::kBF16>);
        return launched(tps::launch_dependent(any, dim3(static_cast<unsigned>(kSMs * 8)), 256u, 0, stream, c.pdl, p, pack));
    }
    return launched(tps::launch_dependent(s.aligned ? pick_pack<true>(dtype, pack) : pick_pack<false>(dtype, pack),
                                          dim3(static_cast<unsigned>(s.blocks)), 256u, 0, stream, c.pdl, p));
}

}  // namespace

extern "C" {

int ar_check_checkpoint(const ar_checkpoint *ck, const void *tensor, int64_t row_bytes, size_t max_elems, int dtype) {
    const size_t es = dtype_bytes(dtype);
    if (!es) return AR_ERR_UNSUPPORTED;
    int st = check_codes(ck, max_elems);
    if (st != AR_OK || ck->ne0 * ck->ne1 == 0) return st;
    if (!tensor || reinterpret_cast<uintptr_t>(tensor) % es || row_bytes < 0 || row_bytes % static_cast<int64_t>(es))
        return AR_ERR_INVALID_ARG;
    const size_t row = ck->ne0 * es, stride = row_bytes ? static_cast<size_t>(row_bytes) : row;
    if (!tps::rows_fit(tensor, ck->ne1, static_cast<int64_t>(stride), row)) return AR_ERR_INVALID_ARG;
    Buffers b;
    b.output(tensor, rows_bytes(ck->ne1, stride, row));
    add_codes(b, ck, true);
    return b.clash() ? AR_ERR_OVERLAP : AR_OK;
}

int ar_checkpoint_pack(const void *src, int64_t row_bytes, const ar_checkpoint *c, int dtype, cudaStream_t stream) {
    return run_checkpoint(c, src, row_bytes, dtype, stream, true);
}

int ar_checkpoint_unpack(const ar_checkpoint *c, void *dst, int64_t row_bytes, int dtype, cudaStream_t stream) {
    return run_checkpoint(c, dst, row_bytes, dtype, stream, false);
}

int ar_check_norm(int R, const void *const *srcs, void *const *dsts, int n_dsts, const ar_layout *L, const ar_norm *norm,
                  const ar_norm_kept *kept, size_t max_elems, int dst_dtype, int wire_dtype) {
    int st = ar_check_layout(R, srcs, dsts, n_dsts, L, max_elems, dst_dtype, wire_dtype);
    if (st != AR_OK) return st;
    const size_t es = dtype_bytes(dst_dtype);
    st = check_norm(norm, es);
    if (st != AR_OK) return st;
    static const ar_norm_kept nothing = {};
    if (!kept) kept = &nothing;
    if (kept->n_sums < 0 || kept->n_sums > AR_MAX_DSTS || (kept->n_sums && !kept->sums)) return AR_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(kept->mean) % sizeof(float) || reinterpret_cast<uintptr_t>(kept->rstd) % sizeof(float))
        return AR_ERR_INVALID_ARG;
    if (kept->checkpoint) {
        if (kept->checkpoint->ne0 != L->ne0 || kept->checkpoint->ne1 != L->ne1) return AR_ERR_INVALID_ARG;
        st = check_codes(kept->checkpoint, max_elems);
        if (st != AR_OK) return st;
    }
    if (L->ne0 * L->ne1 == 0) return AR_OK;
    const size_t row = L->ne0 * es;
    if (kept->n_sums) {
        // against the sources and the residual the sums obey the destinations' rules
        ar_layout sums = *L;
        sums.dst_row_bytes = kept->sum_row_bytes;
        st = ar_check_layout(R, srcs, kept->sums, kept->n_sums, &sums, max_elems, dst_dtype, wire_dtype);
        if (st != AR_OK) return st;
    }
    Buffers outs;
    for (int d = 0; d < n_dsts; ++d) outs.output(dsts[d], rows_bytes(L->ne1, row_stride(L->dst_row_bytes, d, row), row));
    for (int s = 0; s < kept->n_sums; ++s)
        outs.output(kept->sums[s], rows_bytes(L->ne1, row_stride(kept->sum_row_bytes, s, row), row));
    for (const void *r : {norm->weight, norm->shift, norm->bias}) outs.input(r, row);
    if (outs.clash()) return AR_ERR_OVERLAP;
    // what else is written lies apart from everything
    Buffers apart = outs;
    for (int r = 0; r < R; ++r)
        if (!((L->inactive_mask >> r) & 1u)) apart.input(srcs[r], rows_bytes(L->ne1, row_stride(L->src_row_bytes, r, row), row));
    if (L->residual)
        apart.input(L->residual, L->residual_row_bytes ? rows_bytes(L->ne1, static_cast<size_t>(L->residual_row_bytes), row) : row);
    Buffers rest;
    rest.output(kept->mean, L->ne1 * sizeof(float));
    rest.output(kept->rstd, L->ne1 * sizeof(float));
    add_codes(rest, kept->checkpoint, true);
    return rest.clash() || rest.meets(apart) ? AR_ERR_OVERLAP : AR_OK;
}

int ar_reduce_norm(const void *const *srcs, void *const *dsts, int n_dsts, const ar_layout *L, const ar_norm *norm,
                   const ar_norm_kept *kept, int dst_dtype, int wire_dtype, cudaStream_t stream) {
    std::lock_guard<std::mutex> lock(tps::context_mutex());
    tps::CallContext c;
    if (!tps::current_context(&c)) return AR_ERR_NOT_INITIALIZED;
    int st = ar_check_norm(c.R, srcs, dsts, n_dsts, L, norm, kept, c.max_elems, dst_dtype, wire_dtype);
    if (st != AR_OK || L->ne0 * L->ne1 == 0) return st;
    st = tps::check_launch_device(c);
    if (st != AR_OK) return st;

    const size_t packed = L->ne0 * dtype_bytes(dst_dtype);
    tps::NormParams p;
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
        x.src_stride[r] = static_cast<long long>(row_stride(L->src_row_bytes, r, packed));
    }
    for (int d = 0; d < n_dsts; ++d) {
        x.dst[d] = dsts[d];
        x.dst_stride[d] = static_cast<long long>(row_stride(L->dst_row_bytes, d, packed));
    }
    x.residual = L->residual;
    x.res_stride = L->residual_row_bytes;
    if (kept) {
        p.n_sums = kept->n_sums;
        for (int s = 0; s < kept->n_sums; ++s) {
            p.sum[s] = kept->sums[s];
            p.sum_stride[s] = static_cast<long long>(row_stride(kept->sum_row_bytes, s, packed));
        }
        p.mean = kept->mean;
        p.rstd = kept->rstd;
        p.kept = code_rows(kept->checkpoint);
    }
    p.wire = wire_of(dst_dtype, wire_dtype);
    p.rms = norm->kind == AR_NORM_RMS;
    p.eps = norm->eps;
    p.inv_n = 1.0f / static_cast<float>(L->ne0);
    p.weight = norm->weight;
    p.shift = norm->shift;
    p.bias = norm->bias;
    Alignment al;
    for (int r = 0; r < c.R; ++r)
        if (x.src[r]) {
            al.add(x.src[r], x.src_stride[r], x.ne1);
            p.source[p.n_sources++] = source_of(x.src[r], x.src_stride[r], x.ne1, packed);
        }
    for (int d = 0; d < n_dsts; ++d) al.add(x.dst[d], x.dst_stride[d], x.ne1);
    for (int k = 0; k < p.n_sums; ++k) al.add(p.sum[k], p.sum_stride[k], x.ne1);
    al.add(x.residual, x.res_stride, x.ne1);
    if (x.residual) p.source[p.n_sources++] = source_of(x.residual, x.res_stride, x.ne1, packed);
    const size_t es = dtype_bytes(dst_dtype);
    const bool aligned = al.bits % 32 == 0;
    const RowShape s = forward_shape(L->ne0, L->ne1, es, aligned);
    const size_t grid = s.U ? forward_grid(s, L->ne1) : 0;
    if (s.U == 0 || !al.narrow || grid > 0x7FFFFFFF) {
        const NormFn any = by_type<NormFn>(dst_dtype, tps::ar_norm_any_kernel<tps::kF32>, tps::ar_norm_any_kernel<tps::kF16>,
                                           tps::ar_norm_any_kernel<tps::kBF16>);
        const size_t blocks = L->ne1 < 65535 ? L->ne1 : 65535;
        return launched(tps::launch_dependent(any, dim3(static_cast<unsigned>(blocks)), static_cast<unsigned>(kAnyThreads), 0,
                                              stream, c.pdl, p));
    }
    Alignment rows;
    for (const void *row : {p.weight, p.shift, p.bias}) rows.add(row, 0, 1);
    p.rows_aligned = rows.bits % 16 == 0;
    p.apart = 1;
    for (int k = 0; k < p.n_sources; ++k) p.apart &= p.source[k].apart;
    p.bx = s.bx;
    p.units = s.U;
    while (1 << p.cluster_bits < s.cluster) ++p.cluster_bits;
    const NormFn fn = pick_rows<NormFn, Forward>(dst_dtype, aligned, s);
    st = allow_ring(fn, s);
    if (st != AR_OK) return st;
    return launched(tps::launch_clustered(fn, dim3(static_cast<unsigned>(grid)), static_cast<unsigned>(s.cluster), s.threads, s.smem,
                                          stream, c.pdl, p));
}

int ar_reduce_norm_grad_workspace(const ar_layout *L, int n_sums, size_t *bytes) {
    if (!L || !bytes || n_sums < 0 || n_sums > 3) return AR_ERR_INVALID_ARG;
    if (L->ne0 > SIZE_MAX / 16 || (L->ne0 && L->ne1 > SIZE_MAX / L->ne0 / 16)) return AR_ERR_TOO_LARGE;
    // which path a call takes depends on its pointers: room for the larger
    const size_t any = part_ld(2 * L->ne1) + static_cast<size_t>(n_sums) * any_blocks(L->ne1) * part_ld(L->ne0);
    const size_t ring = static_cast<size_t>(n_sums) * ring_blocks(L->ne0, L->ne1) * part_ld(L->ne0);
    *bytes = L->ne0 ? (any > ring ? any : ring) * sizeof(float) : 0;
    return AR_OK;
}

int ar_reduce_norm_grad(const void *dy, const void *h, const ar_checkpoint *ck, const float *mean, const float *rstd,
                        void *const *dxs, int n_dxs, const ar_layout *L, const ar_norm *norm, float *dweight,
                        float *dshift, float *dbias, void *ws, size_t ws_bytes, int dst_dtype, cudaStream_t stream) {
    std::lock_guard<std::mutex> lock(tps::context_mutex());
    tps::CallContext c;
    if (!tps::current_context(&c)) return AR_ERR_NOT_INITIALIZED;
    if (!L || L->inactive_mask || (h != nullptr) == (ck != nullptr)) return AR_ERR_INVALID_ARG;
    const void *srcs[2] = {dy, h};
    int st = ar_check_layout(h ? 2 : 1, srcs, dxs, n_dxs, L, c.max_elems, dst_dtype, dst_dtype);
    if (st != AR_OK) return st;
    const size_t es = dtype_bytes(dst_dtype), packed = L->ne0 * es;
    st = check_norm(norm, es);
    if (st != AR_OK) return st;
    if (ck) {
        if (ck->ne0 != L->ne0 || ck->ne1 != L->ne1) return AR_ERR_INVALID_ARG;
        st = check_codes(ck, c.max_elems);
        if (st != AR_OK) return st;
    }
    if (L->ne0 == 0) return AR_OK;
    float *sums[3] = {dweight, dshift, dbias};
    int n_sums = 0;
    for (float *s : sums) {
        if (reinterpret_cast<uintptr_t>(s) % sizeof(float)) return AR_ERR_INVALID_ARG;
        n_sums += s != nullptr;
    }
    if (L->ne1 == 0 && n_sums == 0) return AR_OK;
    const bool rms = norm->kind == AR_NORM_RMS;
    if (L->ne1 > 0) {
        if (!rstd || (!mean && !rms)) return AR_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(mean) % sizeof(float) || reinterpret_cast<uintptr_t>(rstd) % sizeof(float))
            return AR_ERR_INVALID_ARG;
    }
    size_t need = 0;
    st = ar_reduce_norm_grad_workspace(L, n_sums, &need);
    if (st != AR_OK) return st;
    if (need && (!ws || ws_bytes < need || reinterpret_cast<uintptr_t>(ws) % 16)) return AR_ERR_INVALID_ARG;
    // the results, which obey the layout's rules against dy, h and dsum
    Buffers outs, given, rest;
    for (int d = 0; L->ne1 && d < n_dxs; ++d)
        outs.output(dxs[d], rows_bytes(L->ne1, row_stride(L->dst_row_bytes, d, packed), packed));
    given.input(dy, rows_bytes(L->ne1, row_stride(L->src_row_bytes, 0, packed), packed));
    if (h) given.input(h, rows_bytes(L->ne1, row_stride(L->src_row_bytes, 1, packed), packed));
    if (L->residual)
        given.input(L->residual, L->residual_row_bytes ? rows_bytes(L->ne1, static_cast<size_t>(L->residual_row_bytes), packed) : packed);
    // what else is read, and what else is written
    Buffers apart;
    apart.input(norm->weight, packed);
    if (!rms) apart.input(mean, L->ne1 * sizeof(float));
    apart.input(rstd, L->ne1 * sizeof(float));
    add_codes(apart, ck, false);
    for (float *s : sums) rest.output(s, L->ne0 * sizeof(float));
    rest.output(ws, need);
    if (outs.meets(apart) || rest.clash() || rest.meets(outs) || rest.meets(given) || rest.meets(apart)) return AR_ERR_OVERLAP;
    st = tps::check_launch_device(c);
    if (st != AR_OK) return st;

    tps::NormGradParams p;
    memset(&p, 0, sizeof p);
    size_t blocks = 0;
    p.part_ld = part_ld(L->ne0);
    auto place = [&](float *at) {
        for (int k = 0; k < 3; ++k)
            if (sums[k]) p.part[k] = at, at += blocks * p.part_ld;
    };
    if (L->ne1 > 0) {
        Alignment al;
        auto given_rows = [&](const void *t, long long stride) {
            al.add(t, stride, L->ne1);
            return source_of(t, stride, L->ne1, packed);
        };
        p.dy = given_rows(dy, static_cast<long long>(row_stride(L->src_row_bytes, 0, packed)));
        if (h) p.h = given_rows(h, static_cast<long long>(row_stride(L->src_row_bytes, 1, packed)));
        if (L->residual) p.dsum = given_rows(L->residual, L->residual_row_bytes);
        p.kept = code_rows(ck);
        p.mean = mean;
        p.rstd = rstd;
        for (int d = 0; d < n_dxs; ++d) {
            p.dx[d] = dxs[d];
            p.dx_stride[d] = static_cast<long long>(row_stride(L->dst_row_bytes, d, packed));
            al.add(p.dx[d], p.dx_stride[d], L->ne1);
        }
        al.add(norm->weight, 0, 1);
        p.n_dxs = n_dxs;
        p.rms = rms;
        p.inv_n = 1.0f / static_cast<float>(L->ne0);
        p.ne0 = L->ne0;
        p.ne1 = L->ne1;
        p.weight = norm->weight;
        const bool aligned = al.bits % 32 == 0;
        const size_t cols = aligned ? 32 / es : 8;
        const int v = aligned ? 2 : static_cast<int>(es) / 2 + 1;
        p.status = c.dev_status;
        p.timeout_ns = c.drop_tile < 0 ? tps::kUmmaTimeoutNs : 100ull * 1000 * 1000;
        p.drop_row = c.drop_tile < 0 ? ~0ull : static_cast<unsigned long long>(c.drop_tile);
        // whole vectors of a row that is broadcast could reach behind its end
        const bool copied = aligned && !(L->residual && L->residual_row_bytes == 0 && L->ne1 > 1 && packed % 16);
        const RowShape rows = copied ? copied_shape(L->ne0, L->ne1, es, es + (h ? es : 1) + (L->residual ? es : 0)) : RowShape{};
        const RowShape s =
            rows.U ? rows : row_shape(L->ne0, L->ne1, cols, v + (h ? v : 1) + (L->residual ? v : 0), cols == 16 ? 1 : 2);
        p.rows_aligned = reinterpret_cast<uintptr_t>(norm->weight) % 16 == 0;
        p.apart = p.dy.apart && (!h || p.h.apart) && (!L->residual || p.dsum.apart);
        if (s.U && al.narrow) {
            // no more blocks than the workspace has rows of partial sums for
            const size_t most = ring_blocks(L->ne0, L->ne1), groups = row_grid(s, L->ne1) / s.cluster;
            blocks = groups < most ? groups : most;
            const size_t grid = blocks * s.cluster;
            place(static_cast<float *>(ws));
            p.bx = s.bx;
            p.cluster = s.cluster;
            p.stages = s.stages;
            p.vecs = s.vecs;
            const GradFn fn = rows.U ? (dbias ? pick_copied<true>(dst_dtype) : pick_copied<false>(dst_dtype))
                                     : pick_rows<GradFn, Backward>(dst_dtype, aligned, s);
            st = allow_ring(fn, s);
            if (st != AR_OK) return st;
            st = launched(tps::launch_clustered(fn, dim3(static_cast<unsigned>(grid)), static_cast<unsigned>(s.cluster), s.threads,
                                                s.smem, stream, c.pdl, p));
        } else {
            blocks = any_blocks(L->ne1);
            p.row_sums = static_cast<float *>(ws);
            place(p.row_sums + part_ld(2 * L->ne1));  // on a 16-byte boundary
            p.rows_per_block = static_cast<unsigned>(any_rows(L->ne1));
            const GradFn stats = by_type<GradFn>(dst_dtype, tps::ar_norm_row_sums_kernel<tps::kF32>,
                                                 tps::ar_norm_row_sums_kernel<tps::kF16>, tps::ar_norm_row_sums_kernel<tps::kBF16>);
            const GradFn fn = by_type<GradFn>(dst_dtype, tps::ar_norm_grad_any_kernel<tps::kF32>,
                                              tps::ar_norm_grad_any_kernel<tps::kF16>, tps::ar_norm_grad_any_kernel<tps::kBF16>);
            const size_t rows = L->ne1 < 65535 ? L->ne1 : 65535;
            st = launched(tps::launch_dependent(stats, dim3(static_cast<unsigned>(rows)), static_cast<unsigned>(kAnyThreads), 0,
                                                stream, c.pdl, p));
            if (st != AR_OK) return st;
            st = launched(tps::launch_dependent(fn, dim3(static_cast<unsigned>((L->ne0 + 31) / 32), static_cast<unsigned>(blocks)), 256u,
                                                0, stream, c.pdl, p));
        }
        if (st != AR_OK) return st;
    }
    if (n_sums == 0) return AR_OK;
    tps::NormColumnSums s;
    memset(&s, 0, sizeof s);
    int n = 0;
    for (int k = 0; k < 3; ++k)
        if (sums[k]) s.part[n] = p.part[k], s.out[n++] = sums[k];
    s.ne0 = L->ne0;
    s.ld = p.part_ld;
    s.blocks = static_cast<unsigned>(blocks);
    return launched(tps::launch_dependent(tps::ar_norm_column_sum_kernel,
                                          dim3(static_cast<unsigned>((L->ne0 + 63) / 64), static_cast<unsigned>(n_sums)),
                                          512u, 0, stream, c.pdl, s));
}

}  // extern "C"
