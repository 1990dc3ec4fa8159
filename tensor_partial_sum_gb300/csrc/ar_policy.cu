// Host side of ar_policy_loss.  The operation is specified in include/ar.h.
#include "ar.h"

#include <cmath>
#include <cstring>

#include "ar_buffers.h"
#include "ar_kernels_policy.cuh"

using tps::launched;

namespace {

constexpr size_t kMostBlocks = 608;  // four on each of 152 SMs

// A call's workspace: the counts, those of each sequence or counting block, and the blocks' sums.
struct Plan {
    size_t chunks, blocks, count_blocks, counts, part, bytes;
    bool small;
};

Plan plan_of(const ar_policy *p) {
    Plan w;
    w.small = p->tokens <= tps::kPolicySmall;
    w.chunks = w.small ? 0 : (p->tokens + tps::kPolicyChunk - 1) / tps::kPolicyChunk;
    w.blocks = w.chunks < kMostBlocks ? w.chunks : kMostBlocks;
    // four chunks to a thread of the counting launch, and no more blocks than every later block sums quickly
    w.count_blocks = (w.chunks + 3) / 4 < kMostBlocks ? (w.chunks + 3) / 4 : kMostBlocks;
    w.counts = sizeof(tps::PolicyCounts);
    const size_t counts = p->mean == AR_POLICY_SEQUENCES ? p->sequences : p->mean == AR_POLICY_TOKENS ? w.count_blocks : 0;
    w.part = (w.counts + counts * sizeof(unsigned) + 15) / 16 * 16;
    w.bytes = w.part + w.blocks * 4 * sizeof(double);
    return w;
}

int check_sizes(const ar_policy *p) {
    if (!p) return AR_ERR_INVALID_ARG;
    if (p->mean != AR_POLICY_SUM && p->mean != AR_POLICY_TOKENS && p->mean != AR_POLICY_SEQUENCES) return AR_ERR_INVALID_ARG;
    if (p->tokens > 0xFFFFFFFFull || p->sequences >= (1ull << 31)) return AR_ERR_TOO_LARGE;
    return AR_OK;
}

tps::PolicyLimit limit_of(double v) {
    tps::PolicyLimit l{static_cast<float>(v), 0.0f, 0.0f};
    if (std::isfinite(v)) {
        l.rest = static_cast<float>(v - l.x);
        const double left = v - l.x - l.rest;
        l.sign = left > 0.0 ? 1.0f : left < 0.0 ? -1.0f : 0.0f;
    }
    return l;
}

template <typename T>
bool misplaced(const T *p) {
    return reinterpret_cast<uintptr_t>(p) % alignof(T) != 0;
}

}  // namespace

extern "C" {

int ar_check_policy(const ar_policy *p, size_t max_elems) {
    const int st = check_sizes(p);
    if (st != AR_OK) return st;
    if (p->tokens > max_elems) return AR_ERR_TOO_LARGE;
    if (!(p->clip_low >= 0.0 && p->clip_low <= 1.0) || !(p->clip_high >= 0.0)) return AR_ERR_INVALID_ARG;
    if (!(p->kl_weight >= 0.0) || !std::isfinite(p->kl_weight) || !std::isfinite(p->scale)) return AR_ERR_INVALID_ARG;
    if (p->token_advantages != 0 && p->token_advantages != 1) return AR_ERR_INVALID_ARG;
    if (misplaced(p->offsets) || misplaced(p->nll) || misplaced(p->old_nll) || misplaced(p->ref_nll) || misplaced(p->advantages))
        return AR_ERR_INVALID_ARG;
    if (p->tokens && !p->nll) return AR_ERR_INVALID_ARG;
    if (p->sequences && !p->offsets) return AR_ERR_INVALID_ARG;
    if ((p->token_advantages ? p->tokens : p->sequences) && !p->advantages) return AR_ERR_INVALID_ARG;
    return AR_OK;
}

int ar_policy_workspace(const ar_policy *p, size_t *bytes) {
    const int st = check_sizes(p);
    if (st != AR_OK) return st;
    if (!bytes) return AR_ERR_INVALID_ARG;
    *bytes = plan_of(p).bytes;
    return AR_OK;
}

int ar_policy_loss(const ar_policy *a, float *totals, float *dnll, void *ws, size_t ws_bytes, cudaStream_t stream) {
    std::lock_guard<std::mutex> lock(tps::context_mutex());
    tps::CallContext c;
    if (!tps::current_context(&c)) return AR_ERR_NOT_INITIALIZED;
    int st = ar_check_policy(a, c.max_elems);
    if (st != AR_OK) return st;
    if (!totals || misplaced(totals) || misplaced(dnll)) return AR_ERR_INVALID_ARG;
    const Plan w = plan_of(a);
    if (!ws || ws_bytes < w.bytes || reinterpret_cast<uintptr_t>(ws) % 16) return AR_ERR_INVALID_ARG;
    const size_t T = a->tokens, S = a->sequences, row = T * sizeof(float);
    tps::Buffers b;
    b.output(totals, 4 * sizeof(float));
    b.output(ws, w.bytes);
    b.output(dnll, row);
    if (S) b.input(a->offsets, (S + 1) * sizeof(int64_t));
    for (const float *x : {a->nll, a->old_nll, a->ref_nll})
        if (x != dnll) b.input(x, row);
    b.input(a->advantages, (a->token_advantages ? T : S) * sizeof(float));
    b.input(a->mask, T);
    if (b.clash()) return AR_ERR_OVERLAP;
    st = tps::check_launch_device(c);
    if (st != AR_OK) return st;

    tps::PolicyParams p;
    memset(&p, 0, sizeof p);
    p.tokens = static_cast<unsigned>(T);
    p.sequences = static_cast<unsigned>(S);
    p.offsets = reinterpret_cast<const long long *>(a->offsets);
    p.nll = a->nll;
    p.old_nll = a->old_nll;
    p.ref_nll = a->ref_nll;
    p.adv = a->advantages;
    p.mask = a->mask;
    p.token_adv = a->token_advantages;
    p.mean = a->mean;
    uintptr_t bits = reinterpret_cast<uintptr_t>(a->nll) | reinterpret_cast<uintptr_t>(a->old_nll) |
                     reinterpret_cast<uintptr_t>(a->ref_nll) | reinterpret_cast<uintptr_t>(a->mask) |
                     reinterpret_cast<uintptr_t>(dnll);
    if (a->token_advantages) bits |= reinterpret_cast<uintptr_t>(a->advantages);
    p.vec = bits % 16 == 0;
    p.high = limit_of(std::log1p(a->clip_high));
    p.low = limit_of(std::log1p(-a->clip_low));
    p.limit_high = static_cast<float>(1.0 + a->clip_high);
    p.limit_low = static_cast<float>(1.0 - a->clip_low);
    p.beta = static_cast<float>(a->kl_weight);
    p.kl_weight = a->kl_weight;
    p.scale = a->scale;
    p.totals = totals;
    p.dnll = dnll;
    char *base = static_cast<char *>(ws);
    p.counts = reinterpret_cast<tps::PolicyCounts *>(base);
    p.per_sequence = p.per_block = reinterpret_cast<unsigned *>(base + w.counts);
    p.part = reinterpret_cast<double *>(base + w.part);
    p.blocks = static_cast<unsigned>(w.blocks);
    p.count_blocks = static_cast<unsigned>(w.count_blocks);
    auto go = [&](void (*fn)(tps::PolicyParams), size_t blocks, unsigned threads = tps::kPolicyThreads) {
        return launched(tps::launch_dependent(fn, dim3(static_cast<unsigned>(blocks)), threads, 0, stream, c.pdl, p));
    };
    if (w.small) {
        const size_t threads = (T / tps::kPolicyEach + 32) / 32 * 32;
        return go(tps::ar_policy_small_kernel, 1, threads < tps::kPolicySmallThreads ? static_cast<unsigned>(threads < 64 ? 64 : threads)
                                                                                      : static_cast<unsigned>(tps::kPolicySmallThreads));
    }
    if (a->mean == AR_POLICY_SUM) {
        st = go(tps::ar_policy_kernel<false>, w.blocks);
        return st == AR_OK ? go(tps::ar_policy_join_kernel, 1) : st;
    }
    if (a->mean == AR_POLICY_TOKENS) {
        st = go(tps::ar_policy_count_tokens_kernel, w.count_blocks);
    } else {
        st = go(tps::ar_policy_zero_kernel, S / tps::kPolicyThreads + 1);
        if (st == AR_OK) st = go(tps::ar_policy_count_kernel, w.chunks);
    }
    return st == AR_OK ? go(tps::ar_policy_kernel<true>, w.blocks) : st;
}

}  // extern "C"
