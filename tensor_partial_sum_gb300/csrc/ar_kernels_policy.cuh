// Device code of ar_policy_loss.
//
// The means need counts before the first gradient can be written, so the mask is read once for them and the
// tokens once for the rest.  Few tokens: one block does both.  Many: a launch counts (behind one that zeroes the
// counts of the sequences, where those are wanted), the next computes, and its last block joins the blocks' sums.
// Counts are integers, whose order of adding does not matter; floats are added in a fixed order.
//
// Measured on a GB300 in a graph: 300 tokens 7.3 us (one block: four rounds of dependent loads, an exponential, a sum);
// 262143 tokens in 257 sequences 19.2 us (three launches); four million tokens with an advantage each 33.2 us, 28 of them
// the main launch: 2.7 TB/s, about 100 instructions a token.
#pragma once

#include <climits>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "ar_pairs.cuh"

namespace tps {

constexpr int kPolicyThreads = 256;
constexpr int kPolicyEach = 8;  // adjacent tokens of a thread
constexpr int kPolicyChunk = kPolicyThreads * kPolicyEach;
constexpr int kPolicySmallThreads = 1024;  // of the one block that few tokens take
constexpr int kPolicySmall = 2 * kPolicySmallThreads * kPolicyEach;  // tokens, at most

struct PolicyCounts {
    unsigned ticket;     // blocks that are done
    unsigned sequences;  // sequences that have counted tokens
    unsigned pad[2];
};

// A 64-bit number as floats: rounded, what that leaves rounded, and the sign of what is left then.  Each float
// operation in place of 64-bit ones counts: this GPU has two of those a cycle and SM (with them the kernel was
// bound by them, at 75 us for four million tokens).
struct PolicyLimit {
    float x, rest, sign;
};

struct PolicyParams {
    unsigned tokens;
    unsigned sequences;
    const long long *offsets;
    const float *nll, *old_nll, *ref_nll, *adv;
    const uint8_t *mask;
    int token_adv, mean, vec;  // vec: every array of tokens starts on a 16-byte boundary
    PolicyLimit high, low;  // log(1 + clip_high), log(1 - clip_low)
    float limit_high, limit_low, beta;
    double kl_weight, scale;
    float *totals, *dnll;
    PolicyCounts *counts;
    unsigned *per_sequence;  // counted tokens of each sequence (the mean over sequences)
    unsigned *per_block;     // counted tokens of each block of the counting launch (the mean over tokens)
    double *part;            // [block][4]: gain, kl, clipped, counted
    unsigned blocks, count_blocks;
};

// How many of the sequences + 1 offsets are <= t, found by a warp, 32 probes at a time.  Stays within 0 ..
// sequences + 1 whatever the offsets hold.
__device__ __forceinline__ unsigned offsets_upto_warp(const PolicyParams &p, long long t) {
    unsigned lo = 0, n = p.sequences + 1;
    const unsigned lane = threadIdx.x % 32;
    while (n > 0) {
        const unsigned step = (n + 31) / 32, at = (lane + 1) * step - 1;
        const bool le = at < n && p.offsets[lo + at] <= t;
        const unsigned k = __ffs(~__ballot_sync(~0u, le)) - 1;  // 32 probes true: 32 (ffs of 0 is 0)
        const unsigned found = k > 32 ? 32 : k;
        lo += found * step;
        n -= found * step;
        n = n < step - 1 ? n : step - 1;
    }
    return lo;
}
// The offsets that lie inside a chunk of tokens: `lo` of all are <= its first token, `hi` <= its last.  Few of them
// are held in shared memory.
constexpr unsigned kHeldOffsets = 512;
struct ChunkOffsets {
    unsigned lo, hi;
    long long held[kHeldOffsets];
};

// Walks a thread's tokens through the sequences.  `upto` is the number of offsets <= the token, so the token's
// sequence is upto - 1, none for 0 and sequences + 1.
struct SequenceWalk {
    unsigned upto, lo, hi;
    const long long *at;  // offsets lo, lo + 1, ...
    long long next;       // the offset that ends this sequence
    __device__ __forceinline__ SequenceWalk(const PolicyParams &p, const ChunkOffsets &c) {
        upto = lo = c.lo;
        hi = c.hi;
        at = hi > lo && hi - lo <= kHeldOffsets ? c.held : p.offsets + lo;
    }
    // The first token at or behind the last one sought.
    __device__ __forceinline__ void seek(long long t) {
        unsigned a = upto, b = hi;
        while (a < b) {
            const unsigned mid = a + (b - a) / 2;
            if (at[mid - lo] <= t)
                a = mid + 1;
            else
                b = mid;
        }
        upto = a;
        next = upto < hi ? at[upto - lo] : LLONG_MAX;  // the chunk ends before the offset behind `hi`
    }
    __device__ __forceinline__ void advance(long long t) {
        if (t >= next) seek(t);
    }
    __device__ __forceinline__ bool inside(const PolicyParams &p) const { return upto > 0 && upto <= p.sequences; }
};

// The whole block finds the offsets inside its chunk.
__device__ __forceinline__ void chunk_offsets(const PolicyParams &p, unsigned long long first, unsigned long long last,
                                              ChunkOffsets &c) {
    const int warp = threadIdx.x / 32;
    if (warp < 2) {
        const unsigned n = p.sequences ? offsets_upto_warp(p, static_cast<long long>(warp ? last : first)) : 0;
        if (threadIdx.x % 32 == 0) (warp ? c.hi : c.lo) = n;
    }
    __syncthreads();
    if (c.hi > c.lo && c.hi - c.lo <= kHeldOffsets) {
        for (unsigned k = threadIdx.x; k < c.hi - c.lo; k += blockDim.x) c.held[k] = p.offsets[c.lo + k];
        __syncthreads();
    }
}

static __global__ void __launch_bounds__(256) ar_policy_zero_kernel(const __grid_constant__ PolicyParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const size_t i = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i == 0) *p.counts = PolicyCounts{};
    if (i < p.sequences) p.per_sequence[i] = 0u;
}

// The sum of n over the block, in every thread.  `room`: a word for each warp.
__device__ __forceinline__ unsigned block_count(unsigned n, unsigned *room) {
    n = __reduce_add_sync(~0u, n);
    __syncthreads();
    if (threadIdx.x % 32 == 0) room[threadIdx.x / 32] = n;
    __syncthreads();
    unsigned s = 0;
    for (unsigned k = 0; k < blockDim.x / 32; ++k) s += room[k];
    return s;
}

// Bit k: token t0 + k counts as far as the mask and the array's end say.
__device__ __forceinline__ unsigned mask_bits(const PolicyParams &p, unsigned long long t0, unsigned long long end) {
    if (t0 >= end) return 0u;
    unsigned bits = end - t0 >= 8 ? 0xFFu : (1u << (end - t0)) - 1u;
    if (!p.mask) return bits;
    if (p.vec && bits == 0xFFu) {
        const uint2 m = *reinterpret_cast<const uint2 *>(p.mask + t0);
        bits = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) bits |= static_cast<unsigned>(((k < 4 ? m.x : m.y) >> (8 * (k & 3)) & 0xFFu) != 0) << k;
        return bits;
    }
    unsigned some = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) some |= static_cast<unsigned>((bits >> k & 1u) && p.mask[t0 + k] != 0) << k;
    return some;
}
// Bit k: token t0 + k lies between the first and the last offset.
__device__ __forceinline__ unsigned between_bits(unsigned long long t0, long long first, long long last) {
    const long long t = static_cast<long long>(t0);
    if (t >= first && t + 8 <= last) return 0xFFu;
    unsigned bits = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) bits |= static_cast<unsigned>(t + k >= first && t + k < last) << k;
    return bits;
}

// Adds up the counted tokens of each sequence; the whole block calls, each thread with eight tokens.
__device__ __forceinline__ void count_sequences(const PolicyParams &p, unsigned long long t0, unsigned bits, const ChunkOffsets &c,
                                                unsigned *room) {
    if (c.lo == c.hi) {  // one sequence
        const unsigned n = block_count(__popc(bits), room);
        if (threadIdx.x == 0 && n && c.lo > 0 && c.lo <= p.sequences) atomicAdd(p.per_sequence + c.lo - 1, n);
        return;
    }
    SequenceWalk w(p, c);
    w.seek(static_cast<long long>(t0));
    const unsigned lane0 = __shfl_sync(~0u, w.upto, 0);  // every lane takes part, whatever it finds below
    const bool same = w.next >= static_cast<long long>(t0) + 8 && w.upto == lane0;
    if (__all_sync(~0u, same)) {  // one sequence for the warp
        const unsigned n = __reduce_add_sync(~0u, __popc(bits));
        if (threadIdx.x % 32 == 0 && n && w.inside(p)) atomicAdd(p.per_sequence + w.upto - 1, n);
        return;
    }
    unsigned here = 0, at = w.upto;
    for (int k = 0; k < 8; ++k) {
        w.advance(static_cast<long long>(t0 + k));
        if (w.upto != at) {
            if (here) atomicAdd(p.per_sequence + at - 1, here);
            here = 0;
            at = w.upto;
        }
        here += w.inside(p) && (bits >> k & 1u);
    }
    if (here) atomicAdd(p.per_sequence + at - 1, here);
}

// Sequences with counted tokens, in every thread of the block.
__device__ __forceinline__ unsigned counted_sequences(const PolicyParams &p, unsigned *room) {
    unsigned some = 0;
    for (unsigned s = threadIdx.x; s < p.sequences; s += blockDim.x) some += __ldcg(p.per_sequence + s) > 0;
    return block_count(some, room);
}

// Counted tokens of each block, and the ticket of the launch behind this one.
static __global__ void __launch_bounds__(kPolicyThreads) ar_policy_count_tokens_kernel(const __grid_constant__ PolicyParams p) {
    __shared__ unsigned room[kPolicyThreads / 32];
    pdl_launch_dependents();
    pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.counts = PolicyCounts{};
    const long long first = p.sequences ? p.offsets[0] : 0, last = p.sequences ? p.offsets[p.sequences] : 0;
    unsigned n = 0;
#pragma unroll 4
    for (unsigned long long t = (static_cast<unsigned long long>(blockIdx.x) * kPolicyThreads + threadIdx.x) * 8; t < p.tokens;
         t += static_cast<unsigned long long>(gridDim.x) * kPolicyThreads * 8)
        n += __popc(mask_bits(p, t, p.tokens) & between_bits(t, first, last));
    n = block_count(n, room);
    if (threadIdx.x == 0) p.per_block[blockIdx.x] = n;
}

// Counted tokens of each sequence; the last block counts the sequences that have some.
static __global__ void __launch_bounds__(kPolicyThreads) ar_policy_count_kernel(const __grid_constant__ PolicyParams p) {
    __shared__ ChunkOffsets inner;
    __shared__ unsigned room[kPolicyThreads / 32];
    __shared__ bool last_block;
    pdl_launch_dependents();
    pdl_wait();
    const unsigned long long first = static_cast<unsigned long long>(blockIdx.x) * kPolicyChunk;
    const unsigned long long end = first + kPolicyChunk < p.tokens ? first + kPolicyChunk : p.tokens;
    const unsigned long long t0 = first + threadIdx.x * kPolicyEach;
    const unsigned bits = mask_bits(p, t0, end);
    chunk_offsets(p, first, end - 1, inner);
    if (p.sequences) count_sequences(p, t0, bits, inner, room);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last_block = atomicAdd(&p.counts->ticket, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last_block) return;
    __threadfence();
    const unsigned some = counted_sequences(p, room);
    if (threadIdx.x == 0) p.counts->sequences = some, p.counts->ticket = 0u;  // the ticket of the launch behind this one
}

// exp(d) - d - 1 and its derivative exp(d) - 1.  Near zero the first is d^2 / 2 + d^3 / 6 + ..., of which the
// difference would leave nothing: nine terms are off by less than 2^-27 of it up to |d| = 1/2.
__device__ __forceinline__ void kl_terms(float d, float &kl, float &slope) {
    float s = 1.0f / 3628800.0f;
    s = fmaf(s, d, 1.0f / 362880.0f);
    s = fmaf(s, d, 1.0f / 40320.0f);
    s = fmaf(s, d, 1.0f / 5040.0f);
    s = fmaf(s, d, 1.0f / 720.0f);
    s = fmaf(s, d, 1.0f / 120.0f);
    s = fmaf(s, d, 1.0f / 24.0f);
    s = fmaf(s, d, 1.0f / 6.0f);
    s = fmaf(s, d, 0.5f);
    const float near = s * d * d, far = expf(d) - 1.0f;
    const bool small = fabsf(d) < 0.5f;
    kl = small ? near : far - d;
    slope = small ? near + d : far;
}

// Whether a - b, which rounds to x, lies above (sign 1) or below (sign -1) a 64-bit limit.  x decides unless it is the
// rounded limit itself, because rounding keeps the order; then what rounding took from a - b, which is a float, decides.
__device__ __forceinline__ bool beyond(float x, float a, float b, const PolicyLimit &l, float sign) {
    if (x != l.x) return sign > 0.0f ? x > l.x : x < l.x;
    const float z = __fsub_rn(x, a);
    const float e = __fsub_rn(__fsub_rn(a, __fsub_rn(x, z)), __fadd_rn(b, z));
    const float at = e > l.rest ? 1.0f : e < l.rest ? -1.0f : -l.sign;
    return at * sign > 0.0f;
}

struct PolicySums {
    float gain = 0.0f, kl = 0.0f;
    unsigned clipped = 0, counted = 0;
};

// One counted token: its part of the sums under `weight`, and the gradient of its loss.
__device__ __forceinline__ float policy_token(const PolicyParams &p, float nll, float old_nll, float ref_nll, float adv,
                                              float weight, float beta, PolicySums &s) {
    const float x = p.old_nll ? old_nll - nll : 0.0f;
    const PolicyLimit limit = adv > 0.0f ? p.high : p.low;
    const bool clipped = p.old_nll && (adv > 0.0f || adv < 0.0f) && beyond(x, old_nll, nll, limit, adv);
    const float slope = clipped || adv == 0.0f ? 0.0f : expf(x) * adv;
    const float gain = clipped ? (adv > 0.0f ? p.limit_high : p.limit_low) * adv : slope;
    float kl = 0.0f, dkl = 0.0f;
    if (p.ref_nll) kl_terms(nll - ref_nll, kl, dkl);
    s.gain += weight * gain;
    s.kl += weight * kl;
    s.clipped += clipped;
    s.counted += 1;
    return beta == 0.0f ? slope : fmaf(beta, dkl, slope);
}

// Eight adjacent floats from token t on, those before `end`.
__device__ __forceinline__ void tokens8(const float *a, unsigned long long t, unsigned long long end, int vec, float (&v)[8]) {
    if (vec && t + 8 <= end) {
        const float4 q = *reinterpret_cast<const float4 *>(a + t), r = *reinterpret_cast<const float4 *>(a + t + 4);
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w, v[4] = r.x, v[5] = r.y, v[6] = r.z, v[7] = r.w;
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = t + k < end ? a[t + k] : 0.0f;
    }
}

// The eight tokens from t0 on: their sums, and their gradients.  `base`: scale over what the mean divides by; `bits`: which tokens
// the mask leaves; `c`: the chunk's offsets, where sequences matter.
__device__ __forceinline__ void policy_tokens(const PolicyParams &p, unsigned long long t0, unsigned long long end, unsigned bits,
                                              const float (&nll)[8], const float (&old_nll)[8], const float (&ref_nll)[8],
                                              const float (&adv)[8], float base, const ChunkOffsets &c, long long first, long long last,
                                              PolicySums &s) {
    const float beta = p.beta;
    float out[8];
    if (p.token_adv && p.mean != 2) {
        bits &= between_bits(t0, first, last);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            out[k] = 0.0f;
            if (bits >> k & 1u) out[k] = policy_token(p, nll[k], old_nll[k], ref_nll[k], adv[k], 1.0f, beta, s) * base;
        }
    } else {
        SequenceWalk w(p, c);
        unsigned at = ~0u;
        float a = 0.0f, weight = 1.0f;
        w.seek(static_cast<long long>(t0));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            out[k] = 0.0f;
            if (!(bits >> k & 1u) || !p.sequences) continue;
            w.advance(static_cast<long long>(t0 + k));
            if (!w.inside(p)) continue;
            if (w.upto != at) {
                at = w.upto;
                if (!p.token_adv) a = p.adv[at - 1];
                if (p.mean == 2) weight = 1.0f / static_cast<float>(__ldcg(p.per_sequence + at - 1));
            }
            out[k] = policy_token(p, nll[k], old_nll[k], ref_nll[k], p.token_adv ? adv[k] : a, weight, beta, s) * (base * weight);
        }
    }
    if (!p.dnll) return;
    if (p.vec && t0 + 8 <= end) {
        __stcs(reinterpret_cast<float4 *>(p.dnll + t0), make_float4(out[0], out[1], out[2], out[3]));
        __stcs(reinterpret_cast<float4 *>(p.dnll + t0 + 4), make_float4(out[4], out[5], out[6], out[7]));
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (t0 + k < end) p.dnll[t0 + k] = out[k];
    }
}

// The block's sums in 64 bits, in threads 0 .. 3.  `room`: [4][warps].
__device__ __forceinline__ double policy_block_sums(const PolicySums &s, float *room) {
    const unsigned warps = blockDim.x / 32;
    float v[4] = {s.gain, s.kl, static_cast<float>(s.clipped), static_cast<float>(s.counted)};  // counts: below 2^24
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) v[k] += __shfl_xor_sync(~0u, v[k], m);
        if (threadIdx.x % 32 == 0) room[k * warps + threadIdx.x / 32] = v[k];
    }
    __syncthreads();
    double sum = 0.0;
    if (threadIdx.x < 4)
        for (unsigned q = 0; q < warps; ++q) sum += room[threadIdx.x * warps + q];
    return sum;
}

// The totals from all sums; `some`: sequences with counted tokens.
__device__ __forceinline__ void policy_totals(const PolicyParams &p, double gain_sum, double kl_sum, double clipped, double tokens,
                                              unsigned some) {
    const double counted = tokens > 0.0 ? tokens : 1.0;
    const double n = p.mean == 1 ? counted : p.mean == 2 && some ? some : 1u;
    const double gain = 0.0 - p.scale * gain_sum / n, kl = p.scale * kl_sum / n;
    p.totals[0] = static_cast<float>(p.kl_weight == 0.0 ? gain : gain + p.kl_weight * kl);
    p.totals[1] = static_cast<float>(gain);
    p.totals[2] = static_cast<float>(kl);
    p.totals[3] = static_cast<float>(clipped / counted);
}

// The blocks' sums in a fixed order, by kPolicyThreads threads.
__device__ __forceinline__ void policy_join(const PolicyParams &p, unsigned some, double *room) {
    const int which = threadIdx.x % 4;
    double s = 0.0;
#pragma unroll 8
    for (unsigned b = threadIdx.x / 4; b < p.blocks; b += kPolicyThreads / 4) s += __ldcg(p.part + b * 4ull + which);
    room[threadIdx.x] = s;
    for (int n = kPolicyThreads / 2; n >= 4; n >>= 1) {
        __syncthreads();
        if (threadIdx.x < n) room[threadIdx.x] += room[threadIdx.x + n];
    }
    __syncthreads();
    if (threadIdx.x == 0) policy_totals(p, room[0], room[1], room[2], room[3], some);
}

// The chunks of the tokens in turn.  Behind a counting launch (JOIN) the last block joins the blocks' sums.
template <bool JOIN>
__global__ void __launch_bounds__(kPolicyThreads, 4) ar_policy_kernel(const __grid_constant__ PolicyParams p) {
    __shared__ ChunkOffsets inner;
    __shared__ unsigned counts[kPolicyThreads / 32];
    __shared__ float room[4 * kPolicyThreads / 32], shared_base;
    __shared__ double joined[kPolicyThreads];
    __shared__ float4 long_sums[kPolicyThreads];
    __shared__ bool last_block;
    pdl_launch_dependents();
    pdl_wait();
    long long from = 0, to = 0;
    if (p.sequences) from = p.offsets[0], to = p.offsets[p.sequences];
    unsigned n = 1, some = 1;
    if (p.mean == 1) {
        n = 0;
        for (unsigned b = threadIdx.x; b < p.count_blocks; b += kPolicyThreads) n += p.per_block[b];
        n = block_count(n, counts);
    } else if (p.mean == 2) {
        n = some = p.counts->sequences;
    }
    if (threadIdx.x == 0) shared_base = static_cast<float>(p.scale / (n ? n : 1u));
    __syncthreads();
    const float base = shared_base;
    const bool walk = !(p.token_adv && p.mean != 2);
    // A thread's tokens are added in two steps, those of a chunk and then the chunks, with what that loses: plain sums of equal
    // terms left the totals of 2^28 tokens 1.7e-5 off.  Between chunks the long sums wait in shared memory (in registers they
    // spilled).
    long_sums[threadIdx.x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    PolicySums s;
    for (unsigned long long first = static_cast<unsigned long long>(blockIdx.x) * kPolicyChunk; first < p.tokens;
         first += static_cast<unsigned long long>(gridDim.x) * kPolicyChunk) {
        const unsigned long long end = first + kPolicyChunk < p.tokens ? first + kPolicyChunk : p.tokens;
        const unsigned long long t0 = first + threadIdx.x * kPolicyEach;
        float nll[8], old_nll[8], ref_nll[8], adv[8];
        const unsigned bits = mask_bits(p, t0, end);
        if (t0 < end) {
            tokens8(p.nll, t0, end, p.vec, nll);
            if (p.old_nll) tokens8(p.old_nll, t0, end, p.vec, old_nll);
            if (p.ref_nll) tokens8(p.ref_nll, t0, end, p.vec, ref_nll);
            if (p.token_adv) tokens8(p.adv, t0, end, p.vec, adv);
        }
        if (walk) {
            __syncthreads();  // the offsets of the chunk before have been read
            chunk_offsets(p, first, end - 1, inner);
        }
        if (t0 < end) policy_tokens(p, t0, end, bits, nll, old_nll, ref_nll, adv, base, inner, from, to, s);
        const float4 q = long_sums[threadIdx.x];
        LongSum gain, kl;
        gain.sum = q.x, gain.lost = q.y, kl.sum = q.z, kl.lost = q.w;
        gain.add(s.gain);
        kl.add(s.kl);
        long_sums[threadIdx.x] = make_float4(gain.sum, gain.lost, kl.sum, kl.lost);
        s.gain = s.kl = 0.0f;
    }
    {
        const float4 q = long_sums[threadIdx.x];
        LongSum gain, kl;
        gain.sum = q.x, gain.lost = q.y, kl.sum = q.z, kl.lost = q.w;
        s.gain = gain.value(), s.kl = kl.value();
    }
    const double sum = policy_block_sums(s, room);
    if (threadIdx.x < 4) __stcg(p.part + blockIdx.x * 4ull + threadIdx.x, sum);
    if constexpr (JOIN) {
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) last_block = atomicAdd(&p.counts->ticket, 1u) == gridDim.x - 1;
        __syncthreads();
        if (!last_block) return;
        __threadfence();
        policy_join(p, some, joined);
    }
}

static __global__ void __launch_bounds__(kPolicyThreads) ar_policy_join_kernel(const __grid_constant__ PolicyParams p) {
    __shared__ double joined[kPolicyThreads];
    pdl_launch_dependents();
    pdl_wait();
    policy_join(p, 1u, joined);
}

// Few tokens: everything in one block.
static __global__ void __launch_bounds__(kPolicySmallThreads) ar_policy_small_kernel(const __grid_constant__ PolicyParams p) {
    __shared__ ChunkOffsets inner;
    __shared__ unsigned counts[32];
    __shared__ float room[4 * 32], shared_base;
    pdl_launch_dependents();
    pdl_wait();
    const unsigned chunk = blockDim.x * kPolicyEach;
    const bool walk = p.tokens && !(p.token_adv && p.mean != 2);  // no sequences: the chunk holds no offsets
    long long from = 0, to = 0;
    if (p.sequences) from = p.offsets[0], to = p.offsets[p.sequences];
    if (walk) chunk_offsets(p, 0, p.tokens - 1, inner);
    unsigned n = 1, some = 1;
    if (p.mean == 1) {
        n = 0;
        for (unsigned t0 = threadIdx.x * kPolicyEach; t0 < p.tokens; t0 += chunk)
            n += __popc(mask_bits(p, t0, p.tokens) & between_bits(t0, from, to));
        n = block_count(n, counts);
    } else if (p.mean == 2) {
        for (unsigned q = threadIdx.x; q < p.sequences; q += blockDim.x) p.per_sequence[q] = 0u;
        __threadfence();
        __syncthreads();
        if (p.sequences)
            for (unsigned first = 0; first < p.tokens; first += chunk) {
                const unsigned t0 = first + threadIdx.x * kPolicyEach;
                count_sequences(p, t0, mask_bits(p, t0, p.tokens), inner, counts);
            }
        __threadfence();
        __syncthreads();
        n = some = counted_sequences(p, counts);
    }
    if (threadIdx.x == 0) shared_base = static_cast<float>(p.scale / (n ? n : 1u));
    __syncthreads();
    const float base = shared_base;
    PolicySums s;
    for (unsigned t0 = threadIdx.x * kPolicyEach; t0 < p.tokens; t0 += chunk) {
        float nll[8], old_nll[8], ref_nll[8], adv[8];
        tokens8(p.nll, t0, p.tokens, p.vec, nll);
        if (p.old_nll) tokens8(p.old_nll, t0, p.tokens, p.vec, old_nll);
        if (p.ref_nll) tokens8(p.ref_nll, t0, p.tokens, p.vec, ref_nll);
        if (p.token_adv) tokens8(p.adv, t0, p.tokens, p.vec, adv);
        policy_tokens(p, t0, p.tokens, mask_bits(p, t0, p.tokens), nll, old_nll, ref_nll, adv, base, inner, from, to, s);
    }
    double sum = policy_block_sums(s, room);
    if (threadIdx.x < 32) {
        const double kl = __shfl_sync(~0u, sum, 1), clipped = __shfl_sync(~0u, sum, 2), counted = __shfl_sync(~0u, sum, 3);
        if (threadIdx.x == 0) policy_totals(p, sum, kl, clipped, counted, some);
    }
}

}  // namespace tps
