// Device code of ar_reduce_dropout and ar_reduce_dropout_grad.
//
// Both are bound by memory: the forward pass reads R (+1) tensors and writes
// n_dsts, the backward pass reads one and writes n_dxs.  The generator costs ten
// rounds of two 32x32-bit products for four elements, about a third of the time
// the memory needs at two ranks of bf16, and runs while the loads are in flight.
//
// Measured (graph of launches, three input sets in turn): without sums the backward pass writes and
// reads 6.3 TB/s (bf16 [4096, 8192], four destinations, 53.6 us), with a bias gradient 61.2 us, of which the
// kernel that adds the row blocks takes about 3.
//
// A thread owns eight adjacent columns (two Philox groups, one 16- or 32-byte
// vector) wherever a row starts in memory.  Rows that start off a vector
// boundary are read as the aligned vectors around the eight columns and shifted
// into place, and written as aligned vectors put together with the lane before
// (see load8 and store8), so no layout falls back to element-wise copies and
// columns stay with their threads, which the column sums of the backward pass
// need.
#pragma once

#include "ar_kernels_ex.cuh"
#include "ar_philox.cuh"

namespace tps {

// The dropout of one launch.
struct DropParams {
    PhiloxKeys keys;
    uint32_t off_lo, off_hi;  // counter words 2 and 3
    uint32_t threshold;       // keep a word >= threshold ...
    int any;                  // ... when this is set (0: p = 1, nothing is kept)
    float scale;              // 1 / (1 - p)
};

struct ArDropParams {
    ArExParams ex;
    DropParams drop;
    const void *bias;  // nullptr: none
    int bx, by;        // threads along a row and row groups of a block
    long long stride;  // the row stride of every source and destination, -1: they differ
};

struct ArDropGradParams {
    const void *dy;
    long long dy_stride;
    void *dx[kMaxDsts];
    long long dx_stride[kMaxDsts];
    unsigned long long ne0, ne1;
    int n_dxs;
    unsigned rows_per_block;
    DropParams drop;
    float *part_bias;  // [row block][ne0] partial column sums, nullptr: not wanted
    float *part_res;
    int bx, by;
    long long stride;  // the row stride of every destination, -1: they differ
};

constexpr int kDropCols = 8;   // columns of a thread

// The words of columns 8 * unit .. 8 * unit + 7 of `row`.
__device__ __forceinline__ void words8(const DropParams &d, unsigned row, unsigned long long unit,
                                       uint32_t (&w)[8]) {
#pragma unroll
    for (int g = 0; g < 2; ++g)
        philox4(d.keys, static_cast<uint32_t>(2 * unit + g), row, d.off_lo, d.off_hi,
                reinterpret_cast<uint32_t(&)[4]>(w[4 * g]));
}
// Bit k: column 8 * unit + k of `row` is kept.  One register instead of eight where the mask has to wait for
// loads (forward: 27.2 us against 29.2 at f32 [2048, 4096], two ranks).
__device__ __forceinline__ unsigned keep8(const DropParams &d, unsigned row, unsigned long long unit) {
    uint32_t w[8];
    words8(d, row, unit, w);
    unsigned bits = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) bits |= static_cast<unsigned>(w[k] >= d.threshold) << k;
    return d.any ? bits : 0u;
}
// A dropped element is 0 whatever it held.
__device__ __forceinline__ float dropped(const DropParams &d, uint32_t word, float x) {
    return d.any && word >= d.threshold ? __fmul_rn(x, d.scale) : 0.0f;
}

template <int T>
constexpr int kWords8 = 2 * Elem<T>::bytes;  // 32-bit words of eight elements: 8 or 4

// Eight elements as read: the words of the vector, or of the aligned vectors around it.
template <int T, bool ALIGNED>
struct Raw8 {
    uint32_t w[kWords8<T> + (ALIGNED ? 0 : 4)];
};

// words[k] = the word `bytes` (0..15, whole elements) further on in s.
template <int NW>
__device__ __forceinline__ void shift_words(const uint32_t (&s)[NW + 4], unsigned bytes, uint32_t (&out)[NW]) {
    uint32_t a[NW + 2], b[NW + 1];
#pragma unroll
    for (int k = 0; k < NW + 2; ++k) a[k] = (bytes & 8) ? s[k + 2] : s[k];
#pragma unroll
    for (int k = 0; k < NW + 1; ++k) b[k] = (bytes & 4) ? a[k + 1] : a[k];
#pragma unroll
    for (int k = 0; k < NW; ++k) out[k] = __funnelshift_r(b[k], b[k + 1], (bytes & 3) * 8);
}

// Ask for the eight elements at `at`, the columns from `col` of a row of ne0 (whole: all eight exist).
template <int T, bool ALIGNED>
__device__ __forceinline__ void load8(const char *at, unsigned long long col, unsigned long long ne0, bool whole,
                                      Raw8<T, ALIGNED> &r) {
    constexpr int NW = kWords8<T>, es = Elem<T>::bytes;
    const unsigned off = ALIGNED ? 0 : static_cast<unsigned>(reinterpret_cast<uintptr_t>(at) & 15);
    if (off == 0 && whole) {
        if constexpr (ALIGNED) {
            load_words<4 * NW, false>(at, reinterpret_cast<uint32_t(&)[NW]>(r.w));
        } else {
#pragma unroll
            for (int k = 0; k < NW; k += 4) {
                const uint4 q = *reinterpret_cast<const uint4 *>(at + 4 * k);
                r.w[k] = q.x, r.w[k + 1] = q.y, r.w[k + 2] = q.z, r.w[k + 3] = q.w;
            }
        }
        return;
    }
    if constexpr (!ALIGNED) {
        // the aligned vectors around the eight elements, where they lie inside the row
        if (whole && col > 0 && (ne0 - col - 8) * es >= 16 - off) {
            const char *base = at - off;
#pragma unroll
            for (int k = 0; k < NW + 4; k += 4) {
                const uint4 q = *reinterpret_cast<const uint4 *>(base + 4 * k);
                r.w[k] = q.x, r.w[k + 1] = q.y, r.w[k + 2] = q.z, r.w[k + 3] = q.w;
            }
            return;
        }
    }
    // the row's ends: one element after another, put where raw8_words will look for them
    uint32_t w[NW] = {};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (col + k < ne0) {
            if constexpr (T == kF32) {
                w[k] = *reinterpret_cast<const uint32_t *>(at + 4 * k);
            } else {
                w[k / 2] |= static_cast<uint32_t>(*reinterpret_cast<const unsigned short *>(at + 2 * k)) << (16 * (k & 1));
            }
        }
    if constexpr (ALIGNED) {
#pragma unroll
        for (int k = 0; k < NW; ++k) r.w[k] = w[k];
    } else {
        // moved up by `off` bytes
        uint32_t s[NW + 4], b[NW + 5];
#pragma unroll
        for (int k = 0; k < NW + 4; ++k) s[k] = k < NW ? w[k] : 0u;
        b[0] = 0u;
#pragma unroll
        for (int k = 0; k < NW + 4; ++k) b[k + 1] = s[k];
        uint32_t c[NW + 4], d[NW + 4];
#pragma unroll
        for (int k = 0; k < NW + 4; ++k) c[k] = __funnelshift_l(b[k], b[k + 1], (off & 3) * 8);
#pragma unroll
        for (int k = 0; k < NW + 4; ++k) d[k] = (off & 4) ? (k ? c[k - 1] : 0u) : c[k];
#pragma unroll
        for (int k = 0; k < NW + 4; ++k) r.w[k] = (off & 8) ? (k > 1 ? d[k - 2] : 0u) : d[k];
    }
}

// The words of the eight elements that load8 asked for at `at`.
template <int T, bool ALIGNED>
__device__ __forceinline__ void raw8_words(const Raw8<T, ALIGNED> &r, const char *at, uint32_t (&w)[kWords8<T>]) {
    if constexpr (ALIGNED) {
#pragma unroll
        for (int k = 0; k < kWords8<T>; ++k) w[k] = r.w[k];
    } else {
        shift_words<kWords8<T>>(r.w, static_cast<unsigned>(reinterpret_cast<uintptr_t>(at) & 15), w);
    }
}

// Store eight elements (those below ne0) at `at`.  Off a 16-byte boundary, a lane writes the aligned
// vectors that start with the last bytes of the lane before; `prev` / `next`: the lane before / after
// holds the eight columns before / after of the same row, all of them inside it.  The whole warp calls.
template <int T, bool ALIGNED>
__device__ __forceinline__ void store8(char *at, const uint32_t (&w)[kWords8<T>], unsigned long long col,
                                       unsigned long long ne0, bool whole, bool active, bool prev, bool next) {
    constexpr int NW = kWords8<T>, es = Elem<T>::bytes;
    auto element = [&](int k) {
        if constexpr (T == kF32) {
            *reinterpret_cast<uint32_t *>(at + 4 * k) = w[k];
        } else {
            *reinterpret_cast<unsigned short *>(at + 2 * k) = static_cast<unsigned short>(w[k / 2] >> (16 * (k & 1)));
        }
    };
    if constexpr (ALIGNED) {
        if (active && whole) {
            store_words<4 * NW>(at, w);
        } else if (active) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (col + k < ne0) element(k);
        }
    } else {
        const unsigned off = static_cast<unsigned>(reinterpret_cast<uintptr_t>(at) & 15);
        uint32_t s[NW + 4];
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] = __shfl_up_sync(~0u, w[NW - 4 + k], 1);
#pragma unroll
        for (int k = 0; k < NW; ++k) s[k + 4] = w[k];
        if (!active) return;
        if (!whole) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (col + k < ne0) element(k);
            return;
        }
        if (off == 0) {
#pragma unroll
            for (int k = 0; k < NW; k += 4)
                *reinterpret_cast<uint4 *>(at + 4 * k) = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
            return;
        }
        uint32_t o[NW];
        shift_words<NW>(s, 16 - off, o);  // from 16 - off bytes into [previous, own]: what belongs at at - off
        char *base = at - off;
#pragma unroll
        for (int k = 0; k < NW; k += 4)
            if (k > 0 || prev) *reinterpret_cast<uint4 *>(base + 4 * k) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const unsigned from = static_cast<unsigned>(k * es);  // bytes into the eight elements
            if ((!prev && from < 16 - off) || (!next && from >= 4 * NW - off)) element(k);
        }
    }
}

// Widened values of eight elements' words (no rounding).
template <int T>
__device__ __forceinline__ void widen8(const uint32_t (&w)[kWords8<T>], float (&x)[8]) {
    word_operands<T, T, kWords8<T>>(w, x);
}

// Block (x, y): columns [8 bx x, 8 bx (x+1)) of `by` rows.  A thread's loads of the residual, the
// bias and two ranks (16-bit types: four) are issued before the first is used, and its mask is made
// meanwhile.  The bias (and a broadcast residual) is read anew in every row, from L2.  One row at a
// time in 64 registers: two rows took 116 registers, two blocks of 256 threads an SM, and 31.0 us
// where this takes 27.7 (f32 [2048, 4096], two ranks, two destinations, bias and residual: 168 MB at
// 6.06 TB/s; bf16 [4096, 8192], four and four: 604 MB in 101.5 us, 5.95 TB/s).
template <int Td, int Tw, bool ALIGNED>
__global__ void __launch_bounds__(128, 8) ar_dropout_kernel(const __grid_constant__ ArDropParams p) {
    constexpr int NW = kWords8<Td>, RB = 16 / NW;
    pdl_launch_dependents();
    const ArExParams &x = p.ex;
    const int tx = threadIdx.x % p.bx, ty = threadIdx.x / p.bx;
    const unsigned long long unit = static_cast<unsigned long long>(blockIdx.x) * p.bx + tx, col = unit * kDropCols;
    const bool mine = ty < p.by && col < x.ne0;
    const bool whole = col + kDropCols <= x.ne0;
    const bool prev = tx > 0 && threadIdx.x % 32 > 0;
    const bool next = tx + 1 < p.bx && threadIdx.x % 32 < 31 && col + 16 <= x.ne0;
    const long long at = static_cast<long long>(col) * Elem<Td>::bytes;
    pdl_wait();
    const unsigned long long step = static_cast<unsigned long long>(gridDim.y) * p.by;
    for (unsigned long long row0 = static_cast<unsigned long long>(blockIdx.y) * p.by; row0 < x.ne1; row0 += step) {
        const unsigned row = static_cast<unsigned>(row0) + static_cast<unsigned>(ty);
        const bool on = mine && row0 + ty < x.ne1;
        const long long common = row * p.stride + at;
        auto place = [&](const void *base, long long stride) {
            return static_cast<const char *>(base) + (p.stride >= 0 ? common : row * stride + at);
        };
        Raw8<Td, ALIGNED> res, bias;
        if (on && x.residual) load8<Td, ALIGNED>(static_cast<const char *>(x.residual) + row * x.res_stride + at, col, x.ne0, whole, res);
        if (on && p.bias) load8<Td, ALIGNED>(static_cast<const char *>(p.bias) + at, col, x.ne0, whole, bias);
        float acc[8];
        unsigned keep = 0;
        for (int r0 = 0; r0 < x.R; r0 += RB) {
            Raw8<Td, ALIGNED> in[RB];
#pragma unroll
            for (int j = 0; j < RB; ++j)
                if (on && r0 + j < x.R && !((x.inactive >> (r0 + j)) & 1u))
                    load8<Td, ALIGNED>(place(x.src[r0 + j], x.src_stride[r0 + j]), col, x.ne0, whole, in[j]);
            if (r0 == 0) keep = keep8(p.drop, row, unit);
#pragma unroll
            for (int j = 0; j < RB; ++j) {
                const int r = r0 + j;
                if (r >= x.R) break;
                float v[8] = {};  // an inactive rank adds +0
                if (on && !((x.inactive >> r) & 1u)) {
                    uint32_t w[NW];
                    raw8_words<Td, ALIGNED>(in[j], place(x.src[r], x.src_stride[r]), w);
                    word_operands<Td, Tw, NW>(w, v);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[k] = r == 0 ? v[k] : __fadd_rn(acc[k], v[k]);
            }
        }
        float v[8];
        uint32_t w[NW];
        if (on && p.bias) {
            raw8_words<Td, ALIGNED>(bias, static_cast<const char *>(p.bias) + at, w);
            widen8<Td>(w, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] = __fadd_rn(acc[k], v[k]);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = (keep >> k) & 1u ? __fmul_rn(acc[k], p.drop.scale) : 0.0f;
        if (on && x.residual) {
            raw8_words<Td, ALIGNED>(res, static_cast<const char *>(x.residual) + row * x.res_stride + at, w);
            widen8<Td>(w, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] = __fadd_rn(acc[k], v[k]);
        }
        word_pack<Td, NW>(acc, w);
        for (int d = 0; d < x.n_dsts; ++d)
            store8<Td, ALIGNED>(const_cast<char *>(place(x.dst[d], x.dst_stride[d])), w, col, x.ne0, whole, on, prev, next);
    }
}

// The backward pass: block (x, y) takes eight columns per thread of row block y, its row groups in
// turn; each thread adds up its columns in registers (SUMS: 1 for dbias, 2 for dresidual, 3 for both), and the block
// adds its row groups in order.
template <int Td, bool ALIGNED, int SUMS>
__global__ void __launch_bounds__(512, 2) ar_dropout_grad_kernel(const __grid_constant__ ArDropGradParams p) {
    constexpr int NW = kWords8<Td>;
    __shared__ float sums[SUMS ? 512 * kDropCols : 1];
    pdl_launch_dependents();
    pdl_wait();
    const int tx = threadIdx.x % p.bx, ty = threadIdx.x / p.bx;
    const unsigned long long unit = static_cast<unsigned long long>(blockIdx.x) * p.bx + tx, col = unit * kDropCols;
    const bool mine = ty < p.by && col < p.ne0;
    const bool whole = col + kDropCols <= p.ne0;
    const bool prev = tx > 0 && threadIdx.x % 32 > 0;
    const bool next = tx + 1 < p.bx && threadIdx.x % 32 < 31 && col + 16 <= p.ne0;
    const long long at = static_cast<long long>(col) * Elem<Td>::bytes;
    const unsigned long long first = static_cast<unsigned long long>(blockIdx.y) * p.rows_per_block;
    const unsigned long long end = first + p.rows_per_block < p.ne1 ? first + p.rows_per_block : p.ne1;
    float sb[8] = {}, sr[8] = {};
    // the next row's elements are on their way while this row's words are made
    const unsigned rows = static_cast<unsigned>(end - first);
    const char *from = static_cast<const char *>(p.dy) + static_cast<long long>(first + ty) * p.dy_stride + at;
    const long long from_step = p.by * p.dy_stride, to_step = p.by * p.stride;
    long long to = static_cast<long long>(first + ty) * p.stride + at;
    Raw8<Td, ALIGNED> ahead;
    if (mine && ty < rows) load8<Td, ALIGNED>(from, col, p.ne0, whole, ahead);
    for (unsigned n0 = 0; n0 < rows; n0 += p.by) {
        const unsigned n = n0 + ty, row = static_cast<unsigned>(first) + n;
        const bool on = mine && n < rows;
        const Raw8<Td, ALIGNED> in = ahead;
        const char *here = from;
        from += from_step;
        if (mine && n + p.by < rows) load8<Td, ALIGNED>(from, col, p.ne0, whole, ahead);
        uint32_t rnd[8], w[NW];
        words8(p.drop, row, unit, rnd);
        float g[8] = {}, a[8];
        if (on) {
            raw8_words<Td, ALIGNED>(in, here, w);
            widen8<Td>(w, g);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            a[k] = dropped(p.drop, rnd[k], g[k]);
            if constexpr (SUMS & 1) sb[k] += a[k];
            if constexpr (SUMS & 2) sr[k] += g[k];
        }
        word_pack<Td, NW>(a, w);
        for (int d = 0; d < p.n_dxs; ++d)
            store8<Td, ALIGNED>(static_cast<char *>(p.dx[d]) + (p.stride >= 0 ? to : row * p.dx_stride[d] + at), w, col,
                                p.ne0, whole, on, prev, next);
        to += to_step;
    }
    if constexpr (SUMS) {
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            if (!(SUMS & (1 << which))) continue;
            float *part = which ? p.part_res : p.part_bias;
            __syncthreads();
            if (ty < p.by) {
#pragma unroll
                for (int k = 0; k < 8; ++k) sums[(ty * kDropCols + k) * p.bx + tx] = which ? sr[k] : sb[k];
            }
            __syncthreads();
            // column 8 * unit + k of the block, adjacent threads adjacent columns
            for (int c = threadIdx.x; c < p.bx * kDropCols; c += blockDim.x) {
                const unsigned long long i = static_cast<unsigned long long>(blockIdx.x) * p.bx * kDropCols + c;
                float s = 0.0f;
                for (int y = 0; y < p.by; ++y) s += sums[(y * kDropCols + c % kDropCols) * p.bx + c / kDropCols];
                if (i < p.ne0) part[blockIdx.y * p.ne0 + i] = s;
            }
        }
    }
}

// out[i] = sum over the row blocks of part[block][i]; blockIdx.y picks the sum.  32 columns and
// eight groups of row blocks to a block; the groups are added in order.
struct ColumnSums {
    const float *part[2];
    float *out[2];
    unsigned long long ne0;
    unsigned blocks;
};

static __global__ void __launch_bounds__(256) ar_column_sum_kernel(const __grid_constant__ ColumnSums p) {
    __shared__ float sums[8][32];
    pdl_launch_dependents();
    pdl_wait();
    const float *part = p.part[blockIdx.y];
    const int c = threadIdx.x % 32, g = threadIdx.x / 32;
    const size_t i = static_cast<size_t>(blockIdx.x) * 32 + c;
    float s = 0.0f;
    if (i < p.ne0) {
#pragma unroll 8
        for (unsigned b = g; b < p.blocks; b += 8) s += part[b * p.ne0 + i];
    }
    sums[g][c] = s;
    __syncthreads();
    if (g == 0 && i < p.ne0) {
        for (int q = 1; q < 8; ++q) s += sums[q][c];
        p.out[blockIdx.y][i] = s;
    }
}

}  // namespace tps
