// Device code of ar_reduce_dropout and ar_reduce_dropout_grad.
//
// Both are bound by memory: the forward pass reads R (+1) tensors and writes
// n_dsts, the backward pass reads one and writes n_dxs.  The generator costs ten
// rounds of two 32x32-bit products for four elements, about a third of the time
// the memory needs at two ranks of bf16, and runs while the loads are in flight.
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
};

constexpr int kDropCols = 8;   // columns of a thread
constexpr int kDropRows = 2;   // rows a thread has in flight

// Bit k: column 8 * unit + k of `row` is kept.
__device__ __forceinline__ unsigned keep8(const DropParams &d, unsigned long long row, unsigned long long unit) {
    unsigned bits = 0;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        uint32_t w[4];
        philox4(d.keys, static_cast<uint32_t>(2 * unit + g), static_cast<uint32_t>(row), d.off_lo, d.off_hi, w);
#pragma unroll
        for (int k = 0; k < 4; ++k) bits |= static_cast<unsigned>(w[k] >= d.threshold) << (4 * g + k);
    }
    return d.any ? bits : 0u;
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

// Ask for the `n` (1 to 8) elements at `at`, the columns from `col` of a row of ne0.
template <int T, bool ALIGNED>
__device__ __forceinline__ void load8(const char *at, unsigned long long col, unsigned long long ne0, Raw8<T, ALIGNED> &r) {
    constexpr int NW = kWords8<T>, es = Elem<T>::bytes;
    const unsigned off = ALIGNED ? 0 : static_cast<unsigned>(reinterpret_cast<uintptr_t>(at) & 15);
    const bool whole = col + 8 <= ne0;
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
                                       unsigned long long ne0, bool active, bool prev, bool next) {
    constexpr int NW = kWords8<T>, es = Elem<T>::bytes;
    const bool whole = col + 8 <= ne0;
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

// Block (x, y): columns [8 bx x, 8 bx (x+1)) of row groups of kDropRows rows.
// All loads of two ranks (16-bit types: four) for both rows are issued before the first is used;
// the masks are made meanwhile.  bf16 [4096, 8192], four ranks, four
// destinations and a residual: 604 MB; see the table of measurements.
template <int Td, int Tw, bool ALIGNED>
__global__ void __launch_bounds__(256) ar_dropout_kernel(const __grid_constant__ ArDropParams p) {
    constexpr int NW = kWords8<Td>, N = kDropRows, RB = 16 / NW;
    pdl_launch_dependents();
    const ArExParams &x = p.ex;
    const int tx = threadIdx.x % p.bx, ty = threadIdx.x / p.bx;
    const unsigned long long unit = static_cast<unsigned long long>(blockIdx.x) * p.bx + tx, col = unit * kDropCols;
    const bool mine = ty < p.by && col < x.ne0;
    const bool prev = tx > 0 && threadIdx.x % 32 > 0;
    const bool next = tx + 1 < p.bx && threadIdx.x % 32 < 31 && col + 16 <= x.ne0;
    const long long at = static_cast<long long>(col) * Elem<Td>::bytes;
    pdl_wait();
    float bias[8] = {}, row_res[8] = {};
    const bool broadcast = x.residual && x.res_stride == 0, full = x.residual && x.res_stride != 0;
    if (mine && p.bias) {
        Raw8<Td, ALIGNED> r;
        uint32_t w[NW];
        load8<Td, ALIGNED>(static_cast<const char *>(p.bias) + at, col, x.ne0, r);
        raw8_words<Td, ALIGNED>(r, static_cast<const char *>(p.bias) + at, w);
        widen8<Td>(w, bias);
    }
    if (mine && broadcast) {
        Raw8<Td, ALIGNED> r;
        uint32_t w[NW];
        load8<Td, ALIGNED>(static_cast<const char *>(x.residual) + at, col, x.ne0, r);
        raw8_words<Td, ALIGNED>(r, static_cast<const char *>(x.residual) + at, w);
        widen8<Td>(w, row_res);
    }
    const unsigned long long step = static_cast<unsigned long long>(gridDim.y) * p.by * N;
    for (unsigned long long row0 = static_cast<unsigned long long>(blockIdx.y) * p.by * N; row0 < x.ne1; row0 += step) {
        const unsigned long long row = row0 + static_cast<unsigned long long>(ty) * N;
        bool on[N];
#pragma unroll
        for (int n = 0; n < N; ++n) on[n] = mine && row + n < x.ne1;
        auto place = [&](const void *base, long long stride, int n) {
            return static_cast<const char *>(base) + static_cast<long long>(row + n) * stride + at;
        };
        Raw8<Td, ALIGNED> res[N];
        if (full) {
#pragma unroll
            for (int n = 0; n < N; ++n)
                if (on[n]) load8<Td, ALIGNED>(place(x.residual, x.res_stride, n), col, x.ne0, res[n]);
        }
        float acc[N][8];
        unsigned keep[N];
        for (int r0 = 0; r0 < x.R; r0 += RB) {
            Raw8<Td, ALIGNED> in[RB][N];
#pragma unroll
            for (int j = 0; j < RB; ++j)
                if (r0 + j < x.R && !((x.inactive >> (r0 + j)) & 1u)) {
#pragma unroll
                    for (int n = 0; n < N; ++n)
                        if (on[n]) load8<Td, ALIGNED>(place(x.src[r0 + j], x.src_stride[r0 + j], n), col, x.ne0, in[j][n]);
                }
            if (r0 == 0) {
#pragma unroll
                for (int n = 0; n < N; ++n) keep[n] = on[n] ? keep8(p.drop, row + n, unit) : 0u;
            }
#pragma unroll
            for (int j = 0; j < RB; ++j) {
                const int r = r0 + j;
                if (r >= x.R) break;
                const bool active = !((x.inactive >> r) & 1u);
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    float v[8] = {};  // an inactive rank adds +0
                    if (active && on[n]) {
                        uint32_t w[NW];
                        raw8_words<Td, ALIGNED>(in[j][n], place(x.src[r], x.src_stride[r], n), w);
                        word_operands<Td, Tw, NW>(w, v);
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) acc[n][k] = r == 0 ? v[k] : __fadd_rn(acc[n][k], v[k]);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float v[8];
            if (full && on[n]) {
                uint32_t w[NW];
                raw8_words<Td, ALIGNED>(res[n], place(x.residual, x.res_stride, n), w);
                widen8<Td>(w, v);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = row_res[k];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float a = acc[n][k];
                if (p.bias) a = __fadd_rn(a, bias[k]);
                a = (keep[n] >> k) & 1u ? __fmul_rn(a, p.drop.scale) : 0.0f;
                acc[n][k] = x.residual ? __fadd_rn(a, v[k]) : a;
            }
            uint32_t out[NW];
            word_pack<Td, NW>(acc[n], out);
            for (int d = 0; d < x.n_dsts; ++d)
                store8<Td, ALIGNED>(const_cast<char *>(place(x.dst[d], x.dst_stride[d], n)), out, col, x.ne0, on[n], prev,
                                    next);
        }
    }
}

// The backward pass: block (x, y) takes eight columns per thread of row block y, its row groups in
// turn; with SUMS each thread adds up its columns, and the block adds its row groups in order.
template <int Td, bool ALIGNED, bool SUMS>
__global__ void __launch_bounds__(512) ar_dropout_grad_kernel(const __grid_constant__ ArDropGradParams p) {
    constexpr int NW = kWords8<Td>, N = kDropRows;
    __shared__ float sums[SUMS ? 512 * kDropCols : 1];
    pdl_launch_dependents();
    pdl_wait();
    const int tx = threadIdx.x % p.bx, ty = threadIdx.x / p.bx;
    const unsigned long long unit = static_cast<unsigned long long>(blockIdx.x) * p.bx + tx, col = unit * kDropCols;
    const bool mine = ty < p.by && col < p.ne0;
    const bool prev = tx > 0 && threadIdx.x % 32 > 0;
    const bool next = tx + 1 < p.bx && threadIdx.x % 32 < 31 && col + 16 <= p.ne0;
    const long long at = static_cast<long long>(col) * Elem<Td>::bytes;
    const unsigned long long first = static_cast<unsigned long long>(blockIdx.y) * p.rows_per_block;
    const unsigned long long end = first + p.rows_per_block < p.ne1 ? first + p.rows_per_block : p.ne1;
    float sb[8] = {}, sr[8] = {};
    for (unsigned long long row0 = first; row0 < end; row0 += static_cast<unsigned long long>(p.by) * N) {
        const unsigned long long row = row0 + static_cast<unsigned long long>(ty) * N;
        Raw8<Td, ALIGNED> in[N];
        bool on[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            on[n] = mine && row + n < end;
            if (on[n])
                load8<Td, ALIGNED>(static_cast<const char *>(p.dy) + static_cast<long long>(row + n) * p.dy_stride + at, col,
                                   p.ne0, in[n]);
        }
        unsigned keep[N];
#pragma unroll
        for (int n = 0; n < N; ++n) keep[n] = on[n] ? keep8(p.drop, row + n, unit) : 0u;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float g[8] = {}, a[8];
            if (on[n]) {
                uint32_t w[NW];
                raw8_words<Td, ALIGNED>(in[n], static_cast<const char *>(p.dy) + static_cast<long long>(row + n) * p.dy_stride + at, w);
                widen8<Td>(w, g);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                a[k] = (keep[n] >> k) & 1u ? __fmul_rn(g[k], p.drop.scale) : 0.0f;
                if constexpr (SUMS) sb[k] += a[k], sr[k] += g[k];
            }
            uint32_t out[NW];
            word_pack<Td, NW>(a, out);
            for (int d = 0; d < p.n_dxs; ++d)
                store8<Td, ALIGNED>(static_cast<char *>(p.dx[d]) + static_cast<long long>(row + n) * p.dx_stride[d] + at, out,
                                    col, p.ne0, on[n], prev, next);
        }
    }
    if constexpr (SUMS) {
        for (int which = 0; which < 2; ++which) {
            float *part = which ? p.part_res : p.part_bias;
            if (!part) continue;
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
