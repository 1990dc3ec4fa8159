// Device code of ar_reduce_norm, ar_reduce_norm_grad and the checkpoint calls.
//
// All are bound by memory where there are enough rows.  Measured on a GB300 in a graph of calls over input sets larger than
// L2, against the bytes that a call cannot do without at the copy rate of 6.78 TB/s:
//   forward, R = 2 f32 [n, 4096], two destinations, sum kept, bias, weight, shift, residual: 2048 rows 38.4 us (77%),
//   16384 rows 244 us (97%); R = 2 bf16 [4096, 4096], one destination 34.8 us (71%);
//   backward, f32 [n, 4096] to two, dsum: 2048 rows with three column sums 36.0 us (69%), 4096 rows without sums
//   55.5 us (89%);
//   forward and backward by an e4m3 checkpoint, R = 4 bf16 [4096, 8192] to four: 183 us (87%);
//   checkpoint written and read, f32 [2048, 4096]: 15.7 us (79%), bf16 [4096, 8192]: 33.8 us (89%).
// What is lost at 2048 rows is the start and end of each wave of blocks, and of the backward pass the 4 to 7 us that
// partial column sums take through L2.
#pragma once

#include "ar_codes.cuh"
#include "ar_kernels_ex.cuh"
#include "ar_norm_plan.h"
#include "ar_umma.cuh"
#include "ar_pairs.cuh"
#include "ar_rows8.cuh"

namespace tps {

// A tensor's rows; no byte in front of the first or behind the last element is read.  `apart`: rows are 64 bytes or
// more apart, so that only the first and the last row's vectors can reach outside.
struct RowSource {
    const char *base, *end;
    long long wide;   // the stride, and where it fits 32 bits:
    unsigned stride;
    int apart;
    __device__ __forceinline__ const char *row(unsigned r) const { return base + static_cast<unsigned long long>(r) * stride; }
};

struct NormParams {
    ArExParams ex;
    void *sum[kMaxDsts];
    long long sum_stride[kMaxDsts];
    int n_sums;
    int wire;  // the type operands are rounded through; kF32: none
    int rms;
    float eps, inv_n;
    const void *weight, *shift, *bias;
    float *mean, *rstd;
    CodeRows kept;
    // rows through shared memory
    RowSource source[kMaxRanks + 1];  // the active ranks in order, then the residual
    int n_sources;
    int apart;         // every source's rows are
    int rows_aligned;  // weight, shift and bias start on 16-byte boundaries
    int bx;            // lanes along a row (a warp's)
    int units;         // of a thread
    int cluster_bits;  // log2 of the blocks along a row
};

struct NormGradParams {
    RowSource dy, h, dsum;  // h.base nullptr: kept in 8 bits; dsum.base nullptr: none
    CodeRows kept;
    const float *mean, *rstd;
    void *dx[kMaxDsts];
    long long dx_stride[kMaxDsts];
    int n_dxs;
    int rms;
    float inv_n;
    unsigned long long ne0, ne1;
    const void *weight;
    float *part[3];  // [row block][part_ld] partial column sums of dweight, dshift, dbias; nullptr: not wanted
    unsigned long long part_ld;
    int bx, cluster, stages, vecs;
    int apart, rows_aligned;  // as in NormParams
    unsigned *status;         // a wait that runs out sets bit 1
    unsigned long long timeout_ns;  // bound of every wait
    unsigned long long drop_row;    // test hook: this row's copies are never issued (~0 = none)
    // rows of any length
    float *row_sums;  // [2][ne1]: sum g and sum g x of each row
    unsigned rows_per_block;
};

// x rounded through the wire type, a value of the launch here.
__device__ __forceinline__ float wire_elem(int wire, float x) {
    float y = x;
    if (wire == kF16) wire2<kF32, kF16>(x, y);
    if (wire == kBF16) wire2<kF32, kBF16>(x, y);
    return x;
}

// A sum over the block with what its additions lost, the same in every thread and in a fixed order.  `room`: 64 floats.
__device__ __forceinline__ void block_long_sum(LongSum &s, float *room) {
    auto lanes = [&] {
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) {
            const float a = __shfl_xor_sync(~0u, s.sum, k), b = __shfl_xor_sync(~0u, s.lost, k);
            s.join(a, b);
        }
    };
    lanes();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    __syncthreads();
    if (lane == 0) room[warp] = s.sum, room[32 + warp] = s.lost;
    __syncthreads();
    s.sum = lane < warps ? room[lane] : 0.0f;
    s.lost = lane < warps ? room[32 + lane] : 0.0f;
    lanes();
}

// The sum h of one element before its rounding to T_dst.
template <int Td>
__device__ __forceinline__ float norm_fold(const NormParams &p, size_t row, size_t i) {
    const ArExParams &x = p.ex;
    float acc = 0.0f;
    for (int r0 = 0; r0 < x.R; r0 += 4) {
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = r0 + j;
            v[j] = r < x.R && !((x.inactive >> r) & 1u)
                       ? load_elem<Td, false>(static_cast<const char *>(x.src[r]) + static_cast<long long>(row) * x.src_stride[r],
                                              static_cast<long long>(i))
                       : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (r0 + j < x.R) {
                const float w = wire_elem(p.wire, v[j]);
                acc = r0 + j == 0 ? w : __fadd_rn(acc, w);
            }
    }
    if (p.bias) acc = __fadd_rn(acc, load_elem<Td, false>(p.bias, static_cast<long long>(i)));
    if (x.residual)
        acc = __fadd_rn(acc, load_elem<Td, false>(static_cast<const char *>(x.residual) + static_cast<long long>(row) * x.res_stride,
                                                  static_cast<long long>(i)));
    return acc;
}

// x rounded to T and widened again.
template <int T>
__device__ __forceinline__ float rounded(float x) {
    return wire1<kF32, T>(x);
}

// The first mean m, rounded to T: 16-bit elements' differences to it are exact, and floats' differences from values far
// from zero.  The row's mean is off by what m leaves of the sum; summing the differences again would not tell how much of it,
// because m's last bits lie below those of floats, and elements of one exponent are all rounded the same way.
template <int T>
__device__ __forceinline__ float first_mean(const LongSum &s, float inv_n) {
    return rounded<T>(s.sum * inv_n);
}
__device__ __forceinline__ float mean_rest(const LongSum &s, float m, float n, float inv_n) {
    return (fmaf(-n, m, s.sum) + s.lost) * inv_n;
}
// The mean m + off; an infinite m has no difference to anything.
__device__ __forceinline__ float norm_mean(float m, float off) { return off == off ? m + off : m; }
// 1 / sqrt(variance + eps) from the mean square about a value that is `off` away from the mean.  Not with fmaxf,
// which would make a number of a NaN.
__device__ __forceinline__ float norm_rstd(float square, float off, float eps) {
    const float v = square - off * off;
    return __frsqrt_rn((v < 0.0f ? 0.0f : v) + eps);
}

// A row of any length to a block, element by element: the sum is formed three times (for the mean, the squares,
// the results).  Squares are taken about m: a row far from zero loses nothing to its offset.  They are carried with what their
// additions lose as well: plain sums of a thread's squares left rstd of 30 million bf16 columns 5e-5 off.
template <int Td>
__global__ void __launch_bounds__(512) ar_norm_any_kernel(const __grid_constant__ NormParams p) {
    __shared__ float room[64];
    pdl_launch_dependents();
    pdl_wait();
    const ArExParams &x = p.ex;
    for (size_t row = blockIdx.x; row < x.ne1; row += gridDim.x) {
        float m = 0.0f, off = 0.0f;
        LongSum squares;
        if (!p.rms) {
            LongSum s;
            for (size_t i = threadIdx.x; i < x.ne0; i += blockDim.x) s.add(rounded<Td>(norm_fold<Td>(p, row, i)));
            block_long_sum(s, room);
            m = first_mean<Td>(s, p.inv_n);
            // in 64 bits: not every length is a float
            off = static_cast<float>((static_cast<double>(s.sum) + s.lost) / static_cast<double>(x.ne0) - m);
        }
        for (size_t i = threadIdx.x; i < x.ne0; i += blockDim.x) {
            const float d = rounded<Td>(norm_fold<Td>(p, row, i)) - m;
            squares.add(d * d);
        }
        block_long_sum(squares, room);
        const float rstd = norm_rstd(squares.value() * p.inv_n, off, p.eps);
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[row] = norm_mean(m, off);
            if (p.rstd) p.rstd[row] = rstd;
        }
        const size_t end = (x.ne0 + 31) / 32 * 32;
        for (size_t i = threadIdx.x; i < end; i += blockDim.x) {
            const bool inside = i < x.ne0;
            const float h = inside ? rounded<Td>(norm_fold<Td>(p, row, i)) : 0.0f;
            if (p.kept.codes) encode_block(p.kept, row, i, h, inside);
            if (!inside) continue;
            float y = ((h - m) - off) * rstd;
            if (p.weight) y *= load_elem<Td, false>(p.weight, static_cast<long long>(i));
            if (p.shift) y += load_elem<Td, false>(p.shift, static_cast<long long>(i));
            for (int s = 0; s < p.n_sums; ++s)
                store_elem<Td>(static_cast<char *>(p.sum[s]) + static_cast<long long>(row) * p.sum_stride[s],
                               static_cast<long long>(i), h);
            for (int d = 0; d < x.n_dsts; ++d)
                store_elem<Td>(static_cast<char *>(x.dst[d]) + static_cast<long long>(row) * x.dst_stride[d],
                               static_cast<long long>(i), y);
        }
    }
}

// ---- rows in registers ------------------------------------------------------------

__device__ __forceinline__ void store_remote(const float *mine, unsigned rank, float v) {
    const unsigned at = static_cast<unsigned>(__cvta_generic_to_shared(mine));
    unsigned there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there), "f"(v) : "memory");
}

// Where the warps of a row's blocks leave their parts of sums.  Two rooms in turn need one barrier a sum: the next
// write to a room comes behind the barrier of the other.  (The forward pass takes each of them once.)
struct RowRoom {
    float2 v[kRowBlocks * kRowThreads / 32];
};

// The sums of a (and b) over a row, the same in all its threads and in a fixed order: over the `bx` lanes of a warp
// (WARP), over the block, or over the blocks of a cluster, which write into each other's shared memory.  LONG: a is a sum and
// b what its additions lost.
enum RowSum { kOne, kBoth, kLong };
template <bool WARP, RowSum KIND>
__device__ __forceinline__ void row_sum(float &a, float &b, int bx, int cluster, unsigned rank, RowRoom &room) {
    auto join = [&](float c, float d) {
        if constexpr (KIND == kLong) {
            LongSum s;
            s.sum = a, s.lost = b;
            s.join(c, d);
            a = s.sum, b = s.lost;
        } else {
            a += c;
            if constexpr (KIND == kBoth) b += d;
        }
    };
    auto lane_at = [&](int k) {
        const float c = __shfl_xor_sync(~0u, a, k), d = KIND == kOne ? 0.0f : __shfl_xor_sync(~0u, b, k);
        join(c, d);
    };
    if constexpr (WARP) {
        for (int k = bx / 2; k > 0; k >>= 1) lane_at(k);
    } else {
        auto lanes = [&] {
#pragma unroll KIND == kLong ? 1 : 5
            for (int k = 16; k > 0; k >>= 1) lane_at(k);
        };
        lanes();
        const int lane = threadIdx.x % 32, warps = static_cast<int>(blockDim.x) / 32, warp = threadIdx.x / 32;
        if (cluster == 1) {
            if (lane == 0) room.v[warp] = make_float2(a, b);
            __syncthreads();
            a = room.v[0].x, b = room.v[0].y;
            for (int k = 1; k < warps; ++k) {
                const float2 q = room.v[k];
                join(q.x, q.y);
            }
        } else {
            const int at = static_cast<int>(rank) * warps + warp;
            if (lane < cluster) {
                store_remote(&room.v[at].x, static_cast<unsigned>(lane), a);
                if constexpr (KIND != kOne) store_remote(&room.v[at].y, static_cast<unsigned>(lane), b);
            }
            cluster_sync();
            a = b = 0.0f;
            for (int k = lane; k < cluster * warps; k += 32) join(room.v[k].x, room.v[k].y);
            lanes();
        }
    }
}

// ---- rows through shared memory -----------------------------------------------------
//
// A thread copies the vectors of its own columns into shared memory some rows ahead and reads them back itself, so
// no barrier guards the ring, and what is in flight takes no registers.  Rows that start off a 16-byte boundary
// are copied as the aligned vectors around each unit of eight columns and shifted into place on the way out.

__device__ __forceinline__ void copy_async(unsigned to, const char *from, unsigned bytes) {
    // the bytes after `bytes` become 0
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Wait until all but the newest `ahead` (0..3) groups of this thread have landed.
__device__ __forceinline__ void copy_wait(int ahead) {
    if (ahead == 0)
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (ahead == 1)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    else if (ahead == 2)
        asm volatile("cp.async.wait_group 2;" ::: "memory");
    else
        asm volatile("cp.async.wait_group 3;" ::: "memory");
}

// 32-bit words of a unit: 32 bytes from 32-byte boundaries, else eight columns.
template <int T, bool ALIGNED>
constexpr int kUnitWords = ALIGNED ? 8 : kWords8<T>;
template <int T, bool ALIGNED>
constexpr int kUnitVecs = kUnitWords<T, ALIGNED> / 4 + (ALIGNED ? 0 : 1);  // its 16-byte vectors in the ring

// Copy the vectors of the unit at `at` to `to`, `step` bytes apart; `inner`: those around it lie inside the tensor.
template <int T, bool ALIGNED>
__device__ __forceinline__ void unit_copy(unsigned to, unsigned step, const char *at, const RowSource &s, bool inner) {
    constexpr int V = kUnitVecs<T, ALIGNED>;
    const unsigned off = ALIGNED ? 0u : static_cast<unsigned>(reinterpret_cast<uintptr_t>(at) & 15);
    const char *from = at - off;
    if (inner || (from >= s.base && from + 16 * V <= s.end)) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v < V - 1 || ALIGNED || off)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + v * step), "l"(from + 16 * v) : "memory");
        return;
    }
    // next to the tensor's ends
    for (int v = 0; v < V; ++v, from += 16, to += step) {
        if (from >= s.base && from < s.end) {
            const long long left = s.end - from;
            copy_async(to, from, left < 16 ? static_cast<unsigned>(left) : 16u);
        } else {
            // in front of the first element, or nothing at all: element by element
            for (int e = 0; e < 16; e += Elem<T>::bytes) {
                const bool inside = from + e >= s.base && from + e < s.end;
                if constexpr (T == kF32) {
                    const uint32_t x = inside ? *reinterpret_cast<const uint32_t *>(from + e) : 0u;
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + e), "r"(x) : "memory");
                } else {
                    const unsigned short x = inside ? *reinterpret_cast<const unsigned short *>(from + e) : static_cast<unsigned short>(0);
                    asm volatile("st.shared.b16 [%0], %1;" ::"r"(to + e), "h"(x) : "memory");
                }
            }
        }
    }
}

__device__ __forceinline__ uint4 read_shared(unsigned at) {
    uint4 q;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(at) : "memory");
    return q;
}

// The columns of the unit that unit_copy brought from an address whose low bits are `low`.
template <int T, bool ALIGNED>
__device__ __forceinline__ void unit_read(unsigned from, unsigned step, unsigned low, pair_t (&v)[kCols<T, kUnitWords<T, ALIGNED>> / 2]) {
    constexpr int W = kUnitWords<T, ALIGNED>;
    uint32_t w[W + (ALIGNED ? 0 : 4)];
#pragma unroll
    for (int k = 0; k < W + (ALIGNED ? 0 : 4); k += 4) {
        const uint4 q = read_shared(from + k / 4 * step);
        w[k] = q.x, w[k + 1] = q.y, w[k + 2] = q.z, w[k + 3] = q.w;
    }
    if constexpr (ALIGNED) {
        widen_pairs<T, W>(w, v);
    } else {
        uint32_t o[W];
        shift_words<W>(w, low & 15, o);
        widen_pairs<T, W>(o, v);
    }
}

// Which columns a thread holds: units of C, bx apart, in the bx lanes of a warp (WARP: 1 / bx of the block's
// threads to a row) or in the blocks of a cluster.
template <int C, int U, bool WARP>
struct RowThread {
    int bx, by, tx, ty, cluster;
    unsigned rank, col0;  // of unit 0
    int have[U];          // columns of each unit inside the row, 0..C
    bool prev;            // for store8: the lane before holds the columns before
    size_t group, groups;
    __device__ __forceinline__ RowThread(int p_bx, int p_cluster, unsigned ne0) {
        const int t = static_cast<int>(threadIdx.x);
        bx = WARP ? p_bx : static_cast<int>(blockDim.x);
        by = WARP ? static_cast<int>(blockDim.x) / bx : 1;
        tx = WARP ? t & (bx - 1) : t;
        ty = WARP ? t / bx : 0;
        cluster = WARP ? 1 : p_cluster;
        rank = cluster == 1 ? 0u : cluster_rank();
        col0 = (rank * static_cast<unsigned>(bx) * U + static_cast<unsigned>(tx)) * C;
        prev = tx > 0 && threadIdx.x % 32 > 0;
        group = blockIdx.x / static_cast<unsigned>(cluster);
        groups = gridDim.x / static_cast<unsigned>(cluster);
#pragma unroll
        for (int u = 0; u < U; ++u) have[u] = col(u) >= ne0 ? 0 : ne0 - col(u) >= C ? C : static_cast<int>(ne0 - col(u));
    }
    __device__ __forceinline__ unsigned col(int u) const { return col0 + static_cast<unsigned>(u * bx) * C; }
    __device__ __forceinline__ bool lane_next() const { return tx + 1 < bx && threadIdx.x % 32 < 31; }
};

// A unit as loaded: its own words, or the aligned vectors around it with the bytes to shift by.
template <int T, bool ALIGNED>
struct Unit {
    uint32_t w[kUnitWords<T, ALIGNED> + (ALIGNED ? 0 : 4)];
    unsigned shift;
};

// `have` elements at `at`, one by one.
template <int T, int W>
__device__ __forceinline__ void element_words(const char *at, int have, uint32_t (&w)[W]) {
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] = 0u;
#pragma unroll
    for (int k = 0; k < kCols<T, W>; ++k)
        if (k < have) {
            if constexpr (T == kF32)
                w[k] = *reinterpret_cast<const volatile uint32_t *>(at + 4 * k);
            else
                w[k / 2] |= static_cast<uint32_t>(*reinterpret_cast<const volatile unsigned short *>(at + 2 * k)) << (16 * (k & 1));
        }
}

// Load the unit at `at`, of which `have` columns are inside the row; `inner`: the vectors around it lie inside the
// tensor.
template <int T, bool ALIGNED>
__device__ __forceinline__ void unit_load(Unit<T, ALIGNED> &r, const char *at, const RowSource &s, bool inner, int have) {
    constexpr int W = kUnitWords<T, ALIGNED>;
    if constexpr (ALIGNED) {
        if (have == kCols<T, W>)
            load_words<4 * W, false>(at, r.w);
        else
            element_words<T, W>(at, have, r.w);
    } else {
        const unsigned off = static_cast<unsigned>(reinterpret_cast<uintptr_t>(at) & 15);
        const char *from = at - off;
        r.shift = off;
        if (inner || (from >= s.base && from + 4 * W + 16 <= s.end)) {
#pragma unroll
            for (int k = 0; k < W + 4; k += 4)
                if (k < W || off) load_words<16, false>(from + 4 * k, reinterpret_cast<uint32_t(&)[4]>(r.w[k]));
            return;
        }
        r.shift = 0;
        element_words<T, W>(at, have, reinterpret_cast<uint32_t(&)[W]>(r.w));
    }
}
template <int T, bool ALIGNED>
__device__ __forceinline__ void unit_pairs(const Unit<T, ALIGNED> &r, pair_t (&v)[kCols<T, kUnitWords<T, ALIGNED>> / 2]) {
    constexpr int W = kUnitWords<T, ALIGNED>;
    if constexpr (ALIGNED) {
        widen_pairs<T, W>(r.w, v);
    } else {
        uint32_t w[W];
        shift_words<W>(r.w, r.shift, w);
        widen_pairs<T, W>(w, v);
    }
}
// A unit of a row that every block reads, through L1.
template <int T, int W>
__device__ __forceinline__ void row_unit(const void *row, unsigned col, int have, bool aligned, uint32_t (&w)[W]) {
    const char *at = static_cast<const char *>(row) + col * Elem<T>::bytes;
    if (aligned && have == kCols<T, W>) {
#pragma unroll
        for (int k = 0; k < W; k += 4) {
            const uint4 q = __ldg(reinterpret_cast<const uint4 *>(at + 4 * k));
            w[k] = q.x, w[k + 1] = q.y, w[k + 2] = q.z, w[k + 3] = q.w;
        }
    } else {
        element_words<T, W>(at, have, w);
    }
}

// The first `have` elements of W words, one by one.
template <int T, int W>
__device__ __forceinline__ void element_store(char *at, int have, const uint32_t (&w)[W]) {
#pragma unroll
    for (int k = 0; k < kCols<T, W>; ++k)
        if (k < have) {
            if constexpr (T == kF32)
                *reinterpret_cast<uint32_t *>(at + 4 * k) = w[k];
            else
                *reinterpret_cast<unsigned short *>(at + 2 * k) = static_cast<unsigned short>(w[k / 2] >> (16 * (k & 1)));
        }
}

// Store a unit at `at`; see store8 for units off 16-byte boundaries.  The whole warp calls.
template <int T, bool ALIGNED>
__device__ __forceinline__ void unit_store(char *at, const uint32_t (&w)[kUnitWords<T, ALIGNED>], unsigned col, unsigned ne0, int have,
                                           bool prev, bool lane_next) {
    constexpr int W = kUnitWords<T, ALIGNED>;
    if constexpr (!ALIGNED) {
        store8<T, false>(at, w, col, ne0, have == 8, have > 0, prev, lane_next && col + 16 <= ne0);
    } else if (have == kCols<T, W>) {
        store_words<4 * W>(at, w);
    } else {
        element_store<T, W>(at, have, w);
    }
}

// The codes of a unit's columns from `col` on, of values that are 0 behind the row; the lanes that hold a block of 32
// columns are adjacent.  The whole warp calls.
template <int N>
__device__ __forceinline__ void unit_encode(const CodeRows &c, unsigned row, unsigned col, int have, const pair_t (&v)[N]) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const float2 f = halves(v[k]);
        top = max(top, max(__float_as_uint(f.x) & 0x7FFFFFFFu, __float_as_uint(f.y) & 0x7FFFFFFFu));
    }
    top = max(top, __shfl_xor_sync(~0u, top, 1));
    if constexpr (N == 4) top = max(top, __shfl_xor_sync(~0u, top, 2));
    if (!have) return;
    const unsigned byte = scale_byte(c.format, top);
    const pair_t inv = both(scale_inverse(byte));
    uint32_t w[N / 2] = {};
    if (byte != 255u) encode_pairs(c.format, v, inv, w);
    uint8_t *at = c.codes + row * static_cast<unsigned long long>(c.code_row) + col;
    if (have == 2 * N) {
        if constexpr (N == 8)
            asm volatile("st.global.cs.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
        else
            asm volatile("st.global.cs.v2.b32 [%0], {%1, %2};" ::"l"(at), "r"(w[0]), "r"(w[1]) : "memory");
    } else {
#pragma unroll
        for (int k = 0; k < 2 * N; ++k)
            if (k < have) at[k] = static_cast<uint8_t>(w[k / 4] >> (8 * (k & 3)));
    }
    if (col % kCodeBlock == 0) c.scales[row * static_cast<unsigned long long>(c.scale_row) + col / kCodeBlock] = static_cast<uint8_t>(byte);
}

// Blocks on an SM at least.  The kernel takes 60 registers a thread (eight blocks), 74 where a unit has 16 columns, 72 to 86
// where it is shifted into place.
template <int Td, bool ALIGNED, bool WARP>
constexpr int kNormBlocks = ALIGNED ? (WARP || Td != kF32 ? 6 : 7) : (WARP ? 5 : 7);

// The forward pass: bx lanes of a warp, a block or a cluster's blocks to a row, each thread with `units` units one
// after another; every block takes one turn of rows (a loop over them that ran once took 12 registers more).
// 128 threads a block: with 256 or 512 a row's phases overlap less with other rows' (f32 [2048, 4096]: 42 and 47 us against
// 37).  The sum h of a thread's columns waits in shared memory for the row's statistics, where only the thread itself reads
// it: no barrier, few registers, and enough blocks on an SM that their phases overlap.
template <int Td, bool ALIGNED, bool WARP>
__global__ void __launch_bounds__(kNormThreads, kNormBlocks<Td, ALIGNED, WARP>) ar_norm_kernel(const __grid_constant__ NormParams p) {
    constexpr int W = kUnitWords<Td, ALIGNED>, C = kCols<Td, W>, N = C / 2, RB = 16 / W;
    extern __shared__ uint4 held[];
    __shared__ RowRoom room[WARP ? 1 : 2];
    pdl_launch_dependents();
    const ArExParams &x = p.ex;
    const int T = static_cast<int>(blockDim.x), bx = WARP ? p.bx : T, by = WARP ? T / bx : 1, units = p.units;
    const int tx = WARP ? static_cast<int>(threadIdx.x) & (bx - 1) : static_cast<int>(threadIdx.x);
    const int ty = WARP ? static_cast<int>(threadIdx.x) / bx : 0;
    const int cluster = WARP ? 1 : 1 << p.cluster_bits;
    const unsigned rank = cluster == 1 ? 0u : cluster_rank();
    const unsigned ne0 = static_cast<unsigned>(x.ne0), ne1 = static_cast<unsigned>(x.ne1);
    const unsigned col0 = (rank * static_cast<unsigned>(bx * units) + static_cast<unsigned>(tx)) * C, hop = static_cast<unsigned>(bx) * C;
    const unsigned group = blockIdx.x >> (WARP ? 0 : p.cluster_bits);
    const int ranks = p.n_sources - (x.residual != nullptr);
    // every sum starts from -0, which changes no operand; an inactive rank adds +0, which turns a -0 into +0
    const pair_t start = both(x.inactive ? 0.0f : -0.0f);
    const bool prev = tx > 0 && threadIdx.x % 32 > 0, lane_next = tx + 1 < bx && threadIdx.x % 32 < 31;
    uint4 *const mine = held + threadIdx.x;
    pdl_wait();
    if (!WARP && cluster > 1) cluster_sync();  // every block of the cluster runs before one writes to another
    const unsigned row = group * by + static_cast<unsigned>(ty);
    const bool in_row = row < ne1, inner = p.apart && row > 0 && row + 1 < ne1;
    // how many columns of the unit at `col` are inside the row
    auto inside = [&](unsigned col) { return !in_row || col >= ne0 ? 0 : ne0 - col >= C ? C : static_cast<int>(ne0 - col); };
    auto put = [&](void *base, long long stride, unsigned col, int have, const uint32_t(&w)[W]) {
        unit_store<Td, ALIGNED>(static_cast<char *>(base) + static_cast<unsigned long long>(row) * static_cast<unsigned>(stride) +
                                    col * Elem<Td>::bytes,
                                w, col, ne0, have, prev, lane_next);
    };
    LongSum total;
    unsigned col = col0;
    for (int u = 0; u < units; ++u, col += hop) {
        const int have = inside(col);
        const unsigned at = col * Elem<Td>::bytes;
        pair_t acc[N];
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] = start;
        if (have) {
            Unit<Td, ALIGNED> res;
            pair_t v[N];
            if (x.residual) unit_load<Td, ALIGNED>(res, p.source[ranks].row(row) + at, p.source[ranks], inner, have);
            for (int s0 = 0; s0 < ranks; s0 += RB) {
                Unit<Td, ALIGNED> in[RB];
#pragma unroll
                for (int j = 0; j < RB; ++j)
                    if (s0 + j < ranks) unit_load<Td, ALIGNED>(in[j], p.source[s0 + j].row(row) + at, p.source[s0 + j], inner, have);
#pragma unroll
                for (int j = 0; j < RB; ++j) {
                    if (s0 + j >= ranks) break;
                    unit_pairs<Td, ALIGNED>(in[j], v);
                    wire_pairs<Td>(p.wire, v);
#pragma unroll
                    for (int k = 0; k < N; ++k) acc[k] = add2(acc[k], v[k]);
                }
            }
            if (p.bias) {
                uint32_t w[W];
                row_unit<Td, W>(p.bias, col, have, p.rows_aligned, w);
                widen_pairs<Td, W>(w, v);
#pragma unroll
                for (int k = 0; k < N; ++k) acc[k] = add2(acc[k], v[k]);
            }
            if (x.residual) {
                unit_pairs<Td, ALIGNED>(res, v);
#pragma unroll
                for (int k = 0; k < N; ++k) acc[k] = add2(acc[k], v[k]);
            }
        }
        if (have < C) first_pairs(acc, have);  // nothing behind the row's end, where the sums look
        uint32_t h[W];
        round_pairs<Td, W>(acc, h);
#pragma unroll
        for (int k = 0; k < W; k += 4) mine[(u * (W / 4) + k / 4) * T] = make_uint4(h[k], h[k + 1], h[k + 2], h[k + 3]);
        for (int s = 0; s < p.n_sums; ++s) put(p.sum[s], p.sum_stride[s], col, have, h);
        widen_pairs<Td, W>(h, acc);
        if (p.kept.codes) unit_encode(p.kept, row, col, have, acc);
        if (!p.rms) add_columns<Td>(acc, total);
    }
    auto take = [&](int u, pair_t(&v)[N]) {
        uint32_t h[W];
#pragma unroll
        for (int k = 0; k < W; k += 4) {
            const uint4 q = mine[(u * (W / 4) + k / 4) * T];
            h[k] = q.x, h[k + 1] = q.y, h[k + 2] = q.z, h[k + 3] = q.w;
        }
        widen_pairs<Td, W>(h, v);
    };
    float m = 0.0f, off = 0.0f, square = 0.0f, unused = 0.0f;
    if (!p.rms) {
        row_sum<WARP, kLong>(total.sum, total.lost, bx, cluster, rank, room[0]);
        m = first_mean<Td>(total, p.inv_n);
        off = mean_rest(total, m, static_cast<float>(ne0), p.inv_n);  // ne0 is below 2^24 here
    }
    col = col0;
    const pair_t minus_m = both(-m);
    for (int u = 0; u < units; ++u, col += hop) {
        pair_t v[N], q = 0;
        take(u, v);
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = add2(v[k], minus_m);
        const int have = inside(col);
        if (have < C) first_pairs(v, have);
#pragma unroll
        for (int k = 0; k < N; ++k) q = fma2(v[k], v[k], q);
        const float2 f = halves(q);
        square += f.x + f.y;
    }
    row_sum<WARP, kOne>(square, unused, bx, cluster, rank, room[WARP ? 0 : 1]);
    const float rstd = norm_rstd(square * p.inv_n, off, p.eps);
    if (in_row && col0 == 0) {
        if (p.mean) p.mean[row] = norm_mean(m, off);
        if (p.rstd) p.rstd[row] = rstd;
    }
    // ((h - m) - off) rstd
    const pair_t scale = both(rstd), rest = both(-off * rstd);
    col = col0;
    for (int u = 0; u < units; ++u, col += hop) {
        const int have = inside(col);
        pair_t v[N], f[N];
        uint32_t w[W], g[W];
        if (p.weight) row_unit<Td, W>(p.weight, col, have, p.rows_aligned, w);
        if (p.shift) row_unit<Td, W>(p.shift, col, have, p.rows_aligned, g);
        take(u, v);
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = fma2(add2(v[k], minus_m), scale, rest);
        if (p.weight) {
            widen_pairs<Td, W>(w, f);
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = mul2(v[k], f[k]);
        }
        if (p.shift) {
            widen_pairs<Td, W>(g, f);
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = add2(v[k], f[k]);
        }
        round_pairs<Td, W>(v, w);
        for (int d = 0; d < x.n_dsts; ++d) put(x.dst[d], x.dst_stride[d], col, have, w);
    }
}

// The backward pass in one pass over the rows, for rows off 32-byte boundaries, short ones and few ones: persistent blocks, dy,
// the kept sum and dsum of `stages` rows in the ring.  dy and x stay in registers while the row's two sums are taken; a thread adds up its columns, 16 at most,
// over its block's rows in registers.
template <int Td, bool ALIGNED, int U, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : kRowThreads, WARP ? 2 : 1) ar_norm_grad_kernel(const __grid_constant__ NormGradParams p) {
    constexpr int W = kUnitWords<Td, ALIGNED>, C = kCols<Td, W>, N = C / 2, V = kUnitVecs<Td, ALIGNED>;
    extern __shared__ uint4 ring[];
    __shared__ RowRoom room[WARP ? 1 : 2];
    pdl_launch_dependents();
    const unsigned ne0 = static_cast<unsigned>(p.ne0), ne1 = static_cast<unsigned>(p.ne1);
    const RowThread<C, U, WARP> t(p.bx, p.cluster, ne0);
    const unsigned hop = blockDim.x * 16u, step = hop * U;  // from a unit's vector to the next unit's, and to its own next
    const unsigned mine = static_cast<unsigned>(__cvta_generic_to_shared(ring)) + threadIdx.x * 16u;
    const unsigned stage_bytes = step * static_cast<unsigned>(p.vecs);
    const unsigned at_h = V * step, at_dsum = at_h + (p.kept.codes ? 1u : V) * step;
    pdl_wait();
    if (!WARP && t.cluster > 1) cluster_sync();
    pair_t weight[U][N], sw[U][N], ss[U][N], sb[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int k = 0; k < N; ++k) weight[u][k] = both(1.0f), sw[u][k] = ss[u][k] = sb[u][k] = 0;
        if (p.weight && t.have[u]) {
            uint32_t w[W];
            row_unit<Td, W>(p.weight, t.col(u), t.have[u], p.rows_aligned, w);
            widen_pairs<Td, W>(w, weight[u]);
        }
    }
    auto issue = [&](unsigned row, int stage) {
        if (row < ne1) {
            const unsigned to = mine + static_cast<unsigned>(stage) * stage_bytes;
            const bool inner = p.apart && row > 0 && row + 1 < ne1;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!t.have[u]) continue;
                const unsigned slot = to + u * hop, at = t.col(u) * Elem<Td>::bytes;
                unit_copy<Td, ALIGNED>(slot, step, p.dy.row(row) + at, p.dy, inner);
                if (p.kept.codes)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(slot + at_h),
                                 "l"(p.kept.codes + row * static_cast<unsigned long long>(p.kept.code_row) + t.col(u)), "n"(C == 16 ? 16 : 8),
                                 "r"(t.have[u])
                                 : "memory");
                else
                    unit_copy<Td, ALIGNED>(slot + at_h, step, p.h.row(row) + at, p.h, inner);
                if (p.dsum.base) unit_copy<Td, ALIGNED>(slot + at_dsum, step, p.dsum.row(row) + at, p.dsum, inner);
            }
        }
        copy_commit();
    };
    // what is read straight into registers, a row ahead
    float next_mean = 0.0f, next_rstd = 0.0f;
    unsigned next_scale[U] = {};
    auto fetch = [&](unsigned row) {
        if (row >= ne1) return;
        next_mean = p.rms ? 0.0f : p.mean[row];
        next_rstd = p.rstd[row];
        if (p.kept.codes) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (t.have[u]) next_scale[u] = p.kept.scales[row * static_cast<unsigned long long>(p.kept.scale_row) + t.col(u) / kCodeBlock];
        }
    };
    const unsigned turn = static_cast<unsigned>(t.groups) * t.by;
    unsigned ahead = static_cast<unsigned>(t.group) * t.by + t.ty;
    int put = 0, get = 0, parity = 0;
    fetch(ahead);
    for (int s = 0; s + 1 < p.stages; ++s, ahead += turn) issue(ahead, put++);
    for (unsigned row0 = static_cast<unsigned>(t.group) * t.by; row0 < ne1; row0 += turn, ahead += turn, parity ^= 1) {
        issue(ahead, put);
        if (++put == p.stages) put = 0;
        const unsigned row = row0 + t.ty;
        const bool in_row = row < ne1;
        const pair_t minus_mean = both(-next_mean);
        const float rstd = next_rstd;
        unsigned scale[U];
#pragma unroll
        for (int u = 0; u < U; ++u) scale[u] = next_scale[u];
        fetch(row + turn);
        copy_wait(p.stages - 1);
        const unsigned from = mine + static_cast<unsigned>(get) * stage_bytes;
        if (++get == p.stages) get = 0;
        auto low = [&](const RowSource &s, int u) {
            return static_cast<unsigned>(reinterpret_cast<uintptr_t>(s.base)) + row * s.stride + t.col(u) * Elem<Td>::bytes;
        };
        pair_t dy[U][N], x[U][N], a2 = 0, b2 = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const unsigned slot = from + u * hop;
            unit_read<Td, ALIGNED>(slot, step, low(p.dy, u), dy[u]);
            if (p.kept.codes) {
                uint32_t c[N / 2];
                if constexpr (C == 16) {
                    const uint4 q = read_shared(slot + at_h);
                    c[0] = q.x, c[1] = q.y, c[N / 2 - 2] = q.z, c[N / 2 - 1] = q.w;
                } else {
                    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(c[0]), "=r"(c[1]) : "r"(slot + at_h) : "memory");
                }
                decode_pairs(p.kept.format, c, scale_value(scale[u]), x[u]);
            } else {
                unit_read<Td, ALIGNED>(slot + at_h, step, low(p.h, u), x[u]);
            }
#pragma unroll
            for (int k = 0; k < N; ++k) x[u][k] = mul2(add2(x[u][k], minus_mean), both(rstd));
            if (!in_row || t.have[u] < C) {
                first_pairs(dy[u], in_row ? t.have[u] : 0);
                first_pairs(x[u], in_row ? t.have[u] : 0);
            }
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const pair_t g = mul2(dy[u][k], weight[u][k]);
                a2 = add2(a2, g);
                b2 = fma2(g, x[u][k], b2);
            }
        }
        const float2 af = halves(a2), bf = halves(b2);
        float a = af.x + af.y, b = bf.x + bf.y;
        row_sum<WARP, kBoth>(a, b, t.bx, t.cluster, t.rank, room[WARP ? 0 : parity]);
        // rstd (g - a / n - x b / n)
        const pair_t k0 = both(rstd), k1 = both(p.rms ? 0.0f : -(a * p.inv_n) * rstd), k2 = both(-(b * p.inv_n) * rstd);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool on = in_row && t.have[u];
            pair_t d[N];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const pair_t g = mul2(dy[u][k], weight[u][k]);
                d[k] = fma2(x[u][k], k2, fma2(g, k0, k1));
                sw[u][k] = fma2(dy[u][k], x[u][k], sw[u][k]);
                ss[u][k] = add2(ss[u][k], dy[u][k]);
            }
            if (p.dsum.base) {
                pair_t f[N];
                unit_read<Td, ALIGNED>(from + at_dsum + u * hop, step, low(p.dsum, u), f);
#pragma unroll
                for (int k = 0; k < N; ++k) d[k] = add2(d[k], f[k]);
            }
            if (on) {
#pragma unroll
                for (int k = 0; k < N; ++k) sb[u][k] = add2(sb[u][k], d[k]);  // columns behind the row's end are not looked at
            }
            uint32_t w[W];
            round_pairs<Td, W>(d, w);
            for (int k = 0; k < p.n_dxs; ++k)
                unit_store<Td, ALIGNED>(static_cast<char *>(p.dx[k]) + static_cast<unsigned long long>(row) * static_cast<unsigned>(p.dx_stride[k]) +
                                            t.col(u) * Elem<Td>::bytes,
                                        w, t.col(u), ne0, on ? t.have[u] : 0, t.prev, t.lane_next());
        }
    }
    copy_wait(0);
    // this block's column sums; in the WARP form its row groups' are added in order
#pragma unroll
    for (int which = 0; which < 3; ++which) {
        if (!p.part[which]) continue;
        float *row = p.part[which] + t.group * p.part_ld;
        if constexpr (WARP) {
            float *sums = reinterpret_cast<float *>(ring);
            __syncthreads();
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const float2 f = halves(which == 0 ? sw[u][k] : which == 1 ? ss[u][k] : sb[u][k]);
                    sums[((t.ty * U + u) * C + 2 * k) * t.bx + t.tx] = f.x;
                    sums[((t.ty * U + u) * C + 2 * k + 1) * t.bx + t.tx] = f.y;
                }
            __syncthreads();
            const int width = t.bx * U * C;
            for (int c = threadIdx.x; c < width; c += blockDim.x) {
                // column c of the block: unit c / C, held by lane unit % bx as its unit / bx-th
                const int unit = c / C, at = (unit / t.bx * C + c % C) * t.bx + unit % t.bx;
                float s = 0.0f;
                for (int y = 0; y < t.by; ++y) s += sums[y * width + at];
                if (static_cast<unsigned>(c) < ne0) row[c] = s;
            }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!t.have[u]) continue;
#pragma unroll
                for (int k = 0; k < N; k += 2) {
                    const pair_t(&v)[N] = which == 0 ? sw[u] : which == 1 ? ss[u] : sb[u];
                    const float2 f = halves(v[k]), g = halves(v[k + 1]);
                    *reinterpret_cast<float4 *>(row + t.col(u) + 2 * k) = make_float4(f.x, f.y, g.x, g.y);
                }
            }
        }
    }
}

// The same for rows on 32-byte boundaries that take a block or more: the copy engine brings a row's share of dy, of the
// kept sum and of dsum (cp.async copies held the loads to 3 TB/s, whatever their depth: 4096 rows of 4096 floats took 92 us
// without the sums; this takes 55.5).  Blocks of a cluster that add their column sums before writing them: no gain with two,
// and with four not all blocks are resident (73 us).  A thread holds U 16-byte vectors, 16 columns, blockDim.x vectors apart, so that neither shared memory nor stores
// have bank conflicts or gaps.
template <int Td, bool BIAS>
__global__ void __launch_bounds__(kRowThreads) ar_norm_grad_rows_kernel(const __grid_constant__ NormGradParams p) {
    constexpr int W = 4, C = kCols<Td, W>, N = C / 2, U = 16 / C;
    extern __shared__ uint4 ring[];
    __shared__ RowRoom room[2];
    __shared__ unsigned long long full[4];
    __shared__ volatile unsigned lost;
    __shared__ unsigned stop;  // the row behind which nothing was issued any more, for thread 0
    pdl_launch_dependents();
    const unsigned ne0 = static_cast<unsigned>(p.ne0), ne1 = static_cast<unsigned>(p.ne1), T = blockDim.x;
    const RowThread<C, U, false> t(0, p.cluster, ne0);
    // a stage: dy, the kept sum (or its codes), dsum; this block's share of a row each
    const unsigned share = T * U * 16u, at_h = share, code_bytes = T * U * C, at_dsum = at_h + (p.kept.codes ? code_bytes : share);
    const unsigned stage_bytes = at_dsum + (p.dsum.base ? share : 0u);
    const unsigned base = static_cast<unsigned>(__cvta_generic_to_shared(ring)), first_col = t.rank * T * U * C, hop = T * 16u;
    const bool inside = t.have[U - 1] == C;  // all of this thread's columns are inside the row
    if (threadIdx.x == 0) {
        lost = 0, stop = ~0u;
        for (int s = 0; s < p.stages; ++s) mbar_init(&full[s], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    pdl_wait();
    if (t.cluster > 1) cluster_sync();
    pair_t weight[U][N], sw[U][N], ss[U][N], sb[BIAS ? U : 1][N];  // BIAS: dbias is wanted
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int k = 0; k < N; ++k) weight[u][k] = both(1.0f), sw[u][k] = ss[u][k] = sb[BIAS ? u : 0][k] = 0;
        if (p.weight && t.have[u]) {
            uint32_t w[W];
            row_unit<Td, W>(p.weight, t.col(u), t.have[u], p.rows_aligned, w);
            widen_pairs<Td, W>(w, weight[u]);
        }
    }
    // The bytes of a share that are copied: whole vectors up to the row's end, in the last row those inside the tensor.
    auto vectors = [&](unsigned bytes_before, unsigned row_bytes, bool last, unsigned most) {
        const unsigned end = last ? row_bytes / 16 * 16 : (row_bytes + 15) / 16 * 16;
        return end <= bytes_before ? 0u : end - bytes_before < most ? end - bytes_before : most;
    };
    auto issue = [&](unsigned row, int stage) {  // one thread
        constexpr unsigned es = Elem<Td>::bytes;
        const bool last = row + 1 == ne1;
        const unsigned n = vectors(first_col * es, ne0 * es, last, share);
        const unsigned nc = p.kept.codes ? vectors(first_col, ne0, last, code_bytes) : n;
        if (row == p.drop_row) return;
        char *to = reinterpret_cast<char *>(ring) + static_cast<unsigned>(stage) * stage_bytes;
        mbar_expect_tx(&full[stage], n + nc + (p.dsum.base ? n : 0u));
        if (n) bulk_load(to, p.dy.row(row) + first_col * es, n, &full[stage]);
        if (nc)
            bulk_load(to + at_h,
                      p.kept.codes ? reinterpret_cast<const char *>(p.kept.codes) + row * static_cast<unsigned long long>(p.kept.code_row) + first_col
                                   : p.h.row(row) + first_col * es,
                      nc, &full[stage]);
        if (n && p.dsum.base) bulk_load(to + at_dsum, p.dsum.row(row) + first_col * es, n, &full[stage]);
    };
    // what is read straight into registers, a row ahead
    float next_mean = 0.0f, next_rstd = 0.0f;
    unsigned next_scale[U] = {};
    auto fetch = [&](unsigned row) {
        if (row >= ne1) return;
        next_mean = p.rms ? 0.0f : p.mean[row];
        next_rstd = p.rstd[row];
        if (p.kept.codes) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (t.have[u]) next_scale[u] = p.kept.scales[row * static_cast<unsigned long long>(p.kept.scale_row) + t.col(u) / kCodeBlock];
        }
    };
    const unsigned turn = static_cast<unsigned>(t.groups);
    fetch(static_cast<unsigned>(t.group));
    if (threadIdx.x == 0)
        for (int s = 0; s < p.stages; ++s) {
            const unsigned row = static_cast<unsigned>(t.group) + s * turn;
            if (row < ne1) issue(row, s);
        }
    int stage = 0;
    unsigned phase = 0, parity = 0;
    for (unsigned row = static_cast<unsigned>(t.group); row < ne1; row += turn, parity ^= 1) {
        const pair_t minus_mean = both(-next_mean);
        const float rstd = next_rstd;
        const bool last = row + 1 == ne1;
        unsigned scale[U];
#pragma unroll
        for (int u = 0; u < U; ++u) scale[u] = next_scale[u];
        fetch(row + turn);
        // Behind a copy that came too late nothing is issued any more, and no row waits longer than the first try.
        const unsigned bar = smem_u32(&full[stage]);
        if (!mbar_try(bar, phase, 20000u) && !lost && !mbar_wait_slow(bar, phase, &lost, p.timeout_ns) && !lost) {
            lost = 1;
            atomicOr(p.status, 2u);
        }
        const unsigned from = base + static_cast<unsigned>(stage) * stage_bytes + threadIdx.x * 16u;
        pair_t dy[U][N], x[U][N], a2 = 0, b2 = 0;
        float a = 0.0f, b = 0.0f;
        // EDGE: some columns lie behind the row's end, or in the tensor's last vector, which is not copied
        auto half = [&](const bool edge, unsigned at, const RowSource &s, int u, pair_t(&v)[N]) {
            uint32_t w[W];
            if (edge && last && t.have[u] && t.have[u] < C) {
                element_words<Td, W>(s.row(row) + t.col(u) * Elem<Td>::bytes, t.have[u], w);
            } else {
                const uint4 q = read_shared(from + at + u * hop);
                w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
            }
            widen_pairs<Td, W>(w, v);
        };
        auto sums = [&](const bool edge) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                half(edge, 0, p.dy, u, dy[u]);
                if (p.kept.codes) {
                    uint32_t c[N / 2] = {};
                    const unsigned at = from + at_h - threadIdx.x * (16u - C) + u * (T * C);
                    if (edge && last && t.have[u] && (ne0 - t.col(u)) < 16) {
                        const uint8_t *codes = p.kept.codes + row * static_cast<unsigned long long>(p.kept.code_row) + t.col(u);
#pragma unroll
                        for (int k = 0; k < C; ++k)
                            if (k < t.have[u]) c[k / 4] |= static_cast<uint32_t>(codes[k]) << (8 * (k & 3));
                    } else if constexpr (C == 8) {
                        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(c[0]), "=r"(c[N / 2 - 1]) : "r"(at) : "memory");
                    } else {
                        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(c[0]) : "r"(at) : "memory");
                    }
                    decode_pairs(p.kept.format, c, scale_value(scale[u]), x[u]);
                } else {
                    half(edge, at_h, p.h, u, x[u]);
                }
#pragma unroll
                for (int k = 0; k < N; ++k) x[u][k] = mul2(add2(x[u][k], minus_mean), both(rstd));
                if (edge && t.have[u] < C) {
                    first_pairs(dy[u], t.have[u]);
                    first_pairs(x[u], t.have[u]);
                }
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const pair_t g = mul2(dy[u][k], weight[u][k]);
                    a2 = add2(a2, g);
                    b2 = fma2(g, x[u][k], b2);
                }
            }
            const float2 af = halves(a2), bf = halves(b2);
            a = af.x + af.y, b = bf.x + bf.y;
        };
        auto results = [&](const bool edge) {
            // rstd (g - a / n - x b / n)
            const pair_t k0 = both(rstd), k1 = both(p.rms ? 0.0f : -(a * p.inv_n) * rstd), k2 = both(-(b * p.inv_n) * rstd);
            uint32_t w[U][W];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                pair_t d[N];
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const pair_t g = mul2(dy[u][k], weight[u][k]);
                    d[k] = fma2(x[u][k], k2, fma2(g, k0, k1));
                    sw[u][k] = fma2(dy[u][k], x[u][k], sw[u][k]);
                    ss[u][k] = add2(ss[u][k], dy[u][k]);
                }
                if (p.dsum.base) {
                    pair_t f[N];
                    half(edge, at_dsum, p.dsum, u, f);
#pragma unroll
                    for (int k = 0; k < N; ++k) d[k] = add2(d[k], f[k]);
                }
                if constexpr (BIAS) {  // columns behind the row's end are not looked at
#pragma unroll
                    for (int k = 0; k < N; ++k) sb[u][k] = add2(sb[u][k], d[k]);
                }
                round_pairs<Td, W>(d, w[u]);
            }
            for (int k = 0; k < p.n_dxs; ++k) {
                char *to = static_cast<char *>(p.dx[k]) + static_cast<unsigned long long>(row) * static_cast<unsigned>(p.dx_stride[k]) +
                           t.col(0) * Elem<Td>::bytes;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (!edge || t.have[u] == C)
                        store_words<16>(to + u * hop, w[u]);
                    else
                        element_store<Td, W>(to + u * hop, t.have[u], w[u]);
                }
            }
        };
        if (inside && !last)
            sums(false);
        else
            sums(true);
        row_sum<false, kBoth>(a, b, 0, t.cluster, t.rank, room[parity]);
        const bool gone = lost;  // the whole block has waited; read later it cost 3% of the rows from codes
        if (inside && !last)
            results(false);
        else
            results(true);
        __syncthreads();  // the stage has been read
        if (threadIdx.x == 0) {
            const unsigned next = row + static_cast<unsigned>(p.stages) * turn;
            if (gone)
                stop = stop < row ? stop : row;
            else if (next < ne1 && next > row)
                issue(next, stage);
        }
        if (++stage == p.stages) stage = 0, phase ^= 1;
    }
    if (lost && threadIdx.x == 0) {
        // a copy that comes too late must not find another block's shared memory: the last row of every stage is waited for,
        // at its own parity.  Every row in front of `stop` was followed by the issue of another, if there was one.
        const unsigned stages = static_cast<unsigned>(p.stages), first = static_cast<unsigned>(t.group);
        const unsigned rows = (ne1 - 1 - first) / turn + 1, some = (stop - first) / turn + stages, issued = some < rows ? some : rows;
        for (unsigned k = issued > stages ? issued - stages : 0u; k < issued; ++k)
            mbar_wait(&full[k % stages], k / stages & 1u, p.timeout_ns);
    }
#pragma unroll
    for (int which = 0; which < 3; ++which) {
        if (!p.part[which] || (which == 2 && !BIAS)) continue;
        float *row = p.part[which] + t.group * p.part_ld;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!t.have[u]) continue;
#pragma unroll
            for (int k = 0; k < N; k += 2) {
                const pair_t(&v)[N] = which == 0 ? sw[u] : which == 1 ? ss[u] : sb[BIAS ? u : 0];
                const float2 f = halves(v[k]), g = halves(v[k + 1]);
                *reinterpret_cast<float4 *>(row + t.col(u) + 2 * k) = make_float4(f.x, f.y, g.x, g.y);
            }
        }
    }
}

// dy, g = dy * weight and x of one element of the backward pass.
template <int Td>
__device__ __forceinline__ void grad_elem(const NormGradParams &p, size_t row, size_t i, float mean, float rstd, float &dy,
                                          float &g, float &x) {
    const long long at = static_cast<long long>(i);
    dy = load_elem<Td, false>(p.dy.base + static_cast<long long>(row) * p.dy.wide, at);
    const float h = p.h.base ? load_elem<Td, false>(p.h.base + static_cast<long long>(row) * p.h.wide, at)
                             : decode_elem(p.kept, row, i);
    g = p.weight ? dy * load_elem<Td, false>(p.weight, at) : dy;
    x = (h - mean) * rstd;
}

// Rows of any length, element by element, in two launches.  First a block takes each row's sums.
template <int Td>
__global__ void __launch_bounds__(512) ar_norm_row_sums_kernel(const __grid_constant__ NormGradParams p) {
    __shared__ float room[64];
    pdl_launch_dependents();
    pdl_wait();
    for (size_t row = blockIdx.x; row < p.ne1; row += gridDim.x) {
        const float mean = p.rms ? 0.0f : p.mean[row], rstd = p.rstd[row];
        LongSum a, b;
        for (size_t i = threadIdx.x; i < p.ne0; i += blockDim.x) {
            float dy, g, x;
            grad_elem<Td>(p, row, i, mean, rstd, dy, g, x);
            a.add(g);
            b.add(g * x);
        }
        block_long_sum(a, room);
        block_long_sum(b, room);
        if (threadIdx.x == 0) p.row_sums[row] = a.value(), p.row_sums[p.ne1 + row] = b.value();
    }
}

// Then block (x, y) takes 32 columns of row block y, eight rows at a time: the results, and the columns' sums.
template <int Td>
__global__ void __launch_bounds__(256) ar_norm_grad_any_kernel(const __grid_constant__ NormGradParams p) {
    __shared__ float sums[3][8][32];
    pdl_launch_dependents();
    pdl_wait();
    const int c = threadIdx.x % 32, g0 = threadIdx.x / 32;
    const size_t i = static_cast<size_t>(blockIdx.x) * 32 + c;
    const size_t first = static_cast<size_t>(blockIdx.y) * p.rows_per_block;
    const size_t end = first + p.rows_per_block < p.ne1 ? first + p.rows_per_block : p.ne1;
    float s[3] = {};
    if (i < p.ne0) {
        for (size_t row = first + g0; row < end; row += 8) {
            const float mean = p.rms ? 0.0f : p.mean[row], rstd = p.rstd[row];
            float dy, g, x;
            grad_elem<Td>(p, row, i, mean, rstd, dy, g, x);
            float d = g - x * (p.row_sums[p.ne1 + row] * p.inv_n);
            if (!p.rms) d -= p.row_sums[row] * p.inv_n;
            d *= rstd;
            if (p.dsum.base)
                d += load_elem<Td, false>(p.dsum.base + static_cast<long long>(row) * p.dsum.wide, static_cast<long long>(i));
            s[0] += dy * x;
            s[1] += dy;
            s[2] += d;
            for (int k = 0; k < p.n_dxs; ++k)
                store_elem<Td>(static_cast<char *>(p.dx[k]) + static_cast<long long>(row) * p.dx_stride[k],
                               static_cast<long long>(i), d);
        }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) sums[k][g0][c] = s[k];
    __syncthreads();
    if (g0 < 3 && i < p.ne0 && p.part[g0]) {
        float t = 0.0f;
        for (int q = 0; q < 8; ++q) t += sums[g0][q][c];
        p.part[g0][blockIdx.y * p.part_ld + i] = t;
    }
}

// out[i] = sum over the row blocks of part[block][i]; blockIdx.y picks the sum.  64 columns, four to a lane, and 32
// groups of row blocks to a block; the groups are added in order.
struct NormColumnSums {
    const float *part[3];
    float *out[3];
    unsigned long long ne0, ld;
    unsigned blocks;
};

static __global__ void __launch_bounds__(512) ar_norm_column_sum_kernel(const __grid_constant__ NormColumnSums p) {
    __shared__ float4 sums[32][17];
    pdl_launch_dependents();
    const float *part = p.part[blockIdx.y];
    const int c = threadIdx.x % 16, g = threadIdx.x / 16;
    const size_t i = (static_cast<size_t>(blockIdx.x) * 16 + c) * 4;
    pdl_wait();
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i < p.ne0) {
#pragma unroll 10
        for (unsigned b = g; b < p.blocks; b += 32) {
            const float4 f = *reinterpret_cast<const float4 *>(part + b * p.ld + i);
            s.x += f.x, s.y += f.y, s.z += f.z, s.w += f.w;
        }
    }
    sums[g][c] = s;
    __syncthreads();
    if (threadIdx.x < 64) {
        const size_t out = static_cast<size_t>(blockIdx.x) * 64 + threadIdx.x;
        float t = 0.0f;
#pragma unroll 8
        for (int q = 0; q < 32; ++q) t += reinterpret_cast<const float *>(&sums[q][0])[threadIdx.x];
        if (out < p.ne0) p.out[blockIdx.y][out] = t;
    }
}

// ---- checkpoints ----------------------------------------------------------------

struct PackParams {
    RowSource tensor;
    unsigned long long ne0, ne1;
    unsigned per_row;
    CodeRows kept;
};

// The row of a unit; 64-bit divisions only where they are needed.
__device__ __forceinline__ unsigned unit_row(size_t at, unsigned per_row) {
    return at >> 32 ? static_cast<unsigned>(at / per_row) : static_cast<unsigned>(at) / per_row;
}

// Where a column of a row starts; a flattened tensor's row may have 2^31 - 1 of them.
template <int T>
__device__ __forceinline__ size_t col_bytes(unsigned col) {
    return static_cast<size_t>(col) * Elem<T>::bytes;
}

// A unit of columns to a thread, the rows' units one after another; `per_row` of them (a whole number of blocks).
template <int Td, bool ALIGNED>
__global__ void __launch_bounds__(256) ar_checkpoint_pack_kernel(const __grid_constant__ PackParams p) {
    constexpr int C = kCols<Td, kUnitWords<Td, ALIGNED>>;
    pdl_launch_dependents();
    const size_t at = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    const unsigned row = unit_row(at, p.per_row), col = static_cast<unsigned>(at - static_cast<size_t>(row) * p.per_row) * C;
    const unsigned ne0 = static_cast<unsigned>(p.ne0), ne1 = static_cast<unsigned>(p.ne1);
    const int have = row >= ne1 || col >= ne0 ? 0 : ne0 - col >= C ? C : static_cast<int>(ne0 - col);
    pdl_wait();
    pair_t v[C / 2] = {};
    if (have) {
        Unit<Td, ALIGNED> r;
        unit_load<Td, ALIGNED>(r, p.tensor.row(row) + col_bytes<Td>(col), p.tensor, p.tensor.apart && row > 0 && row + 1 < ne1, have);
        unit_pairs<Td, ALIGNED>(r, v);
        if (have < C) first_pairs(v, have);
    }
    unit_encode(p.kept, row, col, have, v);
}

// At most T's largest finite value in magnitude; NaN stays.
template <int T>
__device__ __forceinline__ float saturated(float x) {
    constexpr float most = T == kF16 ? 65504.0f : T == kBF16 ? 3.3895313892515355e38f : 3.4028234663852886e38f;
    return x > most ? most : x < -most ? -most : x;
}

template <int Td, bool ALIGNED>
__global__ void __launch_bounds__(256) ar_checkpoint_unpack_kernel(const __grid_constant__ PackParams p) {
    constexpr int W = kUnitWords<Td, ALIGNED>, C = kCols<Td, W>, N = C / 2;
    pdl_launch_dependents();
    const size_t at = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    const unsigned row = unit_row(at, p.per_row), unit = static_cast<unsigned>(at - static_cast<size_t>(row) * p.per_row);
    const unsigned ne0 = static_cast<unsigned>(p.ne0), ne1 = static_cast<unsigned>(p.ne1), col = unit * C;
    const int have = row >= ne1 || col >= ne0 ? 0 : ne0 - col >= C ? C : static_cast<int>(ne0 - col);
    pdl_wait();
    uint32_t c[N / 2] = {}, w[W];
    unsigned scale = 0;
    if (have) {
        const uint8_t *from = p.kept.codes + row * static_cast<unsigned long long>(p.kept.code_row) + col;
        scale = p.kept.scales[row * static_cast<unsigned long long>(p.kept.scale_row) + col / kCodeBlock];
        if (have == C) {
            if constexpr (C == 16) {
                load_words<16, false>(from, reinterpret_cast<uint32_t(&)[4]>(c));
            } else {
                const uint2 q = *reinterpret_cast<const uint2 *>(from);
                c[0] = q.x, c[1] = q.y;
            }
        } else {
#pragma unroll
            for (int k = 0; k < C; ++k)
                if (k < have) c[k / 4] |= static_cast<uint32_t>(from[k]) << (8 * (k & 3));
        }
    }
    pair_t v[N];
    decode_pairs(p.kept.format, c, scale_value(scale), v);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const float2 f = halves(v[k]);
        v[k] = make_pair(saturated<Td>(f.x), saturated<Td>(f.y));
    }
    round_pairs<Td, W>(v, w);
    const unsigned prev = threadIdx.x % 32 > 0 && unit > 0, next = threadIdx.x % 32 < 31;
    unit_store<Td, ALIGNED>(const_cast<char *>(p.tensor.row(row)) + col_bytes<Td>(col), w, col, ne0, have, prev, next);
}

// The same for rows and strides past 32 bits: a warp to a block of 32 elements.
template <int Td>
__global__ void __launch_bounds__(256) ar_checkpoint_any_kernel(const __grid_constant__ PackParams p, bool pack) {
    pdl_launch_dependents();
    pdl_wait();
    const size_t per_row = (p.ne0 + 31) / 32, total = per_row * p.ne1;
    const size_t step = static_cast<size_t>(gridDim.x) * (blockDim.x / 32);
    for (size_t b = static_cast<size_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32; b < total; b += step) {
        const size_t row = b / per_row, i = b % per_row * 32 + threadIdx.x % 32;
        char *at = const_cast<char *>(p.tensor.base) + static_cast<long long>(row) * p.tensor.wide;
        const bool inside = i < p.ne0;
        if (pack)
            encode_block(p.kept, row, i, inside ? load_elem<Td, false>(at, static_cast<long long>(i)) : 0.0f, inside);
        else if (inside)
            store_elem<Td>(at, static_cast<long long>(i), saturated<Td>(decode_elem(p.kept, row, i)));
    }
}

}  // namespace tps
