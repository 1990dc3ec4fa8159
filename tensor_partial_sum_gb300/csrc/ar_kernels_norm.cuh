// Device code of ar_reduce_norm and ar_reduce_norm_grad.
#pragma once

#include "ar_codes.cuh"
#include "ar_kernels_ex.cuh"
#include "ar_rows8.cuh"

namespace tps {

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
    int bx;       // threads along a row in a block
    int cluster;  // blocks along a row
};

struct NormGradParams {
    const void *dy, *h, *dsum;  // h nullptr: kept in 8 bits
    long long dy_stride, h_stride, dsum_stride;
    CodeRows kept;
    const float *mean, *rstd;
    void *dx[kMaxDsts];
    long long dx_stride[kMaxDsts];
    int n_dxs;
    int rms;
    float inv_n;
    unsigned long long ne0, ne1;
    const void *weight;
    float *part[3];  // [row block][ne0] partial column sums of dweight, dshift, dbias; nullptr: not wanted
    float *row_sums; // [2][ne1]: sum g and sum g x of each row
    unsigned rows_per_block;
};

// x rounded through the wire type, a value of the launch here.
__device__ __forceinline__ float wire_elem(int wire, float x) {
    float y = x;
    if (wire == kF16) wire2<kF32, kF16>(x, y);
    if (wire == kBF16) wire2<kF32, kBF16>(x, y);
    return x;
}

// Sums of two floats over the block, the same in every thread and in a fixed order.  `room`: 64 floats.
__device__ __forceinline__ void block_sum2(float &a, float &b, float *room) {
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) {
        a += __shfl_xor_sync(~0u, a, k);
        b += __shfl_xor_sync(~0u, b, k);
    }
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    __syncthreads();
    if (lane == 0) room[warp] = a, room[32 + warp] = b;
    __syncthreads();
    a = lane < warps ? room[lane] : 0.0f;
    b = lane < warps ? room[32 + lane] : 0.0f;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) {
        a += __shfl_xor_sync(~0u, a, k);
        b += __shfl_xor_sync(~0u, b, k);
    }
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

// The mean m + off; an infinite m has no difference to anything.
__device__ __forceinline__ float norm_mean(float m, float off) { return off == off ? m + off : m; }
// 1 / sqrt(variance + eps) from the mean square about a value that is `off` away from the mean.  Not with fmaxf,
// which would make a number of a NaN.
__device__ __forceinline__ float norm_rstd(float square, float off, float eps) {
    const float v = square - off * off;
    return 1.0f / sqrtf((v < 0.0f ? 0.0f : v) + eps);
}

// A row of any length to a block, element by element: the sum is formed three times (for the mean, the squares,
// the results).  Squares are taken about the rounded mean m, and sum (h - m) corrects both what rounding the mean left
// and the squares: a row far from zero loses nothing to its offset.
template <int Td>
__global__ void __launch_bounds__(512) ar_norm_any_kernel(const __grid_constant__ NormParams p) {
    __shared__ float room[64];
    pdl_launch_dependents();
    pdl_wait();
    const ArExParams &x = p.ex;
    for (size_t row = blockIdx.x; row < x.ne1; row += gridDim.x) {
        float m = 0.0f, a = 0.0f, b = 0.0f;
        if (!p.rms) {
            for (size_t i = threadIdx.x; i < x.ne0; i += blockDim.x) a += rounded<Td>(norm_fold<Td>(p, row, i));
            block_sum2(a, b, room);
            m = a * p.inv_n;
        }
        a = b = 0.0f;
        for (size_t i = threadIdx.x; i < x.ne0; i += blockDim.x) {
            const float d = rounded<Td>(norm_fold<Td>(p, row, i)) - m;
            a += d;
            b += d * d;
        }
        block_sum2(a, b, room);
        const float off = p.rms ? 0.0f : a * p.inv_n;
        const float rstd = norm_rstd(b * p.inv_n, off, p.eps);
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

constexpr int kRowBlocks = 8;   // most blocks of a cluster along a row
constexpr int kRowThreads = 512;

// A wire rounding chosen at run time, of a unit's eight operands.
template <int Td>
__device__ __forceinline__ void wire8(int wire, float (&v)[8]) {
    if (wire == kF16) {
#pragma unroll
        for (int k = 0; k < 8; k += 2) wire2<Td, kF16>(v[k], v[k + 1]);
    } else if (wire == kBF16) {
#pragma unroll
        for (int k = 0; k < 8; k += 2) wire2<Td, kBF16>(v[k], v[k + 1]);
    }
}

__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_remote(const float *mine, unsigned rank, float v) {
    const unsigned at = static_cast<unsigned>(__cvta_generic_to_shared(mine));
    unsigned there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there), "f"(v) : "memory");
}

// Where the warps of a row's blocks leave their part of two sums.  Two of them in turn need one barrier a sum:
// the next write to a room comes behind the barrier of the other.
struct RowRoom {
    float a[kRowBlocks * kRowThreads / 32], b[kRowBlocks * kRowThreads / 32];
};

// The sums of a and b over a row, the same in all its threads and in a fixed order: over the `bx` lanes of a warp
// (WARP), over the block, or over the blocks of a cluster, which write into each other's shared memory.
template <bool WARP>
__device__ __forceinline__ void row_sum2(float &a, float &b, int bx, int cluster, unsigned rank, RowRoom &room) {
    if constexpr (WARP) {
        for (int k = bx / 2; k > 0; k >>= 1) {
            a += __shfl_xor_sync(~0u, a, k);
            b += __shfl_xor_sync(~0u, b, k);
        }
    } else {
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) {
            a += __shfl_xor_sync(~0u, a, k);
            b += __shfl_xor_sync(~0u, b, k);
        }
        const int lane = threadIdx.x % 32, warps = static_cast<int>(blockDim.x) / 32, warp = threadIdx.x / 32;
        int n = warps;
        if (cluster == 1) {
            if (lane == 0) room.a[warp] = a, room.b[warp] = b;
            __syncthreads();
        } else {
            n *= cluster;
            const int at = static_cast<int>(rank) * warps + warp;
            if (lane < cluster) {
                store_remote(&room.a[at], static_cast<unsigned>(lane), a);
                store_remote(&room.b[at], static_cast<unsigned>(lane), b);
            }
            cluster_barrier();
        }
        a = b = 0.0f;
        for (int k = lane; k < n; k += 32) a += room.a[k], b += room.b[k];
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) {
            a += __shfl_xor_sync(~0u, a, k);
            b += __shfl_xor_sync(~0u, b, k);
        }
    }
}

__device__ __forceinline__ float add8(const float (&v)[8]) {
    return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}

// The codes of eight columns from `col` on, of values that are 0 behind the row; four adjacent lanes hold a block
// of 32 columns.  The whole warp calls.
template <int NW>
__device__ __forceinline__ void encode8(const CodeRows &c, size_t row, unsigned long long col, unsigned long long ne0,
                                        const float (&v)[8], bool on) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(v[k]) & 0x7FFFFFFFu);
    top = max(top, __shfl_xor_sync(~0u, top, 1));
    top = max(top, __shfl_xor_sync(~0u, top, 2));
    if (!on) return;
    const unsigned byte = scale_byte(c.format, top);
    const float inv = scale_inverse(byte);
    uint32_t w[2] = {};
    if (byte != 255u) {
#pragma unroll
        for (int k = 0; k < 8; k += 2) w[k / 4] |= encode2(c.format, v[k] * inv, v[k + 1] * inv) << (8 * (k & 3));
    }
    uint8_t *at = c.codes + static_cast<long long>(row) * c.code_row + static_cast<long long>(col);
    if (col + 8 <= ne0) {
        asm volatile("st.global.cs.v2.b32 [%0], {%1, %2};" ::"l"(at), "r"(w[0]), "r"(w[1]) : "memory");
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (col + k < ne0) at[k] = static_cast<uint8_t>(w[k / 4] >> (8 * (k & 3)));
    }
    if (col % kCodeBlock == 0)
        c.scales[static_cast<long long>(row) * c.scale_row + static_cast<long long>(col / kCodeBlock)] = static_cast<uint8_t>(byte);
}

// A row in the registers of bx lanes (WARP: several rows a block, no barrier), of a block, or of a cluster's
// blocks; a thread holds U units of eight columns.
template <int Td, bool ALIGNED, int U, bool WARP>
__global__ void __launch_bounds__(WARP ? 128 : kRowThreads, WARP ? (U < 4 ? 8 : 4) : U < 4 ? 2 : 1)
    ar_norm_kernel(const __grid_constant__ NormParams p) {
    constexpr int NW = kWords8<Td>, RB = 16 / NW / U > 0 ? 16 / NW / U : 1;
    __shared__ RowRoom room[WARP ? 1 : 2];
    pdl_launch_dependents();
    const ArExParams &x = p.ex;
    const int bx = WARP ? p.bx : static_cast<int>(blockDim.x), by = WARP ? 128 / bx : 1;
    const int tx = WARP ? static_cast<int>(threadIdx.x) & (bx - 1) : static_cast<int>(threadIdx.x);
    const int ty = WARP ? static_cast<int>(threadIdx.x) / bx : 0;
    const int cluster = WARP ? 1 : p.cluster;
    const unsigned rank = WARP || cluster == 1 ? 0u : cluster_rank();
    const unsigned long long unit0 = static_cast<unsigned long long>(rank) * bx * U + tx;
    auto col_of = [&](int u) { return (unit0 + static_cast<unsigned long long>(u) * bx) * 8; };
    pdl_wait();
    if (!WARP && cluster > 1) cluster_barrier();  // every block of the cluster runs before one writes to another
    const size_t group = blockIdx.x / static_cast<unsigned>(cluster), groups = gridDim.x / static_cast<unsigned>(cluster);
    for (size_t row0 = group * by; row0 < x.ne1; row0 += groups * by) {
        const size_t row = row0 + ty;
        const bool in_row = row < x.ne1;
        const long long r64 = static_cast<long long>(row);
        uint32_t h[U][NW];
        {
            float acc[U][8];
            Raw8<Td, ALIGNED> res[U];
            auto res_at = [&](int u) {
                return static_cast<const char *>(x.residual) + r64 * x.res_stride + static_cast<long long>(col_of(u)) * Elem<Td>::bytes;
            };
            if (x.residual) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (in_row && col_of(u) < x.ne0) load8<Td, ALIGNED>(res_at(u), col_of(u), x.ne0, col_of(u) + 8 <= x.ne0, res[u]);
            }
            for (int r0 = 0; r0 < x.R; r0 += RB) {
                Raw8<Td, ALIGNED> in[RB][U];
                auto at = [&](int j, int u) {
                    return static_cast<const char *>(x.src[r0 + j]) + r64 * x.src_stride[r0 + j] +
                           static_cast<long long>(col_of(u)) * Elem<Td>::bytes;
                };
#pragma unroll
                for (int j = 0; j < RB; ++j)
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (in_row && col_of(u) < x.ne0 && r0 + j < x.R && !((x.inactive >> (r0 + j)) & 1u))
                            load8<Td, ALIGNED>(at(j, u), col_of(u), x.ne0, col_of(u) + 8 <= x.ne0, in[j][u]);
#pragma unroll
                for (int j = 0; j < RB; ++j) {
                    if (r0 + j >= x.R) break;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float v[8] = {};  // an inactive rank adds +0
                        if (in_row && col_of(u) < x.ne0 && !((x.inactive >> (r0 + j)) & 1u)) {
                            uint32_t w[NW];
                            raw8_words<Td, ALIGNED>(in[j][u], at(j, u), w);
                            widen8<Td>(w, v);
                            wire8<Td>(p.wire, v);
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k) acc[u][k] = r0 + j == 0 ? v[k] : __fadd_rn(acc[u][k], v[k]);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool on = in_row && col_of(u) < x.ne0;
                float v[8];
                uint32_t w[NW];
                if (on && p.bias) {
                    Raw8<Td, ALIGNED> b;
                    const char *at = static_cast<const char *>(p.bias) + col_of(u) * Elem<Td>::bytes;
                    load8<Td, ALIGNED>(at, col_of(u), x.ne0, col_of(u) + 8 <= x.ne0, b);
                    raw8_words<Td, ALIGNED>(b, at, w);
                    widen8<Td>(w, v);
#pragma unroll
                    for (int k = 0; k < 8; ++k) acc[u][k] = __fadd_rn(acc[u][k], v[k]);
                }
                if (on && x.residual) {
                    raw8_words<Td, ALIGNED>(res[u], res_at(u), w);
                    widen8<Td>(w, v);
#pragma unroll
                    for (int k = 0; k < 8; ++k) acc[u][k] = __fadd_rn(acc[u][k], v[k]);
                }
                word_pack<Td, NW>(acc[u], h[u]);
                if (!on) {
#pragma unroll
                    for (int k = 0; k < NW; ++k) h[u][k] = 0u;
                } else if (col_of(u) + 8 > x.ne0) {
                    // nothing behind the row's end, where the sums look
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (col_of(u) + k >= x.ne0) {
                            if constexpr (Td == kF32)
                                h[u][k] = 0u;
                            else
                                h[u][k / 2] &= k & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                        }
                }
            }
        }
        auto ends = [&](int u, bool &on, bool &whole, bool &prev, bool &next) {
            const unsigned long long col = col_of(u);
            on = in_row && col < x.ne0;
            whole = col + 8 <= x.ne0;
            prev = tx > 0 && threadIdx.x % 32 > 0;
            next = tx + 1 < bx && threadIdx.x % 32 < 31 && col + 16 <= x.ne0;
        };
        if (p.n_sums || p.kept.codes) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                bool on, whole, prev, next;
                ends(u, on, whole, prev, next);
                for (int s = 0; s < p.n_sums; ++s)
                    store8<Td, ALIGNED>(static_cast<char *>(p.sum[s]) + r64 * p.sum_stride[s] +
                                            static_cast<long long>(col_of(u)) * Elem<Td>::bytes,
                                        h[u], col_of(u), x.ne0, whole, on, prev, next);
                if (p.kept.codes) {
                    float v[8];
                    widen8<Td>(h[u], v);
                    encode8<NW>(p.kept, row, col_of(u), x.ne0, v, on);
                }
            }
        }
        float m = 0.0f, a = 0.0f, b = 0.0f;
        if (!p.rms) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float v[8];
                widen8<Td>(h[u], v);
                a += add8(v);
            }
            row_sum2<WARP>(a, b, bx, cluster, rank, room[0]);
            m = a * p.inv_n;
        }
        a = b = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[8], q[8];
            widen8<Td>(h[u], v);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[k] = col_of(u) + k < x.ne0 ? v[k] - m : 0.0f;
                q[k] = v[k] * v[k];
            }
            a += add8(v);
            b += add8(q);
        }
        row_sum2<WARP>(a, b, bx, cluster, rank, room[WARP ? 0 : 1]);
        const float off = p.rms ? 0.0f : a * p.inv_n;
        const float rstd = norm_rstd(b * p.inv_n, off, p.eps);
        if (in_row && unit0 == 0) {
            if (p.mean) p.mean[row] = norm_mean(m, off);
            if (p.rstd) p.rstd[row] = rstd;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            bool on, whole, prev, next;
            ends(u, on, whole, prev, next);
            float v[8], f[8];
            uint32_t w[NW];
            widen8<Td>(h[u], v);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = ((v[k] - m) - off) * rstd;
            auto factors = [&](const void *from) {
                Raw8<Td, ALIGNED> raw;
                const char *at = static_cast<const char *>(from) + col_of(u) * Elem<Td>::bytes;
                load8<Td, ALIGNED>(at, col_of(u), x.ne0, whole, raw);
                raw8_words<Td, ALIGNED>(raw, at, w);
                widen8<Td>(w, f);
            };
            if (on && p.weight) {
                factors(p.weight);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] *= f[k];
            }
            if (on && p.shift) {
                factors(p.shift);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] += f[k];
            }
            word_pack<Td, NW>(v, w);
            for (int d = 0; d < x.n_dsts; ++d)
                store8<Td, ALIGNED>(static_cast<char *>(x.dst[d]) + r64 * x.dst_stride[d] +
                                        static_cast<long long>(col_of(u)) * Elem<Td>::bytes,
                                    w, col_of(u), x.ne0, whole, on, prev, next);
        }
    }
}

// dy, g = dy * weight and x of one element of the backward pass.
template <int Td>
__device__ __forceinline__ void grad_elem(const NormGradParams &p, size_t row, size_t i, float mean, float rstd, float &dy,
                                          float &g, float &x) {
    const long long at = static_cast<long long>(i);
    dy = load_elem<Td, false>(static_cast<const char *>(p.dy) + static_cast<long long>(row) * p.dy_stride, at);
    const float h = p.h ? load_elem<Td, false>(static_cast<const char *>(p.h) + static_cast<long long>(row) * p.h_stride, at)
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
        float a = 0.0f, b = 0.0f;
        for (size_t i = threadIdx.x; i < p.ne0; i += blockDim.x) {
            float dy, g, x;
            grad_elem<Td>(p, row, i, mean, rstd, dy, g, x);
            a += g;
            b += g * x;
        }
        block_sum2(a, b, room);
        if (threadIdx.x == 0) p.row_sums[row] = a, p.row_sums[p.ne1 + row] = b;
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
            if (p.dsum)
                d += load_elem<Td, false>(static_cast<const char *>(p.dsum) + static_cast<long long>(row) * p.dsum_stride,
                                          static_cast<long long>(i));
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
        p.part[g0][blockIdx.y * p.ne0 + i] = t;
    }
}

// out[i] = sum over the row blocks of part[block][i]; blockIdx.y picks the sum.  32 columns and eight groups of
// row blocks to a block; the groups are added in order.
struct NormColumnSums {
    const float *part[3];
    float *out[3];
    unsigned long long ne0;
    unsigned blocks;
};

static __global__ void __launch_bounds__(256) ar_norm_column_sum_kernel(const __grid_constant__ NormColumnSums p) {
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

// ---- checkpoints ----------------------------------------------------------------

struct PackParams {
    void *tensor;
    long long stride;
    unsigned long long ne0, ne1;
    CodeRows kept;
};

// A warp to a block of 32 elements, the blocks of all rows in turn.
template <int Td>
__global__ void __launch_bounds__(256) ar_checkpoint_pack_kernel(const __grid_constant__ PackParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const size_t per_row = (p.ne0 + 31) / 32, total = per_row * p.ne1;
    const size_t step = static_cast<size_t>(gridDim.x) * (blockDim.x / 32);
    for (size_t b = static_cast<size_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32; b < total; b += step) {
        const size_t row = b / per_row, i = b % per_row * 32 + threadIdx.x % 32;
        const bool inside = i < p.ne0;
        const float x = inside ? load_elem<Td, false>(static_cast<const char *>(p.tensor) + static_cast<long long>(row) * p.stride,
                                                      static_cast<long long>(i))
                               : 0.0f;
        encode_block(p.kept, row, i, x, inside);
    }
}

// At most T's largest finite value in magnitude; NaN stays.
template <int T>
__device__ __forceinline__ float saturated(float x) {
    constexpr float most = T == kF16 ? 65504.0f : T == kBF16 ? 3.3895313892515355e38f : 3.4028234663852886e38f;
    return x > most ? most : x < -most ? -most : x;
}

template <int Td>
__global__ void __launch_bounds__(256) ar_checkpoint_unpack_kernel(const __grid_constant__ PackParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const size_t per_row = (p.ne0 + 31) / 32, total = per_row * p.ne1;
    const size_t step = static_cast<size_t>(gridDim.x) * (blockDim.x / 32);
    for (size_t b = static_cast<size_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32; b < total; b += step) {
        const size_t row = b / per_row, i = b % per_row * 32 + threadIdx.x % 32;
        if (i < p.ne0)
            store_elem<Td>(static_cast<char *>(p.tensor) + static_cast<long long>(row) * p.stride, static_cast<long long>(i),
                           saturated<Td>(decode_elem(p.kept, row, i)));
    }
}

}  // namespace tps
