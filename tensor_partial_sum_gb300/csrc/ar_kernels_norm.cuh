// Device code of ar_reduce_norm and ar_reduce_norm_grad.
#pragma once

#include "ar_codes.cuh"
#include "ar_kernels_ex.cuh"

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
