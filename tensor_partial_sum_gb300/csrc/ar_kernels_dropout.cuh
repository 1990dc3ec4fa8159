// Device code of ar_reduce_dropout and ar_reduce_dropout_grad.
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
};

__device__ __forceinline__ bool keep_one(const DropParams &d, unsigned long long row, unsigned long long col) {
    uint32_t w[4];
    philox4(d.keys, static_cast<uint32_t>(col >> 2), static_cast<uint32_t>(row), d.off_lo, d.off_hi, w);
    const uint32_t lo = (col & 1) ? w[1] : w[0], hi = (col & 1) ? w[3] : w[2];
    return d.any && ((col & 2) ? hi : lo) >= d.threshold;
}

// One element per thread.
template <int Td, int Tw>
__global__ void __launch_bounds__(256) ar_dropout_kernel(const __grid_constant__ ArDropParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const ArExParams &x = p.ex;
    const size_t step = static_cast<size_t>(gridDim.x) * blockDim.x;
    for (size_t row = blockIdx.y; row < x.ne1; row += gridDim.y)
        for (size_t i = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < x.ne0; i += step) {
            float a = ex_operand<Td, Tw>(x, 0, row, i);
            for (int r = 1; r < x.R; ++r) a = __fadd_rn(a, ex_operand<Td, Tw>(x, r, row, i));
            if (p.bias) a = __fadd_rn(a, load_elem<Td, false>(p.bias, static_cast<long long>(i)));
            a = keep_one(p.drop, row, i) ? __fmul_rn(a, p.drop.scale) : 0.0f;
            if (x.residual)
                a = __fadd_rn(a, load_elem<Td, false>(static_cast<const char *>(x.residual) +
                                                          static_cast<long long>(row) * x.res_stride,
                                                      static_cast<long long>(i)));
            for (int d = 0; d < x.n_dsts; ++d)
                store_elem<Td>(static_cast<char *>(x.dst[d]) + static_cast<long long>(row) * x.dst_stride[d],
                               static_cast<long long>(i), a);
        }
}

// One column per thread, the rows of one row block after another.
template <int Td>
__global__ void __launch_bounds__(256) ar_dropout_grad_kernel(const __grid_constant__ ArDropGradParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const size_t step = static_cast<size_t>(gridDim.x) * blockDim.x;
    const size_t first = static_cast<size_t>(blockIdx.y) * p.rows_per_block;
    const size_t end = first + p.rows_per_block < p.ne1 ? first + p.rows_per_block : p.ne1;
    for (size_t i = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < p.ne0; i += step) {
        float sb = 0.0f, sr = 0.0f;
        for (size_t row = first; row < end; ++row) {
            const float g = load_elem<Td, false>(static_cast<const char *>(p.dy) +
                                                     static_cast<long long>(row) * p.dy_stride,
                                                 static_cast<long long>(i));
            const float a = keep_one(p.drop, row, i) ? __fmul_rn(g, p.drop.scale) : 0.0f;
            for (int d = 0; d < p.n_dxs; ++d)
                store_elem<Td>(static_cast<char *>(p.dx[d]) + static_cast<long long>(row) * p.dx_stride[d],
                               static_cast<long long>(i), a);
            sb += a;
            sr += g;
        }
        if (p.part_bias) p.part_bias[blockIdx.y * p.ne0 + i] = sb;
        if (p.part_res) p.part_res[blockIdx.y * p.ne0 + i] = sr;
    }
}

// out[i] = sum over the row blocks of part[block][i]; blockIdx.y picks the sum.
struct ColumnSums {
    const float *part[2];
    float *out[2];
    unsigned long long ne0;
    unsigned blocks;
};

static __global__ void __launch_bounds__(256) ar_column_sum_kernel(const __grid_constant__ ColumnSums p) {
    pdl_launch_dependents();
    pdl_wait();
    const float *part = p.part[blockIdx.y];
    float *out = p.out[blockIdx.y];
    const size_t i = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= p.ne0) return;
    float s = 0.0f;
    for (unsigned b = 0; b < p.blocks; ++b) s += part[b * p.ne0 + i];
    out[i] = s;
}

}  // namespace tps
