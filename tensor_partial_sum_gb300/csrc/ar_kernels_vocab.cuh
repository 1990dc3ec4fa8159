// Device code of ar_vocab_loss and ar_vocab_loss_grad.
#pragma once

#include "ar_kernels.cuh"

namespace tps {

// A matrix read element by element: element (i, j) at base + i * row + j * col (in elements).
struct VocabMat {
    const void *base;
    long long row, col;
    const unsigned char *live;  // 0: column j counts as zeros, whatever it holds (nullptr: all count)
};

constexpr int kVT = 64;  // tile edge of the plain product below
constexpr int kVK = 16;

// acc[4][4] of a 64x64 tile of A B^T (A [M][K], B [N][K]) for a thread of 256: rows 4 ty.., columns 4 tx..
template <int Ta, int Tb>
__device__ __forceinline__ void tile_product(const VocabMat &A, const VocabMat &B, size_t M, size_t N, size_t K, size_t m0,
                                             size_t n0, float (&acc)[4][4]) {
    __shared__ float as[kVK][kVT + 1], bs[kVK][kVT + 1];
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    for (size_t k0 = 0; k0 < K; k0 += kVK) {
        for (int e = threadIdx.x; e < kVT * kVK; e += 256) {
            const int i = e / kVK, k = e % kVK;
            as[k][i] = m0 + i < M && k0 + k < K
                           ? load_elem<Ta, false>(A.base, static_cast<long long>(m0 + i) * A.row + static_cast<long long>(k0 + k) * A.col)
                           : 0.0f;
            bs[k][i] = n0 + i < N && k0 + k < K && (!B.live || B.live[k0 + k])
                           ? load_elem<Tb, false>(B.base, static_cast<long long>(n0 + i) * B.row + static_cast<long long>(k0 + k) * B.col)
                           : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kVK; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(as[k][4 * ty + i], bs[k][4 * tx + j], acc[i][j]);
        __syncthreads();
    }
}

struct VocabStatParams {
    VocabMat h, w;
    size_t rows, vocab, dim;      // tokens, vocabulary rows of this piece
    long long first;              // global index of the piece's first row
    const long long *targets;
    float2 *part;                 // [tile][rows]: running maximum and sum of exponentials over the tile
    float *picked;                // [rows]: the target's logit
    unsigned tile0;               // number of the piece's first tile
};

// Logits of a tile, reduced to each row's maximum and sum of exp(z - maximum).
template <int T>
__global__ void __launch_bounds__(256) ar_vocab_stat_kernel(const __grid_constant__ VocabStatParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const size_t m0 = static_cast<size_t>(blockIdx.y) * kVT, n0 = static_cast<size_t>(blockIdx.x) * kVT;
    float acc[4][4] = {};
    tile_product<T, T>(p.h, p.w, p.rows, p.vocab, p.dim, m0, n0, acc);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const size_t t = m0 + 4 * ty + i;
        float m = -INFINITY, s = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n0 + 4 * tx + j < p.vocab) m = fmaxf(m, acc[i][j]);
        for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        const float base = fabsf(m) == INFINITY ? 0.0f : m;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n0 + 4 * tx + j < p.vocab) s += expf(acc[i][j] - base);
        for (int o = 8; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
        if (t >= p.rows) continue;
        if (tx == 0) p.part[(p.tile0 + blockIdx.x) * p.rows + t] = make_float2(m, s);
        const long long at = p.targets[t] - p.first;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (at == static_cast<long long>(n0 + 4 * tx + j) && n0 + 4 * tx + j < p.vocab) p.picked[t] = acc[i][j];
    }
}

struct VocabJoinParams {
    const float2 *part;
    const float *picked;
    const long long *targets;
    long long ignore, vocab;  // vocabulary rows of all pieces
    size_t rows;
    unsigned tiles;
    float *loss, *lse;
};

// Join the tiles of each row: lse = log sum exp, loss = lse - target's logit.
static __global__ void __launch_bounds__(256) ar_vocab_join_kernel(const __grid_constant__ VocabJoinParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const size_t t = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (t >= p.rows) return;
    float m = -INFINITY, s = 0.0f;
    for (unsigned k = 0; k < p.tiles; ++k) m = fmaxf(m, p.part[k * p.rows + t].x);
    const float base = fabsf(m) == INFINITY ? 0.0f : m;
    for (unsigned k = 0; k < p.tiles; ++k) {
        const float2 q = p.part[k * p.rows + t];
        if (q.x != -INFINITY) s += q.y * expf((q.x == INFINITY ? 0.0f : q.x) - base);
    }
    const float lse = base + logf(s);
    p.lse[t] = lse;
    const long long y = p.targets[t];
    p.loss[t] = y == p.ignore ? 0.0f : (y < 0 || y >= p.vocab) ? NAN : lse - p.picked[t];
}

struct VocabGradParams {
    VocabMat h, w;
    size_t rows, vocab, dim;  // tokens, vocabulary rows of this chunk
    long long first, ignore, total;
    const long long *targets;
    const float *lse, *dloss;
    float *d;                 // [rows][vocab] gradient of the chunk's logits
    unsigned char *live;      // [rows] 1: the token is counted
};

// d = dloss * (softmax - [target]) of a tile of the chunk's logits, recomputed.
template <int T>
__global__ void __launch_bounds__(256) ar_vocab_dlogits_kernel(const __grid_constant__ VocabGradParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const size_t m0 = static_cast<size_t>(blockIdx.y) * kVT, n0 = static_cast<size_t>(blockIdx.x) * kVT;
    float acc[4][4] = {};
    tile_product<T, T>(p.h, p.w, p.rows, p.vocab, p.dim, m0, n0, acc);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const size_t t = m0 + 4 * ty + i;
        if (t >= p.rows) continue;
        const long long y = p.targets[t];
        const bool live = y != p.ignore && y >= 0 && y < p.total;
        if (tx == 0 && blockIdx.x == 0) p.live[t] = live;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const size_t v = n0 + 4 * tx + j;
            if (v >= p.vocab) continue;
            const float q = expf(acc[i][j] - p.lse[t]) - (y - p.first == static_cast<long long>(v) ? 1.0f : 0.0f);
            p.d[t * p.vocab + v] = live ? q * p.dloss[t] : 0.0f;
        }
    }
}

struct VocabOutParams {
    VocabMat a, b;
    size_t m, n, k;
    float *sum;       // [m][n] running sum over chunks, nullptr: none
    int begin;        // the first chunk: the running sum starts here
    void *out;        // written when not nullptr
    long long out_row;  // elements
};

// out[m][n] = a b^T (plus the running sum); a is float, b and out T.
template <int T>
__global__ void __launch_bounds__(256) ar_vocab_product_kernel(const __grid_constant__ VocabOutParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const size_t m0 = static_cast<size_t>(blockIdx.y) * kVT, n0 = static_cast<size_t>(blockIdx.x) * kVT;
    float acc[4][4] = {};
    tile_product<kF32, T>(p.a, p.b, p.m, p.n, p.k, m0, n0, acc);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const size_t r = m0 + 4 * ty + i, c = n0 + 4 * tx + j;
            if (r >= p.m || c >= p.n) continue;
            float v = acc[i][j];
            if (p.sum) {
                if (!p.begin) v += p.sum[r * p.n + c];
                p.sum[r * p.n + c] = v;
            }
            if (p.out) store_elem<T>(p.out, static_cast<long long>(r) * p.out_row + static_cast<long long>(c), v);
        }
}

}  // namespace tps
