// Device code of ar_vocab_loss and ar_vocab_loss_grad.
//
// With logits z = H W^T, lse_t = log sum_v exp z_tv and per-token factors g_t,
//     loss_t = lse_t - z_t[y_t],     D = g (softmax(z) - onehot(y)),
//     dH_r = D_r W_r,                dW_r = D_r^T H.
// Three matrix products with reductions of length dim, vocabulary and tokens.
// One kernel does all of them, on a pair of CTAs, and differs in what it does
// with a finished 256x256 tile:
//   kStats   keeps each row's maximum and sum of exponentials (and the
//            target's logit): the logits never leave the chip;
//   kDlogits turns a tile of recomputed logits into a tile of D, held in
//            16 bits for one chunk of the vocabulary;
//   kGrads   stores tiles of dH and dW.
// With 64 tokens or fewer, kStatsFew and kDlogitsFew do the first two the
// other way round, z^T = W H^T: the tensor cores' time goes by the narrow
// side, so tiles of vocabulary rows by a few tokens cost next to nothing and
// reading W is what is left (4 tokens of 5136 elements, six pieces of 1640 rows:
// an eager call 49 -> 40 us; 3 float tokens of 7232, 19671 rows: 489 -> 398).
// Their D of 16-bit inputs is held in two parts (kGradsFew): with few tokens
// the rounding of the targets' entries does not average out (gradients up to
// 1.65 times as far off as a float computation rounded once), and the second
// product is hidden behind W.
// Small kernels around it list the counted tokens, pack rows that the tiled
// copies cannot read in place, and join partial results.
//
// Float32 inputs go through the same tensor cores: x = x1 + x2 + x3 with three
// bf16 parts (exact), and the six largest of the nine products; the ones left
// out are below 2^-25 of the whole.
#pragma once

#include "ar_kernels.cuh"
#include "ar_umma.cuh"
#include "ar_vocab_plan.h"

namespace tps {

enum VocabMode { kStats = 0, kDlogits = 1, kGrads = 2, kStatsFew = 3, kDlogitsFew = 4, kGradsFew = 5 };
template <int MODE>
constexpr bool kVFew = MODE == kStatsFew || MODE == kDlogitsFew;
template <int MODE>
constexpr bool kVGrads = MODE == kGrads || MODE == kGradsFew;

constexpr int kVMaxStages = 32;
constexpr int kVRow = kVK * 2;              // bytes of a row of a stage
constexpr int kVRing = 6 * 256 * kVRow;     // bytes of the stages: six of full height
constexpr int kVEpilogueWarps = 8;
constexpr int kVThreads = 128 + 32 * kVEpilogueWarps;
// The tensor cores' float sums drop what falls below the running sum's last place (they do not round), so
// a long reduction drifts: one token of 4096 elements came out 3.6e-5 off.  Where that would be seen (the
// logits, of the statistics and of D, and everything of float32 inputs) a run of products is kept short and the
// runs are added in registers, rounded to nearest.  The logits of D take the statistics' runs, so that a logit less the
// log-sum-exp holds no drift of its own (in one run, a target with p = 1 - 1e-5 had a gradient of the wrong sign).  Half as long a run is off by half as much and costs one
// hand-over more: with 32 products the prompt's statistics are 2.7e-7 off (a float computation 6.1e-7) in 286 us,
// with 16 they take 306; few tokens wait for W and get 16 for nothing; float32 gets 24 (345 -> 355 us a
// step), which halves the gradients' error to below a float computation's.
template <int MODE, int T>
constexpr bool kVRuns = !kVGrads<MODE> || T == kF32;
template <int MODE, int T>
constexpr int kVRunBlocks = T == kF32 ? 1 : kVFew<MODE> ? 4 : 8;  // blocks of K in a run
// Blocks of K in a stage.  A round of the ring - wait, copies, products, commit - takes the feeding warps about 400
// cycles, more than the products of narrow tiles: those share one between two blocks (three parts fill a
// stage by themselves).
template <int MODE, int T>
constexpr int kVBlocks = kVFew<MODE> && T != kF32 ? 2 : 1;  // a run is whole stages
// Registers of the feeding and of the result warps when a thread adds up 128 columns; the launch's
// kVLaunchRegs for each of 384 threads cover them.
template <int MODE, int T>
constexpr bool kVSplitRegs = kVRuns<MODE, T> && !kVFew<MODE>;
constexpr int kVFeedRegs = 80, kVSumRegs = 208, kVLaunchRegs = 168;
static_assert(128 * kVFeedRegs + 32 * kVEpilogueWarps * kVSumRegs <= kVThreads * kVLaunchRegs, "register split");
constexpr unsigned kVTmemCols = 512;        // two accumulators of 256 columns
constexpr int kVPitch = 80;                 // bytes between a warp's staged output rows of 64 bytes
constexpr int kVOut = kVEpilogueWarps * 32 * kVPitch;
constexpr size_t kVSmem = static_cast<size_t>(kVRing) + kVOut + 1024 + 1024;

// One vocabulary segment of a launch: (part of) a piece.
struct VocabSeg {
    long long first;       // global index of its first vocabulary row
    int rows;
    int tile0;             // first of its column tiles (kStats, kDlogits), of its dW tiles (kGrads)
    long long col0;        // its first column of D
    char *dh;              // kGrads: the piece's dH (nullptr: not now), rows dh_row bytes apart
    long long dh_row;
    char *dw;              // kGrads: dW of the segment's first row, nullptr: not wanted
    long long dw_row;
};

struct VocabGemmParams {
    CUtensorMap b_map[kMaxSegs];  // W of each segment: K-major (kStats, kDlogits) or MN-major (kGrads)
    CUtensorMap b_tail[kMaxSegs]; // kStats, kDlogits: W in boxes of half its last tile's width
    CUtensorMap a_map;            // H (kStats, kDlogits) or D, K-major
    CUtensorMap a_tail_map;       // the same in boxes of a_tail rows
    CUtensorMap at_map;           // kGrads: D, MN-major
    CUtensorMap ht_map;           // kGrads: H, MN-major
    VocabSeg seg[kMaxSegs];
    int nseg;
    int rows;                 // tokens
    int dim;
    int bn;                   // columns of a tile, <= kVN
    // Rows of a K-major A that exist; the last a_rows % 128 of them are copied as a_tail, a multiple of
    // 8.  Copies do not reach past the rows that exist by more than that: rows outside the tensor cost a
    // copy more than rows inside (one token, 127 of 128 rows outside: 115 us, with one box of 8 rows 61),
    // and what a tile holds there goes into results that nobody reads.
    int a_rows, a_tail;
    int a_room;               // rows of A that a stage has room for
    int few_rows;             // kStatsFew, kDlogitsFew: vocabulary rows of a tile in each CTA (b_map's boxes;
                              // b_tail's: the rows left over), and a_map has boxes of bn / 2 tokens
    int stages;               // of a_room + bn / 2 rows each
    int tiles;                // column tiles (kStats, kDlogits) or dW tiles (kGrads) of all segments
    const VocabList *list;    // nullptr: all tokens, in order (kStats)
    const long long *targets; // kStats
    float2 *part;             // kStats: [2 * tile + half][rows]
    float *picked;            // kStats: [rows]
    const VocabRow *row;      // kDlogits: [live]
    const int *index;         // kGrads: original token of list entry i
    unsigned short *d;        // D: [parts][d_rows][d_ld]
    long long d_ld, d_part;   // elements
    int slices;               // kGrads: parts of the reduction over a segment's vocabulary
    int dh_tiles;             // kGrads: column tiles of dH, 0: not wanted
    float *sum;               // kGrads: [segment][slice][sum_rows][sum_ld] partial dH, nullptr: straight to dh
    long long sum_rows, sum_ld;
    int sum_begin;            // the partial sums start here rather than go on
    unsigned *status;
};

// Parts of the operands, and products of parts in a block of K.
template <int MODE, int T>
constexpr int kVPartsA = T == kF32 ? 3 : MODE == kGradsFew ? 2 : 1;
template <int MODE, int T>
constexpr int kVPartsB = T == kF32 ? 3 : 1;
template <int MODE, int T>
constexpr int kVPairs = T == kF32 ? 6 : kVPartsA<MODE, T>;
// Part numbers of A and B in product q, the largest product last, so that the small ones are summed
// while the run is small.
__device__ __forceinline__ constexpr int a_part_of(int pairs, int q) {  // of six: 1 0 2 0 1 0
    return pairs == 6 ? (0x010201 >> (4 * q)) & 0xF : pairs - 1 - q;
}
__device__ __forceinline__ constexpr int b_part_of(int pairs, int q) {  // of six: 1 2 0 1 0 0
    return pairs == 6 ? (0x001021 >> (4 * q)) & 0xF : 0;
}

// A tile: its place, its operands' places and its blocks of K.
struct VocabTile {
    int seg;
    int m, n;        // tile row and column
    int k0, kn;      // first block of K and their number
    int slice;
    int bn;          // columns
    bool dw;
};

template <int MODE>
__host__ __device__ constexpr int tail_width(int rows) {
    return MODE == kStats ? (rows + 15) / 16 * 16 : (rows + 63) / 64 * 64;
}

// A pair's tiles, one after another.  kStats and kDlogits: row tiles of one column tile next to one
// another, so that pairs that run together share W and find H in L2.  kGrads: first the dH tiles (long
// reductions) in turn, then the dW tiles; pairs that got one dH tile fewer first take as many more dW
// tiles as cost the same.
template <int MODE>
struct VocabWalk {
    const VocabGemmParams &p;
    int pair, npairs, mt, kn, nt;
    int i = 0;
    // kGrads: dH tiles of a segment and of this pair, pairs without the last round's dH tile, the dW
    // tiles that each of them takes more
    int per_seg = 0, mine = 0, behind = 0, extra = 0, first = 0;

    __device__ __forceinline__ VocabWalk(const VocabGemmParams &params, int live, int pair_, int npairs_)
        : p(params), pair(pair_), npairs(npairs_), mt((live + kVM - 1) / kVM) {
        if constexpr (!kVGrads<MODE>) {
            kn = (p.dim + kVK - 1) / kVK;
            nt = 0;
        } else {
            kn = (live + kVK - 1) / kVK;
            nt = (p.dim + p.bn - 1) / p.bn;
            per_seg = p.slices * p.dh_tiles * mt;
            const int n_long = p.nseg * per_seg, rem = n_long % npairs;
            mine = n_long / npairs + (pair < rem);
            behind = rem ? npairs - rem : 0;
            if (behind) {
                const int kw = max(kVStoreBlocks, kn), kl = (p.seg[0].rows + kVK * p.slices - 1) / (kVK * p.slices);
                extra = min((kl + kw / 2) / kw, p.tiles / behind);
                first = pair >= rem ? extra : 0;
            }
        }
    }
    __device__ __forceinline__ bool next(VocabTile &t) {
        t.slice = 0;
        t.k0 = 0;
        t.bn = p.bn;
        t.dw = false;
        t.seg = 0;
        if constexpr (!kVGrads<MODE>) {
            const long long id = pair + static_cast<long long>(i++) * npairs;
            if constexpr (kVFew<MODE>) {  // tiles of vocabulary rows by all tokens
                if (mt == 0 || id >= p.tiles) return false;
                while (t.seg + 1 < p.nseg && p.seg[t.seg + 1].tile0 <= id) ++t.seg;
                t.m = static_cast<int>(id) - p.seg[t.seg].tile0;
                t.n = 0;
                t.kn = kn;
                return true;
            }
            if (mt == 0 || id >= static_cast<long long>(p.tiles) * mt) return false;
            const int j = id <= 0x7FFFFFFF ? static_cast<int>(id) / mt : static_cast<int>(id / mt);
            t.m = static_cast<int>(id - static_cast<long long>(j) * mt);
            while (t.seg + 1 < p.nseg && p.seg[t.seg + 1].tile0 <= j) ++t.seg;
            t.n = j - p.seg[t.seg].tile0;
            t.kn = kn;
            // the last tile of a segment is as narrow as its rows allow (D's columns are read in blocks of K)
            t.bn = min(p.bn, tail_width<MODE>(p.seg[t.seg].rows - t.n * p.bn));
            return true;
        } else {
            if (i < mine) {
                int id = pair + i++ * npairs;
                t.seg = id / per_seg;
                id -= t.seg * per_seg;
                t.m = id % mt;
                id /= mt;
                t.n = id % p.dh_tiles;
                t.slice = id / p.dh_tiles;
                const int kb = (p.seg[t.seg].rows + kVK - 1) / kVK, per = (kb + p.slices - 1) / p.slices;
                t.k0 = t.slice * per;
                t.kn = max(0, min(per, kb - t.k0));
            } else {
                const int q = i++ - mine;
                const int id = q < first ? (pair - (npairs - behind)) * extra + q : extra * behind + pair + (q - first) * npairs;
                if (id >= p.tiles) return false;
                const int j = id / nt;
                t.n = id - j * nt;
                while (t.seg + 1 < p.nseg && p.seg[t.seg + 1].tile0 <= j) ++t.seg;
                t.m = j - p.seg[t.seg].tile0;
                t.kn = kn;
                t.dw = true;
            }
            if (p.dim - t.n * p.bn <= kVN / 2) t.bn = kVN / 2;
            return true;
        }
    }
};

// Runs of products of a tile; one without blocks of K still counts as one.
template <int MODE, int T>
__device__ __forceinline__ int vocab_runs(const VocabTile &t) {
    return kVRuns<MODE, T> ? max(1, (t.kn + kVRunBlocks<MODE, T> - 1) / kVRunBlocks<MODE, T>) : 1;
}

// Store a warp's 32x32 values, row `lane` in each thread: `n` (1 to 32) elements of T to each thread's
// `out` (nullptr: no row).  The rows go through shared memory, so that adjacent lanes store adjacent
// bytes: rows of 64 bytes in pieces of 16, of 4 or of one element, whichever all of them allow (each
// lane storing its own row, 2 bytes in 32 places at once, made the dW of odd rows 2.5 times slower).
template <int T>
__device__ __forceinline__ void store_block(unsigned char *stage, char *out, const float (&v)[32], int n, int lane) {
    constexpr int es = Elem<T>::bytes, per = 64 / es;  // elements of a pass
    const unsigned long long mine = reinterpret_cast<unsigned long long>(out);
    const bool vec = __all_sync(~0u, mine % 16 == 0) && n == 32;
    const bool words = es == 4 || (__all_sync(~0u, mine % 4 == 0) && n % 2 == 0);
#pragma unroll
    for (int c = 0; c < 32; c += per) {
        if (c >= n) break;
        uint32_t w[16];
        if constexpr (T == kF32) {
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(v[c + k]);
        } else {
            word_pack<T, 16>(v, w);
        }
        __syncwarp();  // the last pass has been read
#pragma unroll
        for (int k = 0; k < 16; k += 4)
            *reinterpret_cast<uint4 *>(stage + lane * kVPitch + 4 * k) = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
        __syncwarp();
        if (vec) {
#pragma unroll
            for (int r0 = 0; r0 < 32; r0 += 8) {
                const int r = r0 + lane / 4, at = lane % 4 * 16;
                char *to = reinterpret_cast<char *>(__shfl_sync(~0u, mine, r));
                if (to) *reinterpret_cast<uint4 *>(to + c * es + at) = *reinterpret_cast<uint4 *>(stage + r * kVPitch + at);
            }
        } else if (words) {
            const int k = lane % 16;
#pragma unroll 4
            for (int r0 = 0; r0 < 32; r0 += 2) {
                const int r = r0 + lane / 16;
                char *to = reinterpret_cast<char *>(__shfl_sync(~0u, mine, r));
                if (to && c * es + 4 * k < n * es)
                    *reinterpret_cast<uint32_t *>(to + c * es + 4 * k) = *reinterpret_cast<uint32_t *>(stage + r * kVPitch + 4 * k);
            }
        } else if constexpr (T != kF32) {
#pragma unroll 4
            for (int r = 0; r < 32; ++r) {
                char *to = reinterpret_cast<char *>(__shfl_sync(~0u, mine, r));
                if (to && lane < n)
                    reinterpret_cast<unsigned short *>(to)[lane] = *reinterpret_cast<unsigned short *>(stage + r * kVPitch + 2 * lane);
            }
        }
    }
}

// The three bf16 parts of two floats, each the nearest to what is left: the parts have signs of their
// own, so that what the missing products of parts leave out averages out (cut off instead of rounded, a
// step of five tokens had gradients 6.7e-6 off).  ANY: any floats, else finite ones that no rounding
// makes infinite.
template <bool ANY>
__device__ __forceinline__ void split2(float a, float b, uint32_t (&w)[3]) {
    w[0] = pack_bf16x2(a, b);
    if constexpr (ANY) {
        // a finite number that would round to infinity is cut off; an infinity or NaN is all in the first part
        if (fabsf(bf16_lo(w[0])) == INFINITY && fabsf(a) != INFINITY) w[0] = (w[0] & 0xFFFF0000u) | (__float_as_uint(a) >> 16);
        if (fabsf(bf16_hi(w[0])) == INFINITY && fabsf(b) != INFINITY) w[0] = (w[0] & 0xFFFFu) | (__float_as_uint(b) & 0xFFFF0000u);
        a = fabsf(a) <= 3.402823466e38f ? a - bf16_lo(w[0]) : 0.0f;
        b = fabsf(b) <= 3.402823466e38f ? b - bf16_hi(w[0]) : 0.0f;
    } else {
        a -= bf16_lo(w[0]), b -= bf16_hi(w[0]);
    }
    w[1] = pack_bf16x2(a, b);
    w[2] = pack_bf16x2(a - bf16_lo(w[1]), b - bf16_hi(w[1]));
}

// softmax from a logit less the row's log-sum-exp; float inputs want more of it than the fast
// exponential has (its argument's rounding, 1e-6 at -16).
template <int T>
__device__ __forceinline__ float soft(float x) {
    return T == kF32 ? expf(x) : __expf(x);
}

// Combine 32 columns over the warp's lanes: lane k's x[0] becomes column k's result (31 exchanges
// where a reduction of each column would take 160).
template <int O = 16, typename Op>
__device__ __forceinline__ void fold_columns(float (&x)[32], int lane, Op op) {
    const bool high = lane & O;
#pragma unroll
    for (int k = 0; k < O; ++k) {
        const float give = high ? x[k] : x[k + O], keep = high ? x[k + O] : x[k];
        x[k] = op(keep, __shfl_xor_sync(~0u, give, O));
    }
    if constexpr (O > 1) fold_columns<O / 2>(x, lane, op);
}

// x[0] becomes the sum of all 32, added in pairs.
template <int O = 16>
__device__ __forceinline__ void sum_pairs(float (&x)[32]) {
#pragma unroll
    for (int k = 0; k < O; ++k) x[k] += x[k + O];
    if constexpr (O > 1) sum_pairs<O / 2>(x);
}

// ---- the product kernel ---------------------------------------------------------
//
// Warps: 0 copies tiles in, 1 issues the products (in the leader), 2 owns the
// tensor memory, 4..11 turn accumulators into results.  A stage holds 128 rows
// of A and 128 rows of B for 64 elements of K in each CTA; both CTAs' copies
// count on the leader's `full` barrier, and a finished product frees the stage
// in both.  Two accumulators alternate, so the tensor cores work on the next
// tile while the epilogue reads the last.  Every wait is bounded; one that
// runs out sets bit 1 of the status word, and the pair winds down.
//
// bf16, 2048 tokens, dim 4096, 32768 vocabulary rows: statistics 288 us, D 307, dH
// and dW 531 (1.91, 1.79 and 2.07 PFLOP/s; cuBLAS peaks at 1.96), the tensor cores
// 94, 86 and 97% busy: they bound it, and in longer work the power cap does (4096 x
// 4096 x 131072, four products: 10.0 ms, 1.76 PFLOP/s).  D took 297 us with its logits in
// one run; see kVRuns for why it does not.
template <int MODE, int T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kVThreads, 1)
    ar_vocab_gemm_kernel(const __grid_constant__ VocabGemmParams p) {
    extern __shared__ unsigned char raw[];
    const unsigned base = (smem_u32(raw) + 1023u) & ~1023u;
    // barriers behind the stages
    const unsigned bars = base + kVRing + kVOut;
    const unsigned full = bars, empty = bars + 8 * kVMaxStages, tfull = bars + 16 * kVMaxStages, tempty = tfull + 16;
    const unsigned tmem_slot = tempty + 16, abort_slot = tmem_slot + 4, drain = tmem_slot + 8;
    volatile unsigned *abort_flag = reinterpret_cast<volatile unsigned *>(raw + (abort_slot - smem_u32(raw)));
    const unsigned rank = cluster_rank();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int pair = blockIdx.x / 2, npairs = gridDim.x / 2;

    pdl_launch_dependents();
    auto init = [](unsigned bar, unsigned count) {
        asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < kVMaxStages; ++s) init(full + 8 * s, 1), init(empty + 8 * s, 1);
        for (int a = 0; a < 2; ++a) init(tfull + 8 * a, 1), init(tempty + 8 * a, 2 * kVEpilogueWarps);
        init(drain, 1);
        *abort_flag = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) tmem_alloc(tmem_slot, kVTmemCols);
    tmem_fence_before();
    __syncthreads();
    cluster_sync();
    tmem_fence_after();
    const unsigned tmem = *reinterpret_cast<volatile unsigned *>(raw + (tmem_slot - smem_u32(raw)));
    pdl_wait();  // the kernel before this one on the stream has finished
    asm volatile("fence.proxy.async.global;" ::: "memory");  // its plain stores, before this one's copies
    const int live = p.list ? p.list->live : p.rows;
    const unsigned S = static_cast<unsigned>(p.stages);
    // a block of K: the parts of A, then the parts of B
    const unsigned a_size = static_cast<unsigned>(p.a_room) * kVRow, b_size = static_cast<unsigned>(p.bn / 2) * kVRow;
    const unsigned b_at = kVPartsA<MODE, T> * a_size, block = b_at + kVPartsB<MODE, T> * b_size, stage = kVBlocks<MODE, T> * block;

    const volatile unsigned never = 0;  // for waits that follow giving up
    auto give_up = [&] {
        atomicOr(p.status, 2u);
        *abort_flag = 1u;
    };

    if (warp < 4) {
        // the whole warpgroup gives registers up, in the branch that holds its roles' code
        if constexpr (kVSplitRegs<MODE, T>) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kVFeedRegs));
        if (warp == 0) {
            // ---- copies: this CTA's half of each operand ----
            const unsigned lead_full = leader_addr(full);
            unsigned s = 0, round = 0;  // the stage to fill and how often the ring went round
            bool ok = true;
            VocabTile t;
            for (VocabWalk<MODE> walk(p, live, pair, npairs); ok && walk.next(t);) {
                const CUtensorMap *am, *bm;
                int ay, ax, by, bx;  // first element of this CTA's rows (columns) at block 0 of K
                const int row0 = t.m * kVM, arow = row0 + static_cast<int>(rank) * 128;
                const int brow = t.n * p.bn + static_cast<int>(rank) * (t.bn / 2);
                const bool a_mn = kVGrads<MODE> && t.dw, b_mn = kVGrads<MODE>;
                if constexpr (!kVGrads<MODE>) {
                    am = &p.a_map, bm = &p.b_map[t.seg];
                    ax = 0, ay = arow, bx = 0, by = brow;
                } else if (t.dw) {
                    am = &p.at_map, bm = &p.ht_map;
                    ax = static_cast<int>(p.seg[t.seg].col0) + arow, ay = 0, bx = brow, by = 0;
                } else {
                    am = &p.a_map, bm = &p.b_map[t.seg];
                    ax = static_cast<int>(p.seg[t.seg].col0), ay = arow, bx = brow, by = 0;
                }
                // what the first and the second CTA of the pair copy of each operand, in rows of a stage
                auto a_part = [&](int row) { return row + 128 <= p.a_rows ? 128 : row < p.a_rows ? p.a_tail : 0; };
                auto b_part = [&](int col) {  // MN-major: chunks of 64 columns, none of them all outside
                    return t.bn == kVN && col + 64 < p.dim ? 128 : col < p.dim ? 64 : 0;
                };
                int a_mine = a_mn ? 128 : a_part(arow), b_mine = b_mn ? b_part(brow) : t.bn / 2;
                int a_both = a_mn ? 256 : a_part(row0) + a_part(row0 + 128);
                int b_both = b_mn ? b_part(t.n * p.bn) + b_part(t.n * p.bn + t.bn / 2) : t.bn;
                if (!a_mn && a_mine < 128) am = &p.a_tail_map;
                if (!b_mn && t.bn < p.bn) bm = &p.b_tail[t.seg];
                if constexpr (kVFew<MODE>) {  // A: vocabulary rows, B: tokens
                    const int mh = p.few_rows, rows = p.seg[t.seg].rows, w0 = 2 * t.m * mh;
                    auto part = [&](int row) { return row + mh <= rows ? mh : row < rows ? (rows % mh + 7) / 8 * 8 : 0; };
                    ay = w0 + static_cast<int>(rank) * mh, by = static_cast<int>(rank) * (p.bn / 2);
                    a_mine = part(ay), a_both = part(w0) + part(w0 + mh);
                    b_mine = by < p.a_rows ? p.bn / 2 : 0, b_both = p.bn / 2 < p.a_rows ? p.bn : p.bn / 2;
                    am = ay + mh <= rows ? &p.b_map[t.seg] : &p.b_tail[t.seg];
                    bm = &p.a_map;
                }
                const unsigned bytes = static_cast<unsigned>(kVPartsA<MODE, T> * a_both + kVPartsB<MODE, T> * b_both) * kVRow;
                int k = t.k0 * kVK;
                constexpr int U = kVBlocks<MODE, T>;
                for (int n = t.kn; n > 0; n -= U, k += U * kVK) {
                    if (round && !__all_sync(~0u, mbar_wait_bounded(empty + 8 * s, (round - 1) & 1, abort_flag))) {
                        give_up();
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        const unsigned bar = lead_full + 8 * s;
                        if (rank == 0)
                            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full + 8 * s),
                                         "r"(min(n, U) * bytes)
                                         : "memory");
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            if (u >= n) break;
                            const int ku = k + u * kVK;
#pragma unroll
                            for (int q = 0; q < kVPartsA<MODE, T>; ++q) {
                                const unsigned a = base + s * stage + u * block + q * a_size;
                                if (!a_mn) {
                                    if (a_mine) tma_load_3d(a, am, bar, ax + ku, ay, q);
                                } else {  // two chunks of 64 columns, 64 rows each
                                    tma_load_3d(a, am, bar, ax, ay + ku, q);
                                    tma_load_3d(a + 8192, am, bar, ax + 64, ay + ku, q);
                                }
                            }
#pragma unroll
                            for (int q = 0; q < kVPartsB<MODE, T>; ++q) {
                                const unsigned b = base + s * stage + u * block + b_at + q * b_size;
                                if (!b_mn) {
                                    if (b_mine) tma_load_3d(b, bm, bar, bx + ku, by, q);
                                } else {
                                    if (b_mine) tma_load_3d(b, bm, bar, bx, by + ku, q);
                                    if (b_mine > 64) tma_load_3d(b + 8192, bm, bar, bx + 64, by + ku, q);
                                }
                            }
                        }
                    }
                    if (++s == S) s = 0, ++round;
                }
            }
            // the products' last arrivals have to find this CTA still here; after a wait that ran out, the
            // copies in flight (of both CTAs) have to land before the pair leaves
            for (unsigned q = 0; q < S; ++q) {
                const unsigned fills = round + (q < s);  // of stage q
                if (fills == 0) continue;
                if (ok && !__all_sync(~0u, mbar_wait_bounded(empty + 8 * q, (fills - 1) & 1, abort_flag))) {
                    give_up();
                    ok = false;
                }
                if (!ok && rank == 0) mbar_wait_bounded(full + 8 * q, (fills - 1) & 1, &never);
            }
        } else if (warp == 1) {
            if (rank == 0) {
                // ---- products ----
                const uint64_t desc0 = umma_desc(base, 8192);
                unsigned s = 0, phase = 0, acc_it = 0;
                bool ok = true;
                VocabTile t;
                for (VocabWalk<MODE> walk(p, live, pair, npairs); ok && walk.next(t);) {
                    const bool a_mn = kVGrads<MODE> && t.dw, b_mn = kVGrads<MODE>;
                    const uint32_t idesc = umma_idesc(T != kF16, a_mn, b_mn, static_cast<unsigned>(t.bn));
                    // 16 elements of K: 32 bytes along a K-major row, two groups of eight rows otherwise
                    const unsigned a_step = a_mn ? 2048 >> 4 : 32 >> 4, b_step = b_mn ? 2048 >> 4 : 32 >> 4;
                    for (int r = 0, runs = vocab_runs<MODE, T>(t); ok && r < runs; ++r, ++acc_it) {
                        const unsigned acc = acc_it % 2, use = acc_it / 2;
                        if (use && !__all_sync(~0u, mbar_wait_bounded(tempty + 8 * acc, (use - 1) & 1, abort_flag))) {
                            give_up();
                            ok = false;
                            break;
                        }
                        tmem_fence_after();
                        const unsigned d = tmem + acc * 256;
                        bool more = false;  // the first product of a run starts the accumulator
                        int n = t.kn;
                        if constexpr (kVRuns<MODE, T>) n = min(kVRunBlocks<MODE, T>, t.kn - r * kVRunBlocks<MODE, T>);
                        for (; n > 0; n -= kVBlocks<MODE, T>) {
                            if (!__all_sync(~0u, mbar_wait_bounded(full + 8 * s, phase, abort_flag))) {
                                give_up();
                                ok = false;
                                break;
                            }
                            tmem_fence_after();
                            const uint64_t stage0 = desc0 + ((s * stage) >> 4);
                            if (elect_one()) {
#pragma unroll
                                for (int u = 0; u < kVBlocks<MODE, T>; ++u) {
                                    if (u >= n) break;
                                    const uint64_t a0 = stage0 + ((u * block) >> 4), b0 = a0 + (b_at >> 4);
#pragma unroll
                                    for (int q = 0; q < kVPairs<MODE, T>; ++q) {
                                        const uint64_t a = a0 + a_part_of(kVPairs<MODE, T>, q) * (a_size >> 4);
                                        const uint64_t b = b0 + b_part_of(kVPairs<MODE, T>, q) * (b_size >> 4);
#pragma unroll
                                        for (unsigned k = 0; k < kVK / 16; ++k)
                                            umma(d, a + k * a_step, b + k * b_step, idesc, more || u > 0 || q > 0 || k > 0);
                                    }
                                }
                                umma_commit(empty + 8 * s);
                            }
                            __syncwarp();
                            more = true;
                            if (++s == S) s = 0, phase ^= 1;
                        }
                        if (ok && elect_one()) umma_commit(tfull + 8 * acc);
                        __syncwarp();
                    }
                }
                if (!ok) {  // products in flight finish before the tensor memory goes
                    if (elect_one()) umma_commit(drain);
                    __syncwarp();
                    mbar_wait_bounded(drain, 0, &never);
                }
            }
        }
    } else {
        if constexpr (kVSplitRegs<MODE, T>) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kVSumRegs));
        // ---- results: a warp reads the 32 lanes of its quarter and half of the columns ----
        const int quarter = warp % 4, half = (warp - 4) / 4;
        unsigned char *stage_out = raw + (base - smem_u32(raw)) + kVRing + (warp - 4) * 32 * kVPitch;
        unsigned acc_it = 0;
        VocabTile t;
        const float unscale = kVGrads<MODE> && p.list ? p.list->unscale : 1.0f;
        bool ok = true;
        for (VocabWalk<MODE> walk(p, live, pair, npairs); ok && walk.next(t);) {
            const VocabSeg &seg = p.seg[t.seg];
            // row of the product, first column in the tile and number of columns
            const int in_cta = quarter * 32 + lane;
            const int r = kVFew<MODE> ? (2 * t.m + static_cast<int>(rank)) * p.few_rows + in_cta
                                      : t.m * kVM + static_cast<int>(rank) * 128 + in_cta;
            const int c0 = half * (kVFew<MODE> ? 32 : t.bn / 2);
            const int width = kVFew<MODE> ? min(32, t.bn - c0) : t.bn / 2;
            // rows past the end cost nothing (D's are read, as zeros, up to a whole block of K)
            const int rows = MODE == kDlogits ? (live + kVK - 1) / kVK * kVK : kVGrads<MODE> && t.dw ? seg.rows : live;
            const bool idle = kVFew<MODE> ? quarter * 32 >= p.few_rows || (MODE == kStatsFew && c0 >= live) : r - lane >= rows;
            long long y = -1;
            float lse = 0.0f, g = 0.0f;
            if constexpr (MODE == kStats) {
                if (r < live) y = p.targets[r];
            } else if constexpr (MODE == kDlogits) {
                if (r < live) {
                    const VocabRow q = p.row[r];
                    y = q.y, lse = q.lse, g = q.g;
                }
            } else if constexpr (kVFew<MODE>) {  // lane k: token c0 + k
                if (c0 + lane < live) {
                    if constexpr (MODE == kStatsFew) {
                        y = p.targets[c0 + lane];
                    } else {
                        const VocabRow q = p.row[c0 + lane];
                        y = q.y, lse = q.lse, g = q.g;
                    }
                }
            }
            unsigned src = 0;  // the tile's accumulator in tensor memory
            auto next_run = [&] {
                const unsigned acc = acc_it % 2, use = acc_it / 2;
                src = tmem + acc * 256 + static_cast<unsigned>(c0) + (static_cast<unsigned>(quarter * 32) << 16);
                const bool got = mbar_wait_bounded(tfull + 8 * acc, use & 1, abort_flag);
                if (__any_sync(~0u, !got)) {
                    if (lane == 0) give_up();
                    ok = false;
                }
                tmem_fence_after();
            };
            auto done_run = [&] {
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(leader_addr(tempty + 8 * (acc_it % 2)));
                ++acc_it;
            };
            constexpr int kCols = kVFew<MODE> ? 32 : 128;  // of a thread
            float sums[kVRuns<MODE, T> ? kCols : 1];
            if constexpr (kVRuns<MODE, T>) {
#pragma unroll
                for (int k = 0; k < kCols; ++k) sums[k] = 0.0f;
                for (int q = 0, runs = vocab_runs<MODE, T>(t); q < runs; ++q) {
                    next_run();
                    if (!ok) break;
                    if (t.kn && !idle) {
#pragma unroll
                        for (int c = 0; c < kCols; c += 32)
                            if (c < width) tmem_add32(src + c, sums + c);
                    }
                    done_run();
                }
            } else {
                next_run();
            }
            if (!ok) break;
            if (idle) {
                if constexpr (!kVRuns<MODE, T>) done_run();
                continue;
            }
            auto values = [&](int c, float (&v)[32]) {  // columns c .. c + 31 of this thread's row
                if constexpr (kVRuns<MODE, T>) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = sums[c + k];
                } else if (t.kn && width > 0) {
                    tmem_load32(src + c, v);
                } else {  // nothing to sum over
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = 0.0f;
                }
            };
            if constexpr (MODE == kStats) {
                const int col = t.n * p.bn + c0;                 // column in the segment
                const int n = min(width, seg.rows - col);        // columns of this warp that exist
                const long long at = y - seg.first - col;        // the target's column here, if in [0, n)
                float m = -INFINITY, s = 0.0f;
#pragma unroll
                for (int c = 0; c < 128; c += 32) {
                    if (c >= width) break;
                    float v[32];
                    values(c, v);
                    float top = -INFINITY;
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (c + k < n) top = fmaxf(top, v[k]);
                    const float to = fmaxf(m, top);
                    const float ref = fabsf(to) == INFINITY ? 0.0f : to;
                    s = m == -INFINITY ? s : s * __expf((m == INFINITY ? 0.0f : m) - ref);
                    m = to;
                    if (at >= c && at < c + 32 && at < n && r < live) {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (at == c + k) p.picked[r] = v[k];
                    }
                    // The 32 terms in pairs: added to s one after another, terms far below it would all lose their last
                    // bits the same way (a log-sum-exp 3.3e-6 off, in pairs 4.9e-7; a float computation 1.3e-6;
                    // four short sums took 1.5% more time at 2048 x 4096 x 32768).
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = c + k < n ? __expf(v[k] - ref) : 0.0f;
                    sum_pairs(v);
                    s += v[0];
                }
                if (r < live) p.part[(2ll * (seg.tile0 + t.n) + half) * p.rows + r] = make_float2(m, s);
            } else if constexpr (MODE == kDlogits) {
                const int col = t.n * p.bn + c0;
                const int n = min(width, seg.rows - col);
                const long long at = y - seg.first - col;
                unsigned short *out = p.d + static_cast<long long>(r) * p.d_ld + seg.col0 + col;
#pragma unroll
                for (int c = 0; c < 128; c += 32) {
                    if (c >= width) break;
                    float v[32];
                    values(c, v);
                    // the target's probability less one, which keeps its bits where it is nearly sure
                    float target = 0.0f;
                    if (at >= c && at < c + 32) {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (at == c + k) target = v[k];
                        target = expm1f(target - lse);
                    }
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const float q = at == c + k ? target : soft<T>(v[k] - lse);
                        v[k] = r < live && c + k < n ? q * g : 0.0f;
                    }
                    // rows past the list and columns past the segment hold zeros: whole blocks of K are read
                    if constexpr (T != kF32) {
                        uint32_t w[16];
                        word_pack<T, 16>(v, w);
#pragma unroll
                        for (int k = 0; k < 16; k += 4)
                            *reinterpret_cast<uint4 *>(out + c + 2 * k) = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; k += 8) {
                            uint32_t w[4][3];
#pragma unroll
                            for (int e = 0; e < 4; ++e) split2<false>(v[k + 2 * e], v[k + 2 * e + 1], w[e]);
#pragma unroll
                            for (int q = 0; q < 3; ++q)
                                *reinterpret_cast<uint4 *>(out + q * p.d_part + c + k) =
                                    make_uint4(w[0][q], w[1][q], w[2][q], w[3][q]);
                        }
                    }
                }
            } else if constexpr (MODE == kStatsFew) {
                // lane: vocabulary row r, v[k]: token c0 + k.  The maxima of the 32 columns over the 32 lanes by
                // halving: each step gives away half of the columns, until lane k holds column k's.
                const bool exists = in_cta < p.few_rows && r < seg.rows;
                float v[32], top[32];
                values(0, v);
#pragma unroll
                for (int k = 0; k < 32; ++k) top[k] = exists ? v[k] : -INFINITY;
                fold_columns(top, lane, [](float a, float b) { return fmaxf(a, b); });
                float m = top[0], add[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const float mk = __shfl_sync(~0u, m, k), ref = fabsf(mk) == INFINITY ? 0.0f : mk;
                    add[k] = exists ? __expf(v[k] - ref) : 0.0f;
                }
                fold_columns(add, lane, [](float a, float b) { return a + b; });
                const int token = c0 + lane;
                // the target's logit: lane `at` of this warp holds it in v[lane]
                const long long at = y - seg.first - (r - lane);
                const bool here = token < live && at >= 0 && at < 32 && r - lane + at < seg.rows && quarter * 32 + at < p.few_rows;
                if (__any_sync(~0u, here)) {
                    float z = 0.0f;
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const float got = __shfl_sync(~0u, v[k], __shfl_sync(~0u, static_cast<int>(at) & 31, k));
                        if (lane == k) z = got;
                    }
                    if (here) p.picked[token] = z;
                }
                const int quarters = (p.few_rows + 31) / 32;
                if (token < live)
                    p.part[(static_cast<long long>(2 * (seg.tile0 + t.m) + static_cast<int>(rank)) * quarters + quarter) * p.rows + token] =
                        make_float2(m, add[0]);
            } else if constexpr (MODE == kDlogitsFew) {
                float v[32];
                values(0, v);
                const long long at = y - seg.first - (r - lane);
                const int mine_at = at >= 0 && at < 32 ? static_cast<int>(at) : -1;
                const bool some = __any_sync(~0u, mine_at >= 0);
                // D[token][r]: adjacent lanes adjacent columns; zeros up to whole blocks of K either way
                const bool store = in_cta < p.few_rows && r < (seg.rows + kVK - 1) / kVK * kVK;
                unsigned short *out = p.d + seg.col0 + r + static_cast<long long>(c0) * p.d_ld;
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const float l = __shfl_sync(~0u, lse, k), f = __shfl_sync(~0u, g, k);
                    const int a = __shfl_sync(~0u, mine_at, k);
                    float q = soft<T>(v[k] - l);
                    if (some && a == lane) q = expm1f(v[k] - l);  // the target's, see kDlogits
                    const float d = c0 + k < live && r < seg.rows ? q * f : 0.0f;
                    if constexpr (T != kF32) {  // the rounded value and what it lacks
                        float lo, hi;
                        widen2<T>(narrow2<T>(d, d), lo, hi);
                        if (store) {
                            store_elem<T>(out, k * p.d_ld, d);
                            store_elem<T>(out, p.d_part + k * p.d_ld, fabsf(d) <= 3.402823466e38f ? d - lo : 0.0f);
                        }
                    } else {
                        uint32_t w[3];
                        split2<false>(d, 0.0f, w);
#pragma unroll
                        for (int part = 0; part < 3; ++part)
                            if (store) out[part * p.d_part + k * p.d_ld] = static_cast<unsigned short>(w[part] & 0xFFFFu);
                    }
                }
            } else {
                const int col = t.n * p.bn + c0;
                const int n = min(width, p.dim - col);
                const bool mine = r < (t.dw ? seg.rows : live);
                constexpr int es = Elem<T>::bytes;
                char *out = nullptr;
                float *sum = nullptr;
                if (mine && t.dw) {
                    out = seg.dw + static_cast<long long>(r) * seg.dw_row + static_cast<long long>(col) * es;
                } else if (mine) {
                    if (seg.dh) out = seg.dh + static_cast<long long>(p.index[r]) * seg.dh_row + static_cast<long long>(col) * es;
                    if (p.sum)
                        sum = p.sum + ((static_cast<long long>(t.seg) * p.slices + t.slice) * p.sum_rows + r) * p.sum_ld + col;
                }
#pragma unroll
                for (int c = 0; c < 128; c += 32) {
                    if (c >= width) break;
                    float v[32];
                    values(c, v);
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] *= unscale;
                    if (sum) {
                        // rows of partial sums are whole groups of eight
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            if (c + k < n) {
                                float4 *q = reinterpret_cast<float4 *>(sum + c + k);
                                if (!p.sum_begin) {
                                    const float4 o = *q;
                                    v[k] += o.x, v[k + 1] += o.y, v[k + 2] += o.z, v[k + 3] += o.w;
                                }
                                if (!out) *q = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                            }
                    }
                    if (c < n) store_block<T>(stage_out, out ? out + c * es : nullptr, v, min(32, n - c), lane);
                }
            }
            if constexpr (!kVRuns<MODE, T>) done_run();
        }
        if constexpr (MODE == kDlogits || MODE == kDlogitsFew) asm volatile("fence.proxy.async.global;" ::: "memory");
    }
    __syncthreads();
    __syncwarp();
    tmem_fence_before();
    cluster_sync();  // neither CTA leaves or frees its tensor memory while the other may still use it
    tmem_fence_after();
    if (warp == 2) tmem_dealloc(tmem, kVTmemCols);
}

// ---- around the products -----------------------------------------------------------

struct VocabJoinParams {
    const float2 *part;
    const float *picked;
    const long long *targets;
    long long ignore, vocab;  // vocabulary rows of all pieces
    int rows;
    int parts;
    float *loss, *lse;
};

// A running maximum m and sum s of exp(z - m) joined with another; m = -infinity and s = 0 join as nothing.
__device__ __forceinline__ void join_stats(float &m, float &s, float qm, float qs) {
    const float to = fmaxf(m, qm), ref = fabsf(to) == INFINITY ? 0.0f : to;
    auto moved = [&](float a, float x) {  // an infinite maximum's sum is relative to zero
        return a == -INFINITY ? x : x * __expf((a == INFINITY ? 0.0f : a) - ref);
    };
    s = moved(m, s) + moved(qm, qs);
    m = to;
}

// Join the partial statistics of each row: lse = log sum exp, loss = lse - target's logit.  A block
// takes R rows (4, or one of few tokens), 256 / R threads to a row, so that a single row's hundreds of
// parts are loaded at once.
template <int R>
__global__ void __launch_bounds__(256) ar_vocab_join_kernel(const __grid_constant__ VocabJoinParams p) {
    __shared__ float ms[8][R], ss[8][R];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const long long t = static_cast<long long>(blockIdx.x) * R + threadIdx.x % R;
    float m = -INFINITY, s = 0.0f;
    if (t < p.rows) {
        constexpr int U = 4;
        for (int k = threadIdx.x / R; k < p.parts; k += U * (256 / R)) {
            float2 q[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = k + u * (256 / R);
                q[u] = at < p.parts ? p.part[static_cast<long long>(at) * p.rows + t] : make_float2(-INFINITY, 0.0f);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) join_stats(m, s, q[u].x, q[u].y);
        }
    }
    for (int o = 16; o >= R; o /= 2)
        join_stats(m, s, __shfl_xor_sync(~0u, m, o), __shfl_xor_sync(~0u, s, o));
    if (lane < R) ms[warp][lane] = m, ss[warp][lane] = s;
    __syncthreads();
    if (threadIdx.x >= R || t >= p.rows) return;
    for (int w = 1; w < 8; ++w) join_stats(m, s, ms[w][lane], ss[w][lane]);
    const float lse = (fabsf(m) == INFINITY ? 0.0f : m) + logf(s);
    p.lse[t] = lse;
    const long long y = p.targets[t];
    p.loss[t] = y == p.ignore ? 0.0f : (y < 0 || y >= p.vocab) ? NAN : lse - p.picked[t];
}

struct VocabListParams {
    const long long *targets;
    const float *lse, *dloss;
    long long ignore, vocab;
    int rows;
    float gain;       // 2^14 for f16, else 1
    VocabList *list;
    VocabRow *row;    // [live]
    int *index;       // [live] original token
    int *place;       // [rows] list entry, -1: not counted
};

// List the counted tokens in order, one block.  D is held as (softmax - onehot) dloss / max |dloss| (of
// the finite ones), so that rounding it to 16 bits costs the same whatever the scale of dloss, and costs nothing where
// all dloss are alike and the probability is small; f16 moves up by 2^14 so that probabilities keep
// their eleven bits down to 2^-28.
static __global__ void __launch_bounds__(1024) ar_vocab_list_kernel(const __grid_constant__ VocabListParams p) {
    __shared__ int counts[32];
    __shared__ float tops[32];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    auto counted = [&](int t) {
        if (t >= p.rows) return false;
        const long long y = p.targets[t];
        return y != p.ignore && y >= 0 && y < p.vocab;
    };
    // four adjacent tokens to a thread
    constexpr int U = 4;
    float top = 0.0f;
    for (int t0 = U * static_cast<int>(threadIdx.x); t0 < p.rows; t0 += U * 1024)
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (counted(t0 + u)) {
                const float a = fabsf(p.dloss[t0 + u]);
                if (a <= 3.402823466e38f) top = fmaxf(top, a);  // an infinity or NaN is its own token's affair
            }
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    top = tops[lane];
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if (top == 0.0f) top = 1.0f;
    int done = 0;
    for (int b0 = 0; b0 < p.rows; b0 += U * 1024) {
        const int t0 = b0 + U * static_cast<int>(threadIdx.x);
        bool c[U];
        int mine = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) mine += c[u] = counted(t0 + u);
        int upto = mine;  // of this warp's threads up to this one
        for (int o = 1; o < 32; o *= 2) {
            const int q = __shfl_up_sync(~0u, upto, o);
            if (lane >= o) upto += q;
        }
        if (lane == 31) counts[warp] = upto;
        __syncthreads();
        int warps = counts[lane];  // of the warps up to warp `lane`
        for (int o = 1; o < 32; o *= 2) {
            const int q = __shfl_up_sync(~0u, warps, o);
            if (lane >= o) warps += q;
        }
        int at = done + upto - mine + (warp ? __shfl_sync(~0u, warps, warp - 1) : 0);
        done += __shfl_sync(~0u, warps, 31);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t0 + u;
            if (c[u]) {
                p.row[at] = VocabRow{p.lse[t], p.dloss[t] / top * p.gain, p.targets[t]};
                p.index[at] = t;
            }
            if (t < p.rows) p.place[t] = c[u] ? at : -1;
            at += c[u];
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) *p.list = VocabList{done, top / p.gain};
}

struct VocabPackParams {
    const void *src[kMaxSegs];     // matrices of a launch, blockIdx.y picks one
    long long src_row[kMaxSegs];   // bytes
    int rows[kMaxSegs];
    long long dst_at[kMaxSegs];    // where a matrix's rows start in dst
    int dim;
    unsigned short *dst;      // [parts][dst_rows][dst_ld]
    long long dst_ld, dst_part;
    const int *place;         // where row t goes (-1: nowhere), nullptr: in order
    const VocabList *list;    // with place: rows behind the list are zeroed up to a block of K
    char *dh[kMaxSegs];       // outputs whose row t is zeroed when the token is not counted
    long long dh_row[kMaxSegs];
    int n_dh;
};

// Copy rows into 16-byte aligned rows of 16-bit elements (float32: three bf16 parts), one row after
// another per block.  Bound by memory: 50021 f16 rows of 1031, 212 MB in 42 us (5.0 TB/s).
template <int T>
__global__ void __launch_bounds__(256) ar_vocab_pack_kernel(const __grid_constant__ VocabPackParams p) {
    pdl_launch_dependents();
    pdl_wait();
    auto zero_row = [&](long long at) {
        for (int q = 0; q < (T == kF32 ? 3 : 1); ++q)
            for (long long c = threadIdx.x; c < p.dst_ld / 8; c += blockDim.x)
                reinterpret_cast<uint4 *>(p.dst + q * p.dst_part + at * p.dst_ld)[c] = make_uint4(0, 0, 0, 0);
    };
    const int m = blockIdx.y;
    for (int t = blockIdx.x; t < p.rows[m]; t += gridDim.x) {
        const long long at = p.place ? p.place[t] : p.dst_at[m] + t;
        if (at < 0) {
            for (int r = 0; r < p.n_dh; ++r)
                for (int c = threadIdx.x; c < p.dim; c += blockDim.x) store_elem<T>(p.dh[r] + t * p.dh_row[r], c, 0.0f);
            continue;
        }
        const char *src = static_cast<const char *>(p.src[m]) + t * p.src_row[m];
        const bool whole = reinterpret_cast<uintptr_t>(src) % 16 == 0, words = reinterpret_cast<uintptr_t>(src) % 4 == 0;
        for (long long g = threadIdx.x; g < p.dst_ld / 8; g += blockDim.x) {
            if constexpr (T != kF32) {
                if (whole && 8 * g + 8 <= p.dim) {
                    *reinterpret_cast<uint4 *>(p.dst + at * p.dst_ld + 8 * g) = __ldg(reinterpret_cast<const uint4 *>(src) + g);
                    continue;
                }
            }
            if constexpr (T != kF32) {  // rows on a 4-byte boundary
                if (words && 8 * g + 8 <= p.dim) {
                    const uint32_t *from = reinterpret_cast<const uint32_t *>(src) + 4 * g;
                    *reinterpret_cast<uint4 *>(p.dst + at * p.dst_ld + 8 * g) =
                        make_uint4(__ldg(from), __ldg(from + 1), __ldg(from + 2), __ldg(from + 3));
                    continue;
                }
            }
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = 8 * g + k < p.dim ? load_elem<T, true>(src, 8 * g + k) : 0.0f;
            unsigned short *out = p.dst + at * p.dst_ld + 8 * g;
            if constexpr (T != kF32) {
                uint32_t w[4];
                word_pack<T, 4>(v, w);
                *reinterpret_cast<uint4 *>(out) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
                uint32_t w[4][3];
#pragma unroll
                for (int e = 0; e < 4; ++e) split2<true>(v[2 * e], v[2 * e + 1], w[e]);
#pragma unroll
                for (int q = 0; q < 3; ++q)
                    *reinterpret_cast<uint4 *>(out + q * p.dst_part) = make_uint4(w[0][q], w[1][q], w[2][q], w[3][q]);
            }
        }
    }
    if (p.list) {
        const int live = p.list->live, end = (live + kVK - 1) / kVK * kVK;
        for (int at = live + blockIdx.x; at < end; at += gridDim.x) zero_row(at);
    }
    asm volatile("fence.proxy.async.global;" ::: "memory");
}

struct VocabSumParams {
    const float *sum;         // [segment][slice][sum_rows][sum_ld]
    long long sum_rows, sum_ld;
    int slices, dim;
    const VocabList *list;
    const int *index;
    char *dh[kMaxSegs];       // of each segment's piece
    long long dh_row[kMaxSegs];
};

// dH of a piece from its slices, in their order: blockIdx.z picks the segment, blockIdx.y strides over
// rows, a thread takes four columns.
template <int T>
__global__ void __launch_bounds__(256) ar_vocab_sum_kernel(const __grid_constant__ VocabSumParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int live = p.list->live, c = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (c >= p.dim) return;
    for (int r = blockIdx.y; r < live; r += gridDim.y) {
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int s = 0; s < p.slices; ++s) {
            const float4 q = *reinterpret_cast<const float4 *>(
                p.sum + ((static_cast<long long>(blockIdx.z) * p.slices + s) * p.sum_rows + r) * p.sum_ld + c);
            v.x += q.x, v.y += q.y, v.z += q.z, v.w += q.w;
        }
        char *out = p.dh[blockIdx.z] + static_cast<long long>(p.index[r]) * p.dh_row[blockIdx.z];
        const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (c + k < p.dim) store_elem<T>(out, c + k, w[k]);
    }
}

}  // namespace tps
