// linear_xent.cu -- softmax cross entropy of a linear output layer, and its gradients.
//
//     l = H W^T,  lse = log sum_v exp(l_v),  loss = lse - l[target]
//     G = exp(l - lse) - onehot(target),  dH = dloss * (G W),  dW = G^T (dloss * H)
//
// H [N, D] hidden states, W [V, D] output weights, 16-bit.  The N x V logits exist only as
// accumulator tiles in tensor memory: the loss folds each tile into a running maximum and
// sum per row, and the gradient forms them again, one piece of the vocabulary at a time,
// whose G (16-bit, at most about kPieceBytes) goes through the two products behind it.
//
// One kernel does the four products.  A pair of CTAs (one cluster of two SMs) owns a
// 256 x 256 tile: tcgen05.mma.cta_group::2 with both operands in shared memory, 64 of the
// contracted dimension a stage, 128-byte swizzled; each CTA stages its half of A and of B
// (32 KB a stage, a ring of six), so a tile's operands cross from L2 once per pair.  Warp 0
// feeds the ring by TMA, warp 1 of the pair's first CTA issues the MMAs, warps 4..11 (or 4..19) drain
// the accumulator -- of which there are two, 256 TMEM columns each, so that the epilogue of
// one tile runs under the MMAs of the next.  A thread of the epilogue owns one row of the
// tile: row sums need no shuffles.  Tiles are dealt statically to a persistent grid of one
// CTA per SM, in groups of kGroup row tiles that keep their rows of A in L2.
//
// What bounds it: the tensor cores.  A stage's MMAs take 237 ns with operands at hand, 277 ns
// with them coming from L2 (2.1 GHz, one launch); under continuous load the power limit sets
// the clock.  bf16 8,192 x 32,000 x 4,096 over several boards: loss 1,149 to 1,177 us (1,825 to 1,870
// TFLOP/s), gradient 3,690 to 3,760 us (1,715 to 1,745 TFLOP/s; 3,950 us, 1,631, after a second of
// nothing else; a cuBLAS product reaches 1,871 in a burst and 1,707 for seconds).  Short contractions
// are bound by the epilogue, the loads' latency and, below about 450 contracted elements, by G, which is
// written once and read twice: fp16 1,021 x 50,257 x 768, gradient, 158 to 184 us by run, as the buffers
// happen to lie (126 us at 1,871 TFLOP/s); bf16 37 rows against the same weights, loss, 22 us, of which
// about 13 read W at 6 TB/s.
//
// The accumulators are fp32, but tensor cores cut off what an addition shifts below the sum's
// last place, where fp32 arithmetic rounds: a sum comes out smaller by 1e-9 of itself for every contracted
// element.  So an accumulator of the loss's logits takes at most 1,280 elements (kChunkStages), one of dH
// or dW at most kChain, and longer sums are added from those in fp32.
//
// The operands need no transposed copies: dH contracts over the vocabulary, along which W
// is not contiguous, and dW over the tokens, along which neither G nor H is; those operands
// are staged as 64-column boxes and described to the MMA as MN-major.
//
// dloss stays out of the 16-bit G: 1 / rows, the usual dloss, has a rounding of its own that
// every entry of G would share (bf16 1/7168 is 0.19% off, and dH and dW were).  dH takes it in
// fp32 in the epilogue; dW contracts over the rows, so there H is scaled beforehand, by
// dloss / max |dloss|, which is exactly 1 for a mean.  That copy also holds zeros for the rows
// that take no part, whatever their H is.  fp16 lets a power of two of small weights travel in G
// instead (shift_of), where it costs no bits.
//
// Every mbarrier wait is bounded (about one second of %globaltimer).  On expiry the device error
// word is set and the warp goes to its end, where the pair's first CTA waits for all boxes and MMAs that
// either CTA started, however far each had come: at the end of every launch, where it costs nothing, so
// that nothing has to tell the warps of each other's failures.  tb_linear_xent_selftest_timeout runs
// that path.
#include "tensor_core.cuh"

namespace tb {
namespace {

enum Kind { kLse = 0, kGrad = 1, kDH = 2, kDW = 3 };
// What the self-test leaves out, so that waits run out: the boxes of the pair's first or second CTA,
// the word that an accumulator is full, the last word that it is empty again (its barrier counts one
// arrival more).
enum Withheld { kNothing = 0, kBoxes0 = 1, kBoxes1 = 2, kFull = 3, kEmpty = 4 };

// Epilogue warps: two for each quarter of the accumulator's rows, or four where logits have so few
// contracted elements that the epilogue takes longer than a tile's MMAs.  Loss and G of 4,096 x 50,257:
// at 256 contracted elements 97 and 119 us with 8 warps, 77 and 99 with 16; at 384, 100 and 129 against
// 88 and 131; at 512, 117 and 170 against 124 and 170 (a warp of 16 has no second buffer for columns on
// their way).  The loss of few tiles is bound by latency: 100 x 32,000 x 256 took 12.8 us with 8, 14.5
// with 16.
constexpr int kFewWarps = 8, kManyWarps = 16;
constexpr int kShortStages = 384 / kStageK;
constexpr int kThreadsOf(int epi) { return (kEpiWarp + epi) * 32; }
// Contracted elements that one accumulator of the loss's logits takes, at most: what truncation cuts off
// grows with them.  More come in equal chunks, one accumulator after the other, which sixteen epilogue
// warps add up in fp32 registers (64 columns of a row each).  Losses of 1,024 x 32,000 against 64 bits
// at 1,024 / 1,536 / 2,048 / 4,096 / 8,192 contracted elements: in one accumulator 0.63 / 0.91 / 1.13 /
// 1.85 / 2.86e-6 off, in chunks of 1,024 or fewer 0.63 / 0.44 / 0.55 / 0.43 / 0.32e-6 (fp32: 0.22 to
// 0.56e-6).  It costs what the larger epilogue waits for: 64 x 32,000 x 4,096 52.7 -> 54.0 us, 8,192 x
// 32,000 x 4,096 1% and below; with 1,024 as the limit 37 x 50,257 x 1,088 27.9 -> 30.7.
constexpr int kChunkStages = 1280 / kStageK;
constexpr int kSmem = kStages * kStageBytes + kOutboxes * kOutBytes + 1024 + 256;   // alignment, barriers
// Row tiles walked together (see tile_at): bf16 8,192 x 32,000 x 4,096, loss and gradient, took 1,133
// and 3,673 us with 16, 1,170 and 3,704 with 8, 1,180 and 3,943 with 32.
constexpr int kGroup = 16;

// Bytes of G that one piece of the vocabulary may take, and the fewest columns of a piece.  The same
// gradient took 3,673 us with 256 MiB (two pieces), 3,996 with 128, 4,023 with 64, 3,631 with 1,024.
constexpr int64_t kPieceBytes = 256ll << 20;
constexpr int64_t kMinPiece = 2048;
constexpr int64_t kLseRows = 16384;          // rows of one launch of the loss: bounds its workspace

// exp(l - b) is exp2(l log2(e) - b log2(e)) in one FMA, off by a factor of two to the rounding of
// b log2(e): 2^-10 of a power at |b| = 2^14, 16 powers at 2^28, and beyond 2^31 (columns masked by
// -1e10, say) as many as make it inf or 0. The loss takes that rounding out of a group's sum again, where
// the sum is scaled anyway, and above kAlone, where fp32 numbers lie 32 apart, counts the largest logit
// alone. The gradient forms l - lse first where |lse| is above kFar. (So did the loss: a branch in
// every 32 columns, 79 -> 82 us for 4,096 x 50,257 x 256.)
constexpr float kAlone = 268435456.f, kFar = 16384.f;

// ---------------------------------------------------------------- arguments
struct Weigh {
    const float* dloss;
    const void* H;            // [rows][ld], padded where it has to be
    void* scaled;             // [rows][ld]; NULL: dW is not wanted
    float *weight, *top;      // weight NULL: not in this launch
    int64_t rows;
    int ld;
};
struct Product {
    int m_tiles, n_tiles, splits, k_stages;
    int rows, cols;           // of the result
    int chunk;                // kLse: stages of an accumulator, where a tile has more
    int width;                // columns of a tile: at most kTile, fewer where that fills the last wave
    int a_rows;               // K-major A: rows of a box, fewer than kHalf where the result has no more
    int out_map;              // results go out by TMA (16-byte aligned rows), else element by element
    int b_base;               // kGrad, kDH: first vocabulary row of the piece
    int* err;
    unsigned long long wait_ns;   // bound of every wait
    int withhold;             // self-test: a Withheld
    // kLse, kGrad
    const int64_t* target;    // of this launch's rows
    int64_t ignore;
    int vocab;
    float2* part;             // kLse: [parts of a tile * n_tiles][rows] maximum and sum
    float* target_logit;      // kLse: [rows]
    const float *lse, *dloss; // kGrad
    const float* weight;      // kDH: dloss by row, 0 where a row takes no part
    const float* top;         // kDW: the largest |dloss|
    // kDH, kDW
    float* sums;              // [splits][rows][cols] fp32, NULL: the tile is the result
    int first, last;          // piece: starts the sums; writes the result (dW's is always both)
    int sums_map;             // rows of the sums are whole 16 bytes: they go out by TMA
    void* out;                // [rows][cols] 16-bit
    Weigh weigh;              // kGrad
};

// fp16's G is held times 2^14, so that probabilities down to 2^-38 stay above its last step;
// the products undo it in fp32.  bf16 has fp32's range.
template <class Fmt>
constexpr float kGBits = std::is_same<Fmt, F16>::value ? 14.f : 0.f;
template <class Fmt>
constexpr float kGScale = std::is_same<Fmt, F16>::value ? 16384.f : 1.f;

// The power of two by which fp16 holds a row's G smaller and its scaled H larger: dW contracts over the
// rows, so the weights have to be in one of the two, and H times a small weight falls below fp16's
// normal numbers (2^-14) while G has room there.  Three powers stay in H, which is seldom that small,
// and more than eight would take G of ordinary probabilities (2^-20 and above) out of the normal
// numbers.  dH takes it out again with the row's weight.
template <class Fmt>
__device__ __forceinline__ int shift_of(float weight, float top) {
    if constexpr (std::is_same<Fmt, BF16>::value) return 0;
    const int apart = (int)(__float_as_uint(top) >> 23) - (int)(__float_as_uint(weight) << 1 >> 24);
    return min(max(apart - 3, 0), 8);
}
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((127 + e) << 23); }

// An element of dH; a row of weight 0 takes no part, whatever its sums are.
template <class Fmt>
__device__ __forceinline__ float weigh(float sum, float weight) {
    return weight == 0.f ? 0.f : sum * (1.f / kGScale<Fmt>) * weight;
}

// Row tiles in groups of kGroup, the group's tiles column by column: the pairs that run
// together share few column tiles and reuse the group's rows.
__device__ __forceinline__ void tile_at(const Product& p, unsigned t, int* split, int* mt, int* nt) {
    const unsigned per_split = (unsigned)(p.m_tiles * p.n_tiles);
    *split = 0;
    if (p.splits > 1) {
        *split = (int)(t / per_split);
        t -= *split * per_split;
    }
    unsigned first = 0;
    if (p.m_tiles > kGroup) {
        first = t / (unsigned)(kGroup * p.n_tiles);
        t -= first * kGroup * p.n_tiles;
        first *= kGroup;
    }
    const unsigned height = min(kGroup, p.m_tiles - (int)first);
    *nt = (int)(t / height);
    *mt = (int)(first + t - *nt * height);
}
// The contracted stages of a split.
__device__ __forceinline__ void stages_of(const Product& p, int split, int* lo, int* hi) {
    *lo = 0;
    *hi = p.k_stages;
    if (p.splits > 1) {           // (at most 256 splits of 2^24 / 64 stages: no overflow)
        *lo = (int)((unsigned)split * p.k_stages / (unsigned)p.splits);
        *hi = (int)((unsigned)(split + 1) * p.k_stages / (unsigned)p.splits);
    }
}

// What the later products need of dloss: each row's weight (0 where it takes no part), the largest
// magnitude among them, and H with every row times its weight over that.  It runs beside the logits'
// product: the epilogue warps of every CTA find the maximum before their first tile (rows * 12 bytes
// from L2), and two otherwise idle warps copy the CTA's share of the rows.  (A kernel of its own in
// front of the products took 8 us at 1,021 x 768.)
template <class Fmt>
__device__ __forceinline__ float weight_of(const Product& p, int64_t r) {
    const int64_t t = p.target[r];
    const float v = p.weigh.dloss[r];
    return t != p.ignore && t >= 0 && t < p.vocab ? v : 0.f;
}

// Both meet at named barrier 1.
template <int Epi>
constexpr int kWeighThreads = (Epi + 2) * 32;

// By the epilogue warps, `thread` counts theirs.
template <class Fmt, int Epi>
__device__ __forceinline__ void weigh_top(const Product& p, int thread, float* tops) {
    float m = 0.f;
    unsigned owner = 0;               // of the next rows' weights
    const int64_t rows = p.weigh.rows;
#pragma unroll 8
    for (int64_t r = thread; r < rows; r += Epi * 32) {
        const float v = weight_of<Fmt>(p, r);
        if (owner == blockIdx.x) p.weigh.weight[r] = v;
        if (++owner == gridDim.x) owner = 0;
        if (fabsf(v) <= 3.4028235e38f) m = fmaxf(m, fabsf(v));   // neither infinite nor NaN
    }
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (thread % 32 == 0) tops[thread / 32] = m;
    // fp16's G needs the largest weight itself
    if constexpr (std::is_same<Fmt, F16>::value) asm volatile("bar.sync 1, %0;" ::"n"(kWeighThreads<Epi>) : "memory");
    else asm volatile("bar.arrive 1, %0;" ::"n"(kWeighThreads<Epi>) : "memory");
}
template <int Epi>
__device__ __forceinline__ float largest(const float* tops) {
    float m = tops[0];
    for (int i = 1; i < Epi; ++i) m = fmaxf(m, tops[i]);
    return m == 0.f ? 1.f : m;
}

// By the other two; part 0 .. parts - 1 of all CTAs' warps.
template <class Fmt, int Epi>
__device__ __forceinline__ void weigh_rows(const Product& p, int lane, unsigned part, unsigned parts,
                                           const float* tops) {
    using T = typename Fmt::T;
    asm volatile("bar.sync 1, %0;" ::"n"(kWeighThreads<Epi>) : "memory");
    const float m = largest<Epi>(tops);
    if (part == 0 && lane == 0) *p.weigh.top = m;
    if (!p.weigh.scaled) return;
    const uint4* H = static_cast<const uint4*>(p.weigh.H);
    uint4* scaled = static_cast<uint4*>(p.weigh.scaled);
    const int64_t rows = p.weigh.rows;
    const unsigned per_row = (unsigned)p.weigh.ld / 8, first = part * 32 + lane, step = parts * 32;
    int64_t row = first / per_row;
    unsigned col = first % per_row;
    while (row < rows) {              // four vectors at a time, a step apart
        int64_t at[4];
        uint4 x[4];
        float w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            at[k] = -1;
            if (row < rows) {
                at[k] = row * per_row + col;
                x[k] = H[at[k]];
                w[k] = weight_of<Fmt>(p, row);
            }
            row += step / per_row;
            col += step % per_row;
            if (col >= per_row) col -= per_row, ++row;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (at[k] < 0) break;
            const float f = w[k] / m * power_of_two(shift_of<Fmt>(w[k], m));
            float y[8];
            unpack8<Fmt>(x[k], y);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = w[k] == 0.f ? 0.f : y[e] * f;
            scaled[at[k]] = pack8<Fmt>(y);
        }
    }
}

// What one CTA stages of a pair's tiles, stage after stage.
template <int K>
struct Feed {
    static constexpr bool kAMn = K == kDW, kBMn = K == kDH || K == kDW;
    const Product& p;
    const CUtensorMap *a, *b;
    int rank, pairs, tiles, t, k, k_hi, m0, n0;
    int nk, nk_hi, nm0, nn0;      // of the next tile: worked out while the ring is full
    __device__ __forceinline__ Feed(const Product& p_, const CUtensorMap* a_, const CUtensorMap* b_, int rank_,
                                    int pair, int pairs_, int tiles_)
        : p(p_), a(a_), b(b_), rank(rank_), pairs(pairs_), tiles(tiles_), t(pair) {
        look(t);
        take();
    }
    __device__ __forceinline__ bool more() const { return t < tiles; }
    __device__ __forceinline__ void look(int tile) {
        if (tile >= tiles) return;
        int split, mt, nt;
        tile_at(p, (unsigned)tile, &split, &mt, &nt);
        stages_of(p, split, &nk, &nk_hi);
        nm0 = mt * kTile + rank * kHalf;
        nn0 = nt * p.width + rank * (p.width / 2);
    }
    __device__ __forceinline__ void take() { k = nk, k_hi = nk_hi, m0 = nm0, n0 = nn0; }
    __device__ __forceinline__ void next() {
        if (++k < k_hi) return;
        t += pairs;
        take();
    }
    // Calls f(operand 0 or 1, byte offset in it, map, x, y) for the boxes of this stage.
    template <class F>
    __device__ __forceinline__ void boxes(F f) const {
        const int base = K == kGrad || K == kDH ? p.b_base : 0;
        if constexpr (kAMn) {
            f(0, 0, a, m0, k * kStageK);
            f(0, 8192, a, m0 + 64, k * kStageK);
        } else if (p.a_rows == kHalf || rank == 0) {
            f(0, 0, a, k * kStageK, m0);
        }
        if constexpr (kBMn) {
            f(1, 0, b, n0, base + k * kStageK);
            f(1, 8192, b, n0 + 64, base + k * kStageK);
        } else {
            f(1, 0, b, k * kStageK, base + n0);
        }
    }
};

// Folds a group of logits into a row's maximum m and sum s of exp(l - base(m)); base is 0 where the
// maximum is infinite, so that a logit of +inf gives lse = +inf and rows of -inf give -inf.  `off`:
// the powers of two by which the group's sum is too large.
__device__ __forceinline__ float base_of(float m) { return isinf(m) ? 0.f : m; }

__device__ __forceinline__ void fold(float& m, float& s, float m2, float s2, float off = 0.f) {
    const float top = fmaxf(m, m2), b = base_of(top);
    const float x = s == 0.f ? 0.f : s * exp2_fast((base_of(m) - b) * kLog2e);
    const float y = s2 == 0.f ? 0.f : s2 * exp2_fast(__fmaf_rn(base_of(m2) - b, kLog2e, -off));
    m = top;
    s = x + y;
}

// Folds columns c .. c + 31 of a tile into a row's maximum and sum; `hit`, the target's column or -1,
// leaves its logit.
__device__ __forceinline__ void fold_logits(float (&v)[32], int c, int width, int hit, float* target_logit, float& m,
                                            float& s) {
                        if ((hit & ~31) == c) {           // (hit = -1: no chunk)
                            float x = v[0];
    #pragma unroll
                            for (int i = 1; i < 32; ++i) x = c + i == hit ? v[i] : x;
                            *target_logit = x;
                        }
                        if (c + 32 > width) {
    #pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (c + i >= width) v[i] = __int_as_float(0xff800000);
                        }
                        // four chains each: one of 31 maxima and one of 32 sums take longer than the
                        // exponentials
                        float top4[4] = {v[0], v[1], v[2], v[3]};
    #pragma unroll
                        for (int i = 4; i < 32; ++i) top4[i & 3] = fmaxf(top4[i & 3], v[i]);
                        const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
                        // (finite: a column behind the vocabulary's end is -inf)
                        const float base = base_of(top), at = fmaxf(base * kLog2e, -3.4028235e38f),
                                    off = __fmaf_rn(base, kLog2e, -at);
                        const unsigned long long b2 = pair_of(-at, -at), scale = pair_of(kLog2e, kLog2e);
                        unsigned long long sum[4] = {0, 0, 0, 0};
    #pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float lo, hi;
                            split_pair(fma_pair(pair_of(v[2 * i], v[2 * i + 1]), scale, b2), lo, hi);
                            sum[i & 3] = add_pair(sum[i & 3], pair_of(exp2_fast(lo), exp2_fast(hi)));
                        }
                        float part, part2;
                        split_pair(add_pair(add_pair(sum[0], sum[1]), add_pair(sum[2], sum[3])), part, part2);
                        part += part2;
                        const bool alone = fabsf(base) > kAlone;
                        if (alone && part == part) part = 1.f;
                        fold(m, s, top, part, alone ? 0.f : off);
}

// ---------------------------------------------------------------- the product
// Long: kLse of tiles that have more stages than an accumulator takes.
template <class Fmt, int K, int Epi, bool Long>
__global__ void __launch_bounds__(kThreadsOf(Epi), 1)
product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
               const __grid_constant__ CUtensorMap map_out, const __grid_constant__ Product p) {
    using T = typename Fmt::T;
    constexpr bool kAMn = K == kDW, kBMn = K == kDH || K == kDW;
    constexpr int kParts = Epi / 4;         // of a tile's columns
    __shared__ float tops[Epi];       // kGrad: see weigh_top
    extern __shared__ unsigned char raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    unsigned char* outbox = smem + kStages * kStageBytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(outbox + kOutboxes * kOutBytes);
    const uint32_t stage0 = smem_addr(smem), bar0 = smem_addr(bars);
    const uint32_t full = bar0, empty = full + 8 * kStages, acc_full = empty + 8 * kStages,
                   acc_empty = acc_full + 16, drain = acc_empty + 16, done = drain + 8, issued = done + 8,
                   slot = issued + 4;
    // (the shuffle tells the compiler that a warp agrees on its number)
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, p.withhold == kFull ? 2 : 1);
            mbar_init(acc_empty + 8 * i, 2 * Epi + (p.withhold == kEmpty));    // of both CTAs
        }
        mbar_init(drain, 1);
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tmem_fence_before();
    __syncthreads();
    cluster_sync();
    tmem_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + (slot - stage0));
    pdl_wait();
    asm volatile("fence.proxy.async;" ::: "memory");   // what earlier kernels stored, TMA reads
    pdl_trigger();

    const int tiles = p.m_tiles * p.n_tiles * p.splits;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (warp == 0) {
        const uint32_t leader_full = map_to(full, 0);
        const uint32_t a_bytes = (kAMn || p.a_rows == kHalf ? 2 * kHalf : p.a_rows) * kStageK * 2;
        const uint32_t stage_bytes = a_bytes + p.width * kStageK * 2;      // of both CTAs
        int it = 0;
        Feed<K> feed(p, &map_a, &map_b, (int)rank, pair, pairs, tiles);
        if (p.withhold == kBoxes0 + (int)rank) feed.t = tiles;
        for (; feed.more(); feed.next(), ++it) {
            const int s = it % kStages;
            if (it >= kStages && !__all_sync(0xffffffffu, mbar_wait(empty + 8 * s, (it / kStages - 1) & 1, &p)))
                break;
            const uint32_t at = stage0 + s * kStageBytes, bar = leader_full + 8 * s;
            if (elect_one()) {
                if (rank == 0) mbar_expect(full + 8 * s, stage_bytes);
                feed.boxes([&](int operand, int offset, const CUtensorMap* m, int x, int y) {
                    tma_box(at + operand * kOperandBytes + offset, m, x, y, bar);
                });
            }
            if (feed.k + 1 == feed.k_hi) feed.look(feed.t + pairs);
        }
        // The way out: first the MMAs, which the first CTA issues, and the word of them, which goes to both.
        // Then the boxes, which end on the first CTA's barriers.  Stages that both CTAs issued complete by
        // themselves.  After a wait that gave up one may have issued stages, at most a ring of them, that the
        // other has not: such a phase counts the second CTA's boxes, which never come, or lacks the first
        // CTA's arrival.  Both are made good (no MMA waits for them any more), so that every phase ends with
        // its last box.
        if (rank == 1 && elect_one())
            asm volatile("st.shared::cluster.u32 [%0], %1;\n\t"
                         "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%2];" ::"r"(map_to(issued, 0)),
                         "r"(it), "r"(map_to(done, 0))
                         : "memory");
        __syncwarp();
        const bool ended = __all_sync(0xffffffffu, mbar_wait<kEnd>(drain, 0, &p));
        if (rank == 0 && ended && __all_sync(0xffffffffu, mbar_wait<kEnd>(done, 0, &p))) {
            const int peer = *reinterpret_cast<volatile int*>(smem + (issued - stage0));
            const uint32_t bytes1 = ((kAMn || p.a_rows == kHalf ? kHalf : 0) + p.width / 2) * kStageK * 2;
            if (it != peer && elect_one())
                for (int q = min(it, peer); q < max(it, peer); ++q) {
                    const uint32_t bar = full + 8 * (q % kStages);
                    if (q < it)
                        asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes1)
                                     : "memory");
                    else mbar_expect(bar, bytes1);
                }
            __syncwarp();
            for (int q = max(0, max(it, peer) - kStages); q < max(it, peer); ++q)
                mbar_wait<kEnd>(full + 8 * (q % kStages), (q / kStages) & 1, &p);
        }
    } else if (warp == 1) {
        if (rank == 0) {
            // The whole warp walks the stages and one lane issues: the operands of an MMA are uniform
            // registers, which a loop of one lane would have to fill by copies.
            constexpr uint32_t fmt = std::is_same<Fmt, BF16>::value ? 1 : 0;
            const uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)kAMn << 15) |
                                   ((uint32_t)kBMn << 16) | ((uint32_t)(p.width / 8) << 17) | ((kTile / 16) << 24);
            // 16 contracted elements: 32 bytes of a K-major row, 16 rows of an MN-major box
            constexpr uint32_t step_a = (kAMn ? 2048 : 32) >> 4, step_b = (kBMn ? 2048 : 32) >> 4;
            const uint32_t a0 = desc_low<kAMn>(stage0), b0 = desc_low<kBMn>(stage0 + kOperandBytes);
            // One thread issues everything: what stands between two MMAs is kept to a few
            // additions, or the tensor core waits for it (660 clocks a stage instead of the 512
            // of its MMAs, with descriptors and stage numbers worked out each time).
            uint32_t s = 0, parity = 0;
            int n = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                int k, k_hi;
                stages_of(p, p.splits > 1 ? t / (p.m_tiles * p.n_tiles) : 0, &k, &k_hi);
                do {                  // (one accumulator, unless Long)
                    const int buf = n & 1, end = Long ? min(k_hi, k + p.chunk) : k_hi;
                    if (n >= 2 && !__all_sync(0xffffffffu, mbar_wait<kRelaxed>(acc_empty + 8 * buf, (n / 2 - 1) & 1, &p))) {
                        ok = false;
                        break;
                    }
                    tmem_fence_after();
                    const uint32_t d = tmem + buf * kTile;
                    uint32_t accumulate = 0;
                    for (; k < end; ++k) {
                        if (!__all_sync(0xffffffffu, mbar_wait(full + 8 * s, parity, &p))) {
                            ok = false;
                            break;
                        }
                        const uint32_t a = a0 + s * (kStageBytes >> 4), b = b0 + s * (kStageBytes >> 4);
                        if (elect_one()) {
                            mma_pair<false>(d, a, b, idesc, accumulate);
#pragma unroll
                            for (int j = 1; j < kStageK / 16; ++j)
                                mma_pair<true>(d, a + j * step_a, b + j * step_b, idesc, 1);
                            mma_commit(empty + 8 * s);
                        }
                        accumulate = 1;
                        if (++s == kStages) s = 0, parity ^= 1;
                    }
                    if (ok && elect_one()) mma_commit(acc_full + 8 * buf);
                    ++n;
                } while (Long && ok && k < k_hi);
            }
            if (elect_one()) mma_commit(drain);
        }
    } else if (K == kGrad && (warp == 2 || warp == 3)) {
        if (p.weigh.weight) weigh_rows<Fmt, Epi>(p, lane, blockIdx.x * 2 + (warp & 1), gridDim.x * 2, tops);
    } else if (Long && warp >= kEpiWarp) {
        // as below; a tile is long, so its target is there before its logits are
        const int quad = warp & 3, part_no = (warp - kEpiWarp) >> 2;
        const uint32_t leader_empty = map_to(acc_empty, 0);
        int n = 0;
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs) {
            int split, mt, nt;
            tile_at(p, (unsigned)t, &split, &mt, &nt);
            const int row = mt * kTile + (int)rank * kHalf + quad * 32 + lane;
            const bool live = row < p.rows;
            const int64_t target = live ? p.target[row] : p.ignore;
            const int n0 = nt * p.width, all = min(p.width, p.cols - n0);
            const int share = (all + 32 * kParts - 1) / (32 * kParts) * 32;      // 32 or 64
            const int c0 = part_no * share, width = min(all, c0 + share);
            unsigned long long sum[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) sum[i] = 0;
            for (int k = 0; k < p.k_stages; k += p.chunk, ++n) {
                const int buf = n & 1;
                if (!__all_sync(0xffffffffu, mbar_wait<kRelaxed>(acc_full + 8 * buf, (n / 2) & 1, &p))) {
                    ok = false;
                    break;
                }
                tmem_fence_after();
                const uint32_t acc = tmem + buf * kTile + ((uint32_t)(quad * 32) << 16) + c0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t r[16];
                    tmem_read16(acc + 16 * j, r);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        sum[8 * j + i] = add_pair(sum[8 * j + i], pair_of(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])));
                }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(leader_empty + 8 * buf);
            }
            if (!ok) break;
            const int64_t c = target - n0;
            const int hit = target != p.ignore && target >= 0 && target < p.vocab && c >= c0 && c < width ? (int)c : -1;
            float m = __int_as_float(0xff800000), s = 0.f;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                if (c0 + 32 * g >= width) break;
                float v[32];
#pragma unroll
                for (int i = 0; i < 16; ++i) split_pair(sum[16 * g + i], v[2 * i], v[2 * i + 1]);
                fold_logits(v, c0 + 32 * g, width, hit, p.target_logit + row, m, s);
            }
            if (live) p.part[((int64_t)nt * kParts + part_no) * p.rows + row] = make_float2(m, s);
        }
    } else if (warp >= kEpiWarp) {
        // TMEM lanes 32 quad .. 32 quad + 31 (a warp reaches those of its number modulo 4), and
        // one of the parts of the tile's columns
        const int quad = warp & 3, part_no = (warp - kEpiWarp) >> 2;
        const uint32_t leader_empty = map_to(acc_empty, 0);
        if (K == kGrad && p.weigh.weight) weigh_top<Fmt, Epi>(p, threadIdx.x - kEpiWarp * 32, tops);
        constexpr bool kShifts = std::is_same<Fmt, F16>::value && (K == kGrad || K == kDH);
        float top_weight = 1.f;
        if constexpr (K == kGrad && kShifts) top_weight = p.weigh.weight ? largest<Epi>(tops) : *p.top;
        else if constexpr (K == kDW || kShifts) top_weight = *p.top;
        Outbox<Fmt, kOutboxes / Epi> box{outbox + (warp - kEpiWarp) * (kOutboxes / Epi) * kOutBytes, &map_out, lane, 0};
        // What a tile's row needs from memory is asked for while the tile before it is worked on: a
        // load's latency at the start of every tile is as long as the work on one of few stages.
        struct Tile {
            int split, mt, nt, row0;
            int64_t target;
            float lse, weight;
        };
        auto look = [&](int t) {
            Tile x{};
            if (t >= tiles) return x;
            tile_at(p, (unsigned)t, &x.split, &x.mt, &x.nt);
            x.row0 = x.mt * kTile + (int)rank * kHalf + quad * 32;
            if (x.row0 + lane < p.rows) {
                if constexpr (K == kLse || K == kGrad) x.target = p.target[x.row0 + lane];
                if constexpr (K == kGrad) x.lse = p.lse[x.row0 + lane], x.weight = p.dloss[x.row0 + lane];
                if constexpr (K == kDH) x.weight = p.weight[x.row0 + lane];
            }
            return x;
        };
        int n = 0;
        Tile ahead = look(pair);
        for (int t = pair; t < tiles; t += pairs, ++n) {
            const Tile tile = ahead;
            const int buf = n & 1, split = tile.split, nt = tile.nt;
            const int row0 = tile.row0, row = row0 + lane;
            const bool live = row < p.rows;
            const int n0 = nt * p.width, all = min(p.width, p.cols - n0);
            const int share = (all + 32 * kParts - 1) / (32 * kParts) * 32;
            const int c0 = part_no * share, width = min(all, c0 + share);
            const uint32_t acc = tmem + buf * kTile + ((uint32_t)(quad * 32) << 16);
            if (!__all_sync(0xffffffffu, mbar_wait<kRelaxed>(acc_full + 8 * buf, (n / 2) & 1, &p))) break;
            tmem_fence_after();
            ahead = look(t + pairs);
            int hit = -1;                             // the target's column in this tile
            float weight = tile.weight, one_hot = kGScale<Fmt>;
            if constexpr (K == kDH && kShifts) weight *= power_of_two(shift_of<Fmt>(weight, top_weight));
            float lse2 = 0.f;
            bool counts = false, far = false;
            if constexpr (K == kLse || K == kGrad) {
                counts = live && tile.target != p.ignore && tile.target >= 0 && tile.target < p.vocab;
                const int64_t c = tile.target - (K == kGrad ? p.b_base : 0) - n0;
                if (counts && c >= c0 && c < width) hit = (int)c;
                if constexpr (K == kGrad) {
                    far = fabsf(tile.lse) > kFar && !isinf(tile.lse);
                    lse2 = (far ? 0.f : tile.lse * kLog2e) - kGBits<Fmt>;
                    if constexpr (kShifts) {
                        const int e = shift_of<Fmt>(weight, top_weight);
                        lse2 += (float)e;
                        one_hot *= power_of_two(-e);
                    }
                    // a row that is weighted with 0 counts for nothing, not for 0 * NaN (dW)
                    counts = counts && weight != 0.f;
                }
            }

            float m = __int_as_float(0xff800000), s = 0.f;
            auto work = [&](const uint32_t (&r)[32], int c) {
                float v[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
                if constexpr (K == kLse) {
                    fold_logits(v, c, width, hit, p.target_logit + row, m, s);
                } else if constexpr (K == kGrad) {
                    if (far) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] -= tile.lse;
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        split_pair(fma_pair(pair_of(v[i], v[i + 1]), pair_of(kLog2e, kLog2e), pair_of(-lse2, -lse2)),
                                   v[i], v[i + 1]);
                        v[i] = exp2_fast(v[i]);
                        v[i + 1] = exp2_fast(v[i + 1]);
                    }
                    if ((hit & ~31) == c) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = c + i == hit ? v[i] - one_hot : v[i];
                    }
                    if (!counts) {                    // a row that takes no part
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = 0.f;
                    }
                    if (row0 < p.rows) box.put(v, n0 + c, row0);
                } else {
                    T* out = static_cast<T*>(p.out);
                    const int col = n0 + c;
                    const bool keep = !p.last || p.splits > 1;
                    if (p.sums && keep && p.sums_map) {
                        if (row0 < p.rows) put_sums(box.mem, &map_out, lane, v, col, row0, split, !p.first);
                    } else if (p.sums && live) {
                        float* sum = p.sums + ((int64_t)split * p.rows + row) * p.cols + col;
                        if (p.sums_map && c + 32 <= width) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float4 o = *reinterpret_cast<const float4*>(sum + 4 * i);
                                v[4 * i] += o.x, v[4 * i + 1] += o.y, v[4 * i + 2] += o.z, v[4 * i + 3] += o.w;
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (c + i < width) {
                                    if (!p.first) v[i] += sum[i];
                                    if (keep) sum[i] = v[i];
                                }
                        }
                    }
                    __syncwarp();
                    if (!keep) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] = K == kDH ? weigh<Fmt>(v[i], weight) : v[i] * (1.f / kGScale<Fmt>) * top_weight;
                        if (row0 < p.rows) {
                            if (p.out_map) box.put(v, col, row0);
                            else box.put_plain(v, out, col, row0, p.rows, p.cols);
                        }
                    }
                }
            };
            // The next columns come while the present ones are worked on; behind the last ones the
            // accumulator is free for the MMAs of the tile after the next.
            uint32_t one[32];
            auto release = [&] {
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(leader_empty + 8 * buf);
            };
            __syncwarp();
            if constexpr (kParts > 2) {   // four warps a scheduler: the others work while one waits
                if (c0 >= width) release();
                for (int c = c0; c < width; c += 32) {
                    tmem_load32(acc + c, one);
                    tmem_wait(one);
                    if (c + 32 >= width) release();
                    work(one, c);
                    __syncwarp();
                }
            } else {
                uint32_t two[32];
                if (c0 < width) tmem_load32(acc + c0, one);
                else release();
                for (int c = c0; c < width; c += 64) {
                    tmem_wait(one);
                    if (c + 32 < width) tmem_load32(acc + c + 32, two);
                    else release();
                    work(one, c);
                    __syncwarp();
                    if (c + 32 < width) {
                        tmem_wait(two);
                        if (c + 64 < width) tmem_load32(acc + c + 64, one);
                        else release();
                        work(two, c + 32);
                        __syncwarp();
                    }
                }
            }
            if constexpr (K == kLse) {
                if (live) p.part[((int64_t)nt * kParts + part_no) * p.rows + row] = make_float2(m, s);
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    cluster_sync();             // no CTA leaves while the other may signal or read it
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                     : "memory");
}

// ---------------------------------------------------------------- around the products
// A row's parts, two or four for each column tile, in a fixed order.  R rows a CTA, 256 / R lanes a row:
// 32 rows side by side read whole sectors, eight put more loads in flight for calls of few rows.
template <int R>
__global__ void __launch_bounds__(256)
join_kernel(const float2* part, const float* target_logit, const int64_t* target, int64_t ignore,
            int vocab, int rows, int n_parts, float* loss, float* lse, int* err) {
    constexpr int kLanes = 256 / R;
    __shared__ float2 sh[kLanes][R];
    const int r = threadIdx.x % R, w = threadIdx.x / R, row = blockIdx.x * R + r;
    pdl_wait();
    pdl_trigger();
    float m = __int_as_float(0xff800000), s = 0.f;
    if (row < rows) {
        for (int t = w; t < n_parts; t += 8 * kLanes) {
            float2 q[8];              // loaded together, folded one after another
#pragma unroll
            for (int k = 0; k < 8; ++k)
                q[k] = t + k * kLanes < n_parts ? part[(int64_t)(t + k * kLanes) * rows + row]
                                                : make_float2(__int_as_float(0xff800000), 0.f);
#pragma unroll
            for (int k = 0; k < 8; ++k) fold(m, s, q[k].x, q[k].y);
        }
    }
    sh[w][r] = make_float2(m, s);
    __syncthreads();
    for (int k = kLanes / 2; k; k /= 2) {
        if (w < k) {
            fold(m, s, sh[w + k][r].x, sh[w + k][r].y);
            sh[w][r] = make_float2(m, s);
        }
        __syncthreads();
    }
    if (w == 0 && row < rows) {
        const float total = base_of(m) + logf(s);
        lse[row] = total;
        const int64_t tg = target[row];
        if (tg == ignore) {
            loss[row] = 0.f;
        } else if (tg < 0 || tg >= vocab) {
            loss[row] = __int_as_float(0x7fc00000);
            atomicExch(err, (int)TB_ERR_INVALID_VALUE);
        } else {
            loss[row] = total - target_logit[row];
        }
    }
}

// Sums the splits of dH or dW and rounds once: V elements a thread, of one row.  `weight`: by row
// (dH), or one for all (dW: the largest |dloss|, never 0).
template <class Fmt, int V>
__global__ void __launch_bounds__(256)
join_splits_kernel(const float* sums, int splits, int64_t n, int cols, const float* weight, bool by_row,
                   const float* top, typename Fmt::T* out) {
    pdl_wait();
    pdl_trigger();
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V;
    if (i >= n) return;
    float w = by_row ? weight[i / cols] : *weight;
    if (std::is_same<Fmt, F16>::value && by_row) w *= power_of_two(shift_of<Fmt>(w, *top));
    float v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = 0.f;
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
        if constexpr (V == 4) {
            const float4 x = *reinterpret_cast<const float4*>(sums + s * n + i);
            v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
        } else {
            v[0] += sums[s * n + i];
        }
    }
    typename Fmt::T r[V];
#pragma unroll
    for (int e = 0; e < V; ++e) r[e] = Fmt::from_f32(weigh<Fmt>(v[e], w));
    if constexpr (V == 4) *reinterpret_cast<uint2*>(out + i) = *reinterpret_cast<const uint2*>(r);
    else out[i] = r[0];
}

// Rows padded with zeros.  A thread writes one 16-byte vector; what it reads starts on any element,
// so it loads the words around it and shifts.  The matrix itself may start on any element: of the words
// at its two ends, only the half that is inside is read.
struct Pad {
    const void* in[2];        // H, W
    void* out[2];
    int64_t rows[2];
    unsigned ctas;            // of H
    int cols, ld;
};
// Rows of a CTA: a thread finds its row by a 32-bit division, and has a few vectors.
__host__ __device__ constexpr int64_t pad_rows_a_cta(int ld) { return 1024 / (ld / 8) + 1; }
__global__ void __launch_bounds__(256) pad_kernel(const __grid_constant__ Pad p) {
    pdl_wait();
    pdl_trigger();
    const int which = blockIdx.x >= p.ctas;
    const void* in = p.in[which];
    uint4* out = static_cast<uint4*>(p.out[which]);
    const int64_t rows = p.rows[which];
    const int cols = p.cols;
    const unsigned per_row = (unsigned)p.ld / 8;
    const bool odd = reinterpret_cast<uintptr_t>(in) & 2;    // the matrix starts in the middle of a word
    const uint16_t* elements = static_cast<const uint16_t*>(in);
    const unsigned* w = reinterpret_cast<const unsigned*>(elements - odd);
    const int64_t end = rows * cols + odd, words = end >> 1;  // whole words up to the matrix's end
    const int64_t row0 = (int64_t)(blockIdx.x - (which ? p.ctas : 0)) * pad_rows_a_cta(p.ld);
    const int64_t rows_here = min(rows - row0, pad_rows_a_cta(p.ld));
    for (unsigned i = threadIdx.x; i < (unsigned)rows_here * per_row; i += 256) {
        const unsigned r = i / per_row, c = (i - r * per_row) * 8;
        const int64_t at = (row0 + r) * cols + c + odd, word = at >> 1;
        unsigned x[5];
#pragma unroll
        for (int k = 0; k < 5; ++k) {
            if (odd && word + k == 0) x[k] = (unsigned)elements[0] << 16;
            else x[k] = word + k < words ? w[word + k] : word + k == words && (end & 1) ? elements[end - 1 - odd] : 0u;
        }
        if (at & 1) {
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = __funnelshift_r(x[k], x[k + 1], 16);
        }
        const int keep = cols - (int)c;          // elements of this row in the vector, if any
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (2 * k >= keep) x[k] = 0;
            else if (2 * k + 1 >= keep) x[k] &= 0xffffu;
        }
        out[(row0 + r) * per_row + c / 8] = make_uint4(x[0], x[1], x[2], x[3]);
    }
}

// ---------------------------------------------------------------- host
template <class Fmt, int K, int Epi = kFewWarps, bool Long = false>
tb_status launch_product(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& out, Product p, cudaStream_t st,
                         int most_pairs = 1 << 20) {
    if (!p.wait_ns) p.wait_ns = kWaitLimitNs;
    const void* kernel = reinterpret_cast<const void*>(&product_kernel<Fmt, K, Epi, Long>);
    const int pairs = std::min(most_pairs, resident_clusters(kernel, kThreadsOf(Epi), kSmem, 2));
    if (pairs < 1) return TB_ERR_CUDA;
    const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles * p.splits;
    // (pairs without a tile still take their share of weigh_rows)
    const int64_t grid = 2 * (p.weigh.weight ? pairs : std::min<int64_t>(tiles, pairs));
    if (launch_clusters<true>(product_kernel<Fmt, K, Epi, Long>, dim3((unsigned)grid), dim3(kThreadsOf(Epi)), kSmem, st, 2, a,
                              b, out, p) != cudaSuccess)
        return TB_ERR_CUDA;
    return launch_status();
}

// How a call of these sizes is cut up.
struct Cut {
    int lse_width, grad_width;   // columns of a tile of logits
    int64_t lse_tiles;
    int lse_warps, grad_warps;   // of the epilogue of logits
    bool lse_long;            // logits in several accumulators
    int64_t ld;               // padded row length of H and W (D where no copy is needed)
    bool pad;
    int64_t piece, pieces;    // gradient: columns of a piece of the vocabulary
    int64_t ldg;
    int splits, splits_w;     // of dH's contraction, of dW's
    // byte offsets into the workspace
    size_t off_h, off_w, off_scaled, off_weight, off_g, off_sums, off_sums_w, off_top, off_part, off_logit, total;
};

// Parts of the vocabulary (of the rows) that dH's (dW's) products are split into: as many as fill the
// machine when its tiles do not.  The result has n x d elements.  The cost counts in stages (64 contracted elements of a tile, about 0.3 us): waves of
// tiles, about eight more for each one's epilogue, and for the sums that the splits leave a launch and
// their bytes.  (fp16 1,021 x 768 against 50,257: six splits, 160 us; none, 314 us.)
// And as many as keep what one accumulator takes below kChain contracted elements: what its truncated
// additions cut off a sum of one sign grows with them, 1e-9 of the sum an element, 6e-5 at kChain, an
// eighth of fp16's half step (1,048,576 rows in one accumulator: two half steps). The splits are added
// in fp32.
constexpr int64_t kChain = 65536;
int pick_splits(int64_t n, int64_t d, int64_t k_stages, int64_t pairs) {
    const int64_t tiles = ceil_div(n, kTile) * ceil_div(d, kTile);
    const int64_t fewest = ceil_div(k_stages, kChain / kStageK);
    int best = (int)fewest;
    double least = 1e30;
    for (int64_t s = fewest; s <= std::max(fewest, std::min<int64_t>(pairs, k_stages)); ++s) {
        const double cost = (double)ceil_div(tiles * s, pairs) * ((double)ceil_div(k_stages, s) + 8.0) +
                            (s > 1 ? 12.0 + (double)s * (0.05 + (double)(n * d) / 450000.0) : 0.0);
        if (cost < least * 0.97) least = cost, best = (int)s;
    }
    return best;
}

// Columns of a tile of logits: the width among 256, 224, .. 128 that takes the fewest columns' time
// when its tiles are dealt to the pairs in whole waves.  A narrower tile has the same cost per
// column but reads its rows of A more often, so it has to save 3%.  (37 x 50,257: 225 tiles of 224
// columns are three waves of 76 pairs, as are 197 of 256.)
int pick_width(int64_t m_tiles, int64_t cols, int64_t pairs) {
    int best = kTile;
    double least = 1e30;
    for (int w = kTile; w >= 128; w -= 32) {
        const double cost = (double)ceil_div(m_tiles * ceil_div(cols, w), pairs) * w;
        if (cost < least * 0.97) least = cost, best = w;
    }
    return best;
}

Cut cut_call(int64_t n, int64_t d, int64_t v, bool bwd, int sms) {
    Cut c{};
    // TMA wants strides of 16 bytes; a copy that has to be made gets strides of 128, so that no
    // box row lies across two lines
    c.pad = d % 8 != 0;
    c.ld = c.pad ? round_up(d, kStageK) : d;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    if (c.pad) {
        c.off_h = take((size_t)n * c.ld * 2);
        c.off_w = take((size_t)v * c.ld * 2);
    }
    if (!bwd) {
        const int64_t rows = std::min(n, kLseRows);
        c.lse_width = pick_width(ceil_div(rows, kTile), v, sms / 2);
        c.lse_tiles = ceil_div(v, c.lse_width);
        const bool many = ceil_div(d, kStageK) <= kShortStages && ceil_div(rows, kTile) * c.lse_tiles > 8 * (sms / 2);
        c.lse_long = ceil_div(d, kStageK) > kChunkStages;
        c.lse_warps = many || c.lse_long ? kManyWarps : kFewWarps;
        c.off_part = take((size_t)rows * (c.lse_warps / 4) * c.lse_tiles * sizeof(float2));
        c.off_logit = take((size_t)rows * sizeof(float));
    } else {
        int64_t most = std::max(kMinPiece, kPieceBytes / (2 * std::max<int64_t>(n, 1)));
        most = std::max<int64_t>(kTile, most / kTile * kTile);
        c.pieces = ceil_div(v, most);
        c.piece = std::min(round_up(ceil_div(v, c.pieces), kTile), round_up(v, kTile));
        c.pieces = ceil_div(v, c.piece);
        c.ldg = c.piece;
        c.grad_warps = ceil_div(d, kStageK) <= kShortStages ? kManyWarps : kFewWarps;
        c.grad_width = pick_width(ceil_div(n, kTile), std::min(c.piece, v), sms / 2);
        c.splits = pick_splits(n, d, c.piece / kStageK, sms / 2);
        c.splits_w = pick_splits(std::min(c.piece, v), d, ceil_div(n, kStageK), sms / 2);
        c.off_g = take((size_t)n * c.ldg * 2);
        if (c.pieces > 1 || c.splits > 1) c.off_sums = take((size_t)c.splits * n * d * sizeof(float));
        if (c.splits_w > 1) c.off_sums_w = take((size_t)c.splits_w * std::min(c.piece, v) * d * sizeof(float));
        c.off_scaled = take((size_t)n * c.ld * 2);
        c.off_weight = take((size_t)n * sizeof(float));
        c.off_top = take(sizeof(float));
    }
    c.total = at;
    return c;
}

// Rows of a box of K-major A.  A result of at most kHalf rows lies in the pair's first CTA alone: its
// boxes hold those rows and the second CTA loads none.  What the MMAs read in their place is what the
// memory held; it reaches only rows that nothing stores.
int box_rows(int64_t rows) { return rows < kHalf ? (int)round_up(rows, 8) : kHalf; }

// What TMA reads starts on 16 bytes; where it reads a padded copy, the copy does.
uintptr_t operand_alignment(int64_t d) { return d % 8 ? 2 : 16; }

// A tile's MMAs take 0.3 to 0.7 us for 64 contracted elements, and the epilogue waits for a whole
// tile: 2^24 of them stay well inside the wait limit.
constexpr int64_t kMaxSize = 1ll << 24;

tb_status check_sizes(int64_t n, int64_t d, int64_t v, tb_dtype dtype) {
    if (n < 0 || d < 1 || v < 1 || n > kMaxSize || d > kMaxSize || v > kMaxSize) return TB_ERR_INVALID_VALUE;
    if (n * d > (1ll << 40) || v * d > (1ll << 40)) return TB_ERR_INVALID_VALUE;
    if (dtype != TB_BF16 && dtype != TB_F16) return TB_ERR_UNSUPPORTED_DTYPE;
    return TB_OK;
}

tb_status workspace(int64_t n, int64_t d, int64_t v, tb_dtype dtype, bool bwd, size_t* bytes) {
    if (!bytes) return TB_ERR_INVALID_VALUE;
    const tb_status st = check_sizes(n, d, v, dtype);
    if (st != TB_OK) return st;
    *bytes = 0;
    if (n == 0) return TB_OK;
    int dev = 0;
    DeviceInfo info{};
    if (!current_device_info(&dev, &info)) return TB_ERR_CUDA;
    *bytes = cut_call(n, d, v, bwd, info.sm_count).total;
    return TB_OK;
}

tb_status pad_both(const void* H, const void* W, unsigned char* ws, const Cut& c, int64_t n, int64_t v, int64_t d,
                   cudaStream_t st) {
    Pad p{};
    p.in[0] = H, p.in[1] = W;
    p.out[0] = ws + c.off_h, p.out[1] = ws + c.off_w;
    p.rows[0] = n, p.rows[1] = v;
    p.cols = (int)d, p.ld = (int)c.ld;
    p.ctas = (unsigned)ceil_div(n, pad_rows_a_cta(p.ld));
    const int64_t grid = p.ctas + ceil_div(v, pad_rows_a_cta(p.ld));
    return launch_pdl(pad_kernel, dim3((unsigned)grid), dim3(256), 0, st, p) == cudaSuccess ? TB_OK : TB_ERR_CUDA;
}

struct Problem {
    const void *H, *W;
    const int64_t* target;
    const float *lse_in, *dloss;
    float *loss, *lse;
    void *dH, *dW;
    int64_t n, d, v, ignore;
    unsigned char* ws;
    int sms;
    int* err;
    cudaStream_t st;
};

template <class Fmt>
tb_status run_loss(const Problem& q, const Cut& c) {
    constexpr bool bf = std::is_same<Fmt, BF16>::value;
    const void *H = q.H, *W = q.W;
    if (c.pad) {
        if (pad_both(q.H, q.W, q.ws, c, q.n, q.v, q.d, q.st) != TB_OK) return TB_ERR_CUDA;
        H = q.ws + c.off_h;
        W = q.ws + c.off_w;
    }
    CUtensorMap a, b;
    if (!make_map(&b, W, q.v, q.d, c.ld, c.lse_width / 2, bf)) return TB_ERR_CUDA;
    for (int64_t r0 = 0; r0 < q.n; r0 += kLseRows) {
        const int64_t rows = std::min(kLseRows, q.n - r0);
        if (!make_map(&a, static_cast<const char*>(H) + r0 * c.ld * 2, rows, q.d, c.ld, box_rows(rows), bf))
            return TB_ERR_CUDA;
        Product p{};
        p.m_tiles = (int)ceil_div(rows, kTile);
        p.width = c.lse_width;
        p.a_rows = box_rows(rows);
        p.n_tiles = (int)c.lse_tiles;
        p.splits = 1;
        p.k_stages = (int)ceil_div(q.d, kStageK);
        p.rows = (int)rows;
        p.cols = (int)q.v;
        p.err = q.err;
        p.target = q.target + r0;
        p.ignore = q.ignore;
        p.vocab = (int)q.v;
        p.part = reinterpret_cast<float2*>(q.ws + c.off_part);
        p.target_logit = reinterpret_cast<float*>(q.ws + c.off_logit);
        p.chunk = (int)ceil_div(p.k_stages, ceil_div(p.k_stages, kChunkStages));
        const tb_status s = c.lse_long                  ? launch_product<Fmt, kLse, kManyWarps, true>(a, b, a, p, q.st)
                            : c.lse_warps == kManyWarps ? launch_product<Fmt, kLse, kManyWarps>(a, b, a, p, q.st)
                                                        : launch_product<Fmt, kLse>(a, b, a, p, q.st);
        if (s != TB_OK) return s;
        const bool few = rows <= 32 * q.sms;
        const dim3 grid((unsigned)ceil_div(rows, few ? 8 : 32));
        const cudaError_t e = launch_pdl(few ? join_kernel<8> : join_kernel<32>, grid, dim3(256), 0, q.st,
                                         (const float2*)p.part, (const float*)p.target_logit, p.target, p.ignore,
                                         p.vocab, p.rows, c.lse_warps / 4 * p.n_tiles, q.loss + r0, q.lse + r0, q.err);
        if (e != cudaSuccess) return TB_ERR_CUDA;
    }
    return launch_status();
}

template <class Fmt>
bool join_splits(const float* sums, int splits, int64_t n, int64_t cols, const float* weight, bool by_row,
                 const float* top, void* out, cudaStream_t st) {
    using T = typename Fmt::T;
    const bool vec = cols % 4 == 0 && aligned_to(out, 8);
    const dim3 grid((unsigned)ceil_div(n, vec ? 1024 : 256));
    return launch_pdl(vec ? join_splits_kernel<Fmt, 4> : join_splits_kernel<Fmt, 1>, grid, dim3(256), 0, st, sums, splits,
                      n, (int)cols, weight, by_row, top, static_cast<T*>(out)) == cudaSuccess;
}

template <class Fmt>
tb_status run_grad(const Problem& q, const Cut& c) {
    constexpr bool bf = std::is_same<Fmt, BF16>::value;
    const void *H = q.H, *W = q.W;
    if (c.pad) {
        if (pad_both(q.H, q.W, q.ws, c, q.n, q.v, q.d, q.st) != TB_OK) return TB_ERR_CUDA;
        H = q.ws + c.off_h;
        W = q.ws + c.off_w;
    }
    float* weight = reinterpret_cast<float*>(q.ws + c.off_weight);
    float* top = reinterpret_cast<float*>(q.ws + c.off_top);
    using T = typename Fmt::T;
    T* scaled = reinterpret_cast<T*>(q.ws + c.off_scaled);
    void* g = q.ws + c.off_g;
    CUtensorMap h_rows, w_rows, h_cols, w_cols, g_rows, g_cols, out;
    if (!make_map(&h_rows, H, q.n, q.d, c.ld, box_rows(q.n), bf) || !make_map(&w_rows, W, q.v, q.d, c.ld, c.grad_width / 2, bf) ||
        !make_map(&h_cols, scaled, q.n, q.d, c.ld, kStageK, bf) || !make_map(&w_cols, W, q.v, q.d, c.ld, kStageK, bf))
        return TB_ERR_CUDA;
    for (int64_t i = 0; i < c.pieces; ++i) {
        const int64_t v0 = i * c.piece, cols = std::min(c.piece, q.v - v0);
        Product p{};
        p.m_tiles = (int)ceil_div(q.n, kTile);
        p.width = c.grad_width;
        p.a_rows = box_rows(q.n);
        p.n_tiles = (int)ceil_div(cols, p.width);
        p.splits = 1;
        p.out_map = 1;
        p.k_stages = (int)ceil_div(q.d, kStageK);
        p.rows = (int)q.n;
        p.cols = (int)cols;
        p.b_base = (int)v0;
        p.err = q.err;
        p.target = q.target;
        p.ignore = q.ignore;
        p.vocab = (int)q.v;
        p.lse = q.lse_in;
        p.dloss = q.dloss;
        p.weight = weight;
        p.top = top;
        if (i == 0)
            p.weigh = Weigh{q.dloss, H, q.dW ? scaled : nullptr, weight, top, q.n, (int)c.ld};
        if (!make_map(&out, g, q.n, cols, c.ldg, 32, bf, true)) return TB_ERR_CUDA;
        tb_status s = c.grad_warps == kManyWarps ? launch_product<Fmt, kGrad, kManyWarps>(h_rows, w_rows, out, p, q.st)
                                                 : launch_product<Fmt, kGrad>(h_rows, w_rows, out, p, q.st);
        if (s != TB_OK) return s;
        if (q.dH) {
            if (!make_map(&g_rows, g, q.n, cols, c.ldg, box_rows(q.n), bf)) return TB_ERR_CUDA;
            Product r = p;
            r.width = kTile;
            r.out_map = q.d % 8 == 0 && aligned_to(q.dH, 16);
            r.n_tiles = (int)ceil_div(q.d, kTile);
            r.k_stages = (int)ceil_div(cols, kStageK);
            r.splits = std::min(c.splits, r.k_stages);
            r.cols = (int)q.d;
            r.first = i == 0;
            r.last = i == c.pieces - 1;
            // a last piece shorter than the splits leaves slices that it does not add to:
            // the join reads all slices that the first piece wrote
            r.sums = c.pieces > 1 || c.splits > 1 ? reinterpret_cast<float*>(q.ws + c.off_sums) : nullptr;
            r.out = q.dH;
            if (c.splits > 1 && r.splits == 1) r.last = 0;
            r.sums_map = r.sums && q.d % 4 == 0;
            if (r.sums_map && (!r.last || r.splits > 1)) {
                if (!make_sums_map(&out, r.sums, c.splits, q.n, q.d)) return TB_ERR_CUDA;
            } else if (r.out_map && !make_map(&out, q.dH, q.n, q.d, q.d, 32, bf, true)) {
                return TB_ERR_CUDA;
            }
            s = launch_product<Fmt, kDH>(g_rows, w_cols, out, r, q.st);
            if (s != TB_OK) return s;
        }
        if (q.dW) {
            if (!make_map(&g_cols, g, q.n, cols, c.ldg, kStageK, bf)) return TB_ERR_CUDA;
            Product r = p;
            r.m_tiles = (int)ceil_div(cols, kTile);
            r.n_tiles = (int)ceil_div(q.d, kTile);
            r.k_stages = (int)ceil_div(q.n, kStageK);
            r.rows = (int)cols;
            r.cols = (int)q.d;
            r.width = kTile;
            r.out = static_cast<char*>(q.dW) + v0 * q.d * 2;
            r.splits = c.splits_w;
            r.first = r.last = 1;
            r.sums = c.splits_w > 1 ? reinterpret_cast<float*>(q.ws + c.off_sums_w) : nullptr;
            r.sums_map = r.sums && q.d % 4 == 0;
            r.out_map = q.d % 8 == 0 && aligned_to(q.dW, 16);
            if (r.sums_map) {
                if (!make_sums_map(&out, r.sums, r.splits, cols, q.d)) return TB_ERR_CUDA;
            } else if (r.out_map && !make_map(&out, r.out, cols, q.d, q.d, 32, bf, true)) {
                return TB_ERR_CUDA;
            }
            s = launch_product<Fmt, kDW>(g_cols, h_cols, out, r, q.st);
            if (s != TB_OK) return s;
            if (r.sums && !join_splits<Fmt>(r.sums, r.splits, cols * q.d, q.d, top, false, top, r.out, q.st))
                return TB_ERR_CUDA;
        }
    }
    if (q.dH && c.splits > 1) {
        const int used = (int)std::min<int64_t>(c.splits, ceil_div(std::min(c.piece, q.v), kStageK));
        if (!join_splits<Fmt>(reinterpret_cast<const float*>(q.ws + c.off_sums), used, q.n * q.d, q.d, weight, true,
                              top, q.dH, q.st))
            return TB_ERR_CUDA;
    }
    return launch_status();
}

// One pair of CTAs over rows x vocab logits of d elements with something withheld; sets *gave_up to
// whether a wait ran out.
tb_status run_withheld(int64_t rows, int64_t d, int64_t vocab, int withheld, int64_t wait_limit_ns, unsigned char* mem,
                       int* err, cudaStream_t st, bool* gave_up) {
    Product p{};
    p.m_tiles = (int)ceil_div(rows, kTile), p.n_tiles = (int)ceil_div(vocab, kTile), p.splits = 1;
    p.k_stages = (int)ceil_div(d, kStageK);
    p.rows = (int)rows, p.cols = p.vocab = (int)vocab;
    p.width = kTile, p.a_rows = box_rows(rows);
    p.err = err, p.wait_ns = (unsigned long long)wait_limit_ns, p.withhold = withheld;
    auto take = [&](int64_t bytes) {
        unsigned char* at = mem;
        mem += round_up(bytes, 256);
        return at;
    };
    const void* H = take(rows * d * 2);
    const void* W = take(vocab * d * 2);
    p.target = reinterpret_cast<const int64_t*>(take(rows * 8));
    p.target_logit = reinterpret_cast<float*>(take(rows * 4));
    p.part = reinterpret_cast<float2*>(take(rows * (kFewWarps / 4) * p.n_tiles * (int64_t)sizeof(float2)));
    CUtensorMap a, b;
    if (!make_map(&a, H, rows, d, d, p.a_rows, true) || !make_map(&b, W, vocab, d, d, p.width / 2, true)) return TB_ERR_CUDA;
    int word = 0;
    if (cudaMemcpyAsync(err, &word, sizeof(int), cudaMemcpyHostToDevice, st) != cudaSuccess) return TB_ERR_CUDA;
    const tb_status s = launch_product<BF16, kLse>(a, b, a, p, st, 1);
    if (s != TB_OK) return s;
    if (cudaMemcpyAsync(&word, err, sizeof(int), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return TB_ERR_CUDA;
    *gave_up = word == (int)TB_ERR_TIMEOUT;
    return TB_OK;
}

}  // namespace
}  // namespace tb

extern "C" tb_status tb_linear_xent_selftest_timeout(int64_t wait_limit_ns, int* launches, void* stream) {
    using namespace tb;
    if (!launches || wait_limit_ns < 1000 || wait_limit_ns > (int64_t)kWaitLimitNs) return TB_ERR_INVALID_VALUE;
    *launches = 0;
    int* err = device_error_word();
    if (!err) return TB_ERR_CUDA;
    // more stages than the ring has, over four tiles; all stages in the ring; a result in the pair's first
    // CTA alone
    constexpr int64_t kSizes[3][3] = {{256, 512, 1024}, {256, 128, 256}, {40, 320, 1024}};
    constexpr size_t kBytes = 2 << 20;       // the first needs 1.4 MB
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    void* mem = nullptr;
    if (cudaMalloc(&mem, kBytes) != cudaSuccess) {
        cudaGetLastError();
        return TB_ERR_OOM;
    }
    tb_status s = cudaMemsetAsync(mem, 0, kBytes, st) == cudaSuccess ? TB_OK : TB_ERR_CUDA;
    for (const auto& n : kSizes)
        for (int what = kBoxes0; what <= kEmpty && s == TB_OK; ++what) {
            if (what == kEmpty && n[2] <= 2 * kTile) continue;     // nothing waits for a third accumulator
            bool gave_up = false;
            s = run_withheld(n[0], n[1], n[2], what, wait_limit_ns, static_cast<unsigned char*>(mem), err, st, &gave_up);
            if (s == TB_OK && gave_up) ++*launches;
        }
    if (cudaStreamSynchronize(st) != cudaSuccess) s = TB_ERR_CUDA;
    if (cudaFree(mem) != cudaSuccess) s = TB_ERR_CUDA;
    return s;
}

extern "C" tb_status tb_linear_xent_workspace_size(int64_t rows, int64_t D, int64_t vocab, tb_dtype dtype,
                                                   size_t* bytes) {
    return tb::workspace(rows, D, vocab, dtype, false, bytes);
}

extern "C" tb_status tb_linear_xent_bwd_workspace_size(int64_t rows, int64_t D, int64_t vocab,
                                                       tb_dtype dtype, size_t* bytes) {
    return tb::workspace(rows, D, vocab, dtype, true, bytes);
}

extern "C" tb_status tb_linear_xent(const void* H, const void* W, const int64_t* targets, float* loss,
                                    float* lse, int64_t rows, int64_t D, int64_t vocab,
                                    int64_t ignore_index, tb_dtype dtype, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    using namespace tb;
    tb_status s = check_sizes(rows, D, vocab, dtype);
    if (s != TB_OK) return s;
    if (rows == 0) return TB_OK;
    if (!H || !W || !targets || !loss || !lse) return TB_ERR_INVALID_VALUE;
    if (!aligned_to(H, operand_alignment(D)) || !aligned_to(W, operand_alignment(D)) || !aligned_to(targets, 8) || !aligned_to(loss, 4) ||
        !aligned_to(lse, 4))
        return TB_ERR_MISALIGNED;
    const Range in[3] = {range_of(H, rows * D, 2), range_of(W, vocab * D, 2), range_of(targets, rows, 8)};
    const Range out[2] = {range_of(loss, rows, 4), range_of(lse, rows, 4)};
    if (overlap(out[0], out[1])) return TB_ERR_ALIAS;
    for (const Range& o : out)
        for (const Range& i : in)
            if (overlap(o, i)) return TB_ERR_ALIAS;
    int dev = 0;
    DeviceInfo info{};
    if (!current_device_info(&dev, &info)) return TB_ERR_CUDA;
    const Cut c = cut_call(rows, D, vocab, false, info.sm_count);
    if (!workspace || workspace_bytes < c.total) return TB_ERR_WORKSPACE;
    if (!aligned_to(workspace, 16)) return TB_ERR_MISALIGNED;
    const Range ws = range_of(workspace, (int64_t)c.total, 1);
    for (const Range& i : in)
        if (overlap(ws, i)) return TB_ERR_ALIAS;
    for (const Range& o : out)
        if (overlap(ws, o)) return TB_ERR_ALIAS;
    int* err = device_error_word();
    if (!err) return TB_ERR_CUDA;
    Problem q{};
    q.H = H, q.W = W, q.target = targets, q.loss = loss, q.lse = lse;
    q.n = rows, q.d = D, q.v = vocab, q.ignore = ignore_index;
    q.ws = static_cast<unsigned char*>(workspace);
    q.sms = info.sm_count, q.err = err, q.st = static_cast<cudaStream_t>(stream);
    return dtype == TB_BF16 ? run_loss<BF16>(q, c) : run_loss<F16>(q, c);
}

extern "C" tb_status tb_linear_xent_bwd(const float* dloss, const void* H, const void* W,
                                        const int64_t* targets, const float* lse, void* dH, void* dW,
                                        int64_t rows, int64_t D, int64_t vocab, int64_t ignore_index,
                                        tb_dtype dtype, void* workspace, size_t workspace_bytes,
                                        void* stream) {
    using namespace tb;
    tb_status s = check_sizes(rows, D, vocab, dtype);
    if (s != TB_OK) return s;
    if (!dH && !dW) return TB_ERR_INVALID_VALUE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (rows == 0) {                     // no row: dW is a sum over nothing
        if (dW && !aligned_to(dW, 2)) return TB_ERR_MISALIGNED;
        if (dW && cudaMemsetAsync(dW, 0, (size_t)vocab * D * 2, st) != cudaSuccess) return TB_ERR_CUDA;
        return TB_OK;
    }
    if (!dloss || !H || !W || !targets || !lse) return TB_ERR_INVALID_VALUE;
    if (!aligned_to(H, operand_alignment(D)) || !aligned_to(W, operand_alignment(D)) || !aligned_to(targets, 8) || !aligned_to(dloss, 4) ||
        !aligned_to(lse, 4) || !aligned_to(dH, 2) || !aligned_to(dW, 2))
        return TB_ERR_MISALIGNED;
    const Range in[5] = {range_of(H, rows * D, 2), range_of(W, vocab * D, 2), range_of(targets, rows, 8),
                         range_of(dloss, rows, 4), range_of(lse, rows, 4)};
    const Range out[2] = {range_of(dH, dH ? rows * D : 0, 2), range_of(dW, dW ? vocab * D : 0, 2)};
    if (overlap(out[0], out[1])) return TB_ERR_ALIAS;
    for (const Range& o : out)
        for (const Range& i : in)
            if (overlap(o, i)) return TB_ERR_ALIAS;
    int dev = 0;
    DeviceInfo info{};
    if (!current_device_info(&dev, &info)) return TB_ERR_CUDA;
    const Cut c = cut_call(rows, D, vocab, true, info.sm_count);
    if (!workspace || workspace_bytes < c.total) return TB_ERR_WORKSPACE;
    if (!aligned_to(workspace, 16)) return TB_ERR_MISALIGNED;
    const Range ws = range_of(workspace, (int64_t)c.total, 1);
    for (const Range& i : in)
        if (overlap(ws, i)) return TB_ERR_ALIAS;
    for (const Range& o : out)
        if (overlap(ws, o)) return TB_ERR_ALIAS;
    int* err = device_error_word();
    if (!err) return TB_ERR_CUDA;
    Problem q{};
    q.H = H, q.W = W, q.target = targets, q.lse_in = lse, q.dloss = dloss, q.dH = dH, q.dW = dW;
    q.n = rows, q.d = D, q.v = vocab, q.ignore = ignore_index;
    q.ws = static_cast<unsigned char*>(workspace);
    q.sms = info.sm_count, q.err = err, q.st = st;
    return dtype == TB_BF16 ? run_grad<BF16>(q, c) : run_grad<F16>(q, c);
}
