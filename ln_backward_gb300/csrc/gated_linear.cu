// gated_linear.cu -- the gated projections of a decoder's feed-forward block, and their gradients.
//
//     G = X Wg^T,  U = X Wu^T,  H = act(G) * U
//     dG = dH * U * act'(G),  dU = dH * act(G),  dX = dG Wg + dU Wu,  dWg = dG^T X,  dWu = dU^T X
//
// X [N, D] hidden states, Wg and Wu [F, D] weights, 16-bit.  Products are 256 x 256 tiles on pairs of CTAs, a ring of six
// 32 KB stages in each and two accumulators in tensor memory, as the output layer's (linear_xent.cu).
//
// Forward: a tile is 256 rows by 128 columns of G and the same 128 of U; one CTA stages Wg's rows, the other Wu's, so that
// both products of an element meet in one accumulator and H needs no pass of its own.  Few rows read both weights once:
// the columns of a tile are chosen so that the tiles fill the pairs, and where even narrow tiles are fewer, the contraction
// is split into fp32 sums that a second kernel joins (pick_up).
// Gradient: gate_kernel forms dG and dU, 16-bit, side by side in the workspace; one launch has the tiles of dX, which
// contracts over both weights, and of dWg and dWu, which contract over the rows, and deals them out so that the pairs end
// together (deal).  fp16's dG and dU are held times a power of two that a pass before finds.
//
// What bounds it: the tensor cores under the power limit.  bf16 8,192 x 4,096 x 11,008: forward with G and U kept 750 to
// 870 us by board and load (1,700 to 1,970 TFLOP/s, 91 to 105 % of cuBLAS's burst), gradient 1,750 to 1,970 us, of which
// 135 are gate_kernel's 901 MB at 6.7 TB/s and the products run at 1,960 TFLOP/s in a single launch.  16 rows against the same
// weights: 35 us, 5.1 TB/s; 138 tiles of 80 columns on 76 pairs leave 10 % of them idle, and filling the rings about 4 us.
// fp16 1,021 x 768 x 2,048: forward 12 us, gradient 30 us (four launches).
#include "tensor_core.cuh"

namespace tb {
namespace {

// kUp: both projections and the activation.  kBack: the products of the gradient.
enum Kind { kUp = 0, kBack = 1 };
// What the self-test leaves out, so that waits run out: the boxes of the pair's first or second CTA, the word that an
// accumulator is full, the last word that it is empty again.
enum Withheld { kNothing = 0, kBoxes0 = 1, kBoxes1 = 2, kFull = 3, kEmpty = 4 };

constexpr int kThreadsOf(int epi) { return (kEpiWarp + epi) * 32; }
constexpr int kSmem = kStages * kStageBytes + kOutboxes * kOutBytes + 1024 + 256;   // alignment, barriers
constexpr int kGroup = 16;                   // row tiles walked together

// ---------------------------------------------------------------- arguments
// A product's tiles: kGroup row tiles at a time, column by column, split after split of the contraction.
struct Tiles {
    int m, n, splits, stages;
    int count;                // m * n * splits
};
struct Args {
    // kUp: up.  kBack: two products in one launch, the one with the longer tiles first.
    Tiles part[2];
    int first;                // kBack: which product part[0] is, 0: dX, 1: dW
    int light, extra;         // kBack: pairs from `light` on have a tile of part[0] less, and first `extra` of part[1]
    int rows, inner, hidden;  // N, F, D
    int half;                 // kUp: columns of a tile of G and of U; kBack: inner rounded up, columns of dG in the workspace
    int a_rows;               // rows of a box of X or dG by rows: fewer than kHalf where there are no more
    int out_map;              // kUp: results go out by TMA, else in 16-byte vectors
    int sums;                 // bit i: the product's (kUp: bit 0) splits leave fp32 sums
    int act;
    const float* unscale;     // kBack: what fp16's dG is held times, inverted
    void *H, *G, *U;          // kUp; G and U may be NULL
    int* err;
    unsigned long long wait_ns;
    int withhold;             // self-test: a Withheld
};
// kUp: X, Wg, Wu; H, G, U or the sums.  kBack: dG by rows, Wg, Wu, dG and X by columns; dX, dWg, dWu or sums.
struct Maps {
    CUtensorMap in[5];
    CUtensorMap out[3];
};

__device__ __forceinline__ float sigmoid(float x) {   // exact limits: 1 / (1 + inf) = 0
    return __fdividef(1.f, 1.f + exp2_fast(-x * kLog2e));
}

// The activation, and its slope.  (exp's limits give those of the sigmoid; a sigmoid below 2^-126 is 0.)
template <int Act>
__device__ __forceinline__ float act_of(float x) {
    if constexpr (Act == TB_ACT_SILU) return x * sigmoid(x);
    if constexpr (Act == TB_ACT_GELU) return x * normcdff(x);
    const float t = 1.5957691216057308f * x * __fmaf_rn(0.044715f, x * x, 1.f);     // 2 sqrt(2 / pi)
    return x * sigmoid(t);                            // (1 + tanh(t / 2)) / 2 = sigmoid(t)
}
template <int Act>
__device__ __forceinline__ void act_and_slope(float x, float& a, float& slope) {
    if constexpr (Act == TB_ACT_SILU) {
        const float s = sigmoid(x);
        a = x * s;
        slope = s * __fmaf_rn(x, 1.f - s, 1.f);
    } else if constexpr (Act == TB_ACT_GELU) {
        const float c = normcdff(x);
        a = x * c;
        slope = __fmaf_rn(x, 0.3989422804014327f * exp2_fast(-0.5f * kLog2e * x * x), c);
    } else {
        // from 16 on either side the sigmoid is 0 or 1 and the slope with it; x's cube would leave fp32 long before bf16 ends
        const float y = fabsf(x) > 16.f ? copysignf(16.f, x) : x, y2 = y * y;
        const float s = sigmoid(1.5957691216057308f * y * __fmaf_rn(0.044715f, y2, 1.f));
        a = x * s;
        slope = s * __fmaf_rn(1.5957691216057308f * y * (1.f - s), __fmaf_rn(3 * 0.044715f, y2, 1.f), 1.f);
    }
}

// ---------------------------------------------------------------- tiles
struct Where {
    int part, split, mt, nt;
};
__device__ __forceinline__ Where tile_at(const Tiles& g, int part, unsigned t) {
    Where w{part, 0, 0, 0};
    const unsigned per_split = (unsigned)(g.m * g.n);
    if (g.splits > 1) {
        w.split = (int)(t / per_split);
        t -= w.split * per_split;
    }
    unsigned first = 0;
    if (g.m > kGroup) {
        first = t / (unsigned)(kGroup * g.n);
        t -= first * kGroup * g.n;
        first *= kGroup;
    }
    const unsigned height = min(kGroup, g.m - (int)first);
    w.nt = (int)(t / height);
    w.mt = (int)(first + t - w.nt * height);
    return w;
}
// Tile number j of a pair; false behind its last one.
template <int K>
__device__ __forceinline__ bool pair_tile(const Args& p, int pair, int pairs, int j, Where* w) {
    if (K == kUp) {
        const int64_t t = pair + (int64_t)j * pairs;
        if (t >= p.part[0].count) return false;
        *w = tile_at(p.part[0], 0, (unsigned)t);
        return true;
    }
    const int mine = p.part[0].count / pairs + (pair < p.part[0].count % pairs);
    if (j < mine) {
        *w = tile_at(p.part[0], 0, (unsigned)(pair + j * pairs));
        return true;
    }
    j -= mine;
    // the shorter ones begin with the pairs that have a long one less
    const bool light = pair >= p.light;
    const int place = light ? pair - p.light : pair + pairs - p.light;
    int64_t t;
    if (light && j < p.extra) t = (int64_t)place * p.extra + j;
    else t = (int64_t)(pairs - p.light) * p.extra + place + (int64_t)(j - (light ? p.extra : 0)) * pairs;
    if (t >= p.part[1].count) return false;
    *w = tile_at(p.part[1], 1, (unsigned)t);
    return true;
}
__device__ __forceinline__ void stages_of(const Tiles& g, int split, int* lo, int* hi) {
    *lo = 0;
    *hi = g.stages;
    if (g.splits > 1) {           // (at most 256 splits of 2^24 / 64 stages: no overflow)
        *lo = (int)((unsigned)split * g.stages / (unsigned)g.splits);
        *hi = (int)((unsigned)(split + 1) * g.stages / (unsigned)g.splits);
    }
}
// Whether a tile is of dX or of dW.
__device__ __forceinline__ bool is_dw(const Args& p, int part) { return (p.first ^ part) != 0; }

// What one CTA stages of a pair's tiles, stage after stage.
template <int K>
struct Feed {
    const Args& p;
    const Maps& maps;
    int rank, pair, pairs, j;
    bool live, next_live;
    int k, k_hi, m0, n0, part;
    int nk, nk_hi, nm0, nn0, npart;      // of the next tile: worked out while the ring is full
    __device__ __forceinline__ Feed(const Args& p_, const Maps& m_, int rank_, int pair_, int pairs_)
        : p(p_), maps(m_), rank(rank_), pair(pair_), pairs(pairs_), j(0) {
        look(0);
        take();
    }
    __device__ __forceinline__ void look(int at) {
        Where w;
        next_live = pair_tile<K>(p, pair, pairs, at, &w);
        if (!next_live) return;
        stages_of(p.part[w.part], w.split, &nk, &nk_hi);
        npart = w.part;
        if (K == kUp) {
            nm0 = w.mt * kTile + rank * kHalf;
            nn0 = w.nt * p.half;
        } else {
            nn0 = w.nt * kTile + rank * kHalf;
            if (is_dw(p, w.part)) {       // the row tiles of dWg, those of dWu behind them
                const int each = p.part[w.part].m / 2, of_u = w.mt >= each;
                nm0 = of_u * p.half + (w.mt - of_u * each) * kTile + rank * kHalf;
            } else {
                nm0 = w.mt * kTile + rank * kHalf;
            }
        }
    }
    __device__ __forceinline__ void take() { live = next_live, k = nk, k_hi = nk_hi, m0 = nm0, n0 = nn0, part = npart; }
    __device__ __forceinline__ void next() {
        if (++k < k_hi) return;
        ++j;
        take();
    }
    __device__ __forceinline__ uint32_t bytes(int of_rank) const {
        const uint32_t a = (K == kBack && is_dw(p, part)) || p.a_rows == kHalf ? kHalf : of_rank ? 0 : p.a_rows;
        return (a + (K == kUp ? p.half : kHalf)) * kStageK * 2;
    }
    // Calls f(operand 0 or 1, byte offset in it, map, x, y) for the boxes of this stage.
    template <class F>
    __device__ __forceinline__ void boxes(F f) const {
        if constexpr (K == kUp) {
            if (p.a_rows == kHalf || rank == 0) f(0, 0, &maps.in[0], k * kStageK, m0);
            f(1, 0, &maps.in[1 + rank], k * kStageK, n0);     // one CTA stages Wg, the other Wu
        } else if (is_dw(p, part)) {
            f(0, 0, &maps.in[3], m0, k * kStageK);
            f(0, 8192, &maps.in[3], m0 + 64, k * kStageK);
            f(1, 0, &maps.in[4], n0, k * kStageK);
            f(1, 8192, &maps.in[4], n0 + 64, k * kStageK);
        } else {
            if (p.a_rows == kHalf || rank == 0) f(0, 0, &maps.in[0], k * kStageK, m0);
            const int of_u = k * kStageK >= p.half, y = k * kStageK - of_u * p.half;
            f(1, 0, &maps.in[1 + of_u], n0, y);
            f(1, 8192, &maps.in[1 + of_u], n0 + 64, y);
        }
    }
};

// 32 columns of a row to memory in 16-byte vectors; `cols` of them exist (a multiple of 8).
template <class Fmt>
__device__ __forceinline__ void put_vectors(typename Fmt::T* out, const float (&v)[32], int cols) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (8 * i >= cols) break;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = v[8 * i + e];
        *reinterpret_cast<uint4*>(out + 8 * i) = pack8<Fmt>(f);
    }
}

// ---------------------------------------------------------------- the product
template <class Fmt, int K, int Epi, int Act>
__global__ void __launch_bounds__(kThreadsOf(Epi), 1)
gated_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args p) {
    using T = typename Fmt::T;
    constexpr int kParts = Epi / 4;         // of a tile's columns
    extern __shared__ unsigned char raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    unsigned char* outbox = smem + kStages * kStageBytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(outbox + kOutboxes * kOutBytes);
    const uint32_t stage0 = smem_addr(smem), bar0 = smem_addr(bars);
    const uint32_t full = bar0, empty = full + 8 * kStages, acc_full = empty + 8 * kStages,
                   acc_empty = acc_full + 16, drain = acc_empty + 16, done = drain + 8, issued = done + 8,
                   slot = issued + 4;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1 + (p.withhold == kFull));
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

    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (warp == 0) {
        const uint32_t leader_full = map_to(full, 0);
        int it = 0;
        Feed<K> feed(p, maps, (int)rank, pair, pairs);
        if (p.withhold == kBoxes0 + (int)rank) feed.live = false;
        for (; feed.live; feed.next(), ++it) {
            const int s = it % kStages;
            if (it >= kStages && !__all_sync(0xffffffffu, mbar_wait(empty + 8 * s, (it / kStages - 1) & 1, &p)))
                break;
            const uint32_t at = stage0 + s * kStageBytes, bar = leader_full + 8 * s;
            if (elect_one()) {
                if (rank == 0) mbar_expect(full + 8 * s, feed.bytes(0) + feed.bytes(1));
                feed.boxes([&](int operand, int offset, const CUtensorMap* m, int x, int y) {
                    tma_box(at + operand * kOperandBytes + offset, m, x, y, bar);
                });
            }
            if (feed.k + 1 == feed.k_hi) feed.look(feed.j + 1);
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
            if (it != peer) {
                // the stages that one of them lacks, walked again for their bytes
                Feed<K> again(p, maps, 0, pair, pairs);
                for (int q = 0; again.live && q < max(it, peer); ++q) {
                    if (q >= min(it, peer) && elect_one()) {
                        const uint32_t bar = full + 8 * (q % kStages), bytes1 = again.bytes(1);
                        if (q < it)
                            asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar),
                                         "r"(bytes1)
                                         : "memory");
                        else mbar_expect(bar, bytes1);
                    }
                    __syncwarp();
                    if (again.k + 1 == again.k_hi) again.look(again.j + 1);
                    again.next();
                }
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
            const uint32_t width = K == kUp ? 2 * p.half : kTile;
            const uint32_t base = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(K == kBack) << 16) |
                                  ((width / 8) << 17) | ((kTile / 16) << 24);
            // 16 contracted elements: 32 bytes of a K-major row, 16 rows of an MN-major box
            constexpr uint32_t step_b = (K == kBack ? 2048 : 32) >> 4;
            const uint32_t b0 = desc_low<K == kBack>(stage0 + kOperandBytes);
            uint32_t s = 0, parity = 0;
            int n = 0;
            bool ok = true;
            Where w;
            for (int j = 0; ok && pair_tile<K>(p, pair, pairs, j, &w); ++j, ++n) {
                int k, k_hi;
                stages_of(p.part[w.part], w.split, &k, &k_hi);
                const bool a_mn = K == kBack && is_dw(p, w.part);
                const uint32_t idesc = base | ((uint32_t)a_mn << 15), step_a = a_mn ? 2048u >> 4 : 32u >> 4,
                               a0 = a_mn ? desc_low<true>(stage0) : desc_low<false>(stage0);
                const int buf = n & 1;
                if (n >= 2 && !__all_sync(0xffffffffu, mbar_wait<kRelaxed>(acc_empty + 8 * buf, (n / 2 - 1) & 1, &p))) {
                    ok = false;
                    break;
                }
                tmem_fence_after();
                const uint32_t d = tmem + buf * kTile;
                uint32_t accumulate = 0;
                for (; k < k_hi; ++k) {
                    if (!__all_sync(0xffffffffu, mbar_wait(full + 8 * s, parity, &p))) {
                        ok = false;
                        break;
                    }
                    const uint32_t a = a0 + s * (kStageBytes >> 4), b = b0 + s * (kStageBytes >> 4);
                    if (elect_one()) {
                        mma_pair<false>(d, a, b, idesc, accumulate);
#pragma unroll
                        for (int i = 1; i < kStageK / 16; ++i)
                            mma_pair<true>(d, a + i * step_a, b + i * step_b, idesc, 1);
                        mma_commit(empty + 8 * s);
                    }
                    accumulate = 1;
                    if (++s == kStages) s = 0, parity ^= 1;
                }
                if (ok && elect_one()) mma_commit(acc_full + 8 * buf);
            }
            if (elect_one()) mma_commit(drain);
        }
    } else if (warp >= kEpiWarp) {
        // TMEM lanes 32 quad .. 32 quad + 31 (a warp reaches those of its number modulo 4), and
        // one of the parts of the tile's columns
        const int quad = warp & 3, part_no = (warp - kEpiWarp) >> 2;
        const uint32_t leader_empty = map_to(acc_empty, 0);
        Outbox<Fmt, kOutboxes / Epi> box{outbox + (warp - kEpiWarp) * (kOutboxes / Epi) * kOutBytes, &maps.out[0], lane, 0};
        float unscale = 1.f;
        if constexpr (K == kBack && std::is_same<Fmt, F16>::value) unscale = *p.unscale;
        int n = 0;
        bool sums_before = false;
        Where w;
        for (; pair_tile<K>(p, pair, pairs, n, &w); ++n) {
            const int buf = n & 1;
            const uint32_t acc = tmem + buf * kTile + ((uint32_t)(quad * 32) << 16);
            int row0 = w.mt * kTile + (int)rank * kHalf + quad * 32, rows = p.rows, which = 0, z = w.split;
            int n0, all;
            if constexpr (K == kUp) {
                n0 = w.nt * p.half;
                all = min(p.half, p.inner - n0);
            } else {
                n0 = w.nt * kTile;
                all = min(kTile, p.hidden - n0);
                if (is_dw(p, w.part)) {
                    const int each = p.part[w.part].m / 2, of_u = w.mt >= each;
                    row0 -= of_u * each * kTile;
                    rows = p.inner;
                    which = 1 + of_u;
                    z = 2 * w.split + of_u;
                }
            }
            const bool sums = K == kUp ? p.sums : (p.sums >> (which != 0)) & 1;
            const int share = (all + 32 * kParts - 1) / (32 * kParts) * 32;
            const int c0 = part_no * share, width = min(all, c0 + share);
            const int row = row0 + lane;
            if (!__all_sync(0xffffffffu, mbar_wait<kRelaxed>(acc_full + 8 * buf, (n / 2) & 1, &p))) break;
            tmem_fence_after();
            auto release = [&] {
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(leader_empty + 8 * buf);
            };
            __syncwarp();
            if (c0 >= width || row0 >= rows) {         // nothing of this warp's
                release();
                continue;
            }
            if constexpr (K == kUp) {
                for (int c = c0; c < width; c += 32) {
                    uint32_t g[32], u[32];
                    tmem_load32(acc + c, g);
                    tmem_load32(acc + p.half + c, u);
                    tmem_wait(g);
                    tmem_wait(u);
                    if (c + 32 >= width) release();
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(g[i]);
                    if (sums) {
                        put_sums(box.mem, &maps.out[0], lane, v, n0 + c, row0, 2 * z, false);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(u[i]);
                        put_sums(box.mem, &maps.out[0], lane, v, n0 + c, row0, 2 * z + 1, false);
                        continue;
                    }
                    auto put = [&](int to, void* plain) {
                        if (p.out_map) {
                            box.map = &maps.out[to];
                            box.put(v, n0 + c, row0);
                        } else if (row < rows) {
                            put_vectors<Fmt>(static_cast<T*>(plain) + (int64_t)row * p.inner + n0 + c, v, width - c);
                        }
                    };
                    if (p.G) {
                        put(1, p.G);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(u[i]);
                        put(2, p.U);
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = act_of<Act>(__uint_as_float(g[i])) * __uint_as_float(u[i]);
                    put(0, p.H);
                }
            } else {
                box.map = &maps.out[which];
                // Sums fill both boxes and leave in one store; 16-bit results allow for one that still reads the other box.
                if (sums_before && !sums && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                sums_before = sums;
                auto work = [&](const uint32_t (&r)[32], int c) {
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
                    if (sums) {
                        put_sums(box.mem, &maps.out[which], lane, v, n0 + c, row0, z, false);
                    } else {
                        if constexpr (std::is_same<Fmt, F16>::value) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] *= unscale;
                        }
                        box.put(v, n0 + c, row0);
                    }
                };
                // the next columns come while the present ones are worked on
                uint32_t one[32], two[32];
                tmem_load32(acc + c0, one);
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
constexpr int kThreads = 256;

// dG and dU, eight elements a thread.  Top: only the largest finite magnitude among them, for the power of
// two that fp16 holds them times.
struct Gate {
    const void *dH, *G, *U;
    void* out;                // [rows][2][half], zeros behind a row's `inner`
    float* unscale;           // fp16: written by the second pass
    unsigned* tops;           // fp16: magnitude as bits, of each CTA of the first pass
    int n_tops;
    int64_t rows;
    int inner, half;
};
// The power of two that brings a magnitude to 2^14 .. 2^15: no rounding, no overflow.
__device__ __forceinline__ int shift_for(unsigned top) {
    const int e = (int)(top >> 23);                   // 0: nothing, or all below fp32's normal numbers
    return e == 0 ? 0 : min(max(14 + 127 - e, -100), 100);
}
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((127 + e) << 23); }

template <class Fmt, int Act, bool Top>
__global__ void __launch_bounds__(kThreads) gate_kernel(const __grid_constant__ Gate p) {
    pdl_wait();
    pdl_trigger();
    const unsigned per_row = (unsigned)(Top ? p.inner : p.half) / 8;
    const int64_t vectors = p.rows * per_row, step = (int64_t)gridDim.x * kThreads;
    float scale = 1.f;
    if constexpr (!Top && std::is_same<Fmt, F16>::value) {
        __shared__ unsigned most_of[kThreads / 32];
        unsigned m = 0;
        for (int i = threadIdx.x; i < p.n_tops; i += kThreads) m = max(m, p.tops[i]);
        m = __reduce_max_sync(0xffffffffu, m);
        if (threadIdx.x % 32 == 0) most_of[threadIdx.x / 32] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) m = max(m, most_of[i]);
        const int e = shift_for(m);
        scale = power_of_two(e);
        if (blockIdx.x == 0 && threadIdx.x == 0) *p.unscale = power_of_two(-e);
    }
    unsigned most = 0;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < vectors; i += step) {
        const int64_t row = i / per_row;
        const unsigned col = (unsigned)(i - row * per_row) * 8;
        float dg[8], du[8];
        if (col < (unsigned)p.inner) {
            const int64_t at = (row * p.inner + col) * 2;
            float dh[8], g[8], u[8];
            unpack8<Fmt>(ld_stream_u4(static_cast<const char*>(p.dH) + at), dh);
            unpack8<Fmt>(ld_stream_u4(static_cast<const char*>(p.G) + at), g);
            unpack8<Fmt>(ld_stream_u4(static_cast<const char*>(p.U) + at), u);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float a, slope;
                act_and_slope<Act>(g[e], a, slope);
                dg[e] = dh[e] * u[e] * slope;
                du[e] = dh[e] * a;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) dg[e] = du[e] = 0.f;
        }
        if constexpr (Top) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const unsigned x = __float_as_uint(dg[e]) & 0x7fffffffu, y = __float_as_uint(du[e]) & 0x7fffffffu;
                if (x < 0x7f800000u) most = max(most, x);
                if (y < 0x7f800000u) most = max(most, y);
            }
        } else {
            if constexpr (std::is_same<Fmt, F16>::value) {
#pragma unroll
                for (int e = 0; e < 8; ++e) dg[e] *= scale, du[e] *= scale;
            }
            typename Fmt::T* out = static_cast<typename Fmt::T*>(p.out) + row * 2 * p.half + col;
            *reinterpret_cast<uint4*>(out) = pack8<Fmt>(dg);
            *reinterpret_cast<uint4*>(out + p.half) = pack8<Fmt>(du);
        }
    }
    if constexpr (Top) {
        __shared__ unsigned most_of[kThreads / 32];
        most = __reduce_max_sync(0xffffffffu, most);
        if (threadIdx.x % 32 == 0) most_of[threadIdx.x / 32] = most;
        __syncthreads();
        if (threadIdx.x == 0) {
#pragma unroll
            for (int i = 1; i < kThreads / 32; ++i) most = max(most, most_of[i]);
            p.tops[blockIdx.x] = most;
        }
    }
}

// The splits of G and U added, in their order, and what becomes of them; four elements a thread.
template <class Fmt, int Act>
__global__ void __launch_bounds__(kThreads)
join_up_kernel(const float* sums, int splits, int64_t n, typename Fmt::T* H, typename Fmt::T* G, typename Fmt::T* U) {
    pdl_wait();
    pdl_trigger();
    const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4;
    if (i >= n) return;
    float4 g = make_float4(0.f, 0.f, 0.f, 0.f), u = g;
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
        const float4 x = *reinterpret_cast<const float4*>(sums + 2 * s * n + i);
        const float4 y = *reinterpret_cast<const float4*>(sums + (2 * s + 1) * n + i);
        g.x += x.x, g.y += x.y, g.z += x.z, g.w += x.w;
        u.x += y.x, u.y += y.y, u.z += y.z, u.w += y.w;
    }
    auto store = [&](typename Fmt::T* to, float a, float b, float c, float d) {
        typename Fmt::T r[4] = {Fmt::from_f32(a), Fmt::from_f32(b), Fmt::from_f32(c), Fmt::from_f32(d)};
        *reinterpret_cast<uint2*>(to + i) = *reinterpret_cast<const uint2*>(r);
    };
    store(H, act_of<Act>(g.x) * u.x, act_of<Act>(g.y) * u.y, act_of<Act>(g.z) * u.z, act_of<Act>(g.w) * u.w);
    if (G) {
        store(G, g.x, g.y, g.z, g.w);
        store(U, u.x, u.y, u.z, u.w);
    }
}

// The same for dX, dWg and dWu: four elements a thread of one of them.
struct JoinBack {
    const float* sums[3];
    void* out[3];
    int64_t n[3], stride[3];  // elements (0: not split), and from one split to the next
    int splits[3];
    const float* unscale;
};
template <class Fmt>
__global__ void __launch_bounds__(kThreads) join_back_kernel(const __grid_constant__ JoinBack p) {
    pdl_wait();
    pdl_trigger();
    int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4;
    int which = 0;
    while (which < 3 && i >= p.n[which]) i -= p.n[which++];
    if (which == 3) return;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < p.splits[which]; ++s) {
        const float4 x = *reinterpret_cast<const float4*>(p.sums[which] + s * p.stride[which] + i);
        v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
    }
    float f = 1.f;
    if constexpr (std::is_same<Fmt, F16>::value) f = *p.unscale;
    typename Fmt::T r[4] = {Fmt::from_f32(v.x * f), Fmt::from_f32(v.y * f), Fmt::from_f32(v.z * f), Fmt::from_f32(v.w * f)};
    *reinterpret_cast<uint2*>(static_cast<typename Fmt::T*>(p.out[which]) + i) = *reinterpret_cast<const uint2*>(r);
}

// ---------------------------------------------------------------- host
// Contracted elements that one accumulator takes, at most: tensor cores cut off what an addition shifts
// below the sum's last place, 1e-9 of a sum of one sign for every element, 6e-5 at this many.
constexpr int64_t kChain = 65536;

// How a call of these sizes is cut up.
struct Cut {
    int half, splits;         // kUp: columns of a tile of G, parts of the contraction
    int64_t inner;            // kBack: F rounded up to whole stages
    int splits_x, splits_w, gate_ctas;
    size_t off_sums, off_dg, off_sums_x, off_sums_w, off_scale, total;
};

int64_t stages_for(int64_t contracted) { return ceil_div(contracted, kStageK); }

// The columns of a tile and the parts of the contraction, in units of a stage of 128 columns of both weights
// (about 0.28 us): waves of tiles, about eight units for each one's start and epilogue, and for the
// sums that parts leave a launch and their bytes.
void pick_up(int64_t n, int64_t d, int64_t f, int64_t pairs, Cut* c) {
    const int64_t m_tiles = ceil_div(n, kTile), stages = stages_for(d), fewest = ceil_div(stages, kChain / kStageK);
    double least = 1e30;
    for (int half = kHalf; half >= 32; half -= 16) {
        const bool whole = half % 32 == 0;            // of boxes that results go out in
        if (!whole && n >= kHalf) continue;
        const int64_t tiles = m_tiles * ceil_div(f, half);
        const double stage = std::max(0.4, half / 128.0);
        for (int64_t s = fewest; s <= std::max(fewest, std::min<int64_t>(stages, 64)); ++s) {
            if (s > 1 && (!whole || (s > fewest && tiles * s > 2 * pairs))) break;
            const double cost = (double)ceil_div(tiles * s, pairs) * ((double)ceil_div(stages, s) * stage + 8.0) +
                                (s > 1 ? 12.0 + (double)s * (0.05 + (double)(n * f) / 100000.0) : 0.0);
            if (cost < least * 0.97) least = cost, c->half = half, c->splits = (int)s;
        }
    }
}

// Two products' tiles dealt to the pairs: the longer ones round robin, then the shorter, of which the pairs
// with one long tile less first get as many as fill the gap, and then the first of the others.
struct Deal {
    int light, extra;
    double cost;
};
Deal deal(int64_t long_tiles, double long_cost, int64_t short_tiles, double short_cost, int64_t pairs) {
    Deal r{0, 0, 0.0};
    const int64_t heavy = long_tiles % pairs, light = pairs - heavy, base = long_tiles / pairs;
    int64_t extra = 0;
    if (heavy && short_tiles) extra = std::min((int64_t)(long_cost / short_cost + 0.5), short_tiles / light);
    const int64_t rest = short_tiles - extra * light, each = rest / pairs, over = rest % pairs;
    r.light = (int)heavy, r.extra = (int)extra;
    r.cost = std::max((double)base * long_cost + (double)(extra + each + (over > 0)) * short_cost,
                      heavy ? (double)(base + 1) * long_cost + (double)(each + (over > light)) * short_cost : 0.0);
    return r;
}

int64_t dx_tiles(int64_t n, int64_t d) { return ceil_div(n, kTile) * ceil_div(d, kTile); }
int64_t dw_tiles(int64_t f, int64_t d) { return 2 * ceil_div(f, kTile) * ceil_div(d, kTile); }

void pick_back(int64_t n, int64_t d, int64_t f, int64_t pairs, bool dx, bool dw, Cut* c) {
    const int64_t sx = stages_for(2 * c->inner), sw = stages_for(n);
    const int64_t fx = ceil_div(sx, kChain / kStageK), fw = ceil_div(sw, kChain / kStageK);
    const int64_t tx = dx ? dx_tiles(n, d) : 0, tw = dw ? dw_tiles(f, d) : 0;
    c->splits_x = (int)fx, c->splits_w = (int)fw;
    double least = 1e30;
    constexpr int kTry[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32, 48, 64};
    for (const int a0 : kTry) {
        const int64_t a = std::max<int64_t>(a0, fx);
        if (a0 > 1 && (a > sx || !tx || tx * a > 3 * pairs)) break;
        for (const int b0 : kTry) {
            const int64_t b = std::max<int64_t>(b0, fw);
            if (b0 > 1 && (b > sw || !tw || tw * b > 3 * pairs)) break;
            const double lx = (double)ceil_div(sx, a) + 8.0, lw = (double)ceil_div(sw, b) + 8.0;
            double cost = lx >= lw ? deal(tx * a, lx, tw * b, lw, pairs).cost : deal(tw * b, lw, tx * a, lx, pairs).cost;
            if (a > 1 || b > 1) cost += 12.0;
            if (tx && a > 1) cost += (double)a * (0.05 + (double)(n * d) / 450000.0);
            if (tw && b > 1) cost += (double)b * (0.05 + (double)(2 * f * d) / 450000.0);
            if (cost < least * 0.97) least = cost, c->splits_x = (int)a, c->splits_w = (int)b;
        }
    }
}

Cut cut_call(int64_t n, int64_t d, int64_t f, bool back, int sms) {
    Cut c{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    if (!back) {
        pick_up(n, d, f, sms / 2, &c);
        if (c.splits > 1) c.off_sums = take((size_t)c.splits * 2 * n * f * sizeof(float));
    } else {
        c.inner = round_up(f, kStageK);
        pick_back(n, d, f, sms / 2, true, true, &c);
        c.off_dg = take((size_t)n * 2 * c.inner * 2);
        if (c.splits_x > 1) c.off_sums_x = take((size_t)c.splits_x * n * d * sizeof(float));
        if (c.splits_w > 1) c.off_sums_w = take((size_t)c.splits_w * 2 * f * d * sizeof(float));
        c.gate_ctas = (int)std::min<int64_t>(ceil_div(n * c.inner / 8, kThreads), 8ll * sms);
        c.off_scale = take((1 + (size_t)c.gate_ctas) * sizeof(float));
    }
    c.total = at;
    return c;
}

// Rows of a box of K-major A.  A result of at most kHalf rows lies in the pair's first CTA alone: its
// boxes hold those rows and the second CTA loads none.  What the MMAs read in their place is what the
// memory held; it reaches only rows that nothing stores.
int box_rows(int64_t rows) { return rows < kHalf ? (int)round_up(rows, 8) : kHalf; }

constexpr int64_t kMaxSize = 1ll << 24;

tb_status check_sizes(int64_t n, int64_t d, int64_t f, tb_dtype dtype) {
    if (n < 0 || d < 8 || f < 8 || d % 8 || f % 8 || n > kMaxSize || d > kMaxSize || f > kMaxSize) return TB_ERR_INVALID_VALUE;
    if (n * d > (1ll << 38) || f * d > (1ll << 38) || n * f > (1ll << 38)) return TB_ERR_INVALID_VALUE;
    if (dtype != TB_BF16 && dtype != TB_F16) return TB_ERR_UNSUPPORTED_DTYPE;
    return TB_OK;
}

tb_status workspace(int64_t n, int64_t d, int64_t f, tb_dtype dtype, bool back, size_t* bytes) {
    if (!bytes) return TB_ERR_INVALID_VALUE;
    const tb_status st = check_sizes(n, d, f, dtype);
    if (st != TB_OK) return st;
    *bytes = 0;
    if (n == 0) return TB_OK;
    int dev = 0;
    DeviceInfo info{};
    if (!current_device_info(&dev, &info)) return TB_ERR_CUDA;
    *bytes = cut_call(n, d, f, back, info.sm_count).total;
    return TB_OK;
}

struct Problem {
    const void *X, *Wg, *Wu, *dH;
    void *H, *G, *U;          // the gradient reads G and U
    void *dX, *dWg, *dWu;
    int64_t n, d, f;
    unsigned char* ws;
    int sms;
    int* err;
    cudaStream_t st;
};

template <class Fmt, int K, int Act, int Epi = 8>
tb_status launch_product(const Maps& m, Args p, int64_t tiles, cudaStream_t st, int most_pairs = 1 << 20) {
    if (!p.wait_ns) p.wait_ns = kWaitLimitNs;
    const void* kernel = reinterpret_cast<const void*>(&gated_kernel<Fmt, K, Epi, Act>);
    const int pairs = std::min(most_pairs, resident_clusters(kernel, kThreadsOf(Epi), kSmem, 2));
    if (pairs < 1) return TB_ERR_CUDA;
    const int64_t grid = std::min<int64_t>(tiles, pairs);
    if (K == kBack) {
        const Tiles &a = p.part[0], &b = p.part[1];
        const double la = (double)ceil_div(a.stages, std::max(1, a.splits)) + 8.0,
                     lb = (double)ceil_div(b.stages, std::max(1, b.splits)) + 8.0;
        const Deal r = deal(a.count, la, b.count, lb, grid);
        p.light = r.light, p.extra = r.extra;
    }
    if (launch_clusters<true>(gated_kernel<Fmt, K, Epi, Act>, dim3((unsigned)(2 * grid)), dim3(kThreadsOf(Epi)), kSmem, st, 2, m,
                              p) != cudaSuccess)
        return TB_ERR_CUDA;
    return launch_status();
}

// fp32 sums [z][rows][cols], written in boxes of 32 x 32.
bool sums_map(CUtensorMap* m, void* p, int64_t z, int64_t rows, int64_t cols) {
    return make_sums_map(m, static_cast<float*>(p), z, rows, cols);
}

template <class Fmt, int Act>
tb_status run_up(const Problem& q, const Cut& c) {
    constexpr bool bf = std::is_same<Fmt, BF16>::value;
    Maps m{};
    Args p{};
    p.rows = (int)q.n, p.hidden = (int)q.d, p.inner = (int)q.f;
    p.half = c.half;
    p.a_rows = box_rows(q.n);
    p.out_map = c.half % 32 == 0;
    p.sums = c.splits > 1;
    p.H = q.H, p.G = q.G, p.U = q.U;
    p.err = q.err;
    Tiles& g = p.part[0];
    g.m = (int)ceil_div(q.n, kTile), g.n = (int)ceil_div(q.f, c.half), g.splits = c.splits, g.stages = (int)stages_for(q.d);
    g.count = g.m * g.n * g.splits;
    if (!make_map(&m.in[0], q.X, q.n, q.d, q.d, p.a_rows, bf) || !make_map(&m.in[1], q.Wg, q.f, q.d, q.d, c.half, bf) ||
        !make_map(&m.in[2], q.Wu, q.f, q.d, q.d, c.half, bf))
        return TB_ERR_CUDA;
    float* sums = reinterpret_cast<float*>(q.ws + c.off_sums);
    if (p.sums) {
        if (!sums_map(&m.out[0], sums, 2 * c.splits, q.n, q.f)) return TB_ERR_CUDA;
    } else if (!make_map(&m.out[0], q.H, q.n, q.f, q.f, 32, bf, true) ||
               (q.G && (!make_map(&m.out[1], q.G, q.n, q.f, q.f, 32, bf, true) ||
                        !make_map(&m.out[2], q.U, q.n, q.f, q.f, 32, bf, true)))) {
        return TB_ERR_CUDA;
    }
    const tb_status s = launch_product<Fmt, kUp, Act>(m, p, g.count, q.st);
    if (s != TB_OK || !p.sums) return s;
    using T = typename Fmt::T;
    const int64_t n = q.n * q.f;
    return launch_pdl(join_up_kernel<Fmt, Act>, dim3((unsigned)ceil_div(n, 4 * kThreads)), dim3(kThreads), 0, q.st, sums,
                      c.splits, n, static_cast<T*>(q.H), static_cast<T*>(q.G), static_cast<T*>(q.U)) == cudaSuccess
               ? launch_status()
               : TB_ERR_CUDA;
}

template <class Fmt, int Act>
tb_status run_back(const Problem& q, const Cut& c) {
    constexpr bool bf = std::is_same<Fmt, BF16>::value;
    void* dg = q.ws + c.off_dg;
    float* scale = reinterpret_cast<float*>(q.ws + c.off_scale);
    Gate e{};
    e.dH = q.dH, e.G = q.G, e.U = q.U, e.out = dg;
    e.unscale = scale, e.tops = reinterpret_cast<unsigned*>(scale + 1), e.n_tops = c.gate_ctas;
    e.rows = q.n, e.inner = (int)q.f, e.half = (int)c.inner;
    const int ctas = c.gate_ctas;
    if (!bf && launch_pdl(gate_kernel<Fmt, Act, true>, dim3((unsigned)ctas), dim3(kThreads), 0, q.st, e) != cudaSuccess)
        return TB_ERR_CUDA;
    if (launch_pdl(gate_kernel<Fmt, Act, false>, dim3((unsigned)ctas), dim3(kThreads), 0, q.st, e) != cudaSuccess)
        return TB_ERR_CUDA;

    Maps m{};
    Args p{};
    p.rows = (int)q.n, p.hidden = (int)q.d, p.inner = (int)q.f;
    p.half = (int)c.inner;
    p.a_rows = box_rows(q.n);
    p.unscale = scale;
    p.err = q.err;
    Tiles x{}, w{};
    if (q.dX) {
        x.m = (int)ceil_div(q.n, kTile), x.n = (int)ceil_div(q.d, kTile);
        x.splits = c.splits_x, x.stages = (int)stages_for(2 * c.inner);
        x.count = x.m * x.n * x.splits;
    }
    if (q.dWg) {
        w.m = 2 * (int)ceil_div(q.f, kTile), w.n = (int)ceil_div(q.d, kTile);
        w.splits = c.splits_w, w.stages = (int)stages_for(q.n);
        w.count = w.m * w.n * w.splits;
    }
    p.first = !q.dX || (q.dWg && ceil_div(w.stages, w.splits) > ceil_div(x.stages, x.splits));
    p.part[0] = p.first ? w : x;
    p.part[1] = p.first ? x : w;
    p.sums = (q.dX && x.splits > 1) | (q.dWg && w.splits > 1) << 1;
    float *sums_x = reinterpret_cast<float*>(q.ws + c.off_sums_x), *sums_w = reinterpret_cast<float*>(q.ws + c.off_sums_w);
    if (!make_map(&m.in[0], dg, q.n, 2 * c.inner, 2 * c.inner, p.a_rows, bf) ||
        !make_map(&m.in[1], q.Wg, q.f, q.d, q.d, kStageK, bf) || !make_map(&m.in[2], q.Wu, q.f, q.d, q.d, kStageK, bf) ||
        !make_map(&m.in[3], dg, q.n, 2 * c.inner, 2 * c.inner, kStageK, bf) || !make_map(&m.in[4], q.X, q.n, q.d, q.d, kStageK, bf))
        return TB_ERR_CUDA;
    if (q.dX && !(p.sums & 1 ? sums_map(&m.out[0], sums_x, c.splits_x, q.n, q.d)
                             : make_map(&m.out[0], q.dX, q.n, q.d, q.d, 32, bf, true)))
        return TB_ERR_CUDA;
    if (q.dWg) {
        if (p.sums & 2) {
            if (!sums_map(&m.out[1], sums_w, 2 * c.splits_w, q.f, q.d)) return TB_ERR_CUDA;
            m.out[2] = m.out[1];
        } else if (!make_map(&m.out[1], q.dWg, q.f, q.d, q.d, 32, bf, true) ||
                   !make_map(&m.out[2], q.dWu, q.f, q.d, q.d, 32, bf, true)) {
            return TB_ERR_CUDA;
        }
    }
    const tb_status s = launch_product<Fmt, kBack, 0>(m, p, (int64_t)x.count + w.count, q.st);
    if (s != TB_OK || !p.sums) return s;
    JoinBack j{};
    j.unscale = scale;
    if (p.sums & 1)
        j.sums[0] = sums_x, j.out[0] = q.dX, j.n[0] = j.stride[0] = q.n * q.d, j.splits[0] = c.splits_x;
    if (p.sums & 2)
        for (int i = 0; i < 2; ++i) {
            j.sums[1 + i] = sums_w + i * q.f * q.d, j.out[1 + i] = i ? q.dWu : q.dWg;
            j.n[1 + i] = q.f * q.d, j.stride[1 + i] = 2 * q.f * q.d, j.splits[1 + i] = c.splits_w;
        }
    const int64_t n = j.n[0] + j.n[1] + j.n[2];
    return launch_pdl(join_back_kernel<Fmt>, dim3((unsigned)ceil_div(n, 4 * kThreads)), dim3(kThreads), 0, q.st, j) == cudaSuccess
               ? launch_status()
               : TB_ERR_CUDA;
}

template <class Fmt>
tb_status run(const Problem& q, const Cut& c, tb_activation act, bool back) {
    switch (act) {
        case TB_ACT_SILU: return back ? run_back<Fmt, TB_ACT_SILU>(q, c) : run_up<Fmt, TB_ACT_SILU>(q, c);
        case TB_ACT_GELU: return back ? run_back<Fmt, TB_ACT_GELU>(q, c) : run_up<Fmt, TB_ACT_GELU>(q, c);
        default: return back ? run_back<Fmt, TB_ACT_GELU_TANH>(q, c) : run_up<Fmt, TB_ACT_GELU_TANH>(q, c);
    }
}

// Pointers of one call, those that are not given with no elements.
struct Buffers {
    Range in[6], out[3];
    int n_in, n_out;
};
tb_status check_buffers(const Buffers& b) {
    for (int i = 0; i < b.n_out; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(b.out[i], b.out[j])) return TB_ERR_ALIAS;
        for (int j = 0; j < b.n_in; ++j)
            if (overlap(b.out[i], b.in[j])) return TB_ERR_ALIAS;
    }
    return TB_OK;
}
tb_status check_workspace(const Buffers& b, const void* workspace, size_t have, size_t need) {
    if (need == 0) return TB_OK;
    if (!workspace || have < need) return TB_ERR_WORKSPACE;
    if (!aligned_to(workspace, 16)) return TB_ERR_MISALIGNED;
    const Range ws = range_of(workspace, (int64_t)need, 1);
    for (int i = 0; i < b.n_in; ++i)
        if (overlap(ws, b.in[i])) return TB_ERR_ALIAS;
    for (int i = 0; i < b.n_out; ++i)
        if (overlap(ws, b.out[i])) return TB_ERR_ALIAS;
    return TB_OK;
}

// One pair over 256 x 256 of X and 768 x 256 of both weights: more stages than the ring has, over six tiles.
tb_status run_withheld(int64_t wait_limit_ns, int* err, unsigned char* mem, cudaStream_t st, int* launches) {
    constexpr int64_t n = 256, d = 256, f = 768;
    auto take = [&](int64_t bytes) {
        unsigned char* at = mem;
        mem += bytes;
        return at;
    };
    const void *X = take(n * d * 2), *Wg = take(f * d * 2), *Wu = take(f * d * 2), *H = take(n * f * 2), *dg = take(n * 2 * f * 2),
               *dX = take(n * d * 2), *dWg = take(f * d * 2), *dWu = take(f * d * 2);
    for (int k = kUp; k <= kBack; ++k)
        for (int what = kBoxes0; what <= kEmpty; ++what) {
            Maps m{};
            Args p{};
            p.rows = (int)n, p.hidden = (int)d, p.inner = (int)f, p.a_rows = kHalf, p.out_map = 1;
            p.err = err, p.wait_ns = (unsigned long long)wait_limit_ns, p.withhold = what;
            int word = 0;
            if (cudaMemcpyAsync(err, &word, sizeof(int), cudaMemcpyHostToDevice, st) != cudaSuccess) return TB_ERR_CUDA;
            tb_status s;
            if (k == kUp) {
                p.half = kHalf;
                p.H = const_cast<void*>(H);
                p.part[0] = Tiles{1, (int)(f / kHalf), 1, (int)(d / kStageK), (int)(f / kHalf)};
                if (!make_map(&m.in[0], X, n, d, d, kHalf, true) || !make_map(&m.in[1], Wg, f, d, d, kHalf, true) ||
                    !make_map(&m.in[2], Wu, f, d, d, kHalf, true) || !make_map(&m.out[0], H, n, f, f, 32, true, true))
                    return TB_ERR_CUDA;
                s = launch_product<BF16, kUp, TB_ACT_SILU>(m, p, p.part[0].count, st, 1);
            } else {
                p.half = (int)f;
                p.part[0] = Tiles{1, 1, 1, (int)(2 * f / kStageK), 1};
                p.part[1] = Tiles{(int)(2 * f / kTile), 1, 1, (int)(n / kStageK), (int)(2 * f / kTile)};
                if (!make_map(&m.in[0], dg, n, 2 * f, 2 * f, kHalf, true) || !make_map(&m.in[1], Wg, f, d, d, kStageK, true) ||
                    !make_map(&m.in[2], Wu, f, d, d, kStageK, true) || !make_map(&m.in[3], dg, n, 2 * f, 2 * f, kStageK, true) ||
                    !make_map(&m.in[4], X, n, d, d, kStageK, true) || !make_map(&m.out[0], dX, n, d, d, 32, true, true) ||
                    !make_map(&m.out[1], dWg, f, d, d, 32, true, true) || !make_map(&m.out[2], dWu, f, d, d, 32, true, true))
                    return TB_ERR_CUDA;
                s = launch_product<BF16, kBack, 0>(m, p, p.part[0].count + p.part[1].count, st, 1);
            }
            if (s != TB_OK) return s;
            if (cudaMemcpyAsync(&word, err, sizeof(int), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
                cudaStreamSynchronize(st) != cudaSuccess)
                return TB_ERR_CUDA;
            *launches += word == (int)TB_ERR_TIMEOUT;
        }
    return TB_OK;
}

}  // namespace
}  // namespace tb

extern "C" tb_status tb_gated_linear_selftest_timeout(int64_t wait_limit_ns, int* launches, void* stream) {
    using namespace tb;
    if (!launches || wait_limit_ns < 1000 || wait_limit_ns > (int64_t)kWaitLimitNs) return TB_ERR_INVALID_VALUE;
    *launches = 0;
    int* err = device_error_word();
    if (!err) return TB_ERR_CUDA;
    constexpr size_t kBytes = 4 << 20;       // 2.9 MB are needed
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    void* mem = nullptr;
    if (cudaMalloc(&mem, kBytes) != cudaSuccess) {
        cudaGetLastError();
        return TB_ERR_OOM;
    }
    tb_status s = cudaMemsetAsync(mem, 0, kBytes, st) == cudaSuccess ? TB_OK : TB_ERR_CUDA;
    if (s == TB_OK) s = run_withheld(wait_limit_ns, err, static_cast<unsigned char*>(mem), st, launches);
    if (cudaStreamSynchronize(st) != cudaSuccess) s = TB_ERR_CUDA;
    if (cudaFree(mem) != cudaSuccess) s = TB_ERR_CUDA;
    return s;
}

extern "C" tb_status tb_gated_linear_workspace_size(int64_t rows, int64_t D, int64_t F, tb_dtype dtype, size_t* bytes) {
    return tb::workspace(rows, D, F, dtype, false, bytes);
}

extern "C" tb_status tb_gated_linear_bwd_workspace_size(int64_t rows, int64_t D, int64_t F, tb_dtype dtype, size_t* bytes) {
    return tb::workspace(rows, D, F, dtype, true, bytes);
}

extern "C" tb_status tb_gated_linear(const void* X, const void* Wg, const void* Wu, void* H, void* G, void* U, int64_t rows,
                                     int64_t D, int64_t F, tb_activation act, tb_dtype dtype, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    using namespace tb;
    tb_status s = check_sizes(rows, D, F, dtype);
    if (s != TB_OK) return s;
    if (act != TB_ACT_SILU && act != TB_ACT_GELU && act != TB_ACT_GELU_TANH) return TB_ERR_INVALID_VALUE;
    if (!G != !U) return TB_ERR_INVALID_VALUE;
    if (rows == 0) return TB_OK;
    if (!X || !Wg || !Wu || !H) return TB_ERR_INVALID_VALUE;
    for (const void* p : {X, Wg, Wu, (const void*)H, (const void*)G, (const void*)U})
        if (!aligned_to(p, 16)) return TB_ERR_MISALIGNED;
    const int64_t kept = G ? rows * F : 0;
    const Buffers b{{range_of(X, rows * D, 2), range_of(Wg, F * D, 2), range_of(Wu, F * D, 2)},
                    {range_of(H, rows * F, 2), range_of(G, kept, 2), range_of(U, kept, 2)}, 3, 3};
    if ((s = check_buffers(b)) != TB_OK) return s;
    int dev = 0;
    DeviceInfo info{};
    if (!current_device_info(&dev, &info)) return TB_ERR_CUDA;
    const Cut c = cut_call(rows, D, F, false, info.sm_count);
    if ((s = check_workspace(b, workspace, workspace_bytes, c.total)) != TB_OK) return s;
    Problem q{};
    q.X = X, q.Wg = Wg, q.Wu = Wu, q.H = H, q.G = G, q.U = U;
    q.n = rows, q.d = D, q.f = F;
    q.ws = static_cast<unsigned char*>(workspace);
    q.sms = info.sm_count, q.st = static_cast<cudaStream_t>(stream);
    if (!(q.err = device_error_word())) return TB_ERR_CUDA;
    return dtype == TB_BF16 ? run<BF16>(q, c, act, false) : run<F16>(q, c, act, false);
}

extern "C" tb_status tb_gated_linear_bwd(const void* dH, const void* X, const void* Wg, const void* Wu, const void* G,
                                         const void* U, void* dX, void* dWg, void* dWu, int64_t rows, int64_t D, int64_t F,
                                         tb_activation act, tb_dtype dtype, void* workspace, size_t workspace_bytes,
                                         void* stream) {
    using namespace tb;
    tb_status s = check_sizes(rows, D, F, dtype);
    if (s != TB_OK) return s;
    if (act != TB_ACT_SILU && act != TB_ACT_GELU && act != TB_ACT_GELU_TANH) return TB_ERR_INVALID_VALUE;
    if (!dWg != !dWu || (!dX && !dWg)) return TB_ERR_INVALID_VALUE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const Buffers b{{range_of(dH, rows * F, 2), range_of(X, rows * D, 2), range_of(Wg, F * D, 2), range_of(Wu, F * D, 2),
                     range_of(G, rows * F, 2), range_of(U, rows * F, 2)},
                    {range_of(dX, dX ? rows * D : 0, 2), range_of(dWg, dWg ? F * D : 0, 2), range_of(dWu, dWu ? F * D : 0, 2)},
                    6, 3};
    for (const void* p : {(const void*)dX, (const void*)dWg, (const void*)dWu})
        if (!aligned_to(p, 16)) return TB_ERR_MISALIGNED;
    if (rows == 0) {                     // no row: the weights' gradients are sums over nothing
        if ((s = check_buffers(b)) != TB_OK) return s;
        if (dWg && (cudaMemsetAsync(dWg, 0, (size_t)F * D * 2, st) != cudaSuccess ||
                    cudaMemsetAsync(dWu, 0, (size_t)F * D * 2, st) != cudaSuccess))
            return TB_ERR_CUDA;
        return TB_OK;
    }
    if (!dH || !X || !Wg || !Wu || !G || !U) return TB_ERR_INVALID_VALUE;
    for (const void* p : {dH, X, Wg, Wu, G, U})
        if (!aligned_to(p, 16)) return TB_ERR_MISALIGNED;
    if ((s = check_buffers(b)) != TB_OK) return s;
    int dev = 0;
    DeviceInfo info{};
    if (!current_device_info(&dev, &info)) return TB_ERR_CUDA;
    const Cut c = cut_call(rows, D, F, true, info.sm_count);
    if ((s = check_workspace(b, workspace, workspace_bytes, c.total)) != TB_OK) return s;
    Problem q{};
    q.dH = dH, q.X = X, q.Wg = Wg, q.Wu = Wu, q.G = const_cast<void*>(G), q.U = const_cast<void*>(U);
    q.dX = dX, q.dWg = dWg, q.dWu = dWu;
    q.n = rows, q.d = D, q.f = F;
    q.ws = static_cast<unsigned char*>(workspace);
    q.sms = info.sm_count, q.st = st;
    if (!(q.err = device_error_word())) return TB_ERR_CUDA;
    return dtype == TB_BF16 ? run<BF16>(q, c, act, true) : run<F16>(q, c, act, true);
}
