// attention.cu -- causal attention over whole prompts.
//
//     s_ij = scale q_i . k_j for j <= i,  lse_i = log sum_j exp(s_ij),  out_i = sum_j exp(s_ij - lse_i) v_j
//
// One pass over the keys: P = exp(s - m) is taken against a row's maximum of earlier blocks, sums and results are
// fp32, and where a row's sums show that the maximum has grown by much, results and sums are scaled to the new one.
// So P needs no maximum of its own block before it, and is at most kMost, far from fp16's end.
//
// A pair of CTAs (see attention.cuh) takes 512 queries of one head, two tiles of 128 in each CTA, and walks the blocks
// of 128 keys from the last one down.  Each CTA stages half of a block's keys (by rows) and half of its values' columns,
// 16 KB each, in a ring of eight.  Scores lie in tensor memory, P as 16-bit pairs over them, the results beside them:
// 512 columns at heads of 128.  Warp 0 loads, warp 1 of the first CTA issues the MMAs, warp 2 mends sequences' ends,
// warp 3 hands out work, four warps for each tile turn scores into P, a row a lane, and write the results.  While one tile's
// warps work the other's products run: P V of a block and the next scores, 1,024 clocks at heads of 128.
//
// What bounds it: the chain of one tile's block.  At heads of 128 its scores and P V take 1,024 clocks, handing over about
// 400, P 1,100 (512 of them powers, at 32 a clock and SM), so a pair's two tiles need 2,700 where their MMAs need 2,048;
// a piece of work adds the start of its first two blocks and its results, about 10,000.  bf16 4 x 4,096 tokens, 32 heads of
// 128: 407 to 414 us among others in a stream, under the power limit, 1,330 to 1,350 TFLOP/s, 72 % of cuBLAS's burst;
// 372 us, 1,480 TFLOP/s, in tens.
// One CTA with tiles of its own took 466 us there: operands crossed shared memory at its 128 bytes a clock.  Heads of 64
// are bound by P: fp16 16,384 tokens, 8 heads, 266 us, 1,030 TFLOP/s.  Two warps for the same rows instead of one: 449
// against 440 us; a row's maximum before P: the same; registers shared out by setmaxnreg (208 and 88): 641 us, as the
// compiler spills in both shares.
#include "attention.cuh"

namespace tb {
namespace {

constexpr int kItem = 2 * kSpan;             // queries of a pair: two tiles of each CTA share the pair's keys
constexpr int kSoftmaxWarp = 4;              // first of eight: four for each tile
constexpr int kThreads = (kSoftmaxWarp + 8) * 32;
// A block's sum of P, above which a row's maximum is looked for again: far from fp16's end.
constexpr float kMost = 8192.f;
// P is taken in one FMA from a score, 2^(s c - b), b = m c rounded to fp32 for a row's maximum m.  That rounding is a factor
// of all of the row's P, which its sum takes out again: at most 2^(2^-13) below kFar, where the largest P is still 1 in
// fp16, but from |b| = 2^28 on (keys masked by -1e10, say) it leaves P's range.  Beyond kFar m is taken off the scores first,
// exact for scores next to it, in a pass of its own that only warps with such a row make, behind the one for all: a branch
// within that one took 299 us for fp16 16,384 tokens, 8 heads of 64, this 266.
constexpr float kFar = 0x1p12f;

template <int Blocks>                        // of 64 columns of a head
struct Layout {
    static constexpr int kTileBytes = Blocks * kBox;             // of queries
    static constexpr int kKeyBytes = Blocks * kHalfBox;          // half a block's keys
    static constexpr int kValueBytes = kBox;                     // a block's values, half their columns
    static constexpr int kStageBytes = kBox, kRing = 8;
    static constexpr int kStage0 = 2 * kTileBytes;
    static constexpr int kOut = kStage0 + kRing * kStageBytes;
    static constexpr int kBars = kOut + 8 * kOutStage;
    static constexpr int kBytes = kBars + 1024 + 512;            // alignment, barriers
};

struct Args {
    Tokens tokens;
    int heads, group, dim;    // query heads, of which `group` share a key head
    int tiles;                // of kItem queries of a batch entry, without offsets
    float scale, scale_log2;  // and times log2(e)
    void* out;
    int64_t out_batch, out_seq, out_head;    // strides in elements
    float* lse;               // [batch][heads][seq]; NULL: not wanted
    int* err;
    unsigned long long wait_ns;
    int withhold;             // self-test: a Withheld
};

// What a pair works on: kItem queries of one head.  Tile t of CTA r begins 256 t + 128 r behind the first of them.
struct Item {
    Span span;
    int head;
    int blocks0, blocks1;     // of 128 keys that the pair's two tiles read; 0: no such tile
    __device__ __forceinline__ int blocks(int t) const { return t ? blocks1 : blocks0; }
};
__device__ __forceinline__ bool find_item(const Args& p, unsigned index, Item* it) {
    const unsigned heads = (unsigned)p.heads;
    it->head = (int)(index % heads);
    const unsigned slot = index / heads;
    if (p.tokens.offsets) {
        // (there are at least as many slots as sequences)
        if (it->head == 0 && threadIdx.x == 2 * 32 && slot < (unsigned)p.tokens.sequences)
            check_offsets(p.tokens.offsets, slot, p.tokens.seq, p.err);
        // (sorted, short items of few blocks would follow each other, whose latency nothing hides: 147 us, 136 so, of 8,192
        // tokens in 11 sequences, 32 heads of 128)
        if (!find_tile<false>(p.tokens, kItem, (int)slot, false, &it->span)) return false;
    } else {                  // the longest first, over all heads and batch entries
        const unsigned batch = (unsigned)p.tokens.batch;
        it->span = Span{(int)(slot % batch), 0, p.tokens.seq, p.tiles - 1 - (int)(slot / batch)};
    }
    const int all = (it->span.len + kRows - 1) / kRows, left = it->span.len - it->span.tile * kItem;
    it->blocks0 = min(4 * it->span.tile + 2, all);
    it->blocks1 = left > kSpan ? min(4 * it->span.tile + 4, all) : 0;
    return true;
}

// ---------------------------------------------------------------- the kernel
template <class Fmt, int Blocks>
__global__ void __launch_bounds__(kThreads, 1)
attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_out, const __grid_constant__ Args p) {
    using L = Layout<Blocks>;
    using T = typename Fmt::T;
    constexpr bool kBf = std::is_same<Fmt, BF16>::value;
    extern __shared__ unsigned char raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t q0 = smem_addr(smem), ring0 = q0 + L::kStage0, bar0 = q0 + L::kBars;
    const uint32_t answer = bar0, full = answer + 16, empty = full + 8 * L::kRing, q_full = empty + 8 * L::kRing, q_empty = q_full + 16,
                   s_full = q_empty + 16, p_full = s_full + 16, o_full = p_full + 16, o_empty = o_full + 16, tail = o_empty + 16, mended = tail + 8,
                   drain = mended + 8, done = drain + 8, work_full = done + 8, work_empty = work_full + 8, issued = work_empty + 8,
                   slot = issued + 12, stopped = slot + 4;
    static_assert(L::kRing * 16 + 6 * 16 + 6 * 8 + 16 + 20 <= 512);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();

    if (threadIdx.x == 0) {
        for (int i = 0; i < L::kRing; ++i) {
            mbar_init(full + 8 * i, 2);      // an arrival of either CTA, and their bytes
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + 8 * i, 2);
            mbar_init(q_empty + 8 * i, 1);
            mbar_init(s_full + 8 * i, 1 + (p.withhold == kScores));
            mbar_init(p_full + 8 * i, 8 + (p.withhold == kTaken));   // the warps of a tile, of both CTAs
            mbar_init(o_full + 8 * i, 1 + (p.withhold == kResults));
            mbar_init(o_empty + 8 * i, 8);
        }
        mbar_init(tail, 1);
        mbar_init(mended, 1);
        mbar_init(drain, 1);
        mbar_init(done, 1);
        *reinterpret_cast<volatile int*>(smem + (stopped - q0)) = 0;
        init_work(work_full, work_empty, 2 * (2 + 8) + 1);     // the warps that load and mend, those of the softmax, and the MMAs'
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) tmem_alloc_all(slot);
    tmem_fence_before();
    __syncthreads();
    cluster_sync();
    tmem_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + (slot - q0));
    pdl_wait();
    asm volatile("fence.proxy.async;" ::: "memory");   // what earlier kernels stored, TMA reads
    pdl_trigger();

    // The tensor memory: scores of both tiles (their first half becomes P), then results.
    const uint32_t score = tmem, result = tmem + 2 * kRows;
    const int cols = (p.dim + 15) / 16 * 16;
    // What each warp works on, and behind it: asked for when the present work is all under way.  (The answer waits for
    // the slowest warp to have read the one before.)
    Work work{answer, work_full, work_empty, 0};
    Item it, next;
    bool live = find_item(p, blockIdx.x >> 1, &it), next_live = false, more = true;
    auto ask = [&] {
        unsigned cluster;
        more = next_work(work, lane, &cluster, &p);
        next_live = more && find_item(p, cluster, &next);
    };
    auto move_on = [&] { it = next, live = next_live; };
    const Tails ends{tail, mended, stopped};

    if (warp == 0) {
        int n = 0, queries[2] = {0, 0}, tails = 0;       // keys and values staged, tiles of queries, ends
        uint32_t last = 0;                               // barrier of the last end
        bool ok = p.withhold != kLoads0 + (int)rank;
        for (; more; move_on()) {
            if (!ok || !live) {
                ask();
                continue;
            }
            const int blocks = max(it.blocks0, it.blocks1), kv_head = it.head / p.group;
            for (int t = 0; t < 2; ++t) {
                if (!it.blocks(t)) continue;
                if (queries[t] && !__all_sync(0xffffffffu, mbar_wait(q_empty + 8 * t, (queries[t] - 1) & 1, &p))) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    const uint32_t bar = map_to(q_full + 8 * t, 0);
                    mbar_expect_at(bar, L::kTileBytes);
                    for (int b = 0; b < Blocks; ++b)
                        tma_tile(q0 + t * L::kTileBytes + b * kBox, &map_q, 64 * b,
                                 it.span.first + it.span.tile * kItem + t * kSpan + (int)rank * kRows, it.head, it.span.batch, bar);
                }
                __syncwarp();
                ++queries[t];
            }
            // keys, values of the last block, then of the one before
            for (int i = 0; i < 2 * blocks && ok; ++i) {
                const int s = n % L::kRing, block = blocks - 1 - i / 2, row = it.span.first + block * kRows;
                if (n >= L::kRing && !__all_sync(0xffffffffu, mbar_wait(empty + 8 * s, (n / L::kRing - 1) & 1, &p))) {
                    ok = false;
                    break;
                }
                const int rows = it.span.len - block * kRows;
                const uint32_t at = ring0 + s * L::kStageBytes, leader = map_to(full + 8 * s, 0);
                if (i & 1) {
                    // Behind the sequence's end lie other tokens or nothing: P is 0 there, but 0 times what they
                    // hold need not be.
                    const bool mend = rows < kRows;
                    const uint32_t bar = mend ? map_to(tail, rank) : leader;
                    if (mend) {
                        if (!ends.next(tails, &p)) {
                            ok = false;
                            break;
                        }
                        ++tails;
                        last = leader;
                    }
                    if (elect_one()) {
                        mbar_expect_at(bar, L::kValueBytes);
                        tma_tile(at, &map_v, (int)rank * cols / 2, row, kv_head, it.span.batch, bar);
                    }
                    __syncwarp();
                } else if (elect_one()) {
                    mbar_expect_at(leader, L::kKeyBytes);
                    for (int b = 0; b < Blocks; ++b)
                        tma_tile(at + b * kHalfBox, &map_k, 64 * b, row + (int)rank * (kRows / 2), kv_head, it.span.batch, leader);
                }
                __syncwarp();
                ++n;
            }
            ask();
        }
        if (ends.left_over(tails, &p) && lane == 0) mbar_arrive_cluster(last);
        __syncwarp();
        const int mine[3] = {n, queries[0], queries[1]}, rings[3] = {L::kRing, 1, 1};
        way_out<3>(rank, mine, rings, drain, done, issued, smem + (issued - q0), &p, [&](int s, int i, uint32_t* parity) {
            if (s) {
                *parity = i & 1;
                return q_full + 8 * (s - 1);
            }
            *parity = (i / L::kRing) & 1;
            return full + 8 * (i % L::kRing);
        });
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t by_rows = instruction(kBf, kRows, false), by_cols = instruction(kBf, cols, true);
            int n = 0, have[2] = {0, 0}, uses[2] = {0, 0};       // tiles of the ring taken, P taken, items of a tile
            bool ok = true;
            auto wait_ring = [&](int i) { return __all_sync(0xffffffffu, mbar_wait(full + 8 * (i % L::kRing), (i / L::kRing) & 1, &p)); };
            for (; more; move_on()) {
                if (!ok || !live) {
                    ask();
                    continue;
                }
                const int blocks = max(it.blocks0, it.blocks1);
                // block i from the end is read by a tile when it is not behind the tile's last
                auto reads = [&](int t, int i) { return i < blocks && blocks - 1 - i < it.blocks(t); };
                auto scores = [&](int t, int place, bool last) {
                    if (elect_one()) {
                        product_by_rows<Blocks>(score + t * kRows, q0 + t * L::kTileBytes, ring0 + place * L::kStageBytes, cols / 16, by_rows);
                        mma_commit(s_full + 8 * t);
                        if (last) mma_commit(q_empty + 8 * t);
                    }
                    __syncwarp();
                };
                ok = wait_ring(n);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (!ok || !it.blocks(t)) continue;
                    ok = __all_sync(0xffffffffu, mbar_wait(q_full + 8 * t, uses[t] & 1, &p));
                    if (ok && reads(t, 0)) scores(t, n % L::kRing, blocks == 1);
                }
                if (ok && elect_one()) mma_commit(empty + 8 * (n % L::kRing));
                __syncwarp();
                for (int i = 0; i < blocks && ok; ++i) {
                    const int value = n + 1 + 2 * i, key = value + 1;
                    if (!wait_ring(value) || (i + 1 < blocks && !wait_ring(key))) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (ok && reads(t, i)) {
                            const bool first = i == 0 || !reads(t, i - 1);
                            ok = __all_sync(0xffffffffu, mbar_wait(p_full + 8 * t, have[t] & 1, &p)) &&
                                 (!first || !uses[t] || __all_sync(0xffffffffu, mbar_wait<kRelaxed>(o_empty + 8 * t, (uses[t] - 1) & 1, &p)));
                            if (!ok) break;
                            ++have[t];
                            tmem_fence_after();
                            if (elect_one()) {
                                product_over_tokens(result + t * kRows, score + t * kRows, kRows / 4,
                                                    ring0 + value % L::kRing * L::kStageBytes, by_cols, !first);
                                if (i + 1 == blocks) mma_commit(o_full + 8 * t);
                            }
                            __syncwarp();
                        }
                        if (ok && reads(t, i + 1)) scores(t, key % L::kRing, i + 2 == blocks);
                    }
                    if (!ok) break;
                    if (elect_one()) {
                        mma_commit(empty + 8 * (value % L::kRing));
                        if (i + 1 < blocks) mma_commit(empty + 8 * (key % L::kRing));
                    }
                    __syncwarp();
                }
                n += 2 * blocks;
                for (int t = 0; t < 2; ++t) uses[t] += it.blocks(t) != 0;
                ask();
            }
            if (elect_one()) mma_commit(drain);
        }
    } else if (warp == 2) {
        int n = 0, tails = 0;                // tiles of the ring, mended ones
        bool ok = true;
        for (; more; move_on()) {
            if (!ok || !live) {
                ask();
                continue;
            }
            const int blocks = max(it.blocks0, it.blocks1), rows = it.span.len - (blocks - 1) * kRows, s = (n + 1) % L::kRing;
            if (rows < kRows) {              // the first values end with the sequence
                if (!__all_sync(0xffffffffu, mbar_wait(tail, tails++ & 1, &p))) {
                    ends.stop(tails, lane);
                    ok = false;
                    ask();
                    continue;
                }
                clear_behind(smem + L::kStage0 + s * L::kStageBytes, 1, kRows, rows, lane);
                cleared(lane);
                if (lane == 0) {
                    mbar_arrive_cluster(map_to(full + 8 * s, 0));
                    mbar_arrive(mended);
                }
            }
            n += 2 * blocks;
            ask();
        }
    } else if (warp == 3) {
        hand_out(work, rank, &p);
    } else if (warp >= kSoftmaxWarp) {
        const int t = (warp - kSoftmaxWarp) >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t mine = score + t * kRows + lanes, sum = result + t * kRows + lanes;
        const uint32_t taken = map_to(p_full + 8 * t, 0), free = map_to(o_empty + 8 * t, 0);
        const unsigned long long c2 = pair_of(p.scale_log2, p.scale_log2);
        const float lowest = __int_as_float(0xff800000);
        int have = 0, uses = 0;              // scores taken, results
        bool ok = true;
        for (; more; move_on()) {
            if (!ok || !live || !it.blocks(t)) {
                ask();
                continue;
            }
            const int in_seq = it.span.tile * kItem + t * kSpan + (int)rank * kRows;     // the tile's first query
            const int rows = min(32, it.span.len - in_seq - quad * 32);                  // of this warp, none: 0 or less
            // P is 2^((score - m) * scale_log2), m = `top`, a maximum of the row's scores.  (lowest: none yet, or all were;
            // m is 0 and P too.)
            float top = lowest;
            unsigned long long total = 0;
            auto anchor = [&] { return top == lowest ? 0.f : top; };
            auto beyond = [&] { return !(fabsf(anchor() * p.scale_log2) < kFar); };
            // the power of two that P has too much by the rounding of m * scale_log2
            auto rest = [&] {
                const float m = anchor(), b = __fmul_rn(m, p.scale_log2);
                return beyond() ? 0.f : __fmaf_rn(m, p.scale_log2, -b);
            };
            for (int i = 0; i < it.blocks(t); ++i, ++have) {
                if (!__all_sync(0xffffffffu, mbar_wait(s_full + 8 * t, have & 1, &p))) {
                    ok = false;
                    break;
                }
                tmem_fence_after();
                const int ahead = in_seq - (it.blocks(t) - 1 - i) * kRows;       // of the tile's first query before the block
                uint32_t w[2][32];
                if (rows <= 0 || ahead < 0) {        // nobody's queries (whatever P holds stays in their rows), or a block
                                                     // that begins behind the tile's last
#pragma unroll
                    for (int e = 0; e < 32; ++e) w[0][e] = w[1][e] = 0;
                } else {
                    unsigned long long sums[2];
                    auto hide = [&](uint32_t (&x)[32], int at) {     // tokens behind the row's own
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = at + e > row ? 0xff800000u : x[e];
                    };
                    // P of the block, and its sum; Any: of rows that may lie far from zero
                    auto all_powers = [&](auto any, bool hides) {
                        constexpr bool kAny = decltype(any)::value;
                        sums[0] = sums[1] = 0;
                        const float m = anchor(), less = kAny && beyond() ? m : 0.f, b = kAny && beyond() ? 0.f : __fmul_rn(m, -p.scale_log2);
                        const unsigned long long b2 = pair_of(b, b);
                        auto powers = [&](uint32_t (&x)[32], int g) {
                            if (hides) hide(x, 32 * g);
                            if constexpr (kAny) {
#pragma unroll
                                for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) - less);
                            }
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float lo, hi;
                                split_pair(fma_pair(pair_of(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), c2, b2), lo, hi);
                                lo = exp2_fast(lo);
                                hi = exp2_fast(hi);
                                sums[e & 1] = add_pair(sums[e & 1], pair_of(lo, hi));
                                w[g / 2][16 * (g & 1) + e] = pack2<Fmt>(lo, hi);
                            }
                        };
                        uint32_t x[32], y[32];       // the next columns come meanwhile
                        tmem_load32(mine, x);
                        tmem_wait(x);
                        tmem_load32(mine + 32, y);
                        powers(x, 0);
                        tmem_wait(y);
                        tmem_load32(mine + 64, x);
                        powers(y, 1);
                        tmem_wait(x);
                        tmem_load32(mine + 96, y);
                        powers(x, 2);
                        tmem_wait(y);
                        powers(y, 3);
                    };
                    auto highest = [&](bool hides) {                 // (by the whole warp)
                        float m4[4] = {lowest, lowest, lowest, lowest};
#pragma unroll 1         // (four blocks of scores at once would take all registers)
                        for (int g = 0; g < 4; ++g) {
                            uint32_t x[32];
                            tmem_load32(mine + 32 * g, x);
                            tmem_wait(x);
                            if (hides) hide(x, 32 * g);
#pragma unroll
                            for (int e = 0; e < 32; e += 2)
                                m4[e / 2 & 3] = fmaxf(m4[e / 2 & 3], fmaxf(__uint_as_float(x[e]), __uint_as_float(x[e + 1])));
                        }
                        return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    };
                    // The block of the tile's own tokens first: up to there nothing is to be rescaled.  Then P against what it
                    // was taken against before; where a row's sum shows that it grew beyond kMost, everything is taken
                    // against the new maximum.  (One row's growth leaves the others as they are.)  So it is where a row has no
                    // maximum yet, and in every block of rows far from zero: a log sum is a multiple of large steps
                    // there, and less than a score would make the gradient's P more than 1.
                    bool again;
                    if (ahead == 0) {
                        top = highest(true);
                        all_powers(std::false_type{}, true);
                        again = beyond();
                    } else {
                        all_powers(std::false_type{}, false);
                        float lo, hi;
                        split_pair(add_pair(sums[0], sums[1]), lo, hi);
                        again = !(lo + hi <= kMost) || top == lowest || beyond();
                    }
                    if (__any_sync(0xffffffffu, again)) {
                        if (ahead) {
                            const float before = anchor(), before_rest = rest(), most = highest(false);
                            const bool first = top == lowest;
                            if (again) top = fmaxf(top, most);
                            const float f = first ? 0.f : exp2_fast(__fmaf_rn(before - anchor(), p.scale_log2, rest() - before_rest));
                            total = mul_pair(total, pair_of(f, f));
                            for (int x = 0; x < cols; x += 16) {
                                uint32_t o[16];
                                tmem_read16(sum + x, o);
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tmem_store16(sum + x, o);
                            }
                        }
                        all_powers(std::true_type{}, ahead == 0);
                    }
                    total = add_pair(total, add_pair(sums[0], sums[1]));
                }
                tmem_store32(mine, w[0]);    // over scores that are done with
                tmem_store32(mine + 32, w[1]);
                tmem_stored();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(taken);
            }
            ask();
            if (!ok) continue;
            if (!__all_sync(0xffffffffu, mbar_wait(o_full + 8 * t, uses++ & 1, &p))) {
                ok = false;
                continue;
            }
            tmem_fence_after();
            float l0, l1;
            split_pair(total, l0, l1);
            const float l = l0 + l1;
            const int token = it.span.first + in_seq + quad * 32;
            // (the gradient rounds a score to fp32 and takes its row's log sum off: rounded alike here, a row of one large
            // key has the very score, whatever its size)
            if (p.lse && lane < rows)
                p.lse[((int64_t)it.span.batch * p.heads + it.head) * p.tokens.seq + token + lane] =
                    __fmaf_rn(0.693147180559945309f, log2f(l) - rest(), __fmul_rn(anchor(), p.scale));
            if (rows > 0) {
                const Place to{&map_out, static_cast<T*>(p.out) + it.span.batch * p.out_batch + token * p.out_seq + it.head * p.out_head,
                               p.out_seq, token, it.head, it.span.batch};
                store_rows<Fmt>(smem + L::kOut + (warp - kSoftmaxWarp) * kOutStage, sum, 1.f / l, to, rows, 0, p.dim, lane, free);
            } else {
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(free);
            }
        }
        stored_all(lane);
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    cluster_sync();             // no CTA leaves while the other may signal or read it
    if (warp == 2) tmem_free_all(tmem);
}

// ---------------------------------------------------------------- host
template <class Fmt, int Blocks>
tb_status launch(const CUtensorMap (&m)[4], const Args& p, int64_t items, cudaStream_t st) {
    using L = Layout<Blocks>;
    if (resident_clusters(reinterpret_cast<const void*>(&attention_kernel<Fmt, Blocks>), kThreads, L::kBytes, 2) < 1) return TB_ERR_CUDA;
    return launch_clusters<true>(attention_kernel<Fmt, Blocks>, dim3((unsigned)(2 * items)), dim3(kThreads), L::kBytes, st, 2, m[0], m[1], m[2],
                                 m[3], p) == cudaSuccess
               ? launch_status()
               : TB_ERR_CUDA;
}

// The self-test's share of this kernel.
template <int Blocks>
tb_status withheld(int64_t wait_limit_ns, int* err, unsigned char* mem, cudaStream_t st, int* launches) {
    const int64_t dim = 64 * Blocks;
    tb_heads h[4];
    for (int i = 0; i < 4; ++i) h[i] = self_heads(&mem, i == 1 || i == 2 ? 1 : kSelfHeads, dim);
    CUtensorMap m[4];
    for (int i = 0; i < 4; ++i)
        if (!make_heads_map(&m[i], h[i], 1, kSelfTokens, dim, i == 1 ? kRows / 2 : kRows, true, i == 3)) return TB_ERR_CUDA;
    Args p{};
    p.tokens = Tokens{nullptr, 0, 1, (int)kSelfTokens, err};
    p.heads = p.group = (int)kSelfHeads, p.dim = (int)dim;
    p.tiles = (int)ceil_div(kSelfTokens, kItem);
    p.scale = p.scale_log2 = 1.f;
    p.out = h[3].data, p.out_batch = h[3].stride_batch, p.out_seq = h[3].stride_seq, p.out_head = h[3].stride_head;
    p.err = err, p.wait_ns = (unsigned long long)wait_limit_ns;
    return run_withheld(err, st, launches, [&](int what) {
        p.withhold = what;
        return launch<BF16, Blocks>(m, p, p.tiles * kSelfHeads, st);
    });
}

}  // namespace

tb_status attention_withheld(int64_t wait_limit_ns, int* err, unsigned char* mem, cudaStream_t st, int* launches) {
    const tb_status s = withheld<1>(wait_limit_ns, err, mem, st, launches);
    return s == TB_OK ? withheld<2>(wait_limit_ns, err, mem, st, launches) : s;
}

}  // namespace tb

extern "C" tb_status tb_attention(const tb_heads* q, const tb_heads* k, const tb_heads* v, const tb_heads* out, float* lse,
                                  int64_t batch, int64_t seq, int64_t head_dim, const int64_t* offsets, int64_t sequences,
                                  float scale, tb_dtype dtype, void* stream) {
    using namespace tb;
    tb_status s = check_call(batch, seq, head_dim, offsets, sequences, scale, dtype);
    if (s != TB_OK) return s;
    View view[4];
    const tb_heads* given[4] = {q, k, v, out};
    for (int i = 0; i < 4; ++i)
        if ((s = check_heads(given[i], batch, seq, head_dim, i == 3, &view[i])) != TB_OK) return s;
    if (out->heads != q->heads || v->heads != k->heads) return TB_ERR_INVALID_VALUE;
    if (batch == 0 || seq == 0 || q->heads == 0) return TB_OK;
    if (k->heads == 0 || q->heads % k->heads) return TB_ERR_INVALID_VALUE;
    if (!aligned_to(lse, 4)) return TB_ERR_MISALIGNED;
    const Range sums = range_of(lse, lse ? batch * q->heads * seq : 0, 4);
    const Range starts = range_of(offsets, offsets ? sequences + 1 : 0, 8);
    for (int i = 0; i < 4; ++i) {
        if (i < 3 && shares(view[3], view[i], head_dim, 2)) return TB_ERR_ALIAS;
        if (overlap(sums, range_of_view(view[i], head_dim))) return TB_ERR_ALIAS;
    }
    if (overlap(sums, starts) || overlap(starts, range_of_view(view[3], head_dim))) return TB_ERR_ALIAS;
    if (offsets && sequences == 0) return TB_OK;
    const int64_t tiles = ceil_div(seq, kItem), slots = offsets ? slots_of(seq, sequences, kItem) : tiles * batch;
    if (slots > ((1ll << 30) - 1) / q->heads) return TB_ERR_INVALID_VALUE;
    const bool bf = dtype == TB_BF16;
    CUtensorMap m[4];
    for (int i = 0; i < 4; ++i)
        if (!make_heads_map(&m[i], *given[i], batch, seq, head_dim, i == 1 ? kRows / 2 : kRows, bf, i == 3)) return TB_ERR_CUDA;
    Args p{};
    if (!(p.err = device_error_word())) return TB_ERR_CUDA;
    p.tokens = Tokens{offsets, (int)sequences, (int)batch, (int)seq, p.err};
    p.heads = (int)q->heads, p.group = (int)(q->heads / k->heads), p.dim = (int)head_dim;
    p.tiles = (int)tiles;
    p.scale = scale, p.scale_log2 = scale * kLog2e;
    p.out = out->data;
    p.out_batch = view[3].s[0], p.out_seq = view[3].s[1], p.out_head = view[3].s[2];
    p.lse = lse;
    p.wait_ns = kWaitLimitNs;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t items = slots * q->heads;
    if (head_dim <= 64) return bf ? launch<BF16, 1>(m, p, items, st) : launch<F16, 1>(m, p, items, st);
    return bf ? launch<BF16, 2>(m, p, items, st) : launch<F16, 2>(m, p, items, st);
}
