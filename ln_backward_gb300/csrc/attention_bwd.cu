// attention_bwd.cu -- the gradient of causal attention over whole prompts.
//
//     p_ij = exp(s_ij - lse_i),  dp_ij = dout_i . v_j,  ds_ij = p_ij (dp_ij - dout_i . out_i)
//     dv_j = sum_i p_ij dout_i,  dk_j = scale sum_i ds_ij q_i,  dq_i = scale sum_j ds_ij k_j
//
// Three kernels: rows_kernel forms dout . out of every row; dkv_kernel walks the queries of a tile of keys (four
// products: scores, dP, dV, dK), dq_kernel the keys of a tile of queries (three: scores and dP again, dQ).  Five products
// would do if one walk gave all three gradients, but then dQ of a tile is a sum over CTAs: of atomics, whose order
// changes its bits, or of fp32 partial sums in memory.  Sums here stay in tensor memory, in one order; only where tiles of
// keys are fewer than SMs do several pieces share a key head's query heads, whose fp32 sums join_kernel adds in their order.
//
// Pairs of CTAs work on 256 keys or queries (see attention.cuh).  Tiles that stream by are staged in both forms, by rows for
// scores and dP, by columns for the sums over tokens.  P and dS are first operands of the products over tokens and go from
// the warps back to tensor memory, over the scores and dP (dkv), or over the scores of which there are two (dq).  Eight
// warps work, two for the same rows, 64 columns each.  The key heads' gradients are summed over their group's query heads in
// the same accumulators.
//
// What bounds them at heads of 128 (bf16 4 x 4,096 tokens, 32 heads): dkv 2,750 clocks a tile of 128 queries where the MMAs
// need 2,048: P takes 990 and dS 900, mostly powers, and reads of tensor memory whose port the MMAs share; 745 us, 1,475
// TFLOP/s of its four products.  dq 1,800 clocks where 1,536 are needed; 533 us, 1,550 TFLOP/s of its three.  Together with the
// rows 1,360 us while the clocks last, 1,010 TFLOP/s of the formula's five products, 54 % of cuBLAS's burst; 1,500 to 1,535 us, 900
// to 920 TFLOP/s, call after call under the power limit.  A piece of work
// adds 4,000 to 6,000 clocks, which tells on short sequences: 8,192 packed tokens of 1 to 2,047 396 us, 605 TFLOP/s.
// One CTA with tiles of its own: 965 and 998 us.  Log sums and deltas taken off by the tensor cores, as products over three
// parts of 8 or 11 bits: P 840 and dS 400 clocks, but the parts' way to the other CTA and the added products took
// that back (1,360 us at best).
#include "attention.cuh"

namespace tb {
namespace {

constexpr int kWorkWarp = 4;                 // first of the eight that turn scores into P and dS
constexpr int kThreads = (kWorkWarp + 8) * 32;
constexpr int kHalfCols = kRows / 2;         // columns of a tile that one of the two warps of some rows takes

// Shared memory: two tiles that stay while a CTA works on its rows, and the tiles that stream by.  Those are staged in
// both of the forms that products take them in, each CTA half: 64 tokens with all columns, to be multiplied by rows,
// and 128 tokens with half the columns, to be summed over the tokens.
template <int Blocks, int... Rings>          // of 64 columns of a head; places of each stream
struct Layout {
    static constexpr int kStreams = sizeof...(Rings);
    static constexpr int kTileBytes = Blocks * kBox;
    static constexpr int kStageBytes = kBox;
    static constexpr int kStages = (Rings + ...);
    static constexpr int kStage0 = 2 * kTileBytes;
    static constexpr int kOut = kStage0 + kStages * kStageBytes;
    static constexpr int kAux = kOut + 8 * kOutStage;
    static constexpr int kBars = kAux + 2 * kRows * 4;           // log sums and deltas of a query tile
    static constexpr int kBytes = kBars + 1024 + 512;            // alignment, barriers
    static __host__ __device__ constexpr int ring(int s) {
        constexpr int r[kStreams] = {Rings...};
        return r[s];
    }
    static __host__ __device__ constexpr int first(int s) {      // stage of a stream
        int n = 0;
        for (int i = 0; i < s; ++i) n += ring(i);
        return n;
    }
};
// Queries and gradients of the output by rows, then both summed over.
template <int Blocks>
using LayoutKv = Layout<Blocks, 2, 2, 2, 2>;
// Keys and values by rows, keys summed over.
template <int Blocks>
using LayoutQ = Layout<Blocks, 2, 2, 3>;

struct Args {
    Tokens tokens;
    int heads, kv_heads, group, dim;
    int tiles;                // of 256 tokens of a batch entry, without offsets
    float scale, scale_log2;
    const float2* aux;        // [batch][heads][seq]: lse, dout . out
    const unsigned* norms;    // fp16: the largest norms of a dout and of a v, as bits
    void *grad0, *grad1;      // dQ; or dK and dV
    int parts;                // dkv: pieces of work that share a key head's query heads
    float* sums;              // [parts][batch][seq][kv_heads][2][dim]: dK's and dV's where there are several
    int64_t stride[2][3];     // of batch, seq, head in elements
    int* err;
    unsigned long long wait_ns;
    int withhold;             // self-test: a Withheld
};

// fp16 holds P times 2^14 and dS times the power of two that keeps it below 2^15 whatever the scores are:
// |dS| <= |dout_i . (v_j - out_i)| <= 2 |dout_i| max |v|.  (bf16 has fp32's range.)
template <class Fmt>
constexpr int kPShift = std::is_same<Fmt, F16>::value ? 14 : 0;
template <class Fmt>
__device__ __forceinline__ int ds_shift(const unsigned* norms) {
    if constexpr (std::is_same<Fmt, BF16>::value) return 0;
    const float bound = 2.f * __uint_as_float(__ldcg(norms)) * __uint_as_float(__ldcg(norms + 1));
    const int e = (int)(__float_as_uint(bound) >> 23);
    return e == 0 || e == 255 ? 0 : min(max(13 + 127 - e, -100), 100);
}
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((127 + e) << 23); }

// P is one FMA and a power of a score, 2^(s c - lse log2(e)): off by the rounding of either product, 2^-24 of |s| and of |lse|,
// which is 2^-13 of P at kFarSum, a fourth of fp16's own rounding.  Beyond it the score is rounded to fp32 first, as the
// forward's log sums have it, and the log sum taken off: exact next to each other, so that a row's one large key has P = 1
// whatever its size.  (Without that P was off by 14 % at 1e6 and by a factor of 8 at 1e7.)
constexpr float kFarSum = 1024.f;
__device__ __forceinline__ bool far_sum(float lse) { return !(fabsf(lse) <= kFarSum); }
// That is done to 64 columns of scores where they lie, before P is taken; column c's log sum is that of aux[step * c], and
// from column `left` on 0.  (Done to the registers on P's way, the branch alone cost 2.6 % of the gradient of 8,192 packed
// tokens.)
__device__ __noinline__ void take_off_sums(uint32_t tmem, float scale, const float2* aux, int step, int left) {
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        uint32_t x[32];
        tmem_load32(tmem + 32 * half, x);
        tmem_wait(x);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            const int c = 32 * half + e;
            const float sum = c < left ? __ldcg(&aux[step * c]).x : 0.f;
            x[e] = __float_as_uint(__fadd_rn(__fmul_rn(__uint_as_float(x[e]), scale), -sum));
        }
        tmem_store32(tmem + 32 * half, x);
    }
    tmem_stored();
}

// Barriers of either kernel.
struct Bars {
    uint32_t answer, keep, keep_free, full, free, first, second, first_taken, second_taken, aux, aux_free, acc, acc_free, tail, mended, drain,
        done, work_full, work_empty, words, slot, far, stopped;
};
template <class L>
__device__ __forceinline__ Bars bars_at(uint32_t at) {
    Bars b;
    auto take = [&](int n) {
        const uint32_t x = at;
        at += 8 * n;
        return x;
    };
    b.answer = take(2);                      // (16-byte aligned)
    b.keep = take(2), b.keep_free = take(2);
    b.full = take(L::kStages), b.free = take(L::kStages);
    b.first = take(2), b.second = take(1), b.first_taken = take(1), b.second_taken = take(1);
    b.aux = take(2), b.aux_free = take(2), b.acc = take(1), b.acc_free = take(1);
    b.tail = take(1), b.mended = take(1), b.drain = take(1), b.done = take(1), b.work_full = take(1), b.work_empty = take(1);
    b.words = take(3), b.slot = at, b.far = at + 4, b.stopped = at + 8;
    static_assert((2 + 4 + 2 * L::kStages + 5 + 6 + 6 + 3) * 8 + 12 <= 512 && L::kStreams + 2 <= 6);
    return b;
}
template <class L>
__device__ __forceinline__ void init_bars(const Bars& b, volatile int* stopped, int readers, int withhold) {
    *stopped = 0;
    for (int i = 0; i < L::kStages; ++i) {
        mbar_init(b.full + 8 * i, 2);        // an arrival of either CTA, and their bytes
        mbar_init(b.free + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
        mbar_init(b.keep + 8 * i, 2);
        mbar_init(b.keep_free + 8 * i, 1);
        mbar_init(b.first + 8 * i, 1 + (withhold == kScores));
        mbar_init(b.aux + 8 * i, 1);
        mbar_init(b.aux_free + 8 * i, 8);
    }
    mbar_init(b.second, 1);
    mbar_init(b.first_taken, 16 + (withhold == kTaken));         // the warps of both CTAs
    mbar_init(b.second_taken, 16 + (withhold == kTaken));
    mbar_init(b.acc, 1 + (withhold == kResults));
    mbar_init(b.acc_free, 16);
    mbar_init(b.tail, 1);
    mbar_init(b.mended, 1);
    mbar_init(b.drain, 1);
    mbar_init(b.done, 1);
    init_work(b.work_full, b.work_empty, readers);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// What the loading warp of a CTA has staged, by stream, and the tiles that stay.
template <class L, int Blocks>
struct Loader {
    const Args& p;
    const Bars& bar;
    unsigned char* smem;
    uint32_t smem0, rank;
    Tails ends;
    int lane, loaded[L::kStreams], kept[2], tails, last;      // ends, and the tile number of the last one
    __device__ __forceinline__ Loader(const Args& p_, const Bars& b_, unsigned char* s_, uint32_t s0_, uint32_t r_, int l_)
        : p(p_), bar(b_), smem(s_), smem0(s0_), rank(r_),
          ends{b_.tail, b_.mended, b_.stopped}, lane(l_), loaded{}, kept{}, tails(0), last(0) {}
    // One of the tiles that stay: this CTA's 128 tokens from `token` on.
    __device__ __forceinline__ bool keep(int i, const CUtensorMap* map, int token, int head, int batch) {
        if (kept[i] && !__all_sync(0xffffffffu, mbar_wait(bar.keep_free + 8 * i, (kept[i] - 1) & 1, &p))) return false;
        if (elect_one()) {
            const uint32_t to = map_to(bar.keep + 8 * i, 0);
            mbar_expect_at(to, L::kTileBytes);
            for (int b = 0; b < Blocks; ++b) tma_tile(smem0 + i * L::kTileBytes + b * kBox, map, 64 * b, token, head, batch, to);
        }
        __syncwarp();
        ++kept[i];
        return true;
    }
    __device__ __forceinline__ uint32_t place(int s) const { return L::first(s) + loaded[s] % L::ring(s); }
    __device__ __forceinline__ bool room(int s) const {
        const int ring = L::ring(s);
        return loaded[s] < ring || __all_sync(0xffffffffu, mbar_wait(bar.free + 8 * place(s), (loaded[s] / ring - 1) & 1, &p));
    }
    // The next tile of stream s (the map's box is half the tokens, by rows, or all of them and half the `cols`
    // columns): counted on the first CTA's barrier, or on this CTA's own while its end is to be mended.
    __device__ __forceinline__ void load(int s, bool by_rows, const CUtensorMap* map, int token, int head, int batch, int cols, bool mend) {
        if (elect_one()) {
            const uint32_t to = mend ? map_to(bar.tail, rank) : map_to(bar.full + 8 * place(s), 0);
            const uint32_t at = smem0 + L::kStage0 + place(s) * L::kStageBytes;
            // (of a tile to be mended, the bytes of all streams are counted before)
            if (!mend) mbar_expect_at(to, bytes(by_rows));
            if (by_rows)
                for (int b = 0; b < Blocks; ++b) tma_tile(at + b * kHalfBox, map, 64 * b, token + (int)rank * (kRows / 2), head, batch, to);
            else tma_tile(at, map, (int)rank * cols / 2, token, head, batch, to);
        }
        __syncwarp();
    }
    static __device__ __forceinline__ int bytes(bool by_rows) { return by_rows ? Blocks * kHalfBox : kBox; }
    // Before a tile to be mended: `n` bytes in all streams.  (One at a time.)
    __device__ __forceinline__ bool expect_mended(int n) {
        if (!ends.next(tails, &p)) return false;
        ++tails;
        last = loaded[0];
        if (elect_one()) mbar_expect_at(map_to(bar.tail, rank), n);
        __syncwarp();
        return true;
    }
    // `first`: the streams from it on are mended.
    __device__ __forceinline__ void leave(int first) const {
        if (ends.left_over(tails, &p) && lane == 0) {
#pragma unroll
            for (int s = 0; s < L::kStreams; ++s)
                if (s >= first) mbar_arrive_cluster(map_to(bar.full + 8 * (L::first(s) + last % L::ring(s)), 0));
        }
        __syncwarp();
        constexpr int n = L::kStreams + 2;
        int mine[n], rings[n];
        for (int s = 0; s < L::kStreams; ++s) mine[s] = loaded[s], rings[s] = L::ring(s);
        for (int i = 0; i < 2; ++i) mine[L::kStreams + i] = kept[i], rings[L::kStreams + i] = 1;
        way_out<n>(rank, mine, rings, bar.drain, bar.done, bar.words, smem + (bar.words - smem0), &p, [&](int s, int i, uint32_t* parity) {
            if (s >= L::kStreams) {
                *parity = i & 1;
                return bar.keep + 8 * (s - L::kStreams);
            }
            *parity = (i / L::ring(s)) & 1;
            return bar.full + 8 * (L::first(s) + i % L::ring(s));
        });
    }
};

// The warp that mends tiles at a sequence's end.  `rows`: tokens of the tile that are the sequence's.
template <class L, int Blocks>
struct Mender {
    const Args& p;
    const Bars& bar;
    unsigned char* smem;
    uint32_t rank;
    Tails ends;
    int lane, tails;
    __device__ __forceinline__ bool wait() {
        if (!__all_sync(0xffffffffu, mbar_wait(bar.tail, tails & 1, &p))) {
            stop();
            return false;
        }
        ++tails;
        return true;
    }
    __device__ __forceinline__ void stop() const { ends.stop(tails + 1, lane); }
    // Tile n of the streams from `first` on, those below 2 by rows.
    __device__ __forceinline__ void mend(int first, int n, int rows) const {
#pragma unroll
        for (int s = 0; s < L::kStreams; ++s)
            if (s >= first)
                clear_behind(smem + L::kStage0 + (L::first(s) + n % L::ring(s)) * L::kStageBytes, s < 2 ? Blocks : 1, s < 2 ? kRows / 2 : kRows,
                             s < 2 ? rows - (int)rank * (kRows / 2) : rows, lane);
        cleared(lane);
        if (lane == 0) {
#pragma unroll
            for (int s = 0; s < L::kStreams; ++s)
                if (s >= first) mbar_arrive_cluster(map_to(bar.full + 8 * (L::first(s) + n % L::ring(s)), 0));
            mbar_arrive(bar.mended);
        }
        __syncwarp();
    }
};

// What the warp that issues the MMAs takes from a stream: place n.
template <class L>
struct Stages {
    const Args& p;
    const Bars& bar;
    uint32_t smem0;
    __device__ __forceinline__ uint32_t tile(int s, int n) const {
        return smem0 + L::kStage0 + (L::first(s) + n % L::ring(s)) * L::kStageBytes;
    }
    __device__ __forceinline__ bool wait(int s, int n) const {
        return __all_sync(0xffffffffu, mbar_wait(bar.full + 8 * (L::first(s) + n % L::ring(s)), (n / L::ring(s)) & 1, &p));
    }
    __device__ __forceinline__ void free(int s, int n) const { mma_commit(bar.free + 8 * (L::first(s) + n % L::ring(s))); }
};

struct Maps {
    CUtensorMap q, q_rows, k, k_rows, v, v_rows, dout, dout_rows;    // 128 tokens a box; _rows: 64
    CUtensorMap out0, out1;
};

// ---------------------------------------------------------------- dK and dV
// A pair has 256 keys of one key head, and walks the query tiles of the sequence from its own on, of every
// query head of the group.  Transposed: keys are rows, so that P^T and dS^T are first operands as they come.
struct Keys {
    Span span;
    int head, part;
    int first, each, steps;   // query tiles: the first, of a head, of all heads
    int query0;               // the first query head
    __device__ __forceinline__ int tile(int i) const { return first + i % each; }
    __device__ __forceinline__ int query_head(int i) const { return query0 + i / each; }
};
__device__ __forceinline__ bool find_keys(const Args& p, unsigned index, Keys* k) {
    const unsigned heads = (unsigned)(p.kv_heads * p.parts), slot = index / heads, which = index - slot * heads;
    k->head = (int)(which / (unsigned)p.parts);
    k->part = (int)(which - (unsigned)(k->head * p.parts));
    k->query0 = k->head * p.group + k->part * (p.group / p.parts);
    if (p.tokens.offsets) {
        if (!find_tile<true>(p.tokens, kSpan, (int)slot, true, &k->span)) return false;
    } else {                  // the longest first
        const unsigned batch = (unsigned)p.tokens.batch;
        k->span = Span{(int)(slot % batch), 0, p.tokens.seq, (int)(slot / batch)};
    }
    k->first = 2 * k->span.tile;
    k->each = (k->span.len + kRows - 1) / kRows - k->first;
    k->steps = k->each * (p.group / p.parts);
    return true;
}

// 32 rows of sums, a row a lane, to memory.
__device__ __forceinline__ void store_sums(float* out, uint32_t tmem, bool live, int dim, int lane, uint32_t free) {
#pragma unroll 1
    for (int x = 0; x < dim; x += 32) {
        uint32_t o[32];
        tmem_load32(tmem + x, o);
        tmem_wait(o);
        if (x + 32 >= dim) {
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(free);
        }
        if (live) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (x + 4 * i < dim) *reinterpret_cast<uint4*>(out + x + 4 * i) = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
    }
}

template <class Fmt, int Blocks>
__global__ void __launch_bounds__(kThreads, 1) dkv_kernel(const __grid_constant__ Maps m, const __grid_constant__ Args p) {
    using L = LayoutKv<Blocks>;
    using T = typename Fmt::T;
    constexpr bool kBf = std::is_same<Fmt, BF16>::value;
    enum { kQRows, kDoRows, kDoSum, kQSum };
    extern __shared__ unsigned char raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t smem0 = smem_addr(smem);
    const Bars bar = bars_at<L>(smem0 + L::kBars);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();
    if (threadIdx.x == 0)                    // loads, log sums, work; the MMAs
        init_bars<L>(bar, reinterpret_cast<volatile int*>(smem + (bar.stopped - smem0)), 2 * 10 + 1, p.withhold);
    if (warp == 3) tmem_alloc_all(bar.slot);
    tmem_fence_before();
    __syncthreads();
    cluster_sync();
    tmem_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + (bar.slot - smem0));
    pdl_wait();
    asm volatile("fence.proxy.async;" ::: "memory");
    pdl_trigger();

    const uint32_t score = tmem, dprob = tmem + kRows, dv = tmem + 2 * kRows, dk = tmem + 3 * kRows;
    const int cols = (p.dim + 15) / 16 * 16;
    Work work{bar.answer, bar.work_full, bar.work_empty, 0};
    Keys it, next;
    bool live = find_keys(p, blockIdx.x >> 1, &it), next_live = false, more = true;
    auto ask = [&] {
        unsigned cluster;
        more = next_work(work, lane, &cluster, &p);
        next_live = more && find_keys(p, cluster, &next);
    };
    auto move_on = [&] { it = next, live = next_live; };

    if (warp == 0) {
        Loader<L, Blocks> load(p, bar, smem, smem0, rank, lane);
        bool ok = p.withhold != kLoads0 + (int)rank;
        for (; more; move_on()) {
            if (!ok || !live) {
                ask();
                continue;
            }
            const int token = it.span.first + it.span.tile * kSpan + (int)rank * kRows, batch = it.span.batch;
            ok = load.keep(0, &m.k, token, it.head, batch) && load.keep(1, &m.v, token, it.head, batch);
            for (int i = 0; i < it.steps && ok; ++i) {
                const int row = it.tile(i) * kRows, head = it.query_head(i), rows = it.span.len - row;
                const bool mend = rows < kRows;
                if (mend) {                      // all of it, or nothing
#pragma unroll
                    for (int s = 0; s < 4; ++s) ok = ok && load.room(s);
                    ok = ok && load.expect_mended(2 * load.bytes(true) + 2 * load.bytes(false));
                    if (!ok) break;
                }
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    ok = ok && load.room(s);
                    if (!ok) break;
                    const bool by_rows = s < 2;
                    load.load(s, by_rows, s == kQRows ? &m.q_rows : s == kDoRows ? &m.dout_rows : s == kDoSum ? &m.dout : &m.q,
                              it.span.first + row, head, batch, cols, mend);
                    ++load.loaded[s];
                }
            }
            ask();
        }
        load.leave(0);
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t by_rows = instruction(kBf, kRows, false), by_cols = instruction(kBf, cols, true);
            const Stages<L> st{p, bar, smem0};
            int n = 0, items = 0;            // query tiles taken, in all
            bool ok = true;
            auto scores = [&](int at, bool last) {
                if (!st.wait(kQRows, at)) return false;
                if (elect_one()) {
                    product_by_rows<Blocks>(score, smem0, st.tile(kQRows, at), cols / 16, by_rows);
                    mma_commit(bar.first);
                    st.free(kQRows, at);
                    if (last) mma_commit(bar.keep_free);
                }
                __syncwarp();
                return true;
            };
            auto dprobs = [&](int at, bool last) {
                if (!st.wait(kDoRows, at)) return false;
                if (elect_one()) {
                    product_by_rows<Blocks>(dprob, smem0 + L::kTileBytes, st.tile(kDoRows, at), cols / 16, by_rows);
                    mma_commit(bar.second);
                    st.free(kDoRows, at);
                    if (last) mma_commit(bar.keep_free + 8);
                }
                __syncwarp();
                return true;
            };
            for (; more; move_on()) {
                if (!ok || !live) {
                    ask();
                    continue;
                }
                ok = __all_sync(0xffffffffu, mbar_wait(bar.keep, items & 1, &p)) && scores(n, it.steps == 1) &&
                     __all_sync(0xffffffffu, mbar_wait(bar.keep + 8, items & 1, &p)) && dprobs(n, it.steps == 1);
                for (int i = 0; i < it.steps && ok; ++i, ++n) {
                    // P^T lies over the scores: the next ones follow its product, in order
                    const bool more_tiles = i + 1 < it.steps, last = i + 2 == it.steps;
                    ok = st.wait(kDoSum, n) && __all_sync(0xffffffffu, mbar_wait<kRelaxed>(bar.first_taken, n & 1, &p)) &&
                         (i || !items || __all_sync(0xffffffffu, mbar_wait<kRelaxed>(bar.acc_free, (items - 1) & 1, &p)));
                    if (!ok) break;
                    tmem_fence_after();
                    if (elect_one()) {
                        product_over_tokens(dv, score, kHalfCols, st.tile(kDoSum, n), by_cols, i > 0);
                        st.free(kDoSum, n);
                    }
                    __syncwarp();
                    if (more_tiles && !scores(n + 1, last)) ok = false;
                    ok = ok && st.wait(kQSum, n) && __all_sync(0xffffffffu, mbar_wait<kRelaxed>(bar.second_taken, n & 1, &p));
                    if (!ok) break;
                    tmem_fence_after();
                    if (elect_one()) {
                        product_over_tokens(dk, dprob, kHalfCols, st.tile(kQSum, n), by_cols, i > 0);
                        st.free(kQSum, n);
                        if (!more_tiles) mma_commit(bar.acc);
                    }
                    __syncwarp();
                    if (more_tiles && !dprobs(n + 1, last)) ok = false;
                }
                ++items;
                ask();
            }
            if (elect_one()) mma_commit(bar.drain);
        }
    } else if (warp == 2) {
        // The ends of sequences; log sums and deltas of the next query tile, negated.  A query behind the end has P = 0.
        Mender<L, Blocks> ends{p, bar, smem, rank, {bar.tail, bar.mended, bar.stopped}, lane, 0};
        const float f = power_of_two(ds_shift<Fmt>(p.norms) - kPShift<Fmt>);
        float* table = reinterpret_cast<float*>(smem + L::kAux);
        int n = 0;
        bool ok = true;
        for (; more; move_on()) {
            if (!ok || !live) {
                ask();
                continue;
            }
            for (int i = 0; i < it.steps; ++i, ++n) {
                float2 x[4];
                const int row0 = it.tile(i) * kRows;
                if (it.span.len - row0 < kRows) {        // (before the loads, which its release would wait for)
                    if (!ends.wait()) {
                        ok = false;
                        break;
                    }
                    ends.mend(0, n, it.span.len - row0);
                }
                const float2* aux = p.aux + ((int64_t)it.span.batch * p.heads + it.query_head(i)) * p.tokens.seq + it.span.first;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int row = row0 + 32 * k + lane;
                    x[k] = row < it.span.len ? aux[row] : make_float2(0.f, 0.f);
                }
                const bool far = __any_sync(0xffffffffu, far_sum(x[0].x) || far_sum(x[1].x) || far_sum(x[2].x) || far_sum(x[3].x));
                // the log sums are read with the scores, the deltas with dP: each is free for the next tile behind that
                if (n && !__all_sync(0xffffffffu, mbar_wait(bar.aux_free, (n - 1) & 1, &p))) {
                    ends.stop();
                    ok = false;
                    break;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float sum = far ? 0.f : x[k].x;        // (a far tile's are taken off the scores)
                    table[32 * k + lane] = row0 + 32 * k + lane < it.span.len ? __fmaf_rn(-sum, kLog2e, (float)kPShift<Fmt>) : __int_as_float(0xff800000);
                }
                if (lane == 0) *reinterpret_cast<volatile int*>(smem + (bar.far - smem0)) = far;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar.aux);
                if (n && !__all_sync(0xffffffffu, mbar_wait(bar.aux_free + 8, (n - 1) & 1, &p))) {
                    ends.stop();
                    ok = false;
                    break;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) table[kRows + 32 * k + lane] = -x[k].y * f;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar.aux + 8);
            }
            ask();
        }
    } else if (warp == 3) {
        hand_out(work, rank, &p);
    } else {
        const int half = (warp - kWorkWarp) >> 2, quad = warp & 3;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t s_at = score + lanes + half * kHalfCols, d_at = dprob + lanes + half * kHalfCols;
        const uint32_t s_taken = map_to(bar.first_taken, 0), d_taken = map_to(bar.second_taken, 0), acc_free = map_to(bar.acc_free, 0);
        const int shift = ds_shift<Fmt>(p.norms);
        const float f = power_of_two(shift - kPShift<Fmt>);
        const unsigned long long f2 = pair_of(f, f);
        // (a lane's columns are 8 k + lane % 4 * 2 and the next, of four rows: a quarter of the table's values that a lane
        // with a row of its own needs, which took 1,500 of a tile's 3,100 clocks of shared memory)
        const float2 *sums = reinterpret_cast<const float2*>(smem + L::kAux) + half * kHalfCols / 2 + lane % 4, *deltas = sums + kRows / 2;
        int n = 0, items = 0;
        bool ok = true;
        for (; more; move_on()) {
            if (!ok || !live) {
                ask();
                continue;
            }
            const int mine = it.first + (int)rank;           // this CTA's keys as a query tile
            for (int i = 0; i < it.steps; ++i, ++n) {
                if (!__all_sync(0xffffffffu, mbar_wait(bar.aux, n & 1, &p)) || !__all_sync(0xffffffffu, mbar_wait<kRelaxed>(bar.first, n & 1, &p))) {
                    ok = false;
                    break;
                }
                tmem_fence_after();
                const int tile = it.tile(i);
                unsigned long long prob[2][16];
                if (tile >= mine) {
                    const int row = quad * 32 + lane / 4, col = half * kHalfCols + lane % 4 * 2;
                    const bool far = *reinterpret_cast<volatile int*>(smem + (bar.far - smem0));
                    if (far) {
                        const int query = tile * kRows + half * kHalfCols;
                        take_off_sums(s_at, p.scale, p.aux + ((int64_t)it.span.batch * p.heads + it.query_head(i)) * p.tokens.seq + it.span.first + query,
                                      1, it.span.len - query);
                    }
                    uint32_t x[2][32];
                    tmem_load_16x64(s_at, x[0]);
                    tmem_load_16x64(s_at + (16u << 16), x[1]);
                    tmem_wait(x[0]);
                    tmem_wait(x[1]);
                    const float c = far ? kLog2e : p.scale_log2;
                    const unsigned long long c2 = pair_of(c, c);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        if (tile == mine) {      // queries before the row's own token
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (col + e / 4 * 8 + (e & 1) < row + 16 * g + (e & 2 ? 8 : 0)) x[g][e] = 0xff800000u;
                        }
                        uint32_t w[16];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float2 l = sums[4 * k];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float lo, hi;
                                split_pair(fma_pair(pair_of(__uint_as_float(x[g][4 * k + 2 * h]), __uint_as_float(x[g][4 * k + 2 * h + 1])), c2,
                                                    pair_of(l.x, l.y)), lo, hi);
                                lo = exp2_fast(lo);
                                hi = exp2_fast(hi);
                                prob[g][2 * k + h] = pair_of(lo, hi);
                                w[2 * k + h] = pack2<Fmt>(lo, hi);
                            }
                        }
                        tmem_store_16x64(s_at + ((uint32_t)(16 * g) << 16), w);
                    }
                } else {                         // all before the keys
                    const uint32_t none[16] = {};
                    tmem_store_16x64(s_at, none);
                    tmem_store_16x64(s_at + (16u << 16), none);
                }
                tmem_stored();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_cluster(s_taken);
                    mbar_arrive(bar.aux_free);
                }
                if (!__all_sync(0xffffffffu, mbar_wait(bar.aux + 8, n & 1, &p)) || !__all_sync(0xffffffffu, mbar_wait<kRelaxed>(bar.second, n & 1, &p))) {
                    ok = false;
                    break;
                }
                tmem_fence_after();
                if (tile >= mine) {
                    uint32_t x[2][32];
                    tmem_load_16x64(d_at, x[0]);
                    tmem_load_16x64(d_at + (16u << 16), x[1]);
                    tmem_wait(x[0]);
                    tmem_wait(x[1]);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        uint32_t w[16];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float2 d = deltas[4 * k];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const unsigned long long dp = pair_of(__uint_as_float(x[g][4 * k + 2 * h]), __uint_as_float(x[g][4 * k + 2 * h + 1]));
                                float lo, hi;
                                split_pair(mul_pair(prob[g][2 * k + h], kBf ? add_pair(dp, pair_of(d.x, d.y)) : fma_pair(dp, f2, pair_of(d.x, d.y))), lo, hi);
                                w[2 * k + h] = pack2<Fmt>(lo, hi);
                            }
                        }
                        tmem_store_16x64(d_at + ((uint32_t)(16 * g) << 16), w);
                    }
                } else {
                    const uint32_t none[16] = {};
                    tmem_store_16x64(d_at, none);
                    tmem_store_16x64(d_at + (16u << 16), none);
                }
                tmem_stored();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_cluster(d_taken);
                    mbar_arrive(bar.aux_free + 8);
                }
            }
            ask();
            if (!ok) continue;
            if (!__all_sync(0xffffffffu, mbar_wait<kRelaxed>(bar.acc, items++ & 1, &p))) {
                ok = false;
                continue;
            }
            tmem_fence_after();
            const int in_seq = it.span.tile * kSpan + (int)rank * kRows + quad * 32, rows = min(32, it.span.len - in_seq);
            if (rows > 0 && p.sums) {
                const int64_t token = ((int64_t)it.part * p.tokens.batch + it.span.batch) * p.tokens.seq + it.span.first + in_seq + lane;
                store_sums(p.sums + ((token * p.kv_heads + it.head) * 2 + !half) * p.dim, (half ? dk : dv) + lanes, lane < rows, p.dim, lane,
                           acc_free);
            } else if (rows > 0) {
                const int token = it.span.first + in_seq, g = !half;     // dV, dK
                const Place to{half ? &m.out0 : &m.out1,
                               static_cast<T*>(half ? p.grad0 : p.grad1) + it.span.batch * p.stride[g][0] + token * p.stride[g][1] + it.head * p.stride[g][2],
                               p.stride[g][1], token, it.head, it.span.batch};
                store_rows<Fmt>(smem + L::kOut + (warp - kWorkWarp) * kOutStage, (half ? dk : dv) + lanes,
                                half ? p.scale * power_of_two(-shift) : power_of_two(-kPShift<Fmt>), to, rows, 0, p.dim, lane, acc_free);
            } else {
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(acc_free);
            }
        }
        stored_all(lane);
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    cluster_sync();             // no CTA leaves while the other may signal or read it
    if (warp == 3) tmem_free_all(tmem);
}

// ---------------------------------------------------------------- dQ
// A pair has 256 queries of one head, and walks the key tiles up to its own, the last first.
struct Queries {
    Span span;
    int head, steps;          // key tiles
};
__device__ __forceinline__ bool find_queries(const Args& p, unsigned index, Queries* q) {
    q->head = (int)(index % (unsigned)p.heads);
    const unsigned slot = index / (unsigned)p.heads;
    if (p.tokens.offsets) {
        if (!find_tile<true>(p.tokens, kSpan, (int)slot, false, &q->span)) return false;
    } else {
        const unsigned batch = (unsigned)p.tokens.batch;
        q->span = Span{(int)(slot % batch), 0, p.tokens.seq, p.tiles - 1 - (int)(slot / batch)};
    }
    q->steps = min(2 * q->span.tile + 2, (q->span.len + kRows - 1) / kRows);
    return true;
}

template <class Fmt, int Blocks>
__global__ void __launch_bounds__(kThreads, 1) dq_kernel(const __grid_constant__ Maps m, const __grid_constant__ Args p) {
    using L = LayoutQ<Blocks>;
    using T = typename Fmt::T;
    constexpr bool kBf = std::is_same<Fmt, BF16>::value;
    enum { kKRows, kVRows, kKSum };
    extern __shared__ unsigned char raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t smem0 = smem_addr(smem);
    const Bars bar = bars_at<L>(smem0 + L::kBars);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();
    if (threadIdx.x == 0) init_bars<L>(bar, reinterpret_cast<volatile int*>(smem + (bar.stopped - smem0)), 2 * 10 + 1, p.withhold);
    if (warp == 3) tmem_alloc_all(bar.slot);
    tmem_fence_before();
    __syncthreads();
    cluster_sync();
    tmem_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + (bar.slot - smem0));
    // This kernel follows dkv_kernel, whose results it does not touch, and starts as that one's CTAs end: every CTA of it
    // had seen all earlier kernels complete before it let this one start.  It ends after it (see the end).
    asm volatile("fence.proxy.async;" ::: "memory");
    pdl_trigger();

    // scores in two places, the second for the next key tile; dS lies over them
    const uint32_t score = tmem, dprob = tmem + 2 * kRows, dq = tmem + 3 * kRows;
    const int cols = (p.dim + 15) / 16 * 16;
    Work work{bar.answer, bar.work_full, bar.work_empty, 0};
    Queries it, next;
    bool live = find_queries(p, blockIdx.x >> 1, &it), next_live = false, more = true;
    auto ask = [&] {
        unsigned cluster;
        more = next_work(work, lane, &cluster, &p);
        next_live = more && find_queries(p, cluster, &next);
    };
    auto move_on = [&] { it = next, live = next_live; };

    if (warp == 0) {
        Loader<L, Blocks> load(p, bar, smem, smem0, rank, lane);
        bool ok = p.withhold != kLoads0 + (int)rank;
        for (; more; move_on()) {
            if (!ok || !live) {
                ask();
                continue;
            }
            const int token = it.span.first + it.span.tile * kSpan + (int)rank * kRows, batch = it.span.batch, kv_head = it.head / p.group;
            ok = load.keep(0, &m.q, token, it.head, batch) && load.keep(1, &m.dout, token, it.head, batch);
            for (int i = 0; i < it.steps && ok; ++i) {
                const int row = (it.steps - 1 - i) * kRows, rows = it.span.len - row;
                // (scores of keys behind the end are hidden)
                const bool mend = rows < kRows;
                if (mend) {                      // all of it, or nothing
#pragma unroll
                    for (int s = 0; s < 3; ++s) ok = ok && load.room(s);
                    ok = ok && load.expect_mended(load.bytes(true) + load.bytes(false));
                    if (!ok) break;
                }
#pragma unroll
                for (int s = 0; s < 3; ++s) {
                    ok = ok && load.room(s);
                    if (!ok) break;
                    load.load(s, s < 2, s == kKRows ? &m.k_rows : s == kVRows ? &m.v_rows : &m.k, it.span.first + row, kv_head, batch, cols,
                              mend && s != kKRows);
                    ++load.loaded[s];
                }
            }
            ask();
        }
        load.leave(kVRows);
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t by_rows = instruction(kBf, kRows, false), by_cols = instruction(kBf, cols, true);
            const Stages<L> st{p, bar, smem0};
            int n = 0, items = 0;            // key tiles taken, in all
            bool ok = true;
            auto scores = [&](int at, bool last) {
                if (!st.wait(kKRows, at)) return false;
                if (elect_one()) {
                    product_by_rows<Blocks>(score + (at & 1) * kRows, smem0, st.tile(kKRows, at), cols / 16, by_rows);
                    mma_commit(bar.first + 8 * (at & 1));
                    st.free(kKRows, at);
                    if (last) mma_commit(bar.keep_free);
                }
                __syncwarp();
                return true;
            };
            auto dprobs = [&](int at, bool last) {
                if (!st.wait(kVRows, at)) return false;
                if (elect_one()) {
                    product_by_rows<Blocks>(dprob, smem0 + L::kTileBytes, st.tile(kVRows, at), cols / 16, by_rows);
                    mma_commit(bar.second);
                    st.free(kVRows, at);
                    if (last) mma_commit(bar.keep_free + 8);
                }
                __syncwarp();
                return true;
            };
            for (; more; move_on()) {
                if (!ok || !live) {
                    ask();
                    continue;
                }
                ok = __all_sync(0xffffffffu, mbar_wait(bar.keep, items & 1, &p)) && scores(n, it.steps == 1) &&
                     __all_sync(0xffffffffu, mbar_wait(bar.keep + 8, items & 1, &p)) && dprobs(n, it.steps == 1);
                for (int i = 0; i < it.steps && ok; ++i, ++n) {
                    // The place of the scores of n + 1 held dS of n - 1, whose product came before.
                    const bool more_tiles = i + 1 < it.steps, last = i + 2 == it.steps;
                    if (more_tiles && !scores(n + 1, last)) ok = false;
                    ok = ok && __all_sync(0xffffffffu, mbar_wait<kRelaxed>(bar.second_taken, n & 1, &p));
                    if (!ok) break;
                    tmem_fence_after();
                    if (more_tiles && !dprobs(n + 1, last)) ok = false;
                    ok = ok && st.wait(kKSum, n) &&
                         (i || !items || __all_sync(0xffffffffu, mbar_wait<kRelaxed>(bar.acc_free, (items - 1) & 1, &p)));
                    if (!ok) break;
                    tmem_fence_after();
                    if (elect_one()) {
                        product_over_tokens(dq, score + (n & 1) * kRows, kHalfCols, st.tile(kKSum, n), by_cols, i > 0);
                        st.free(kKSum, n);
                        if (!more_tiles) mma_commit(bar.acc);
                    }
                    __syncwarp();
                }
                ++items;
                ask();
            }
            if (elect_one()) mma_commit(bar.drain);
        }
    } else if (warp == 2) {
        Mender<L, Blocks> ends{p, bar, smem, rank, {bar.tail, bar.mended, bar.stopped}, lane, 0};
        int n = 0;
        bool ok = true;
        for (; more; move_on()) {
            if (!ok || !live) {
                ask();
                continue;
            }
            const int rows = it.span.len - (it.steps - 1) * kRows;
            if (rows < kRows) {              // the first keys and values end with the sequence
                if (!ends.wait()) {
                    ok = false;
                    ask();
                    continue;
                }
                ends.mend(kVRows, n, rows);
            }
            n += it.steps;
            ask();
        }
    } else if (warp == 3) {
        hand_out(work, rank, &p);
    } else if (warp >= kWorkWarp) {
        const int half = (warp - kWorkWarp) >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t d_at = dprob + lanes + half * kHalfCols;
        const uint32_t taken = map_to(bar.second_taken, 0), acc_free = map_to(bar.acc_free, 0);
        const int shift = ds_shift<Fmt>(p.norms);
        const int share = (cols / 2 + 31) / 32 * 32, from = half * share, to_col = min(p.dim, from + share);  // of dQ's columns
        int n = 0, items = 0;
        bool ok = true;
        for (; more; move_on()) {
            if (!ok || !live) {
                ask();
                continue;
            }
            const int in_seq = it.span.tile * kSpan + (int)rank * kRows + quad * 32, rows = min(32, it.span.len - in_seq);
            const int mine = 2 * it.span.tile + (int)rank;       // this CTA's queries as a key tile
            float2 aux = make_float2(0.f, 0.f);
            const float2* own = &p.aux[((int64_t)it.span.batch * p.heads + it.head) * p.tokens.seq + it.span.first + in_seq + lane];
            if (lane < rows) aux = __ldcg(own);
            const bool far = __any_sync(0xffffffffu, far_sum(aux.x));
            const float base = far ? (float)shift : __fmaf_rn(-aux.x, kLog2e, (float)shift), c = far ? kLog2e : p.scale_log2;
            const unsigned long long b2 = pair_of(base, base), c2 = pair_of(c, c), delta = pair_of(-aux.y, -aux.y);
            for (int i = 0; i < it.steps; ++i, ++n) {
                const uint32_t s_at = score + (n & 1) * kRows + lanes + half * kHalfCols;
                const int tile = it.steps - 1 - i;
                if (!__all_sync(0xffffffffu, mbar_wait<kRelaxed>(bar.first + 8 * (n & 1), (n / 2) & 1, &p))) {
                    ok = false;
                    break;
                }
                tmem_fence_after();
                unsigned long long prob[32];
                uint32_t a[32], b[32];
                if (tile <= mine) {
                    if (far) take_off_sums(s_at, p.scale, own, 0, lane < rows ? 2 * kHalfCols : 0);
                    tmem_load32(s_at, a);
                    tmem_load32(s_at + 32, b);
                    auto powers = [&](uint32_t (&x)[32], int at) {
                        if (tile == mine) {      // tokens behind the row's own
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[e] = half * kHalfCols + at + e > row ? 0xff800000u : x[e];
                        }
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float lo, hi;
                            split_pair(fma_pair(pair_of(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), c2, b2), lo, hi);
                            prob[at / 2 + e] = pair_of(exp2_fast(lo), exp2_fast(hi));
                        }
                    };
                    tmem_wait(a);
                    tmem_wait(b);
                    powers(a, 0);
                    powers(b, 32);
                }
                if (!__all_sync(0xffffffffu, mbar_wait<kRelaxed>(bar.second, n & 1, &p))) {
                    ok = false;
                    break;
                }
                tmem_fence_after();
                if (tile <= mine) {
                    tmem_load32(d_at, a);
                    tmem_load32(d_at + 32, b);
                    auto slopes = [&](const uint32_t (&x)[32], int at) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const unsigned long long dp = pair_of(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
                            float lo, hi;
                            split_pair(mul_pair(prob[at / 2 + e], add_pair(dp, delta)), lo, hi);
                            w[e] = pack2<Fmt>(lo, hi);
                        }
                        tmem_store16(s_at + at / 2, w);
                    };
                    tmem_wait(a);
                    tmem_wait(b);
                    slopes(a, 0);
                    slopes(b, 32);
                } else {                         // all keys behind the queries
                    const uint32_t none[32] = {};
                    tmem_store32(s_at, none);
                }
                tmem_stored();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(taken);
            }
            ask();
            if (!ok) continue;
            if (!__all_sync(0xffffffffu, mbar_wait<kRelaxed>(bar.acc, items++ & 1, &p))) {
                ok = false;
                continue;
            }
            tmem_fence_after();
            if (rows > 0 && from < to_col) {
                const int token = it.span.first + in_seq;
                const Place to{&m.out0,
                               static_cast<T*>(p.grad0) + it.span.batch * p.stride[0][0] + token * p.stride[0][1] + it.head * p.stride[0][2],
                               p.stride[0][1], token, it.head, it.span.batch};
                store_rows<Fmt>(smem + L::kOut + (warp - kWorkWarp) * kOutStage, dq + lanes, p.scale * power_of_two(-shift), to, rows, from,
                                to_col, lane, acc_free);
            } else {
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(acc_free);
            }
        }
        stored_all(lane);
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    cluster_sync();             // no CTA leaves while the other may signal or read it
    if (warp == 3) tmem_free_all(tmem);
    pdl_wait();                 // what waits for this kernel waits for both
}

// ---------------------------------------------------------------- before the products
// A row's log sum and dout . out; fp16: the largest norms of the rows of dout and of v in any
// sequence too.  The call's offsets are checked here.  Eight lanes a row, 16 bytes at a time, kRowsAtOnce rows in flight.
struct Rows {
    const void *dout, *out, *v;
    int64_t stride[3][3];     // of batch, seq, head
    const float* lse;         // [batch][heads][seq]
    float2* aux;
    unsigned* norms;
    const int64_t* offsets;
    int* err;
    int sequences, batch, seq, heads, kv_heads, dim;
    unsigned chunks, ctas;    // of a head's tokens; of rows of dout, the others have rows of v
};
constexpr int kRowThreads = 256, kRowsAtOnce = 2, kRowsCta = kRowThreads / 8 * kRowsAtOnce;

template <class Fmt>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const __grid_constant__ Rows p) {
    constexpr bool kNorms = std::is_same<Fmt, F16>::value;
    pdl_wait();
    pdl_trigger();
    const bool of_v = blockIdx.x >= p.ctas;
    const unsigned heads = of_v ? p.kv_heads : p.heads, part = threadIdx.x & 7;
    const unsigned cta = blockIdx.x - (of_v ? p.ctas : 0), row = cta / p.chunks, chunk = cta - row * p.chunks;   // of a head's tokens
    const unsigned batch = row / heads, head = row - batch * heads;
    auto start = [&](const void* x, int i) {
        return static_cast<const char*>(x) + (batch * p.stride[i][0] + head * p.stride[i][2] + part * 8) * 2;
    };
    const char *a = start(of_v ? p.v : p.dout, of_v ? 2 : 0), *b = start(p.out, 1);
    const int64_t step_a = p.stride[of_v ? 2 : 0][1] * 2, step_b = p.stride[1][1] * 2;
    const int at = (int)chunk * kRowsCta + threadIdx.x / 8;
    uint4 x[kRowsAtOnce][2], y[kRowsAtOnce][2];
#pragma unroll
    for (int i = 0; i < kRowsAtOnce; ++i) {
        const int s = at + i * (kRowThreads / 8);
#pragma unroll
        for (int c = 0; c < 2; ++c) {    // 64 columns each
            x[i][c] = y[i][c] = make_uint4(0, 0, 0, 0);
            if (s < p.seq && (int)part * 8 + 64 * c < p.dim) {
                x[i][c] = ld_stream_u4(a + s * step_a + 128 * c);
                if (!of_v) y[i][c] = ld_stream_u4(b + s * step_b + 128 * c);
            }
        }
    }
    unsigned most = 0;
#pragma unroll
    for (int i = 0; i < kRowsAtOnce; ++i) {
        const int s = at + i * (kRowThreads / 8);
        float dot = 0.f, square = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float u[8], v[8];
            unpack8<Fmt>(x[i][c], u);
            unpack8<Fmt>(y[i][c], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dot = __fmaf_rn(u[e], v[e], dot);
                if constexpr (kNorms) square = __fmaf_rn(u[e], u[e], square);
            }
        }
#pragma unroll
        for (int o = 4; o; o >>= 1) {
            dot += __shfl_xor_sync(0xffffffffu, dot, o);
            if constexpr (kNorms) square += __shfl_xor_sync(0xffffffffu, square, o);
        }
        if (s < p.seq && !of_v && part == 0) {
            const int64_t k = (int64_t)row * p.seq + s;
            p.aux[k] = make_float2(p.lse[k], dot);
        }
        if constexpr (kNorms) {
            const bool counts = s < p.seq && square <= 3.4028235e38f && (!p.offsets || (s >= p.offsets[0] && s < p.offsets[p.sequences]));
            if (counts) most = max(most, __float_as_uint(sqrtf(square) * 1.0001f));
        }
    }
    if constexpr (kNorms) {
        most = __reduce_max_sync(0xffffffffu, most);
        if ((threadIdx.x & 31) == 0 && most) atomicMax(p.norms + of_v, most);
    }
    if (p.offsets)
        for (int64_t i = (int64_t)blockIdx.x * kRowThreads + threadIdx.x; i < p.sequences; i += (int64_t)gridDim.x * kRowThreads)
            check_offsets(p.offsets, i, p.seq, p.err);
}

// dK and dV from the sums of several pieces, in their order; eight elements a thread.
struct Join {
    const float* sums;
    void* out[2];             // dK, dV
    int64_t stride[2][3];
    const unsigned* norms;
    const int64_t* offsets;
    int sequences, parts, batch, seq, heads, dim;
    float scale;
};
template <class Fmt>
__global__ void __launch_bounds__(kRowThreads) join_kernel(const __grid_constant__ Join p) {
    pdl_wait();
    pdl_trigger();
    const unsigned each = (unsigned)p.dim / 8;
    const int64_t i = (int64_t)blockIdx.x * kRowThreads + threadIdx.x, row = i / (2 * each);       // of [batch][seq][heads]
    const unsigned at = (unsigned)(i - row * (2 * each)), which = at >= each, c = (at - which * each) * 8;
    const int64_t token = row / p.heads, rows = (int64_t)p.batch * p.seq * p.heads;
    const int head = (int)(row - token * p.heads), batch = (int)(token / p.seq), s = (int)(token - (int64_t)batch * p.seq);
    if (row >= rows || (p.offsets && (s < p.offsets[0] || s >= p.offsets[p.sequences]))) return;
    float v[8] = {};
    for (int k = 0; k < p.parts; ++k) {
        const float4* x = reinterpret_cast<const float4*>(p.sums + ((k * rows + row) * 2 + which) * p.dim + c);
        const float4 a = __ldcs(x), b = __ldcs(x + 1);
        v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w, v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
    }
    const float f = which ? power_of_two(-kPShift<Fmt>) : p.scale * power_of_two(-ds_shift<Fmt>(p.norms));
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= f;
    typename Fmt::T* out = static_cast<typename Fmt::T*>(p.out[which]) + batch * p.stride[which][0] + s * p.stride[which][1] + head * p.stride[which][2] + c;
    *reinterpret_cast<uint4*>(out) = pack8<Fmt>(v);
}

// ---------------------------------------------------------------- host
// Pieces that the query heads of a key head are dealt to, where the tiles of keys are too few for the machine and have
// enough to do that the sums pay.  bf16, heads of 128, in one piece and as this says: 2,048 tokens of 8 heads over one
// 204 and 54 us, 8,192 767 and 341, 4,096 of 32 over four 404 and 358; 600 tokens of 8 heads of 64 over one 77 and 28.
constexpr int kSms = 152;                    // of a GB300: the cut, and the workspace, do not ask the device
// Grids, and with them the bytes of a workspace, stay within their types.
bool fits(int64_t batch, int64_t seq, int64_t heads) { return ceil_div(seq, kRowsCta) * batch <= (1ll << 30) / heads; }
int parts_for(int64_t batch, int64_t seq, int64_t heads, int64_t kv_heads) {
    const int64_t pieces = ceil_div(seq, kSpan) * batch * kv_heads, group = heads / kv_heads;
    if (ceil_div(seq, kRows) * group < 16) return 1;
    int64_t parts = 1;
    while (parts < group && (pieces * parts < kSms || group % parts)) ++parts;   // two for each pair of SMs
    return (int)parts;
}
size_t padded(size_t bytes) { return (bytes + 255) / 256 * 256; }
size_t aux_bytes(int64_t batch, int64_t seq, int64_t heads) { return padded((size_t)(batch * heads * seq) * sizeof(float2)); }
size_t workspace_bytes_for(int64_t batch, int64_t seq, int64_t heads, int64_t kv_heads, int64_t dim, int parts) {
    return 256 + aux_bytes(batch, seq, heads) +      // norms, aux, sums
           (parts > 1 ? (size_t)parts * batch * seq * kv_heads * 2 * dim * sizeof(float) : 0);
}

// The products of dK and dV, and of dQ.
template <class Fmt, int Blocks, bool Kv, bool Dq>
tb_status launch_products(Maps& m, Args p, const tb_heads* const (&grads)[3], const View (&grad)[3], int64_t batch, int64_t seq,
                          int64_t slots, cudaStream_t st) {
    constexpr bool bf = std::is_same<Fmt, BF16>::value;
    constexpr int kv_bytes = LayoutKv<Blocks>::kBytes, q_bytes = LayoutQ<Blocks>::kBytes;
    if (resident_clusters(reinterpret_cast<const void*>(&dkv_kernel<Fmt, Blocks>), kThreads, kv_bytes, 2) < 1 ||
        resident_clusters(reinterpret_cast<const void*>(&dq_kernel<Fmt, Blocks>), kThreads, q_bytes, 2) < 1)
        return TB_ERR_CUDA;
    auto gradient = [&](int i, int of, void** data, CUtensorMap* map) {
        *data = const_cast<char*>(grad[of].p);
        for (int k = 0; k < 3; ++k) p.stride[i][k] = grad[of].s[k];
        return make_heads_map(map, *grads[of], batch, seq, p.dim, 32, bf, true);
    };
    if (!gradient(0, 1, &p.grad0, &m.out0) || !gradient(1, 2, &p.grad1, &m.out1)) return TB_ERR_CUDA;
    if (Kv && launch_clusters<true>(dkv_kernel<Fmt, Blocks>, dim3((unsigned)(2 * slots * p.kv_heads * p.parts)), dim3(kThreads), kv_bytes, st, 2, m, p) !=
        cudaSuccess)
        return TB_ERR_CUDA;
    if (!gradient(0, 0, &p.grad0, &m.out0)) return TB_ERR_CUDA;
    if (Dq && launch_clusters<true>(dq_kernel<Fmt, Blocks>, dim3((unsigned)(2 * slots * p.heads)), dim3(kThreads), q_bytes, st, 2, m, p) !=
        cudaSuccess)
        return TB_ERR_CUDA;
    return launch_status();
}

template <class Fmt, int Blocks>
tb_status launch(Maps& m, Args p, const Rows& r, const tb_heads* const (&grads)[3], const View (&grad)[3], int64_t batch, int64_t seq,
                 cudaStream_t st) {
    constexpr bool bf = std::is_same<Fmt, BF16>::value;
    int64_t ctas = (int64_t)r.chunks * batch * r.heads;
    if (!bf) {
        if (cudaMemsetAsync(r.norms, 0, 2 * sizeof(unsigned), st) != cudaSuccess) return TB_ERR_CUDA;
        ctas += (int64_t)r.chunks * batch * r.kv_heads;
    }
    if (launch_pdl(rows_kernel<Fmt>, dim3((unsigned)ctas), dim3(kRowThreads), 0, st, r) != cudaSuccess) return TB_ERR_CUDA;
    const int64_t slots = r.offsets ? slots_of(seq, r.sequences, kSpan) : p.tiles * batch;
    const tb_status s = launch_products<Fmt, Blocks, true, true>(m, p, grads, grad, batch, seq, slots, st);
    if (s != TB_OK || p.parts == 1) return s;
    Join j{};
    j.sums = p.sums, j.norms = p.norms, j.offsets = r.offsets, j.sequences = r.sequences;
    j.parts = p.parts, j.batch = (int)batch, j.seq = (int)seq, j.heads = p.kv_heads, j.dim = p.dim, j.scale = p.scale;
    for (int i = 0; i < 2; ++i) {
        j.out[i] = const_cast<char*>(grad[1 + i].p);
        for (int k = 0; k < 3; ++k) j.stride[i][k] = grad[1 + i].s[k];
    }
    // (behind dq_kernel, which ends behind dkv_kernel)
    return launch_pdl(join_kernel<Fmt>, dim3((unsigned)ceil_div(batch * seq * p.kv_heads * 2 * (p.dim / 8), kRowThreads)), dim3(kRowThreads), 0, st,
                      j) == cudaSuccess
               ? launch_status()
               : TB_ERR_CUDA;
}

// The self-test's share of these kernels.
template <int Blocks>
tb_status withheld(int64_t wait_limit_ns, int* err, unsigned char* mem, cudaStream_t st, int* launches) {
    const int64_t dim = 64 * Blocks;
    tb_heads h[7];                       // q, k, v, dout; dq, dk, dv
    for (int i = 0; i < 7; ++i) h[i] = self_heads(&mem, i == 0 || i == 3 || i == 4 ? kSelfHeads : 1, dim);
    Maps m{};
    CUtensorMap* const whole[4] = {&m.q, &m.k, &m.v, &m.dout};
    CUtensorMap* const by_rows[4] = {&m.q_rows, &m.k_rows, &m.v_rows, &m.dout_rows};
    for (int i = 0; i < 4; ++i)
        if (!make_heads_map(whole[i], h[i], 1, kSelfTokens, dim, kRows, true) || !make_heads_map(by_rows[i], h[i], 1, kSelfTokens, dim, kRows / 2, true))
            return TB_ERR_CUDA;
    const tb_heads* const grads[3] = {&h[4], &h[5], &h[6]};
    View grad[3];
    for (int i = 0; i < 3; ++i) grad[i] = view_of(grads[i], 1, kSelfTokens);
    Args p{};
    p.tokens = Tokens{nullptr, 0, 1, (int)kSelfTokens, err};
    p.heads = p.group = (int)kSelfHeads, p.kv_heads = p.parts = 1, p.dim = (int)dim;
    p.tiles = (int)ceil_div(kSelfTokens, kSpan);
    p.scale = p.scale_log2 = 1.f;
    p.aux = reinterpret_cast<const float2*>(mem);
    p.err = err, p.wait_ns = (unsigned long long)wait_limit_ns;
    tb_status s = run_withheld(err, st, launches, [&](int what) {
        p.withhold = what;
        return launch_products<BF16, Blocks, true, false>(m, p, grads, grad, 1, kSelfTokens, p.tiles, st);
    });
    if (s == TB_OK)
        s = run_withheld(err, st, launches, [&](int what) {
            p.withhold = what;
            return launch_products<BF16, Blocks, false, true>(m, p, grads, grad, 1, kSelfTokens, p.tiles, st);
        });
    return s;
}

}  // namespace

tb_status attention_withheld(int64_t wait_limit_ns, int* err, unsigned char* mem, cudaStream_t st, int* launches);   // attention.cu

}  // namespace tb

extern "C" tb_status tb_attention_selftest_timeout(int64_t wait_limit_ns, int* launches, void* stream) {
    using namespace tb;
    if (!launches || wait_limit_ns < 1000 || wait_limit_ns > (int64_t)kWaitLimitNs) return TB_ERR_INVALID_VALUE;
    *launches = 0;
    int* err = device_error_word();
    if (!err) return TB_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    void* data = nullptr;
    if (cudaMalloc(&data, kSelfBytes) != cudaSuccess) {
        cudaGetLastError();
        return TB_ERR_OOM;
    }
    unsigned char* mem = static_cast<unsigned char*>(data);
    tb_status s = cudaMemsetAsync(data, 0, kSelfBytes, st) == cudaSuccess ? TB_OK : TB_ERR_CUDA;
    if (s == TB_OK) s = attention_withheld(wait_limit_ns, err, mem, st, launches);
    if (s == TB_OK) s = withheld<1>(wait_limit_ns, err, mem, st, launches);
    if (s == TB_OK) s = withheld<2>(wait_limit_ns, err, mem, st, launches);
    if (cudaStreamSynchronize(st) != cudaSuccess) s = TB_ERR_CUDA;
    if (cudaFree(data) != cudaSuccess) s = TB_ERR_CUDA;
    return s;
}

extern "C" tb_status tb_attention_bwd_workspace_size(int64_t batch, int64_t seq, int64_t heads_q, int64_t heads_k, int64_t head_dim,
                                                     tb_dtype dtype, size_t* bytes) {
    using namespace tb;
    if (!bytes || heads_q < 0 || heads_k < 0 || heads_q > (1 << 20) || heads_k > (1 << 20)) return TB_ERR_INVALID_VALUE;
    const tb_status s = check_call(batch, seq, head_dim, nullptr, 0, 1.f, dtype);
    if (s != TB_OK) return s;
    *bytes = 0;
    if (batch == 0 || seq == 0 || heads_q == 0) return TB_OK;
    if (heads_k == 0 || heads_q % heads_k || !fits(batch, seq, heads_q)) return TB_ERR_INVALID_VALUE;
    *bytes = workspace_bytes_for(batch, seq, heads_q, heads_k, head_dim, parts_for(batch, seq, heads_q, heads_k));
    return TB_OK;
}

extern "C" tb_status tb_attention_bwd(const tb_heads* dout, const tb_heads* q, const tb_heads* k, const tb_heads* v, const tb_heads* out,
                                      const float* lse, const tb_heads* dq, const tb_heads* dk, const tb_heads* dv, int64_t batch,
                                      int64_t seq, int64_t head_dim, const int64_t* offsets, int64_t sequences, float scale,
                                      tb_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace tb;
    tb_status s = check_call(batch, seq, head_dim, offsets, sequences, scale, dtype);
    if (s != TB_OK) return s;
    const tb_heads* in[5] = {q, k, v, dout, out};
    const tb_heads* grads[3] = {dq, dk, dv};
    View read[5], grad[3];
    for (int i = 0; i < 5; ++i)
        if ((s = check_heads(in[i], batch, seq, head_dim, false, &read[i])) != TB_OK) return s;
    for (int i = 0; i < 3; ++i)
        if ((s = check_heads(grads[i], batch, seq, head_dim, true, &grad[i])) != TB_OK) return s;
    for (const tb_heads* t : {dout, out, dq})
        if (t->heads != q->heads) return TB_ERR_INVALID_VALUE;
    for (const tb_heads* t : {v, dk, dv})
        if (t->heads != k->heads) return TB_ERR_INVALID_VALUE;
    if (batch == 0 || seq == 0 || (q->heads == 0 && k->heads == 0)) return TB_OK;
    if (q->heads == 0 || k->heads == 0 || q->heads % k->heads || !lse) return TB_ERR_INVALID_VALUE;
    if (!aligned_to(lse, 4)) return TB_ERR_MISALIGNED;
    const int64_t rows = batch * seq * q->heads;
    const Range sums = range_of(lse, rows, 4), starts = range_of(offsets, offsets ? sequences + 1 : 0, 8);
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 5; ++j)
            if (shares(grad[i], read[j], head_dim, 2)) return TB_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (shares(grad[i], grad[j], head_dim, 2)) return TB_ERR_ALIAS;
        const Range g = range_of_view(grad[i], head_dim);
        if (overlap(g, sums) || overlap(g, starts)) return TB_ERR_ALIAS;
    }
    const int parts = parts_for(batch, seq, q->heads, k->heads);
    const size_t need = workspace_bytes_for(batch, seq, q->heads, k->heads, head_dim, parts);
    if (!workspace || workspace_bytes < need) return TB_ERR_WORKSPACE;
    if (!aligned_to(workspace, 16)) return TB_ERR_MISALIGNED;
    const Range ws = range_of(workspace, (int64_t)need, 1);
    for (int i = 0; i < 5; ++i)
        if (overlap(ws, range_of_view(read[i], head_dim))) return TB_ERR_ALIAS;
    for (int i = 0; i < 3; ++i)
        if (overlap(ws, range_of_view(grad[i], head_dim))) return TB_ERR_ALIAS;
    if (overlap(ws, sums) || overlap(ws, starts)) return TB_ERR_ALIAS;
    if (offsets && sequences == 0) return TB_OK;
    const int64_t tiles = ceil_div(seq, kSpan), slots = offsets ? slots_of(seq, sequences, kSpan) : tiles * batch;
    if (slots > ((1ll << 30) - 1) / q->heads || !fits(batch, seq, q->heads)) return TB_ERR_INVALID_VALUE;
    const bool bf = dtype == TB_BF16;
    Maps m{};
    CUtensorMap* const whole[4] = {&m.q, &m.k, &m.v, &m.dout};
    CUtensorMap* const by_rows[4] = {&m.q_rows, &m.k_rows, &m.v_rows, &m.dout_rows};
    for (int i = 0; i < 4; ++i)
        if (!make_heads_map(whole[i], *in[i], batch, seq, head_dim, kRows, bf) ||
            !make_heads_map(by_rows[i], *in[i], batch, seq, head_dim, kRows / 2, bf))
            return TB_ERR_CUDA;
    Args p{};
    if (!(p.err = device_error_word())) return TB_ERR_CUDA;
    unsigned char* mem = static_cast<unsigned char*>(workspace);
    p.tokens = Tokens{offsets, (int)sequences, (int)batch, (int)seq, p.err};
    p.heads = (int)q->heads, p.kv_heads = (int)k->heads, p.group = (int)(q->heads / k->heads), p.dim = (int)head_dim;
    p.tiles = (int)tiles;
    p.scale = scale, p.scale_log2 = scale * kLog2e;
    p.norms = reinterpret_cast<unsigned*>(mem);
    p.aux = reinterpret_cast<float2*>(mem + 256);
    p.parts = parts;
    if (parts > 1) p.sums = reinterpret_cast<float*>(mem + 256 + aux_bytes(batch, seq, q->heads));
    p.wait_ns = kWaitLimitNs;
    Rows r{};
    const int of[3] = {3, 4, 2};
    const void** to[3] = {&r.dout, &r.out, &r.v};
    for (int i = 0; i < 3; ++i) {
        *to[i] = read[of[i]].p;
        for (int j = 0; j < 3; ++j) r.stride[i][j] = read[of[i]].s[j];
    }
    r.lse = lse, r.aux = const_cast<float2*>(p.aux), r.norms = const_cast<unsigned*>(p.norms);
    r.err = p.err, r.offsets = offsets, r.sequences = (int)sequences;
    r.batch = (int)batch, r.seq = (int)seq, r.heads = p.heads, r.kv_heads = p.kv_heads, r.dim = p.dim;
    r.chunks = (unsigned)ceil_div(seq, kRowsCta), r.ctas = r.chunks * (unsigned)(batch * q->heads);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (head_dim <= 64) return bf ? launch<BF16, 1>(m, p, r, grads, grad, batch, seq, st) : launch<F16, 1>(m, p, r, grads, grad, batch, seq, st);
    return bf ? launch<BF16, 2>(m, p, r, grads, grad, batch, seq, st) : launch<F16, 2>(m, p, r, grads, grad, batch, seq, st);
}
