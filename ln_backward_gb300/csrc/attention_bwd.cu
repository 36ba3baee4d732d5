// attention_bwd.cu -- the gradient of causal attention over whole prompts.
//
//     p_ij = exp(s_ij - lse_i),  dp_ij = dout_i . v_j,  ds_ij = p_ij (dp_ij - dout_i . out_i)
//     dv_j = sum_i p_ij dout_i,  dk_j = scale sum_i ds_ij q_i,  dq_i = scale sum_j ds_ij k_j
#include "attention.cuh"

namespace tb {
namespace {

constexpr int kWorkWarp = 4;                 // first of the eight that turn scores into P and dS
constexpr int kThreads = (kWorkWarp + 8) * 32;
constexpr int kHalfCols = kRows / 2;         // columns of a tile that one of the two warps of a row quarter takes

template <int Blocks>
struct Layout {
    static constexpr int kTileBytes = Blocks * kBox;
    static constexpr int kRing0 = Blocks == 1 ? 5 : 3;           // tiles of the stream that is read last
    static constexpr int kRing1 = Blocks == 1 ? 4 : 2;           // and of the other
    static constexpr int kStream = 2 * kTileBytes;               // behind the two tiles that stay
    static constexpr int kAux = kStream + (kRing0 + kRing1) * kTileBytes;
    static constexpr int kBars = kAux + 2 * kRows * 4;           // log sums and deltas of a query tile
    static __device__ __forceinline__ int ring(int i) { return i ? kRing1 : kRing0; }
    static __device__ __forceinline__ int at(int i, int n) { return kStream + (i * kRing0 + n % ring(i)) * kTileBytes; }
    static constexpr int kBytes = kBars + 1024 + 256;            // alignment, barriers
};

struct Args {
    Tokens tokens;
    int heads, kv_heads, group, dim;
    int tiles;                // of a batch entry, without offsets
    float scale, scale_log2;
    const float2* aux;        // [batch][heads][seq]: lse * log2(e), dout . out
    const unsigned* norms;    // fp16: the largest norms of a dout and of a v, as bits
    void *grad0, *grad1;      // dQ; or dK and dV
    int64_t stride[2][3];     // of batch, seq, head in elements
    int* err;
    unsigned long long wait_ns;
};

// fp16 holds P times 2^14 and dS times the power of two that keeps it below 2^15 whatever the scores are:
// |dS| <= |dout_i . (v_j - out_i)| <= 2 |dout_i| max |v|.  (bf16 has fp32's range.)
template <class Fmt>
constexpr int kPShift = std::is_same<Fmt, F16>::value ? 14 : 0;
template <class Fmt>
__device__ __forceinline__ int ds_shift(const unsigned* norms) {
    if constexpr (std::is_same<Fmt, BF16>::value) return 0;
    const float bound = 2.f * __uint_as_float(norms[0]) * __uint_as_float(norms[1]);
    const int e = (int)(__float_as_uint(bound) >> 23);
    return e == 0 || e == 255 ? 0 : min(max(13 + 127 - e, -100), 100);
}
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((127 + e) << 23); }

// What both kernels set up and take down.
struct Bars {
    uint32_t keep, ring[2], ring_free[2], first, second, first_taken, second_taken, aux, aux_free, all, tail, drain, slot;
};
template <class L>
__device__ __forceinline__ Bars bars_at(uint32_t at) {
    Bars b;
    auto take = [&](int n) {
        const uint32_t x = at;
        at += 8 * n;
        return x;
    };
    b.keep = take(2);
    b.ring[0] = take(L::kRing0), b.ring[1] = take(L::kRing1), b.ring_free[0] = take(L::kRing0), b.ring_free[1] = take(L::kRing1);
    b.first = take(2), b.second = take(1), b.first_taken = take(1), b.second_taken = take(1);
    b.aux = take(2), b.aux_free = take(2), b.all = take(1), b.tail = take(1), b.drain = take(1), b.slot = at;
    return b;
}
template <class L>
__device__ __forceinline__ void init_bars(const Bars& b) {
    for (int i = 0; i < 2; ++i) {
        mbar_init(b.keep + 8 * i, 1);
        for (int s = 0; s < L::ring(i); ++s) {
            mbar_init(b.ring[i] + 8 * s, 1);
            mbar_init(b.ring_free[i] + 8 * s, 1);
        }
        mbar_init(b.first + 8 * i, 1);
        mbar_init(b.aux + 8 * i, 1);
        mbar_init(b.aux_free + 8 * i, 8);
    }
    mbar_init(b.second, 1);
    mbar_init(b.first_taken, 8);
    mbar_init(b.second_taken, 8);
    mbar_init(b.all, 1);
    mbar_init(b.tail, 1);
    mbar_init(b.drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// Loads a tile of 128 tokens, those behind the sequence's end as zeros, by a whole warp.
template <int Blocks, class P>
__device__ __forceinline__ void load_tile(unsigned char* smem, uint32_t smem0, uint32_t at, const CUtensorMap* map, int token,
                                          int head, int batch, int rows, uint32_t bar, uint32_t tail, int* tails, int lane,
                                          const P* p) {
    const bool mend = rows < kRows;
    if (elect_one()) {
        mbar_expect(mend ? tail : bar, Blocks * kBox);
        for (int b = 0; b < Blocks; ++b) tma_tile(at + b * kBox, map, 64 * b, token, head, batch, mend ? tail : bar);
    }
    __syncwarp();
    if (!mend) return;
    mbar_wait<kEnd>(tail, *tails & 1, p);
    ++*tails;
    clear_behind<Blocks>(smem + (at - smem0), rows, lane);
    if (lane == 0) mbar_arrive(bar);
    __syncwarp();
}

// ---------------------------------------------------------------- dK and dV
// A CTA has 128 keys of one key head, and walks the query tiles of the sequence from its own on, of every
// query head of the group.  Transposed: keys are rows, so that P^T and dS^T are left operands as they come.
template <class Fmt, int Blocks>
__global__ void __launch_bounds__(kThreads, 1)
dkv_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
           const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do, const __grid_constant__ Args p) {
    using L = Layout<Blocks>;
    using T = typename Fmt::T;
    constexpr bool kBf = std::is_same<Fmt, BF16>::value;
    extern __shared__ unsigned char raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t smem0 = smem_addr(smem);
    const Bars bar = bars_at<L>(smem0 + L::kBars);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) init_bars<L>(bar);
    if (warp == 3) tmem_alloc_all(bar.slot);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + (bar.slot - smem0));
    pdl_wait();
    asm volatile("fence.proxy.async;" ::: "memory");
    pdl_trigger();

    const uint32_t score = tmem, dprob = tmem + kRows, dv = tmem + 2 * kRows, dk = tmem + 3 * kRows;
    Span span;
    const int kv_head = (int)(blockIdx.x % (unsigned)p.kv_heads);
    const unsigned place = blockIdx.x / (unsigned)p.kv_heads;
    bool live = true;
    if (p.tokens.offsets) live = find_tile(p.tokens, kRows, (int)place, false, &span);
    else span = Span{(int)(place % (unsigned)p.tokens.batch), 0, p.tokens.seq, (int)(place / (unsigned)p.tokens.batch)};
    const int each = live ? (span.len + kRows - 1) / kRows - span.tile : 0;   // query tiles of a head
    const int steps = each * p.group;
    auto tile_of = [&](int n) { return span.tile + n % each; };
    auto head_of = [&](int n) { return kv_head * p.group + n / each; };

    if (warp == 0) {
        int tails = 0, n = 0;
        bool ok = true;
        if (live) {
            const int token = span.first + span.tile * kRows;
            load_tile<Blocks>(smem, smem0, smem0, &map_k, token, kv_head, span.batch, kRows, bar.keep, 0, nullptr, lane, &p);
            for (; n < steps && ok; ++n) {
                const int row = tile_of(n) * kRows;
                for (int i = 0; i < 2; ++i) {      // queries, gradients
                    const int ring = L::ring(i), s = n % ring;
                    if (n >= ring && !__all_sync(0xffffffffu, mbar_wait(bar.ring_free[i] + 8 * s, (n / ring - 1) & 1, &p))) {
                        ok = false;
                        break;
                    }
                    load_tile<Blocks>(smem, smem0, smem0 + L::at(i, n), i ? &map_do : &map_q,
                                      span.first + row, head_of(n), span.batch, span.len - row, bar.ring[i] + 8 * s, bar.tail, &tails,
                                      lane, &p);
                    if (n == 0 && i == 0)
                        load_tile<Blocks>(smem, smem0, smem0 + L::kTileBytes, &map_v, token, kv_head, span.batch, kRows, bar.keep + 8,
                                          0, nullptr, lane, &p);
                }
            }
        }
        // The way out: the MMAs, then the loads that no MMA waited for.
        mbar_wait<kEnd>(bar.drain, 0, &p);
        if (live)
            for (int i = 0; i < 2; ++i) {
                mbar_wait<kEnd>(bar.keep + 8 * i, 0, &p);
                for (int q = max(0, n - L::ring(i)); q < n; ++q)
                    mbar_wait<kEnd>(bar.ring[i] + 8 * (q % L::ring(i)), (q / L::ring(i)) & 1, &p);
            }
    } else if (warp == 1) {
        const int cols = (p.dim + 15) / 16 * 16;
        const uint32_t by_rows = instruction(kBf, kRows, false), by_cols = instruction(kBf, cols, true);
        const uint32_t k_tile = tile_desc(smem0, false), v_tile = tile_desc(smem0 + L::kTileBytes, false);
        auto tile = [&](int i, int n) { return smem0 + L::at(i, n); };
        auto wait_ring = [&](int i, int n) {
            return __all_sync(0xffffffffu, mbar_wait(bar.ring[i] + 8 * (n % L::ring(i)), (n / L::ring(i)) & 1, &p));
        };
        auto scores = [&](int n) {
            if (!wait_ring(0, n)) return false;
            if (elect_one()) {
                product_by_rows<Blocks>(score, k_tile, tile_desc(tile(0, n), false), cols / 16, by_rows);
                mma_done(bar.first);
            }
            __syncwarp();
            return true;
        };
        auto dprobs = [&](int n) {
            if (!wait_ring(1, n)) return false;
            if (elect_one()) {
                product_by_rows<Blocks>(dprob, v_tile, tile_desc(tile(1, n), false), cols / 16, by_rows);
                mma_done(bar.second);
            }
            __syncwarp();
            return true;
        };
        bool ok = live && __all_sync(0xffffffffu, mbar_wait(bar.keep, 0, &p)) && scores(0) &&
                  __all_sync(0xffffffffu, mbar_wait(bar.keep + 8, 0, &p)) && dprobs(0);
        for (int n = 0; n < steps && ok; ++n) {
            // P^T lies over the scores: the next ones follow its product, in order
            if (!__all_sync(0xffffffffu, mbar_wait(bar.first_taken, n & 1, &p))) break;
            tmem_fence_after();
            if (elect_one()) product_over_tokens(dv, score, kHalfCols, tile_desc(tile(1, n), true), by_cols, n > 0);
            __syncwarp();
            if (n + 1 < steps && !scores(n + 1)) break;
            if (!__all_sync(0xffffffffu, mbar_wait(bar.second_taken, n & 1, &p))) break;
            tmem_fence_after();
            if (elect_one()) {
                product_over_tokens(dk, dprob, kHalfCols, tile_desc(tile(0, n), true), by_cols, n > 0);
                mma_done(bar.ring_free[0] + 8 * (n % L::kRing0));
                mma_done(bar.ring_free[1] + 8 * (n % L::kRing1));
                if (n + 1 == steps) mma_done(bar.all);
            }
            __syncwarp();
            if (n + 1 < steps && !dprobs(n + 1)) break;
        }
        if (elect_one()) mma_done(bar.drain);
    } else if (warp == 2) {
        // log sums and deltas of the next query tile; a query behind the end has P = 0
        const float f = power_of_two(ds_shift<Fmt>(p.norms) - kPShift<Fmt>);
        float* table = reinterpret_cast<float*>(smem + L::kAux);
        for (int n = 0; n < steps; ++n) {
            float2 x[4];
            const int row0 = tile_of(n) * kRows;
            const float2* aux = p.aux + ((int64_t)span.batch * p.heads + head_of(n)) * p.tokens.seq + span.first;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = row0 + 32 * i + lane;
                x[i] = row < span.len ? aux[row] : make_float2(__int_as_float(0x7f800000), 0.f);
            }
            // the log sums are read with the scores, the deltas with dP: each is free for the next tile behind that
            if (n && !__all_sync(0xffffffffu, mbar_wait(bar.aux_free, (n - 1) & 1, &p))) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) table[32 * i + lane] = x[i].x - kPShift<Fmt>;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar.aux);
            if (n && !__all_sync(0xffffffffu, mbar_wait(bar.aux_free + 8, (n - 1) & 1, &p))) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) table[kRows + 32 * i + lane] = x[i].y * f;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar.aux + 8);
        }
    } else if (warp >= kWorkWarp && live) {
        const int half = (warp - kWorkWarp) >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t s_at = score + lanes + half * kHalfCols, d_at = dprob + lanes + half * kHalfCols;
        const int shift = ds_shift<Fmt>(p.norms);
        const float f = power_of_two(shift - kPShift<Fmt>);
        const unsigned long long c2 = pair_of(p.scale_log2, p.scale_log2), f2 = pair_of(f, f), minus = pair_of(-1.f, -1.f);
        const float4 *sums = reinterpret_cast<const float4*>(smem + L::kAux) + half * kHalfCols / 4, *deltas = sums + kRows / 4;
        bool ok = true;
        for (int n = 0; n < steps; ++n) {
            if (!__all_sync(0xffffffffu, mbar_wait(bar.aux, n & 1, &p)) ||
                !__all_sync(0xffffffffu, mbar_wait(bar.first, n & 1, &p))) {
                ok = false;
                break;
            }
            tmem_fence_after();
            unsigned long long prob[32];
            uint32_t a[32], b[32];
            tmem_load32(s_at, a);
            tmem_load32(s_at + 32, b);
            const bool own = tile_of(n) == span.tile;
            auto powers = [&](uint32_t (&x)[32], int from) {
                if (own) {       // queries before the row's own token
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = half * kHalfCols + from + e < row ? 0xff800000u : x[e];
                }
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float4 l = sums[(from + 2 * e) / 4];
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        float lo, hi;
                        split_pair(fma_pair(pair_of(__uint_as_float(x[2 * (e + g)]), __uint_as_float(x[2 * (e + g) + 1])), c2,
                                            mul_pair(g ? pair_of(l.z, l.w) : pair_of(l.x, l.y), minus)), lo, hi);
                        lo = exp2_fast(lo);
                        hi = exp2_fast(hi);
                        prob[from / 2 + e + g] = pair_of(lo, hi);
                        w[e + g] = pack2<Fmt>(lo, hi);
                    }
                }
                tmem_store16(s_at + from / 2, w);
            };
            // (the first half's P lies over scores that both halves of this warp have in registers)
            tmem_wait(a);
            tmem_wait(b);
            powers(a, 0);
            powers(b, 32);
            tmem_stored();
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar.first_taken);
                mbar_arrive(bar.aux_free);
            }
            if (!__all_sync(0xffffffffu, mbar_wait(bar.aux + 8, n & 1, &p)) ||
                !__all_sync(0xffffffffu, mbar_wait(bar.second, n & 1, &p))) {
                ok = false;
                break;
            }
            tmem_fence_after();
            tmem_load32(d_at, a);
            tmem_load32(d_at + 32, b);
            auto slopes = [&](const uint32_t (&x)[32], int from) {
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float4 d = deltas[(from + 2 * e) / 4];
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const unsigned long long dp = pair_of(__uint_as_float(x[2 * (e + g)]), __uint_as_float(x[2 * (e + g) + 1]));
                        const unsigned long long delta = mul_pair(g ? pair_of(d.z, d.w) : pair_of(d.x, d.y), minus);
                        float lo, hi;
                        split_pair(mul_pair(prob[from / 2 + e + g], kBf ? add_pair(dp, delta) : fma_pair(dp, f2, delta)), lo, hi);
                        w[e + g] = pack2<Fmt>(lo, hi);
                    }
                }
                tmem_store16(d_at + from / 2, w);
            };
            tmem_wait(a);
            tmem_wait(b);
            slopes(a, 0);
            slopes(b, 32);
            tmem_stored();
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar.second_taken);
                mbar_arrive(bar.aux_free + 8);
            }
        }
        if (ok && __all_sync(0xffffffffu, mbar_wait(bar.all, 0, &p))) {
            tmem_fence_after();
            const int in_seq = span.tile * kRows + quad * 32, rows = min(32, span.len - in_seq);
            T* out = static_cast<T*>(half ? p.grad0 : p.grad1) + span.batch * p.stride[!half][0] +
                     (int64_t)(span.first + in_seq) * p.stride[!half][1] + kv_head * p.stride[!half][2];
            const float factor = half ? p.scale * power_of_two(-shift) : power_of_two(-kPShift<Fmt>);
            store_rows<Fmt>(smem + (warp - kWorkWarp) * kOutStage, (half ? dk : dv) + lanes, factor, out, p.stride[!half][1], rows,
                            p.dim, lane);
        }
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    if (warp == 3) tmem_free_all(tmem);
}

// ---------------------------------------------------------------- dQ
// A CTA has 128 queries of one head, and walks the key tiles up to its own.
template <class Fmt, int Blocks>
__global__ void __launch_bounds__(kThreads, 1)
dq_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
          const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do, const __grid_constant__ Args p) {
    using L = Layout<Blocks>;
    using T = typename Fmt::T;
    constexpr bool kBf = std::is_same<Fmt, BF16>::value;
    extern __shared__ unsigned char raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t smem0 = smem_addr(smem);
    const Bars bar = bars_at<L>(smem0 + L::kBars);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) init_bars<L>(bar);
    if (warp == 3) tmem_alloc_all(bar.slot);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + (bar.slot - smem0));
    pdl_wait();
    asm volatile("fence.proxy.async;" ::: "memory");
    pdl_trigger();

    // scores in two places, the second for the next key tile; dS lies over them
    const uint32_t score = tmem, dprob = tmem + 2 * kRows, dq = tmem + 3 * kRows;
    Span span;
    const int head = (int)(blockIdx.x % (unsigned)p.heads), kv_head = head / p.group;
    const unsigned place = blockIdx.x / (unsigned)p.heads;
    bool live = true;
    if (p.tokens.offsets) live = find_tile(p.tokens, kRows, (int)place, true, &span);
    else span = Span{(int)(place % (unsigned)p.tokens.batch), 0, p.tokens.seq, p.tiles - 1 - (int)(place / (unsigned)p.tokens.batch)};
    const int steps = live ? span.tile + 1 : 0;       // key tiles, the last first

    if (warp == 0) {
        int tails = 0, n = 0;
        bool ok = true;
        if (live) {
            const int token = span.first + span.tile * kRows;
            load_tile<Blocks>(smem, smem0, smem0, &map_q, token, head, span.batch, kRows, bar.keep, 0, nullptr, lane, &p);
            for (; n < steps && ok; ++n) {
                const int row = (steps - 1 - n) * kRows;
                for (int i = 0; i < 2; ++i) {      // keys, values
                    const int ring = L::ring(i), s = n % ring;
                    if (n >= ring && !__all_sync(0xffffffffu, mbar_wait(bar.ring_free[i] + 8 * s, (n / ring - 1) & 1, &p))) {
                        ok = false;
                        break;
                    }
                    load_tile<Blocks>(smem, smem0, smem0 + L::at(i, n), i ? &map_v : &map_k,
                                      span.first + row, kv_head, span.batch, span.len - row, bar.ring[i] + 8 * s, bar.tail, &tails,
                                      lane, &p);
                    if (n == 0 && i == 0)
                        load_tile<Blocks>(smem, smem0, smem0 + L::kTileBytes, &map_do, token, head, span.batch, kRows, bar.keep + 8, 0,
                                          nullptr, lane, &p);
                }
            }
        }
        mbar_wait<kEnd>(bar.drain, 0, &p);
        if (live)
            for (int i = 0; i < 2; ++i) {
                mbar_wait<kEnd>(bar.keep + 8 * i, 0, &p);
                for (int q = max(0, n - L::ring(i)); q < n; ++q)
                    mbar_wait<kEnd>(bar.ring[i] + 8 * (q % L::ring(i)), (q / L::ring(i)) & 1, &p);
            }
    } else if (warp == 1) {
        const int cols = (p.dim + 15) / 16 * 16;
        const uint32_t by_rows = instruction(kBf, kRows, false), by_cols = instruction(kBf, cols, true);
        const uint32_t q_tile = tile_desc(smem0, false), do_tile = tile_desc(smem0 + L::kTileBytes, false);
        auto tile = [&](int i, int n) { return smem0 + L::at(i, n); };
        auto wait_ring = [&](int i, int n) {
            return __all_sync(0xffffffffu, mbar_wait(bar.ring[i] + 8 * (n % L::ring(i)), (n / L::ring(i)) & 1, &p));
        };
        auto scores = [&](int n) {
            if (!wait_ring(0, n)) return false;
            if (elect_one()) {
                product_by_rows<Blocks>(score + (n & 1) * kRows, q_tile, tile_desc(tile(0, n), false), cols / 16, by_rows);
                mma_done(bar.first + 8 * (n & 1));
            }
            __syncwarp();
            return true;
        };
        auto dprobs = [&](int n) {
            if (!wait_ring(1, n)) return false;
            if (elect_one()) {
                product_by_rows<Blocks>(dprob, do_tile, tile_desc(tile(1, n), false), cols / 16, by_rows);
                mma_done(bar.second);
                mma_done(bar.ring_free[1] + 8 * (n % L::kRing1));
            }
            __syncwarp();
            return true;
        };
        bool ok = live && __all_sync(0xffffffffu, mbar_wait(bar.keep, 0, &p)) && scores(0) &&
                  __all_sync(0xffffffffu, mbar_wait(bar.keep + 8, 0, &p)) && dprobs(0);
        for (int n = 0; n < steps && ok; ++n) {
            // The place of the scores of n + 1 held dS of n - 1, whose product came before.
            if (n + 1 < steps && !scores(n + 1)) break;
            if (!__all_sync(0xffffffffu, mbar_wait(bar.second_taken, n & 1, &p))) break;
            tmem_fence_after();
            if (n + 1 < steps && !dprobs(n + 1)) break;
            if (elect_one()) {
                product_over_tokens(dq, score + (n & 1) * kRows, kHalfCols, tile_desc(tile(0, n), true), by_cols, n > 0);
                mma_done(bar.ring_free[0] + 8 * (n % L::kRing0));
                if (n + 1 == steps) mma_done(bar.all);
            }
            __syncwarp();
        }
        if (elect_one()) mma_done(bar.drain);
    } else if (warp >= kWorkWarp && live) {
        const int half = (warp - kWorkWarp) >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t d_at = dprob + lanes + half * kHalfCols;
        const int shift = ds_shift<Fmt>(p.norms);
        const int in_seq = span.tile * kRows + quad * 32, rows = min(32, span.len - in_seq);
        float2 aux = make_float2(0.f, 0.f);
        if (lane < rows) aux = p.aux[((int64_t)span.batch * p.heads + head) * p.tokens.seq + span.first + in_seq + lane];
        const float base = (float)shift - aux.x;
        const unsigned long long c2 = pair_of(p.scale_log2, p.scale_log2), b2 = pair_of(base, base), delta = pair_of(-aux.y, -aux.y);
        bool ok = true;
        for (int n = 0; n < steps; ++n) {
            const uint32_t s_at = score + (n & 1) * kRows + lanes + half * kHalfCols;
            if (!__all_sync(0xffffffffu, mbar_wait(bar.first + 8 * (n & 1), (n / 2) & 1, &p))) {
                ok = false;
                break;
            }
            tmem_fence_after();
            unsigned long long prob[32];
            uint32_t a[32], b[32];
            tmem_load32(s_at, a);
            tmem_load32(s_at + 32, b);
            auto powers = [&](uint32_t (&x)[32], int from) {
                if (n == 0) {    // tokens behind the row's own
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = half * kHalfCols + from + e > row ? 0xff800000u : x[e];
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float lo, hi;
                    split_pair(fma_pair(pair_of(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), c2, b2), lo, hi);
                    prob[from / 2 + e] = pair_of(exp2_fast(lo), exp2_fast(hi));
                }
            };
            tmem_wait(a);
            tmem_wait(b);
            powers(a, 0);
            powers(b, 32);
            if (!__all_sync(0xffffffffu, mbar_wait(bar.second, n & 1, &p))) {
                ok = false;
                break;
            }
            tmem_fence_after();
            tmem_load32(d_at, a);
            tmem_load32(d_at + 32, b);
            auto slopes = [&](const uint32_t (&x)[32], int from) {
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const unsigned long long dp = pair_of(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
                    float lo, hi;
                    split_pair(mul_pair(prob[from / 2 + e], add_pair(dp, delta)), lo, hi);
                    w[e] = pack2<Fmt>(lo, hi);
                }
                tmem_store16(s_at + from / 2, w);
            };
            tmem_wait(a);
            tmem_wait(b);
            slopes(a, 0);
            slopes(b, 32);
            tmem_stored();
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar.second_taken);
        }
        // (the keys' and values' places are free once all products are done)
        if (ok && __all_sync(0xffffffffu, mbar_wait(bar.all, 0, &p)) && half == 0) {
            tmem_fence_after();
            T* out = static_cast<T*>(p.grad0) + span.batch * p.stride[0][0] + (int64_t)(span.first + in_seq) * p.stride[0][1] +
                     head * p.stride[0][2];
            store_rows<Fmt>(smem + L::kStream + quad * kOutStage, dq + lanes, p.scale * power_of_two(-shift), out, p.stride[0][1], rows,
                            p.dim, lane);
        }
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    if (warp == 3) tmem_free_all(tmem);
}

// ---------------------------------------------------------------- before the products
// A row's log sum in powers of two and dout . out; fp16: the largest norms of the rows of dout and of v in any
// sequence too.  Eight lanes a row, 16 bytes at a time.
struct Rows {
    const void *dout, *out, *v;
    int64_t stride[3][3];     // of batch, seq, head
    const float* lse;         // [batch][heads][seq]
    float2* aux;
    unsigned* norms;
    const int64_t* offsets;
    int sequences, batch, seq, heads, kv_heads, dim;
    int64_t ctas;             // of rows of dout; the others have rows of v
};
constexpr int kRowThreads = 256;

template <class Fmt>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const __grid_constant__ Rows p) {
    constexpr bool kNorms = std::is_same<Fmt, F16>::value;
    pdl_wait();
    pdl_trigger();
    const bool of_v = blockIdx.x >= p.ctas;
    const int heads = of_v ? p.kv_heads : p.heads, part = threadIdx.x & 7;
    const int64_t row = ((int64_t)blockIdx.x - (of_v ? p.ctas : 0)) * (kRowThreads / 8) + threadIdx.x / 8;
    const int64_t token = row / heads;
    const int head = (int)(row - token * heads);
    const int batch = (int)(token / p.seq), at = (int)(token - (int64_t)batch * p.seq);
    const bool live = batch < p.batch;
    float dot = 0.f, square = 0.f;
    if (live) {
        auto row_of = [&](const void* x, int i) {
            return static_cast<const char*>(x) + (batch * p.stride[i][0] + at * p.stride[i][1] + head * p.stride[i][2]) * 2;
        };
        const char *a = row_of(of_v ? p.v : p.dout, of_v ? 2 : 0), *b = of_v ? nullptr : row_of(p.out, 1);
        for (int c = part * 8; c < p.dim; c += 64) {
            float x[8], y[8];
            unpack8<Fmt>(*reinterpret_cast<const uint4*>(a + 2 * c), x);
            if (!of_v) unpack8<Fmt>(*reinterpret_cast<const uint4*>(b + 2 * c), y);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (!of_v) dot = __fmaf_rn(x[e], y[e], dot);
                if constexpr (kNorms) square = __fmaf_rn(x[e], x[e], square);
            }
        }
    }
#pragma unroll
    for (int o = 4; o; o >>= 1) {
        dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if constexpr (kNorms) square += __shfl_xor_sync(0xffffffffu, square, o);
    }
    if (live && !of_v && part == 0) {
        const int64_t i = ((int64_t)batch * heads + head) * p.seq + at;
        p.aux[i] = make_float2(p.lse[i] * kLog2e, dot);
    }
    if constexpr (kNorms) {
        const bool counts = live && square <= 3.4028235e38f &&
                            (!p.offsets || (at >= p.offsets[0] && at < p.offsets[p.sequences]));
        const unsigned most = __reduce_max_sync(0xffffffffu, counts ? __float_as_uint(sqrtf(square) * 1.0001f) : 0u);
        if ((threadIdx.x & 31) == 0 && most) atomicMax(p.norms + of_v, most);
    }
}

// ---------------------------------------------------------------- host
size_t padded(size_t bytes) { return (bytes + 255) / 256 * 256; }
size_t workspace_bytes_for(int64_t batch, int64_t seq, int64_t heads) {
    return 256 + padded((size_t)(batch * heads * seq) * sizeof(float2));      // norms, aux
}

template <class Fmt, int Blocks>
tb_status launch(const CUtensorMap (&m)[4], Args p, const Rows& r, const View (&grad)[3], int64_t batch, int64_t seq, cudaStream_t st) {
    using L = Layout<Blocks>;
    const void *a = reinterpret_cast<const void*>(&dkv_kernel<Fmt, Blocks>), *b = reinterpret_cast<const void*>(&dq_kernel<Fmt, Blocks>);
    if (resident_ctas_per_sm(a, kThreads, L::kBytes) < 1 || resident_ctas_per_sm(b, kThreads, L::kBytes) < 1) return TB_ERR_CUDA;
    int64_t ctas = r.ctas;
    if (std::is_same<Fmt, F16>::value) {
        if (cudaMemsetAsync(r.norms, 0, 2 * sizeof(unsigned), st) != cudaSuccess) return TB_ERR_CUDA;
        ctas += ceil_div(batch * seq * r.kv_heads, kRowThreads / 8);
    }
    if (launch_pdl(rows_kernel<Fmt>, dim3((unsigned)ctas), dim3(kRowThreads), 0, st, r) != cudaSuccess) return TB_ERR_CUDA;
    const int64_t slots = r.offsets ? slots_of(seq, r.sequences, kRows) : p.tiles * batch;
    auto gradient = [&](int i, const View& v, void** to) {
        *to = const_cast<char*>(v.p);
        for (int k = 0; k < 3; ++k) p.stride[i][k] = v.s[k];
    };
    gradient(0, grad[1], &p.grad0);
    gradient(1, grad[2], &p.grad1);
    if (launch_pdl(dkv_kernel<Fmt, Blocks>, dim3((unsigned)(slots * p.kv_heads)), dim3(kThreads), L::kBytes, st, m[0], m[1], m[2], m[3],
                   p) != cudaSuccess)
        return TB_ERR_CUDA;
    gradient(0, grad[0], &p.grad0);
    if (launch_pdl(dq_kernel<Fmt, Blocks>, dim3((unsigned)(slots * p.heads)), dim3(kThreads), L::kBytes, st, m[0], m[1], m[2], m[3], p) !=
        cudaSuccess)
        return TB_ERR_CUDA;
    return launch_status();
}

}  // namespace
}  // namespace tb

extern "C" tb_status tb_attention_bwd_workspace_size(int64_t batch, int64_t seq, int64_t heads_q, int64_t heads_k, int64_t head_dim,
                                                     tb_dtype dtype, size_t* bytes) {
    using namespace tb;
    if (!bytes || heads_q < 0 || heads_k < 0 || heads_q > (1 << 20) || heads_k > (1 << 20)) return TB_ERR_INVALID_VALUE;
    const tb_status s = check_call(batch, seq, head_dim, nullptr, 0, 1.f, dtype);
    if (s != TB_OK) return s;
    *bytes = 0;
    if (batch == 0 || seq == 0 || heads_q == 0) return TB_OK;
    if (heads_k == 0 || heads_q % heads_k) return TB_ERR_INVALID_VALUE;
    *bytes = workspace_bytes_for(batch, seq, heads_q);
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
    if (batch == 0 || seq == 0 || q->heads == 0) return TB_OK;
    if (k->heads == 0 || q->heads % k->heads || !lse) return TB_ERR_INVALID_VALUE;
    if (!aligned_to(lse, 4)) return TB_ERR_MISALIGNED;
    const int64_t rows = batch * seq * q->heads;
    const size_t need = workspace_bytes_for(batch, seq, q->heads);
    const Range sums = range_of(lse, rows, 4), starts = range_of(offsets, offsets ? sequences + 1 : 0, 8);
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 5; ++j)
            if (shares(grad[i], read[j], head_dim, 2)) return TB_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (shares(grad[i], grad[j], head_dim, 2)) return TB_ERR_ALIAS;
        const Range g = range_of_view(grad[i], head_dim);
        if (overlap(g, sums) || overlap(g, starts)) return TB_ERR_ALIAS;
    }
    if (!workspace || workspace_bytes < need) return TB_ERR_WORKSPACE;
    if (!aligned_to(workspace, 16)) return TB_ERR_MISALIGNED;
    const Range ws = range_of(workspace, (int64_t)need, 1);
    for (int i = 0; i < 5; ++i)
        if (overlap(ws, range_of_view(read[i], head_dim))) return TB_ERR_ALIAS;
    for (int i = 0; i < 3; ++i)
        if (overlap(ws, range_of_view(grad[i], head_dim))) return TB_ERR_ALIAS;
    if (overlap(ws, sums) || overlap(ws, starts)) return TB_ERR_ALIAS;
    if (offsets && sequences == 0) return TB_OK;
    const int64_t tiles = ceil_div(seq, kRows), slots = offsets ? slots_of(seq, sequences, kRows) : tiles * batch;
    if (slots > ((1ll << 31) - 1) / q->heads || rows > (1ll << 35)) return TB_ERR_INVALID_VALUE;
    const bool bf = dtype == TB_BF16;
    CUtensorMap m[4];
    for (int i = 0; i < 4; ++i)
        if (!make_heads_map(&m[i], *in[i], batch, seq, head_dim, bf)) return TB_ERR_CUDA;
    Args p{};
    if (!(p.err = device_error_word())) return TB_ERR_CUDA;
    unsigned char* mem = static_cast<unsigned char*>(workspace);
    p.tokens = Tokens{offsets, (int)sequences, (int)batch, (int)seq, p.err};
    p.heads = (int)q->heads, p.kv_heads = (int)k->heads, p.group = (int)(q->heads / k->heads), p.dim = (int)head_dim;
    p.tiles = (int)tiles;
    p.scale = scale, p.scale_log2 = scale * kLog2e;
    p.norms = reinterpret_cast<unsigned*>(mem);
    p.aux = reinterpret_cast<float2*>(mem + 256);
    p.wait_ns = kWaitLimitNs;
    Rows r{};
    const int of[3] = {3, 4, 2};
    const void** to[3] = {&r.dout, &r.out, &r.v};
    for (int i = 0; i < 3; ++i) {
        *to[i] = read[of[i]].p;
        for (int j = 0; j < 3; ++j) r.stride[i][j] = read[of[i]].s[j];
    }
    r.lse = lse, r.aux = const_cast<float2*>(p.aux), r.norms = const_cast<unsigned*>(p.norms);
    r.offsets = offsets, r.sequences = (int)sequences;
    r.batch = (int)batch, r.seq = (int)seq, r.heads = p.heads, r.kv_heads = p.kv_heads, r.dim = p.dim;
    r.ctas = ceil_div(rows, kRowThreads / 8);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (head_dim <= 64) return bf ? launch<BF16, 1>(m, p, r, grad, batch, seq, st) : launch<F16, 1>(m, p, r, grad, batch, seq, st);
    return bf ? launch<BF16, 2>(m, p, r, grad, batch, seq, st) : launch<F16, 2>(m, p, r, grad, batch, seq, st);
}
