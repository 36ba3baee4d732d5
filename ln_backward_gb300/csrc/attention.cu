// attention.cu -- causal attention over whole prompts.
//
//     s_ij = scale q_i . k_j for j <= i,  lse_i = log sum_j exp(s_ij),  out_i = sum_j exp(s_ij - lse_i) v_j
#include "attention.cuh"

namespace tb {
namespace {

constexpr int kPair = 2 * kRows;             // queries of a CTA: two tiles that share its keys
constexpr int kSoftmaxWarp = 4;              // first of eight: four for each tile
constexpr int kThreads = (kSoftmaxWarp + 8) * 32;

// A block's sum of P, above which a row's maximum is looked for again: far from fp16's end.
constexpr float kMost = 8192.f;

template <int Blocks>                        // of 64 columns of a head
struct Layout {
    static constexpr int kTileBytes = Blocks * kBox;
    static constexpr int kRing = Blocks == 1 ? 8 : 4;            // tiles of keys and values
    static constexpr int kOut = (2 + kRing) * kTileBytes;        // behind the queries and the ring
    static constexpr int kBars = kOut + 8 * kOutStage;
    static constexpr int kBytes = kBars + 1024 + 256;            // alignment, barriers
};

struct Args {
    Tokens tokens;
    int heads, group, dim;    // query heads, of which `group` share a key head
    int tiles;                // pairs of query tiles of a batch entry, without offsets
    float scale_log2;         // scale * log2(e)
    void* out;
    int64_t out_batch, out_seq, out_head;    // strides in elements
    float* lse;               // [batch][heads][seq]; NULL: not wanted
    int* err;
    unsigned long long wait_ns;
};

// What a CTA works on: the queries of tile `tile` (256 of them) and of the tile behind, of one head.
struct Item {
    Span span;
    int head;
    int blocks0, blocks1;     // of keys that the two tiles of 128 read; 0: no such tile
    __device__ __forceinline__ int blocks(int t) const { return t ? blocks1 : blocks0; }
};
__device__ __forceinline__ bool find_item(const Args& p, unsigned index, Item* it) {
    const unsigned heads = (unsigned)p.heads;
    it->head = (int)(index % heads);
    const unsigned slot = index / heads;
    if (p.tokens.offsets) {
        if (!find_tile(p.tokens, kPair, (int)slot, true, &it->span)) return false;
    } else {                  // the longest first, over all heads and batch entries
        const unsigned batch = (unsigned)p.tokens.batch;
        it->span = Span{(int)(slot % batch), 0, p.tokens.seq, p.tiles - 1 - (int)(slot / batch)};
    }
    const int left = it->span.len - it->span.tile * kPair;
    it->blocks0 = 2 * it->span.tile + 1;
    it->blocks1 = left > kRows ? 2 * it->span.tile + 2 : 0;
    return true;
}

// ---------------------------------------------------------------- the kernel
template <class Fmt, int Blocks>
__global__ void __launch_bounds__(kThreads, 1)
attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v, const __grid_constant__ Args p) {
    using L = Layout<Blocks>;
    using T = typename Fmt::T;
    constexpr bool kBf = std::is_same<Fmt, BF16>::value;
    extern __shared__ unsigned char raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t q0 = smem_addr(smem), ring0 = q0 + 2 * L::kTileBytes, bar0 = q0 + L::kBars;
    const uint32_t full = bar0, empty = full + 8 * L::kRing, q_full = empty + 8 * L::kRing, q_empty = q_full + 16,
                   s_full = q_empty + 16, p_full = s_full + 16, o_full = p_full + 16, o_empty = o_full + 16,
                   tail = o_empty + 16, drain = tail + 8, slot = drain + 8;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < L::kRing; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + 8 * i, 1);
            mbar_init(q_empty + 8 * i, 1);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(p_full + 8 * i, 4);
            mbar_init(o_full + 8 * i, 1);
            mbar_init(o_empty + 8 * i, 4);
        }
        mbar_init(tail, 1);
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) tmem_alloc_all(slot);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + (slot - q0));
    pdl_wait();
    asm volatile("fence.proxy.async;" ::: "memory");   // what earlier kernels stored, TMA reads
    pdl_trigger();

    // The tensor memory: scores of both tiles (their first half becomes P), then results.
    const uint32_t score = tmem, result = tmem + 2 * kRows;
    const int cols = (p.dim + 15) / 16 * 16;
    Item it;
    bool more = find_item(p, blockIdx.x, &it);

    if (warp == 0) {
        int n = 0, items = 0, tails = 0;     // tiles staged, items, tails mended
        bool ok = true;
        for (; more && ok; more = false, ++items) {
            const int blocks = max(it.blocks0, it.blocks1), kv_head = it.head / p.group;
            const int q_row = it.span.first + it.span.tile * kPair;
            for (int t = 0; t < 2; ++t) {
                if (!it.blocks(t)) continue;
                // (one item: the queries' place is free)
                if (elect_one()) {
                    mbar_expect(q_full + 8 * t, L::kTileBytes);
                    for (int b = 0; b < Blocks; ++b)
                        tma_tile(q0 + t * L::kTileBytes + b * kBox, &map_q, 64 * b, q_row + t * kRows, it.head, it.span.batch,
                                 q_full + 8 * t);
                }
                __syncwarp();
            }
            for (int i = 0; i < 2 * blocks && ok; ++i, ++n) {      // keys, values of the last block, then the one before
                const int s = n % L::kRing, block = blocks - 1 - i / 2;
                const bool values = i & 1;
                if (n >= L::kRing && !__all_sync(0xffffffffu, mbar_wait(empty + 8 * s, (n / L::kRing - 1) & 1, &p))) {
                    ok = false;
                    break;
                }
                const int rows = it.span.len - block * kRows;
                // Behind the sequence's end lie other tokens or nothing: P is 0 there, but 0 times what they
                // hold need not be.
                const bool mend = values && rows < kRows;
                const uint32_t at = ring0 + s * L::kTileBytes, bar = mend ? tail : full + 8 * s;
                if (elect_one()) {
                    mbar_expect(bar, L::kTileBytes);
                    for (int b = 0; b < Blocks; ++b)
                        tma_tile(at + b * kBox, values ? &map_v : &map_k, 64 * b, it.span.first + block * kRows, kv_head,
                                 it.span.batch, bar);
                }
                __syncwarp();
                if (mend) {
                    if (!__all_sync(0xffffffffu, mbar_wait<kEnd>(tail, tails & 1, &p))) ok = false;
                    ++tails;
                    clear_behind<Blocks>(smem + (at - q0), rows, lane);
                    if (lane == 0) mbar_arrive(full + 8 * s);
                }
            }
        }
        // The way out: the MMAs, then the loads that no MMA waited for.
        __syncwarp();
        mbar_wait<kEnd>(drain, 0, &p);
        if (items)
            for (int t = 0; t < 2; ++t)
                if (it.blocks(t)) mbar_wait<kEnd>(q_full + 8 * t, (items - 1) & 1, &p);
        for (int i = max(0, n - L::kRing); i < n; ++i) mbar_wait<kEnd>(full + 8 * (i % L::kRing), (i / L::kRing) & 1, &p);
    } else if (warp == 1) {
        const uint32_t by_rows = instruction(kBf, kRows, false), by_cols = instruction(kBf, cols, true);
        const int steps = cols / 16;
        int n = 0, items = 0;                // tiles of the ring taken
        int have[2] = {0, 0};                // P taken
        bool ok = true;
        for (; more && ok; more = false, ++items) {
            const int blocks = max(it.blocks0, it.blocks1);
            // block i from the end is read by a tile when it is not behind the tile's last
            auto reads = [&](int t, int i) { return it.blocks(t) && i < blocks && blocks - 1 - i < it.blocks(t); };
            auto scores = [&](int t, int place) {
                if (elect_one()) {
                    product_by_rows<Blocks>(score + t * kRows, tile_desc(q0 + t * L::kTileBytes, false),
                                            tile_desc(ring0 + place * L::kTileBytes, false), steps, by_rows);
                    mma_done(s_full + 8 * t);
                }
                __syncwarp();
            };
            auto wait_ring = [&](int i) { return __all_sync(0xffffffffu, mbar_wait(full + 8 * (i % L::kRing), (i / L::kRing) & 1, &p)); };
            for (int t = 0; t < 2 && ok; ++t)
                if (it.blocks(t)) ok = __all_sync(0xffffffffu, mbar_wait(q_full + 8 * t, items & 1, &p));
            if (!ok || !wait_ring(n)) break;
            for (int t = 0; t < 2; ++t)
                if (reads(t, 0)) scores(t, n % L::kRing);
            if (elect_one()) mma_done(empty + 8 * (n % L::kRing));
            __syncwarp();
            for (int i = 0; i < blocks && ok; ++i) {
                const int value = n + 1 + 2 * i, key = value + 1;
                if (!wait_ring(value) || (i + 1 < blocks && !wait_ring(key))) {
                    ok = false;
                    break;
                }
                for (int t = 0; t < 2; ++t) {
                    if (reads(t, i)) {
                        if (!__all_sync(0xffffffffu, mbar_wait(p_full + 8 * t, have[t] & 1, &p))) {
                            ok = false;
                            break;
                        }
                        ++have[t];
                        tmem_fence_after();
                        const bool first = i == 0 || !reads(t, i - 1);
                        if (elect_one()) {
                            product_over_tokens(result + t * kRows, score + t * kRows, kRows / 4,
                                                tile_desc(ring0 + value % L::kRing * L::kTileBytes, true), by_cols, !first);
                            if (i + 1 == blocks) mma_done(o_full + 8 * t);
                        }
                        __syncwarp();
                    }
                    if (reads(t, i + 1)) scores(t, key % L::kRing);
                }
                if (!ok) break;
                if (elect_one()) {
                    mma_done(empty + 8 * (value % L::kRing));
                    if (i + 1 < blocks) mma_done(empty + 8 * (key % L::kRing));
                }
                __syncwarp();
            }
            n += 2 * blocks;
        }
        if (elect_one()) mma_done(drain);
    } else if (warp >= kSoftmaxWarp) {
        const int t = (warp - kSoftmaxWarp) >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t mine = score + t * kRows + lanes, sum = result + t * kRows + lanes;
        const unsigned long long c2 = pair_of(p.scale_log2, p.scale_log2);
        int have = 0, items = 0;
        bool ok = true;
        for (; more && ok && it.blocks(t); more = false, ++items) {
            float base = 0.f;                // P is 2^(score * scale_log2 - base)
            unsigned long long total = 0;
            for (int i = 0; i < it.blocks(t); ++i, ++have) {
                if (!__all_sync(0xffffffffu, mbar_wait(s_full + 8 * t, have & 1, &p))) {
                    ok = false;
                    break;
                }
                tmem_fence_after();
                uint32_t a[32], b[32], w[4][16];
                unsigned long long sums[2];
                // 32 columns from g * 32 on: P, and its sum
                auto powers = [&](const uint32_t (&x)[32], int g) {
                    const unsigned long long b2 = pair_of(-base, -base);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float lo, hi;
                        split_pair(fma_pair(pair_of(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), c2, b2), lo, hi);
                        lo = exp2_fast(lo);
                        hi = exp2_fast(hi);
                        sums[e & 1] = add_pair(sums[e & 1], pair_of(lo, hi));
                        w[g][e] = pack2<Fmt>(lo, hi);
                    }
                };
                auto hide = [&](uint32_t (&x)[32], int from) {       // tokens behind the row's own
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = from + e > row ? 0xff800000u : x[e];
                };
                auto all_powers = [&](bool own) {                    // the next columns come meanwhile
                    sums[0] = sums[1] = 0;
                    tmem_load32(mine, a);
                    tmem_load32(mine + 32, b);
                    tmem_wait(a);
                    if (own) hide(a, 0);
                    powers(a, 0);
                    tmem_wait(b);
                    tmem_load32(mine + 64, a);
                    if (own) hide(b, 32);
                    powers(b, 1);
                    tmem_wait(a);
                    tmem_load32(mine + 96, b);
                    if (own) hide(a, 64);
                    powers(a, 2);
                    tmem_wait(b);
                    if (own) hide(b, 96);
                    powers(b, 3);
                };
                auto highest = [&](bool own) {
                    float m4[4] = {__int_as_float(0xff800000), __int_as_float(0xff800000), __int_as_float(0xff800000), __int_as_float(0xff800000)};
                    for (int x = 0; x < kRows; x += 32) {
                        tmem_load32(mine + x, a);
                        tmem_wait(a);
                        if (own) hide(a, x);
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            m4[e / 2 & 3] = fmaxf(m4[e / 2 & 3], fmaxf(__uint_as_float(a[e]), __uint_as_float(a[e + 1])));
                    }
                    return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                };
                if (i == 0) {                // the block of the tile's own tokens
                    const float m = highest(true);
                    base = m == __int_as_float(0xff800000) ? 0.f : m * p.scale_log2;
                    all_powers(true);
                } else {
                    // P against what it was taken against before; where a row's sum shows that it grew beyond
                    // kMost, everything is taken against the new maximum.
                    all_powers(false);
                    float lo, hi;
                    split_pair(add_pair(sums[0], sums[1]), lo, hi);
                    const bool grew = !(lo + hi <= kMost);       // (one row's growth leaves the others as they are)
                    if (__any_sync(0xffffffffu, grew)) {
                        const float most = highest(false) * p.scale_log2, next = grew ? fmaxf(base, most) : base,
                                    f = exp2_fast(base - next);
                        base = next;
                        total = mul_pair(total, pair_of(f, f));
                        for (int x = 0; x < cols; x += 16) {
                            uint32_t o[16];
                            tmem_read16(sum + x, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_store16(sum + x, o);
                        }
                        all_powers(false);
                    }
                }
                total = add_pair(total, add_pair(sums[0], sums[1]));
#pragma unroll
                for (int g = 0; g < 4; ++g) tmem_store16(mine + 16 * g, w[g]);       // over scores that are done with
                tmem_stored();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * t);
            }
            if (!ok) break;
            float l0, l1;
            split_pair(total, l0, l1);
            const float l = l0 + l1, inv = 1.f / l;
            if (!__all_sync(0xffffffffu, mbar_wait(o_full + 8 * t, items & 1, &p))) break;
            tmem_fence_after();
            const int in_seq = it.span.tile * kPair + t * kRows + quad * 32, rows = min(32, it.span.len - in_seq);
            const int64_t token = it.span.first + in_seq;
            if (p.lse && lane < rows)
                p.lse[((int64_t)it.span.batch * p.heads + it.head) * p.tokens.seq + token + lane] =
                    0.693147180559945309f * (base + log2f(l));
            T* out = static_cast<T*>(p.out) + it.span.batch * p.out_batch + token * p.out_seq + it.head * p.out_head;
            unsigned char* box = smem + L::kOut + (warp - kSoftmaxWarp) * kOutStage;
            store_rows<Fmt>(box, sum, inv, out, p.out_seq, rows, p.dim, lane);
        }
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    if (warp == 2) tmem_free_all(tmem);
}

// ---------------------------------------------------------------- host
template <class Fmt, int Blocks>
tb_status launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const Args& p, int64_t items, cudaStream_t st) {
    using L = Layout<Blocks>;
    if (resident_ctas_per_sm(reinterpret_cast<const void*>(&attention_kernel<Fmt, Blocks>), kThreads, L::kBytes) < 1) return TB_ERR_CUDA;
    return launch_pdl(attention_kernel<Fmt, Blocks>, dim3((unsigned)items), dim3(kThreads), L::kBytes, st, q, k, v, p) == cudaSuccess
               ? launch_status()
               : TB_ERR_CUDA;
}

}  // namespace
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
    const int64_t tiles = ceil_div(seq, kPair), slots = offsets ? slots_of(seq, sequences, kPair) : tiles * batch;
    if (slots > ((1ll << 31) - 1) / q->heads) return TB_ERR_INVALID_VALUE;
    const bool bf = dtype == TB_BF16;
    CUtensorMap maps[3];
    for (int i = 0; i < 3; ++i)
        if (!make_heads_map(&maps[i], *given[i], batch, seq, head_dim, bf)) return TB_ERR_CUDA;
    Args p{};
    if (!(p.err = device_error_word())) return TB_ERR_CUDA;
    p.tokens = Tokens{offsets, (int)sequences, (int)batch, (int)seq, p.err};
    p.heads = (int)q->heads, p.group = (int)(q->heads / k->heads), p.dim = (int)head_dim;
    p.tiles = (int)tiles;
    p.scale_log2 = scale * kLog2e;
    p.out = out->data;
    p.out_batch = view[3].s[0], p.out_seq = view[3].s[1], p.out_head = view[3].s[2];
    p.lse = lse;
    p.wait_ns = kWaitLimitNs;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t items = slots * q->heads;
    if (head_dim <= 64) return bf ? launch<BF16, 1>(maps[0], maps[1], maps[2], p, items, st) : launch<F16, 1>(maps[0], maps[1], maps[2], p, items, st);
    return bf ? launch<BF16, 2>(maps[0], maps[1], maps[2], p, items, st) : launch<F16, 2>(maps[0], maps[1], maps[2], p, items, st);
}
