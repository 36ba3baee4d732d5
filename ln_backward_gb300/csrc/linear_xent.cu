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
// (32 KB a stage, six stages), so a tile's operands cross from L2 once per pair.  Warp 0
// feeds the stages by TMA, warp 1 of the pair's first CTA issues the MMAs, warps 4..7 drain
// the accumulator -- of which there are two, 256 TMEM columns each, so that the epilogue of
// one tile runs under the MMAs of the next.  A thread of the epilogue owns one row of the
// tile: row sums need no shuffles.  Tiles are dealt statically to a persistent grid of one
// CTA per SM, in groups of kGroup row tiles that keep their rows of A in L2.
//
// The operands need no transposed copies: dH contracts over the vocabulary, along which W
// is not contiguous, and dW over the tokens, along which neither G nor H is; those operands
// are staged as 64-column boxes and described to the MMA as MN-major.
//
// dloss stays out of the 16-bit G: 1 / rows, the usual dloss, has a rounding of its own that
// every entry of G would share (bf16 1/7168 is 0.19% off, and dH and dW were).  dH takes it in
// fp32 in the epilogue; dW contracts over the rows, so there H is scaled beforehand, by
// dloss / max |dloss|, which is exactly 1 for a mean.  That copy also holds zeros for the rows
// that take no part, whatever their H is.
//
// Every mbarrier wait is bounded (about one second of %globaltimer); on expiry the device
// error word is set and the CTAs drain what they issued and return.
#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "tb_common.cuh"

namespace tb {
namespace {

enum Kind { kLse = 0, kGrad = 1, kDH = 2, kDW = 3 };

constexpr int kTile = 256;                   // rows and columns of a CTA pair's tile
constexpr int kHalf = 128;                   // of which one CTA stages and drains
constexpr int kStageK = 64;                  // contracted elements a stage: 128 bytes
constexpr int kStages = 6;
constexpr int kOperandBytes = kHalf * kStageK * 2;
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kThreads = 256;
constexpr int kEpiWarp = 4;                  // first of the four epilogue warps
constexpr int kSmem = kStages * kStageBytes + 1024 + 256;   // alignment, barriers
constexpr int kTmemCols = 512;               // two accumulators
constexpr int kGroup = 16;                   // row tiles walked together (see tile_at)
constexpr unsigned long long kWaitLimitNs = 1000000000ull;

// Bytes of G that one piece of the vocabulary may take, and the fewest columns of a piece.
constexpr int64_t kPieceBytes = 256ll << 20;
constexpr int64_t kMinPiece = 2048;
constexpr int64_t kLseRows = 16384;          // rows of one launch of the loss (workspace)
constexpr int kMaxSplits = 16;

// ---------------------------------------------------------------- PTX
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// The address of the same shared-memory offset in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_to(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t remote_bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote_bar)
                 : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ unsigned long long now_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __noinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, int* err) {
    const unsigned long long t0 = now_ns();
    for (uint32_t it = 1; it < (1u << 30); ++it) {
        if (mbar_try(bar, parity)) return true;
        if ((it & 63u) == 0 && now_ns() - t0 > kWaitLimitNs) break;
    }
    atomicExch(err, (int)TB_ERR_TIMEOUT);
    return false;
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, int* err) {
    return mbar_try(bar, parity) || mbar_wait_slow(bar, parity, err);
}
// A box of `map` at column x (a multiple of 64), row y into this CTA's shared memory,
// counted on the mbarrier of the pair's first CTA.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int y,
                                        uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// Shared-memory operand descriptor: 128-byte swizzle.  K-major: 8-row groups every 1,024
// bytes.  MN-major: 64-column blocks every 8,192 bytes (one box), 8-row groups along the
// contracted dimension every 1,024.
template <bool MnMajor>
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
    constexpr uint64_t lbo = MnMajor ? 8192 >> 4 : 1, sbo = 1024 >> 4;
    return (uint64_t)((addr & 0x3FFFF) >> 4) | (lbo << 16) | (sbo << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
// Arrives on the mbarrier at this offset in both CTAs when the MMAs issued so far are done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
        "%30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {   // 2 ulp, 0 below -126
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.44269504088896341f;

// ---------------------------------------------------------------- arguments
struct Product {
    int m_tiles, n_tiles, splits, k_stages;
    int rows, cols;           // of the result
    int b_base;               // kGrad, kDH: first vocabulary row of the piece
    int* err;
    // kLse, kGrad
    const int64_t* target;    // of this launch's rows
    int64_t ignore;
    int vocab;
    float2* part;             // kLse: [n_tiles][rows] maximum and sum
    float* target_logit;      // kLse: [rows]
    const float* lse;         // kGrad
    const float* weight;      // kDH: dloss by row, 0 where a row takes no part
    const float* top;         // kDW: the largest |dloss|
    void* g;                  // kGrad: [rows][ldg]
    int ldg;
    // kDH, kDW
    float* sums;              // kDH: [splits][rows][cols] fp32, NULL: one split, one piece
    int first, last;          // piece: starts the sums; writes the result
    void* out;                // [rows][cols] 16-bit
};

// fp16's G is held times 2^14, so that probabilities down to 2^-38 stay above its last step;
// the products undo it in fp32.  bf16 has fp32's range.
template <class Fmt>
constexpr float kGBits = std::is_same<Fmt, F16>::value ? 14.f : 0.f;
template <class Fmt>
constexpr float kGScale = std::is_same<Fmt, F16>::value ? 16384.f : 1.f;

// An element of dH; a row of weight 0 takes no part, whatever its sums are.
template <class Fmt>
__device__ __forceinline__ float weigh(float sum, float weight) {
    return weight == 0.f ? 0.f : sum * (1.f / kGScale<Fmt>) * weight;
}

// Row tiles in groups of kGroup, the group's tiles column by column: the pairs that run
// together share few column tiles and reuse the group's rows.
__device__ __forceinline__ void tile_at(const Product& p, int t, int* split, int* mt, int* nt) {
    const int per_split = p.m_tiles * p.n_tiles;
    *split = t / per_split;
    t -= *split * per_split;
    const int group = t / (kGroup * p.n_tiles), first = group * kGroup;
    const int height = min(kGroup, p.m_tiles - first);
    t -= group * kGroup * p.n_tiles;
    *nt = t / height;
    *mt = first + t - *nt * height;
}

template <class Fmt>
__device__ __forceinline__ void store16(typename Fmt::T* row, int col, int cols, bool vec,
                                        const float (&v)[32]) {
    if (vec && col + 32 <= cols) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = v[8 * i + e];
            *reinterpret_cast<uint4*>(row + col + 8 * i) = pack8<Fmt>(f);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (col + i < cols) row[col + i] = Fmt::from_f32(v[i]);
    }
}

// Folds 32 logits into a row's maximum m and sum s of exp(l - base(m)); base is 0 where the
// maximum is infinite, so that a logit of +inf gives lse = +inf and rows of -inf give -inf.
__device__ __forceinline__ float base_of(float m) { return isinf(m) ? 0.f : m; }

__device__ __forceinline__ void fold(float& m, float& s, float m2, float s2) {
    const float top = fmaxf(m, m2), b = base_of(top);
    const float x = s == 0.f ? 0.f : s * exp2_fast((base_of(m) - b) * kLog2e);
    const float y = s2 == 0.f ? 0.f : s2 * exp2_fast((base_of(m2) - b) * kLog2e);
    m = top;
    s = x + y;
}

// ---------------------------------------------------------------- the product
template <class Fmt, int K>
__global__ void __launch_bounds__(kThreads, 1)
product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
               const __grid_constant__ Product p) {
    using T = typename Fmt::T;
    constexpr bool kAMn = K == kDW, kBMn = K == kDH || K == kDW;
    extern __shared__ unsigned char raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
    const uint32_t stage0 = smem_addr(smem), bar0 = smem_addr(bars);
    const uint32_t full = bar0, empty = full + 8 * kStages, acc_full = empty + 8 * kStages,
                   acc_empty = acc_full + 16, drain = acc_empty + 16, slot = drain + 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, 8);      // four warps of each CTA
        }
        mbar_init(drain, 1);
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
    pdl_trigger();

    const int tiles = p.m_tiles * p.n_tiles * p.splits;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (warp == 0) {
        if (lane == 0) {
            const uint32_t leader_full = map_to(full, 0);
            int it = 0, failed = 0;
            for (int t = pair; t < tiles && !failed; t += pairs) {
                int split, mt, nt;
                tile_at(p, t, &split, &mt, &nt);
                const int k_lo = (int)((int64_t)split * p.k_stages / p.splits);
                const int k_hi = (int)((int64_t)(split + 1) * p.k_stages / p.splits);
                const int m0 = mt * kTile + (int)rank * kHalf, n0 = nt * kTile + (int)rank * kHalf;
                for (int k = k_lo; k < k_hi; ++k, ++it) {
                    const int s = it % kStages;
                    if (it >= kStages && !mbar_wait(empty + 8 * s, (it / kStages - 1) & 1, p.err)) {
                        failed = 1;
                        break;
                    }
                    if (rank == 0) mbar_expect(full + 8 * s, 2 * kStageBytes);
                    const uint32_t a = stage0 + s * kStageBytes, b = a + kOperandBytes;
                    const uint32_t bar = leader_full + 8 * s;
                    if constexpr (kAMn) {
                        tma_box(a, &map_a, m0, k * kStageK, bar);
                        tma_box(a + 8192, &map_a, m0 + 64, k * kStageK, bar);
                    } else {
                        tma_box(a, &map_a, k * kStageK, m0, bar);
                    }
                    const int base = K == kGrad || K == kDH ? p.b_base : 0;
                    if constexpr (kBMn) {
                        tma_box(b, &map_b, n0, base + k * kStageK, bar);
                        tma_box(b + 8192, &map_b, n0 + 64, base + k * kStageK, bar);
                    } else {
                        tma_box(b, &map_b, k * kStageK, base + n0, bar);
                    }
                }
            }
            if (failed && rank == 0)      // what both CTAs issued ends on these barriers
                for (int q = max(0, it - kStages); q < it; ++q)
                    mbar_wait(full + 8 * (q % kStages), (q / kStages) & 1, p.err);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            constexpr uint32_t fmt = std::is_same<Fmt, BF16>::value ? 1 : 0;
            constexpr uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)kAMn << 15) |
                                       ((uint32_t)kBMn << 16) | ((kTile / 8) << 17) | ((kTile / 16) << 24);
            // 16 contracted elements: 32 bytes of a K-major row, 16 rows of an MN-major box
            constexpr uint32_t step_a = kAMn ? 2048 : 32, step_b = kBMn ? 2048 : 32;
            int it = 0, n = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs, ++n) {
                const int split = t / (p.m_tiles * p.n_tiles);
                const int k_lo = (int)((int64_t)split * p.k_stages / p.splits);
                const int k_hi = (int)((int64_t)(split + 1) * p.k_stages / p.splits);
                const int buf = n & 1;
                if (n >= 2 && !mbar_wait(acc_empty + 8 * buf, (n / 2 - 1) & 1, p.err)) {
                    ok = false;
                    break;
                }
                tmem_fence_after();
                for (int k = k_lo; k < k_hi; ++k, ++it) {
                    const int s = it % kStages;
                    if (!mbar_wait(full + 8 * s, (it / kStages) & 1, p.err)) {
                        ok = false;
                        break;
                    }
                    tmem_fence_after();
                    const uint32_t a = stage0 + s * kStageBytes, b = a + kOperandBytes;
#pragma unroll
                    for (int j = 0; j < kStageK / 16; ++j)
                        mma_pair(tmem + buf * kTile, operand_desc<kAMn>(a + j * step_a),
                                 operand_desc<kBMn>(b + j * step_b), idesc, k > k_lo || j > 0);
                    mma_commit(empty + 8 * s);
                }
                if (ok) mma_commit(acc_full + 8 * buf);
            }
            if (!ok) {
                mma_commit(drain);
                mbar_wait(drain, 0, p.err);
            }
        }
    } else if (warp >= kEpiWarp) {
        const int quad = warp - kEpiWarp;             // TMEM lanes 32 quad .. 32 quad + 31
        const uint32_t leader_empty = map_to(acc_empty, 0);
        const float top_weight = K == kDW ? *p.top : 1.f;
        int n = 0;
        for (int t = pair; t < tiles; t += pairs, ++n) {
            int split, mt, nt;
            tile_at(p, t, &split, &mt, &nt);
            const int buf = n & 1;
            const int row = mt * kTile + (int)rank * kHalf + quad * 32 + lane;
            const bool live = row < p.rows;
            const int n0 = nt * kTile, width = min(kTile, p.cols - n0);
            const uint32_t acc = tmem + buf * kTile + ((uint32_t)(quad * 32) << 16);

            // what the row needs, on its way before the accumulator is done
            int hit = -1;                             // the target's column in this tile
            float lse2 = 0.f, weight = 0.f;
            if constexpr (K == kDH) {
                if (live) weight = p.weight[row];
            }
            if constexpr (K == kLse || K == kGrad) {
                if (live) {
                    const int64_t tg = p.target[row];
                    const bool counts = tg != p.ignore && tg >= 0 && tg < p.vocab;
                    const int64_t c = tg - (K == kGrad ? p.b_base : 0) - n0;
                    if (counts && c >= 0 && c < width) hit = (int)c;
                    if constexpr (K == kGrad) {
                        lse2 = p.lse[row] * kLog2e - kGBits<Fmt>;
                        weight = counts ? 1.f : 0.f;
                    }
                }
            }
            if (!__all_sync(0xffffffffu, mbar_wait(acc_full + 8 * buf, (n / 2) & 1, p.err))) break;
            tmem_fence_after();

            float m = __int_as_float(0xff800000), s = 0.f;
            for (int c = 0; c < width; c += 32) {
                float v[32];
                __syncwarp();
                tmem_load32(acc + c, v);
                if constexpr (K == kLse) {
                    if (c + 32 > width) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c + i >= width) v[i] = __int_as_float(0xff800000);
                    }
                    float top = v[0];
#pragma unroll
                    for (int i = 1; i < 32; ++i) top = fmaxf(top, v[i]);
                    const float b = base_of(top) * kLog2e;
                    float part = 0.f;
#pragma unroll
                    for (int i = 0; i < 32; ++i) part += exp2_fast(fmaf(v[i], kLog2e, -b));
                    fold(m, s, top, part);
                    if ((hit & ~31) == c) {           // (hit = -1: no chunk)
                        float x = v[0];
#pragma unroll
                        for (int i = 1; i < 32; ++i) x = c + i == hit ? v[i] : x;
                        p.target_logit[row] = x;
                    }
                } else if constexpr (K == kGrad) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float e = exp2_fast(fmaf(v[i], kLog2e, -lse2));
                        v[i] = c + i == hit ? e - kGScale<Fmt> : e;
                    }
                    if (weight == 0.f) {              // a row that takes no part
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = 0.f;
                    }
                    if (live)                         // ldg is a multiple of 64: whole vectors
                        store16<Fmt>(static_cast<T*>(p.g) + (int64_t)row * p.ldg, n0 + c, p.ldg, true, v);
                } else if constexpr (K == kDH) {
                    const int col = n0 + c;
                    if (p.sums) {
                        float* sum = p.sums + ((int64_t)split * p.rows + row) * p.cols + col;
                        const bool vec = c + 32 <= width && (p.cols & 3) == 0;
                        if (live && vec) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                                if (!p.first) o = *reinterpret_cast<float4*>(sum + 4 * i);
                                o.x += v[4 * i], o.y += v[4 * i + 1], o.z += v[4 * i + 2], o.w += v[4 * i + 3];
                                v[4 * i] = o.x, v[4 * i + 1] = o.y, v[4 * i + 2] = o.z, v[4 * i + 3] = o.w;
                                if (!p.last || p.splits > 1) *reinterpret_cast<float4*>(sum + 4 * i) = o;
                            }
                        } else if (live) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (c + i < width) {
                                    if (!p.first) v[i] += sum[i];
                                    if (!p.last || p.splits > 1) sum[i] = v[i];
                                }
                        }
                    }
                    if (live && p.last && p.splits == 1) {
                        T* out = static_cast<T*>(p.out);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = weigh<Fmt>(v[i], weight);
                        store16<Fmt>(out + (int64_t)row * p.cols, col, p.cols,
                                     (p.cols & 7) == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0, v);
                    }
                } else {
                    T* out = static_cast<T*>(p.out);
                    if (live) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = v[i] * (1.f / kGScale<Fmt>) * top_weight;
                        store16<Fmt>(out + (int64_t)row * p.cols, n0 + c, p.cols,
                                     (p.cols & 7) == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0, v);
                    }
                }
            }
            if constexpr (K == kLse) {
                if (live) p.part[(int64_t)nt * p.rows + row] = make_float2(m, s);
            }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(leader_empty + 8 * buf);
        }
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
// A row's parts, one per column tile, in a fixed order: 32 rows a CTA, eight lanes a row.
__global__ void __launch_bounds__(256)
join_kernel(const float2* part, const float* target_logit, const int64_t* target, int64_t ignore,
            int vocab, int rows, int n_tiles, float* loss, float* lse, int* err) {
    __shared__ float2 sh[8][32];
    const int row = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    float m = __int_as_float(0xff800000), s = 0.f;
    if (row < rows) {
#pragma unroll 4
        for (int t = w; t < n_tiles; t += 8) {
            const float2 q = part[(int64_t)t * rows + row];
            fold(m, s, q.x, q.y);
        }
    }
    sh[w][threadIdx.x & 31] = make_float2(m, s);
    __syncthreads();
    if (w == 0 && row < rows) {
        for (int i = 1; i < 8; ++i) fold(m, s, sh[i][threadIdx.x].x, sh[i][threadIdx.x].y);
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

// What the gradient needs of dloss: each row's weight (0 where it takes no part), the largest
// magnitude among them, and H with every row times its weight over that.  Each CTA finds the
// maximum by itself (rows * 12 bytes from L2), which saves a launch.
template <class Fmt>
__global__ void __launch_bounds__(256)
weigh_kernel(const float* dloss, const int64_t* target, int64_t ignore, int vocab, int64_t rows,
             const typename Fmt::T* H, int cols, int ld, typename Fmt::T* scaled, float* weight, float* top) {
    __shared__ float sh[8];
    pdl_wait();
    pdl_trigger();
    auto weight_of = [&](int64_t r) {
        const int64_t t = target[r];
        return t != ignore && t >= 0 && t < vocab ? dloss[r] : 0.f;
    };
    float m = 0.f;
#pragma unroll 4
    for (int64_t r = threadIdx.x; r < rows; r += 256) {
        const float w = weight_of(r);
        if (blockIdx.x == 0) weight[r] = w;
        if (fabsf(w) <= 3.4028235e38f) m = fmaxf(m, fabsf(w));   // neither infinite nor NaN
    }
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = m;
    __syncthreads();
    m = sh[0];
    for (int i = 1; i < 8; ++i) m = fmaxf(m, sh[i]);
    if (m == 0.f) m = 1.f;
    if (blockIdx.x == 0 && threadIdx.x == 0) *top = m;
    if (!scaled) return;
    if (cols == ld) {                 // whole 16-byte vectors
        const int per_row = ld / 8;
        const int64_t n = rows * per_row;
        for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
            const float w = weight_of(i / per_row);
            float f[8];
            unpack8<Fmt>(reinterpret_cast<const uint4*>(H)[i], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = w == 0.f ? 0.f : f[e] * (w / m);
            reinterpret_cast<uint4*>(scaled)[i] = pack8<Fmt>(f);
        }
    } else {
        const int64_t n = rows * ld;
        for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
            const int64_t r = i / ld;
            const int c = (int)(i - r * ld);
            const float w = weight_of(r);
            scaled[i] = Fmt::from_f32(c < cols && w != 0.f ? Fmt::to_f32(H[r * cols + c]) * (w / m) : 0.f);
        }
    }
}

// Sums the splits of dH and rounds once.
template <class Fmt>
__global__ void __launch_bounds__(256)
join_dh_kernel(const float* sums, int splits, int64_t n, int cols, const float* weight,
               typename Fmt::T* out) {
    pdl_wait();
    pdl_trigger();
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        float v = 0.f;
        for (int s = 0; s < splits; ++s) v += sums[s * n + i];
        out[i] = Fmt::from_f32(weigh<Fmt>(v, weight[i / cols]));
    }
}

// Rows padded with zeros to a multiple of eight elements: TMA wants strides of 16 bytes.
__global__ void __launch_bounds__(256)
pad_kernel(const uint16_t* in, uint16_t* out, int64_t rows, int cols, int ld) {
    pdl_wait();
    pdl_trigger();
    const int64_t n = rows * ld;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / ld;
        const int c = (int)(i - r * ld);
        out[i] = c < cols ? in[r * cols + c] : (uint16_t)0;
    }
}

// ---------------------------------------------------------------- host
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// A row-major 16-bit matrix, read in boxes of 64 columns by `box_rows` rows, swizzled over
// 128 bytes; what lies outside reads as zeros.
bool make_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_rows,
              bool bf16) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {(cuuint32_t)kStageK, (cuuint32_t)box_rows};
    const cuuint32_t ones[2] = {1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
              const_cast<void*>(p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class Fmt, int K>
tb_status launch_product(const CUtensorMap& a, const CUtensorMap& b, const Product& p, cudaStream_t st) {
    const void* kernel = reinterpret_cast<const void*>(&product_kernel<Fmt, K>);
    const int pairs = resident_clusters(kernel, kThreads, kSmem, 2);
    if (pairs < 1) return TB_ERR_CUDA;
    const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles * p.splits;
    const int64_t grid = 2 * std::min<int64_t>(tiles, pairs);
    if (launch_cluster(product_kernel<Fmt, K>, dim3((unsigned)grid), dim3(kThreads), kSmem, st, 2, a, b, p) !=
        cudaSuccess)
        return TB_ERR_CUDA;
    return launch_status();
}

// How a call of these sizes is cut up.
struct Cut {
    int64_t ld;               // padded row length of H and W (D where no copy is needed)
    bool pad;
    int64_t piece, pieces;    // gradient: columns of a piece of the vocabulary
    int64_t ldg;
    int splits;               // of dH's contraction
    // byte offsets into the workspace
    size_t off_h, off_w, off_scaled, off_weight, off_g, off_sums, off_top, off_part, off_logit, total;
};

// Parts of the vocabulary that dH's products are split into: as many as fill the machine
// when its tiles do not.  One more split saves a share of the contraction and costs one
// more pass over dH in fp32; the cost below counts both in stages (64 contracted elements
// of a tile, about 0.3 us).
int pick_splits(int64_t m_tiles, int64_t n_tiles, int64_t k_stages, int64_t pairs) {
    int best = 1;
    double least = 1e30;
    for (int s = 1; s <= kMaxSplits && s <= k_stages; ++s) {
        const double waves = (double)ceil_div(m_tiles * n_tiles * s, pairs);
        const double cost = waves * ((double)ceil_div(k_stages, s) + 8.0) + (s > 1 ? 12.0 + 2.0 * s : 0.0);
        if (cost < least * 0.97) least = cost, best = s;
    }
    return best;
}

Cut cut_call(int64_t n, int64_t d, int64_t v, bool bwd, int sms) {
    Cut c{};
    c.ld = round_up(d, 8);
    c.pad = c.ld != d;
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
        c.off_part = take((size_t)rows * ceil_div(v, kTile) * sizeof(float2));
        c.off_logit = take((size_t)rows * sizeof(float));
    } else {
        int64_t most = std::max(kMinPiece, kPieceBytes / (2 * std::max<int64_t>(n, 1)));
        most = std::max<int64_t>(kTile, most / kTile * kTile);
        c.pieces = ceil_div(v, most);
        c.piece = std::min(round_up(ceil_div(v, c.pieces), kTile), round_up(v, kTile));
        c.pieces = ceil_div(v, c.piece);
        c.ldg = c.piece;
        c.splits = pick_splits(ceil_div(n, kTile), ceil_div(d, kTile), c.piece / kStageK, sms / 2);
        c.off_g = take((size_t)n * c.ldg * 2);
        if (c.pieces > 1 || c.splits > 1) c.off_sums = take((size_t)c.splits * n * d * sizeof(float));
        c.off_scaled = take((size_t)n * c.ld * 2);
        c.off_weight = take((size_t)n * sizeof(float));
        c.off_top = take(sizeof(float));
    }
    c.total = at;
    return c;
}

constexpr int64_t kMaxSize = (1ll << 31) - 512;

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

tb_status pad_rows(const void* in, void* out, int64_t rows, int64_t cols, int64_t ld, int sms,
                   cudaStream_t st) {
    const int64_t grid = std::min<int64_t>(ceil_div(rows * ld, 256), (int64_t)sms * 8);
    return launch_pdl(pad_kernel, dim3((unsigned)grid), dim3(256), 0, st, static_cast<const uint16_t*>(in),
                      static_cast<uint16_t*>(out), rows, (int)cols, (int)ld) == cudaSuccess
               ? TB_OK
               : TB_ERR_CUDA;
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
        if (pad_rows(q.H, q.ws + c.off_h, q.n, q.d, c.ld, q.sms, q.st) != TB_OK ||
            pad_rows(q.W, q.ws + c.off_w, q.v, q.d, c.ld, q.sms, q.st) != TB_OK)
            return TB_ERR_CUDA;
        H = q.ws + c.off_h;
        W = q.ws + c.off_w;
    }
    CUtensorMap a, b;
    if (!make_map(&b, W, q.v, q.d, c.ld, kHalf, bf)) return TB_ERR_CUDA;
    for (int64_t r0 = 0; r0 < q.n; r0 += kLseRows) {
        const int64_t rows = std::min(kLseRows, q.n - r0);
        if (!make_map(&a, static_cast<const char*>(H) + r0 * c.ld * 2, rows, q.d, c.ld, kHalf, bf))
            return TB_ERR_CUDA;
        Product p{};
        p.m_tiles = (int)ceil_div(rows, kTile);
        p.n_tiles = (int)ceil_div(q.v, kTile);
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
        const tb_status s = launch_product<Fmt, kLse>(a, b, p, q.st);
        if (s != TB_OK) return s;
        if (launch_pdl(join_kernel, dim3((unsigned)ceil_div(rows, 32)), dim3(256), 0, q.st,
                       (const float2*)p.part, (const float*)p.target_logit, p.target, p.ignore, p.vocab,
                       p.rows, p.n_tiles, q.loss + r0, q.lse + r0, q.err) != cudaSuccess)
            return TB_ERR_CUDA;
    }
    return launch_status();
}

template <class Fmt>
tb_status run_grad(const Problem& q, const Cut& c) {
    constexpr bool bf = std::is_same<Fmt, BF16>::value;
    const void *H = q.H, *W = q.W;
    if (c.pad) {
        if (pad_rows(q.H, q.ws + c.off_h, q.n, q.d, c.ld, q.sms, q.st) != TB_OK ||
            pad_rows(q.W, q.ws + c.off_w, q.v, q.d, c.ld, q.sms, q.st) != TB_OK)
            return TB_ERR_CUDA;
        H = q.ws + c.off_h;
        W = q.ws + c.off_w;
    }
    float* weight = reinterpret_cast<float*>(q.ws + c.off_weight);
    float* top = reinterpret_cast<float*>(q.ws + c.off_top);
    using T = typename Fmt::T;
    T* scaled = reinterpret_cast<T*>(q.ws + c.off_scaled);
    const int64_t copy_ctas = q.dW ? ceil_div(q.n * c.ld, 256 * 8 * 4) : 1;
    if (launch_pdl(weigh_kernel<Fmt>, dim3((unsigned)std::min<int64_t>(copy_ctas, (int64_t)q.sms * 4)), dim3(256),
                   0, q.st, q.dloss, q.target, q.ignore, (int)q.v, q.n, static_cast<const T*>(q.H), (int)q.d,
                   (int)c.ld, q.dW ? scaled : (T*)nullptr, weight, top) != cudaSuccess)
        return TB_ERR_CUDA;
    void* g = q.ws + c.off_g;
    CUtensorMap h_rows, w_rows, h_cols, w_cols, g_rows, g_cols;
    if (!make_map(&h_rows, H, q.n, q.d, c.ld, kHalf, bf) || !make_map(&w_rows, W, q.v, q.d, c.ld, kHalf, bf) ||
        !make_map(&h_cols, scaled, q.n, q.d, c.ld, kStageK, bf) || !make_map(&w_cols, W, q.v, q.d, c.ld, kStageK, bf))
        return TB_ERR_CUDA;
    for (int64_t i = 0; i < c.pieces; ++i) {
        const int64_t v0 = i * c.piece, cols = std::min(c.piece, q.v - v0);
        Product p{};
        p.m_tiles = (int)ceil_div(q.n, kTile);
        p.n_tiles = (int)ceil_div(cols, kTile);
        p.splits = 1;
        p.k_stages = (int)ceil_div(q.d, kStageK);
        p.rows = (int)q.n;
        p.cols = (int)cols;
        p.b_base = (int)v0;
        p.err = q.err;
        p.target = q.target;
        p.ignore = q.ignore;
        p.vocab = (int)q.v;
        p.lse = q.lse_in;
        p.weight = weight;
        p.top = top;
        p.g = g;
        p.ldg = (int)c.ldg;
        tb_status s = launch_product<Fmt, kGrad>(h_rows, w_rows, p, q.st);
        if (s != TB_OK) return s;
        if (q.dH) {
            if (!make_map(&g_rows, g, q.n, cols, c.ldg, kHalf, bf)) return TB_ERR_CUDA;
            Product r = p;
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
            s = launch_product<Fmt, kDH>(g_rows, w_cols, r, q.st);
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
            r.out = static_cast<char*>(q.dW) + v0 * q.d * 2;
            s = launch_product<Fmt, kDW>(g_cols, h_cols, r, q.st);
            if (s != TB_OK) return s;
        }
    }
    if (q.dH && c.splits > 1) {
        const int64_t n = q.n * q.d, grid = std::min<int64_t>(ceil_div(n, 256), (int64_t)q.sms * 8);
        const int used = (int)std::min<int64_t>(c.splits, ceil_div(std::min(c.piece, q.v), kStageK));
        if (launch_pdl(join_dh_kernel<Fmt>, dim3((unsigned)grid), dim3(256), 0, q.st,
                       (const float*)(q.ws + c.off_sums), used, n, (int)q.d, (const float*)weight,
                       static_cast<T*>(q.dH)) != cudaSuccess)
            return TB_ERR_CUDA;
    }
    return launch_status();
}

}  // namespace
}  // namespace tb

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
    if (!aligned_to(H, 16) || !aligned_to(W, 16) || !aligned_to(targets, 8) || !aligned_to(loss, 4) ||
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
    if (!aligned_to(H, 16) || !aligned_to(W, 16) || !aligned_to(targets, 8) || !aligned_to(dloss, 4) ||
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
