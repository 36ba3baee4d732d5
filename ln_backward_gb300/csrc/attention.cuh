// attention.cuh -- what the kernels of causal attention share: the sequences of a call, tcgen05
// products of a pair of CTAs with the first operand in shared or tensor memory, and loads by TMA.
#pragma once

#include "heads_view.cuh"
#include "tensor_core.cuh"

namespace tb {
namespace {

constexpr int kRows = 128;                   // queries or keys of a CTA's tile: TMEM's lanes
constexpr int kSpan = 2 * kRows;             // of a pair of CTAs
constexpr int kBox = kRows * 64 * 2;         // 64 columns of a tile, swizzled over 128 bytes
constexpr int kHalfBox = kBox / 2;           // and of half its rows

// A pair of CTAs (a cluster of two SMs) works on 256 rows, 128 each, against tiles of 128 tokens that both need.
// tcgen05.mma.cta_group::2 takes each CTA's rows from its own shared or tensor memory and half of the other
// operand from either: the operands' way through shared memory, 128 bytes a clock, would bound products of one
// CTA (128 x 128 x 16: 64 clocks of MMA, 64 of reading both operands, and the next tiles come in beside).

// What a self-test leaves out, so that waits run out: the loads of the pair's first or second CTA, or the last
// arrival that says that scores (and dP) are complete, that P (and dS) is there, that results are complete.
enum Withheld { kNothing = 0, kLoads0 = 1, kLoads1 = 2, kScores = 3, kTaken = 4, kResults = 5 };

// ---------------------------------------------------------------- PTX
// Hands shared memory that this CTA's threads wrote to the pair's first CTA.  (What lies in tensor memory is handed
// over between tcgen05 fences by mbar_arrive_cluster: a release waits about 900 clocks.)
__device__ __forceinline__ void mbar_arrive_release(uint32_t remote_bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote_bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect_at(uint32_t remote_bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(remote_bar), "r"(bytes) : "memory");
}
// A box of 64 columns from x on of the map's number of rows from y on of one head of one batch entry; zeros
// outside the tensor.  Counted on an mbarrier of either CTA.
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, int x, int y, int head, int batch, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(head), "r"(batch), "r"(bar)
        : "memory");
}
// Instruction descriptor of 256 rows by `cols`; b_mn: the second operand's rows are contracted.
__host__ __device__ constexpr uint32_t instruction(bool bf16, int cols, bool b_mn) {
    return (1u << 4) | ((uint32_t)bf16 << 7) | ((uint32_t)bf16 << 10) | ((uint32_t)b_mn << 16) | ((uint32_t)(cols / 8) << 17) |
           ((uint32_t)(kSpan / 16) << 24);
}
// 16 contracted elements, the first operand 16-bit pairs in tensor memory.  Add: onto what d holds; otherwise `add`
// says whether.
template <bool Add>
__device__ __forceinline__ void mma_pair_tmem(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add = 1) {
    if constexpr (Add)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.eq.u32 p, 0, 0;\n\t"
            "mov.b64 y, {%2, %4};\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(idesc), "r"(kDescHigh)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.u32 p, %5, 0;\n\t"
            "mov.b64 y, {%2, %4};\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(idesc), "r"(kDescHigh), "r"(add)
            : "memory");
}
// 256 rows against 128 over `steps` times 16 of a head's elements.  a: 128 rows of each CTA, b: 64, by the addresses
// of their first boxes.  One thread issues all MMAs, each of 64 clocks: no loop where the head is whole.
template <int Blocks>
__device__ __forceinline__ void product_by_rows(uint32_t d, uint32_t a_tile, uint32_t b_tile, int steps, uint32_t idesc) {
    const uint32_t a = desc_low<false>(a_tile), b = desc_low<false>(b_tile);
    mma_pair<false>(d, a, b, idesc, 0);
    if (steps == 4 * Blocks) {
#pragma unroll
        for (int k = 1; k < 4 * Blocks; ++k)
            mma_pair<true>(d, a + (k < 4 ? 0 : kBox >> 4) + k % 4 * 2, b + (k < 4 ? 0 : kHalfBox >> 4) + k % 4 * 2, idesc, 1);
    } else {
        for (int k = 1; k < steps; ++k)
            mma_pair<true>(d, a + (k < 4 ? 0 : kBox >> 4) + k % 4 * 2, b + (k < 4 ? 0 : kHalfBox >> 4) + k % 4 * 2, idesc, 1);
    }
}
// d (+)= A B over the 128 tokens of B's rows, of which each CTA has half the columns.  A lies in tensor memory,
// 64 tokens (32 columns) and the others `apart` columns behind.
__device__ __forceinline__ void product_over_tokens(uint32_t d, uint32_t a, uint32_t apart, uint32_t b_tile, uint32_t idesc, bool add) {
    const uint32_t b = desc_low<true>(b_tile);
    mma_pair_tmem<false>(d, a, b, idesc, add);
#pragma unroll
    for (int k = 1; k < kRows / 16; ++k) mma_pair_tmem<true>(d, a + (k < 4 ? 8 * k : apart + 8 * (k - 4)), b + k * (2048 >> 4), idesc);
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
        "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
        "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
        "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
        : "memory");
}
// A quarter of the lanes' 16 (those of `addr`) by 64 columns, as a matrix instruction's accumulator lies in a warp:
// r[4 k + 2 h + b] is row lane / 4 + 8 h, column 8 k + lane % 4 * 2 + b.  There after tmem_wait.
__device__ __forceinline__ void tmem_load_16x64(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
        "%30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
// The same 16 rows by 64 columns as 16-bit pairs, 32 columns: r[2 k + h] is row lane / 4 + 8 h, columns 8 k +
// lane % 4 * 2 and the one behind.
__device__ __forceinline__ void tmem_store_16x64(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_alloc_all(uint32_t slot) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_all(uint32_t tmem) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}
__device__ __forceinline__ unsigned long long mul_pair(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// Two values as 16-bit pairs lie in TMEM and in registers: the first in the low half.  (Volatile: it stays where it is
// written.  Sunk behind a branch to where the pairs are stored, it keeps twice the registers alive.)
template <class Fmt>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if constexpr (std::is_same<Fmt, BF16>::value) asm volatile("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm volatile("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Where a result's rows go: by TMA in boxes of 32 columns by 32 rows, or, where fewer rows are a sequence's, one by one.
struct Place {
    const CUtensorMap* map;
    void* data;               // of the warp's first row
    int64_t stride;           // from one row to the next, in elements
    int token, head, batch;   // of that row
};
// Columns from .. dim - 1 of 32 rows of a result from tensor memory, a row a lane, times the lane's factor and rounded,
// to the first `rows` rows of `to`, through the warp's two boxes of shared memory, in turn.  Of stores before the call any
// may still read either box: they are waited for, which costs nothing, as a piece of work lies between.  A lane's 16-byte pieces lie at piece ^ (row / 2 & 3), the
// pattern of a 64-byte swizzle: no two lanes of a quarter warp share banks.  Arrives on `free` when the last columns
// are in registers.  (Stores from registers held the warps up for the time that the memory took: 4,000 clocks for
// 64 KB of every CTA at once.)
constexpr int kOutBox = 32 * 64, kOutStage = 2 * kOutBox;
template <class Fmt>
__device__ __forceinline__ void store_rows(unsigned char* boxes, uint32_t tmem, float factor, const Place& to, int rows, int from,
                                           int dim, int lane, uint32_t free) {
    for (int x = from; x < dim; x += 32) {
        unsigned char* box = boxes + (x & 32 ? kOutBox : 0);
        uint32_t o[32];
        tmem_load32(tmem + x, o);
        if (lane == 0) {         // the box is free
            if (x == from) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            else asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        }
        tmem_wait(o);
        __syncwarp();
        if (x + 32 >= dim) {
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(free);
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                h[e] = pack2<Fmt>(__uint_as_float(o[8 * g + 2 * e]) * factor, __uint_as_float(o[8 * g + 2 * e + 1]) * factor);
            *reinterpret_cast<uint4*>(box + lane * 64 + ((g ^ (lane / 2 & 3)) * 16)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
        if (rows >= 32) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(to.map),
                             "r"(x), "r"(to.token), "r"(to.head), "r"(to.batch), "r"(smem_addr(box))
                             : "memory");
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
        } else {
            __syncwarp();
            const int c = lane & 3;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int y = lane / 4 + 8 * i;
                if (y < rows && x + 8 * c < dim)
                    *reinterpret_cast<uint4*>(static_cast<typename Fmt::T*>(to.data) + y * to.stride + x + 8 * c) =
                        *reinterpret_cast<const uint4*>(box + y * 64 + ((c ^ (y / 2 & 3)) * 16));
            }
            __syncwarp();
        }
    }
}
__device__ __forceinline__ void stored_all(int lane) {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// Rows from `rows` on of `boxes` boxes as zeros: whatever lies behind a sequence's end need not be 0 times 0.  By
// a whole warp, which waits for the tile's loads and hands it to the MMAs; another than the one that loads, which
// goes on meanwhile.
__device__ __forceinline__ void clear_behind(unsigned char* tile, int boxes, int box_rows, int rows, int lane) {
    for (int b = 0; b < boxes; ++b)
        for (int x = max(rows, 0) * 8 + lane; x < box_rows * 8; x += 32)
            *reinterpret_cast<uint4*>(tile + (b * box_rows * 8 + x) * 16) = make_uint4(0, 0, 0, 0);
}
// Behind it, before the arrivals: what the warp wrote is there for the MMAs of either CTA.  (One release for all
// arrivals, each of which would wait about 900 clocks for its own.)
__device__ __forceinline__ void cleared(int lane) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) asm volatile("fence.acq_rel.cluster;" ::: "memory");
}

__device__ __forceinline__ int load_shared(uint32_t at) {
    int x;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
    return x;
}
// Waits until tail number `loaded` is mended or the mending warp has stopped: then `mended` may be two phases further,
// and a wait for that one's parity would not see it.
template <class P>
__device__ __noinline__ bool tail_settled(uint32_t mended, uint32_t stopped, int loaded, unsigned long long limit, const P* p) {
    const unsigned long long t0 = now_ns();
    for (uint32_t it = 1; it < (1u << 30); ++it) {
        if (load_shared(stopped) || mbar_try<true>(mended, (loaded - 1) & 1)) return true;
        if ((it & 63u) == 0 && now_ns() - t0 > limit) break;
    }
    atomicExch(p->err, (int)TB_ERR_TIMEOUT);
    return false;
}
// A tile that ends with its sequence is counted on its CTA's own barrier (`tail`) while the mending warp clears what
// lies behind, one at a time; that warp then arrives in the loading warp's place, and on `mended`.  Where its wait gave up it
// leaves the number of the tile, counted from 1, that it mends no more, and ends that one's phase of `mended`: the loading
// warp loads no other, and on its way out arrives itself for the one that it may have loaded meanwhile, behind its bytes.
struct Tails {
    uint32_t tail, mended;
    uint32_t stopped;         // a word, 0 at first
    __device__ __forceinline__ void stop(int number, int lane) const {     // by the mending warp, once
        if (lane == 0) {
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(stopped), "r"(number) : "memory");
            mbar_arrive(mended);
        }
        __syncwarp();
    }
    // Before the loading warp's tail number `loaded` + 1.
    template <class P>
    __device__ __forceinline__ bool next(int loaded, const P* p) const {
        return (!loaded || __all_sync(0xffffffffu, mbar_wait(mended, (loaded - 1) & 1, p))) && __all_sync(0xffffffffu, load_shared(stopped) == 0);
    }
    // On its way out: whether it has to arrive for the last one.
    template <class P>
    __device__ __forceinline__ bool left_over(int loaded, const P* p) const {
        return loaded && __all_sync(0xffffffffu, mbar_wait<kEnd>(tail, (loaded - 1) & 1, p)) &&
               __all_sync(0xffffffffu, tail_settled(mended, stopped, loaded, 4 * kWaitLimitNs, p)) && __all_sync(0xffffffffu, load_shared(stopped) == loaded);
    }
};

// ---------------------------------------------------------------- work
// A pair stays on its SMs: its first CTA asks for the next cluster of the grid that has not started, whose work
// the pair then does.  (A cluster's launch, set-up and first loads take longer than short tiles.)  Both CTAs get the
// answer, one at a time: each warp that needs it reads it and says so, then the first CTA asks again.  The answers
// come to the clusters as they get done, so uneven sequences even out.  A warp whose wait gave up reads on without
// working, so that the others come to their end.
struct Work {
    uint32_t answer, full, empty;    // 16 bytes, 16-byte aligned; barriers
    uint32_t parity;
};
__device__ __forceinline__ void init_work(uint32_t full, uint32_t empty, int readers) {   // warps of both CTAs that work
    mbar_init(full, 1);
    mbar_init(empty, readers + 1);                   // and the second CTA's that hands out
}
// By one warp of each CTA: asks until there is nothing left.
template <class P>
__device__ __forceinline__ void hand_out(const Work& w, uint32_t rank, const P* p) {
    for (uint32_t n = 0;; ++n) {
        if (elect_one()) {
            mbar_expect(w.full, 16);
        }
        __syncwarp();
        if (rank == 0) {
            if (n && !__all_sync(0xffffffffu, mbar_wait<kWork>(w.empty, (n - 1) & 1, p))) return;
            if (elect_one())
                asm volatile(
                    "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.multicast::cluster::all.b128"
                    " [%0], [%1];" ::"r"(w.answer),
                    "r"(w.full)
                    : "memory");
            __syncwarp();
        }
        if (!__all_sync(0xffffffffu, mbar_wait<kWork>(w.full, n & 1, p))) return;
        uint32_t more;
        asm volatile(
            "{\n\t.reg .b128 r;\n\t.reg .pred q;\n\tld.shared.b128 r, [%1];\n\t"
            "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 q, r;\n\tselp.u32 %0, 1, 0, q;\n\t}"
            : "=r"(more)
            : "r"(w.answer)
            : "memory");
        __syncwarp();
        if (rank == 1 && elect_one()) mbar_arrive_release(map_to(w.empty, 0));
        if (!more) return;
    }
}
// By every warp that works: the next cluster's number; false when there is none, or a wait gave up.
template <class P>
__device__ __forceinline__ bool next_work(Work& w, int lane, unsigned* cluster, const P* p) {
    if (!__all_sync(0xffffffffu, mbar_wait<kWork>(w.full, w.parity, p))) return false;
    w.parity ^= 1;
    uint32_t more, x = 0;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred q;\n\tld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 q, r;\n\tselp.u32 %0, 1, 0, q;\n\t"
        "mov.u32 %1, 0;\n\t@q clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
        : "=r"(more), "=r"(x)
        : "r"(w.answer)
        : "memory");
    // (the arrival names what was read, and so comes behind it)
    __syncwarp();
    if (lane == 0)
        asm volatile("{\n\t.reg .b32 t;\n\tand.b32 t, %1, 0;\n\tadd.u32 t, t, %0;\n\t"
                     "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [t];\n\t}" ::"r"(map_to(w.empty, 0)), "r"(x + more)
                     : "memory");
    *cluster = x >> 1;
    return more != 0;
}

// The way out of the warp that loads: the MMAs, which the first CTA issues, then the boxes, which end on the first
// CTA's barriers.  Each phase of those counts an arrival of either CTA.  After a wait that gave up one may have
// loaded what the other has not: the first CTA arrives in its place, so that every phase ends with its last box.
// `mine`: loads of this CTA by stream, bar_of(stream, i, &parity): the barrier of load i, rings: how many a stream
// has open at most.  `words`: the streams' counts of the second CTA, in the first one's shared memory.
template <int Streams, class P, class F>
__device__ __forceinline__ void way_out(uint32_t rank, const int (&mine)[Streams], const int (&rings)[Streams], uint32_t drain,
                                        uint32_t done, uint32_t words, const unsigned char* words_at, const P* p, F bar_of) {
    if (rank == 1 && elect_one()) {
#pragma unroll
        for (int s = 0; s < Streams; ++s)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to(words + 4 * s, 0)), "r"(mine[s]) : "memory");
        mbar_arrive_release(map_to(done, 0));
    }
    __syncwarp();
    const bool ended = __all_sync(0xffffffffu, mbar_wait<kWork>(drain, 0, p));
    if (rank != 0 || !ended || !__all_sync(0xffffffffu, mbar_wait<kEnd>(done, 0, p))) return;
#pragma unroll
    for (int s = 0; s < Streams; ++s) {
        const int peer = reinterpret_cast<const volatile int*>(words_at)[s], all = max(mine[s], peer);
        uint32_t parity;
        if (elect_one())
            for (int i = min(mine[s], peer); i < all; ++i) mbar_arrive(bar_of(s, i, &parity));
        __syncwarp();
        for (int i = max(0, all - rings[s]); i < all; ++i) {
            const uint32_t bar = bar_of(s, i, &parity);
            mbar_wait<kEnd>(bar, parity, p);
        }
    }
}

// ---------------------------------------------------------------- sequences
// The tokens of a call: `batch` rows of `seq` tokens.  With offsets, sequences packed into the one row:
// number i is tokens offsets[i] .. offsets[i + 1] - 1.
struct Tokens {
    const int64_t* offsets;   // NULL: every batch entry is a sequence
    int sequences, batch, seq;
    int* err;
};
// A tile of one sequence.  Its tokens are first .. first + len - 1 of its batch entry.
struct Span {
    int batch, first, len, tile;
};

// A call's tiles of `size` tokens are dealt out by slots, at least as many as there are tiles.
__host__ __device__ inline int64_t slots_of(int64_t tokens, int64_t sequences, int size) { return tokens / size + sequences; }

// The tile in a slot, by a whole warp; false: none.  Tiles are the longer to work on the further they lie from one end
// of their sequence, the first one (from_last false: a query's keys begin there) or the last.  Sorted, and of up to
// kSorted sequences: those that take longest are in the first slots, over all sequences, so that the pairs' work ends
// together.  (The gradient of 8,192 tokens in 11 sequences, 32 heads of 128 over 8: 463 us unsorted, 452 sorted.)
// Otherwise sequence after sequence, the longest tiles of each first, numbered so that a sequence is found without
// adding up the lengths before it: sequence i's slots are floor(offsets[i] / size) + i and on, as floor((o + n) / size) -
// floor(o / size) + 1 is at least ceil(n / size).
// Offsets that do not count up within the row are cut to it: tiles stay inside, whatever they share or miss.  check_offsets
// reports them in the device error word, of sequence i, tiles or none.
__device__ __forceinline__ void check_offsets(const int64_t* offsets, int64_t i, int seq, int* err) {
    const int64_t a = __ldcg((const long long*)offsets + i), b = __ldcg((const long long*)offsets + i + 1);
    if (a < 0 || b < a || b > seq) atomicExch(err, (int)TB_ERR_INVALID_VALUE);
}
constexpr int kSorted = 128;
template <bool Sorted>
__device__ __forceinline__ bool find_tile(const Tokens& t, int size, int slot, bool from_last, Span* s) {
    const int lane = threadIdx.x & 31;
    // (from L2: dq_kernel starts before the kernel in front of it has ended)
    auto offset = [&](int i) { return (int)min(max((int64_t)__ldcg((const long long*)t.offsets + i), (int64_t)0), (int64_t)t.seq); };
    auto tiles_of = [&](int i) { return (max(offset(i + 1) - offset(i), 0) + size - 1) / size; };
    int seq, far;                        // the sequence, and how far from the end the tile lies
    if (Sorted && t.sequences <= kSorted) {
        int n[kSorted / 32];
#pragma unroll
        for (int i = 0; i < kSorted / 32; ++i) n[i] = 32 * i + lane < t.sequences ? tiles_of(32 * i + lane) : 0;
        auto as_far = [&](int d) {       // tiles at least that far away
            int c = 0;
#pragma unroll
            for (int i = 0; i < kSorted / 32; ++i) c += max(n[i] - d, 0);
            return (int)__reduce_add_sync(0xffffffffu, (unsigned)c);
        };
        if (slot >= as_far(0)) return false;
        int most = 0;
#pragma unroll
        for (int i = 0; i < kSorted / 32; ++i) most = max(most, n[i]);
        int lo = 0, hi = (int)__reduce_max_sync(0xffffffffu, (unsigned)most);    // as_far(lo) > slot >= as_far(hi)
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (as_far(mid) > slot) lo = mid;
            else hi = mid;
        }
        int k = slot - as_far(lo + 1);   // of the sequences that have one there
        far = lo;
        seq = 0;
#pragma unroll
        for (int i = 0; i < kSorted / 32; ++i) {
            const unsigned has = __ballot_sync(0xffffffffu, n[i] > far);
            const int c = __popc(has);
            if (k >= 0 && k < c) seq = 32 * i + (int)__fns(has, 0, k + 1);
            k -= c;
        }
    } else {
        int lo = 0, hi = t.sequences;    // the sequence is the last whose first slot is not behind `slot`
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32, at = lo + lane * step;
            const bool before = at < hi && offset(at) / size + at <= slot;
            const int c = __popc(__ballot_sync(0xffffffffu, before));
            if (c == 0) return false;
            lo += (c - 1) * step;
            hi = min(lo + step, hi);
        }
        seq = lo;
        const int k = slot - (offset(seq) / size + seq), tiles = tiles_of(seq);
        if (k < 0 || k >= tiles) return false;
        far = tiles - 1 - k;
    }
    const int first = offset(seq), len = max(offset(seq + 1) - first, 0);
    *s = Span{0, first, len, from_last ? (len + size - 1) / size - 1 - far : far};
    return true;
}

// ---------------------------------------------------------------- host
// A tensor of heads as a caller describes it, [batch, seq, heads, head_dim], as boxes of 64 columns by some tokens,
// swizzled over 128 bytes; `out`: of 32 columns by 32 tokens, swizzled over 64.
inline bool make_heads_map(CUtensorMap* map, const tb_heads& h, int64_t batch, int64_t seq, int64_t dim, int tokens, bool bf16,
                           bool out = false) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)dim, (cuuint64_t)seq, (cuuint64_t)h.heads, (cuuint64_t)batch};
    const cuuint64_t row = (cuuint64_t)dim * 2;      // of a dimension of size 1, whose stride is anything
    const cuuint64_t strides[3] = {seq > 1 ? (cuuint64_t)h.stride_seq * 2 : row, h.heads > 1 ? (cuuint64_t)h.stride_head * 2 : row,
                                   batch > 1 ? (cuuint64_t)h.stride_batch * 2 : row};
    const cuuint32_t box[4] = {out ? 32u : 64u, out ? 32u : (cuuint32_t)tokens, 1, 1};
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, h.data, dims, strides, box, ones,
              CU_TENSOR_MAP_INTERLEAVE_NONE, out ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Runs launch() with each of the Withheld left out; counts those whose waits gave up.
template <class F>
inline tb_status run_withheld(int* err, cudaStream_t st, int* launches, F launch) {
    for (int what = kLoads0; what <= kResults; ++what) {
        int word = 0;
        if (cudaMemcpyAsync(err, &word, sizeof(int), cudaMemcpyHostToDevice, st) != cudaSuccess) return TB_ERR_CUDA;
        const tb_status s = launch(what);
        if (s != TB_OK) return s;
        if (cudaMemcpyAsync(&word, err, sizeof(int), cudaMemcpyDeviceToHost, st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess)
            return TB_ERR_CUDA;
        *launches += word == (int)TB_ERR_TIMEOUT;
    }
    return TB_OK;
}
// The problem of the self-tests: three whole tiles and one that ends with the sequence, two query heads of one key head,
// zeros in `mem` (kSelfBytes of them).
constexpr int64_t kSelfTokens = 500, kSelfHeads = 2;
constexpr size_t kSelfBytes = 4 << 20;
inline tb_heads self_heads(unsigned char** mem, int64_t heads, int64_t dim) {
    const tb_heads h{*mem, kSelfTokens * heads * dim, heads * dim, dim, heads};
    *mem += kSelfTokens * heads * dim * 2;
    return h;
}

// What every entry point checks of a call's sizes.
constexpr int64_t kMaxTokens = 1ll << 25;    // of a batch entry: a tile's work stays well inside the limit of its waits
constexpr int64_t kMaxHeadDim = 128;
inline tb_status check_call(int64_t batch, int64_t seq, int64_t dim, const int64_t* offsets, int64_t sequences, float scale,
                            tb_dtype dtype) {
    if (batch < 0 || seq < 0 || batch > (1 << 20) || seq > kMaxTokens) return TB_ERR_INVALID_VALUE;
    if (dim < 8 || dim % 8 || dim > kMaxHeadDim) return TB_ERR_INVALID_VALUE;
    if (!(scale > 0.f && scale <= 0x1p127f)) return TB_ERR_INVALID_VALUE;   // times log2(e) is finite too
    if (offsets ? batch != 1 || sequences < 0 || sequences > (1 << 24) : sequences != 0) return TB_ERR_INVALID_VALUE;
    if (!aligned_to(offsets, 8)) return TB_ERR_MISALIGNED;
    if (dtype != TB_BF16 && dtype != TB_F16) return TB_ERR_UNSUPPORTED_DTYPE;
    return TB_OK;
}
// A view that TMA reads, or results that are written by 16-byte vectors.
inline tb_status check_heads(const tb_heads* t, int64_t batch, int64_t seq, int64_t dim, bool output, View* v) {
    if (!t) return TB_ERR_INVALID_VALUE;
    const tb_status s = check_view(t, batch, seq, dim, 2, v);
    if (s != TB_OK) return s;
    for (int i = 0; i < 3; ++i)
        if (v->n[i] > 1 && (v->s[i] == 0 || v->s[i] >= (1ll << 39))) return TB_ERR_INVALID_VALUE;
    if (!aligned_to(v->p, 16)) return TB_ERR_MISALIGNED;
    for (int i = 0; i < 3; ++i)
        if (v->s[i] % 8) return TB_ERR_MISALIGNED;
    int order[3], count = 0;
    if (output && !nested(*v, dim, order, &count)) return TB_ERR_ALIAS;
    return TB_OK;
}
inline Range range_of_view(const View& v, int64_t dim) {
    int64_t e = 0;
    extent(v, dim, &e);       // (checked before)
    return range_of(v.p, v.n[0] && v.n[1] && v.n[2] ? e : 0, 2);
}

}  // namespace
}  // namespace tb
