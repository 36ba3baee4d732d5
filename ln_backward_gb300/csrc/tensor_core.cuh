// tensor_core.cuh -- what the kernels on the tensor cores share: mbarriers with bounded waits, TMA,
// tcgen05 and packed fp32 in inline PTX, operand descriptors, the way out of an epilogue warp, and
// tensor maps on the host.
#pragma once

#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "tb_common.cuh"

namespace tb {
namespace {

constexpr int kTile = 256;                   // rows and columns of a CTA pair's tile
constexpr int kHalf = 128;                   // of which one CTA stages and drains
constexpr int kStageK = 64;                  // contracted elements a stage: 128 bytes
constexpr int kStages = 6;
constexpr int kOperandBytes = kHalf * kStageK * 2;
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kEpiWarp = 4;                  // first of the epilogue warps
constexpr int kOutCols = 32;
constexpr int kOutBytes = 32 * kOutCols * 2; // what an epilogue warp stores at once: 32 rows
constexpr int kOutboxes = 16;                // one or two for each epilogue warp
constexpr int kTmemCols = 512;               // two accumulators
constexpr unsigned long long kWaitLimitNs = 1000000000ull;

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
// Accumulators change hands between tcgen05 fences, which order the tcgen05 instructions: the
// barrier itself need not order anything else.  (A release waited for the lane's stores before every
// hand-over: fp16 gradient of 1,021 x 50,257 x 768 in 168 us, 158 without; loss of 4,096 x 50,257 x
// 512, 137 and 108.)
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t remote_bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote_bar)
                 : "memory");
}
template <bool Acquire>
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t done;
    if constexpr (Acquire)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
    return done != 0;
}
// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(yes));
    return yes != 0;
}
__device__ __forceinline__ unsigned long long now_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// kEnd: waits at a warp's end, for what the warps that may still be waiting themselves finish.  kWork: for other
// warps to finish a whole piece of work, of many waits of theirs.
enum Waits { kRelaxed, kAcquire, kEnd, kWork };
// P: a kernel's arguments, with the bound of its waits (wait_ns) and the device error word (err).
template <int How, class P>
__device__ __noinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, const P* p) {
    const unsigned long long t0 = now_ns(), limit = How == kWork ? 64 * kWaitLimitNs : How == kEnd ? 4 * kWaitLimitNs : p->wait_ns;
    for (uint32_t it = 1; it < (1u << 30); ++it) {
        if (mbar_try<How != kRelaxed>(bar, parity)) return true;
        if ((it & 63u) == 0 && now_ns() - t0 > limit) break;
    }
    atomicExch(p->err, (int)TB_ERR_TIMEOUT);
    return false;
}
template <int How = kAcquire, class P>
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, const P* p) {
    return mbar_try<How != kRelaxed>(bar, parity) || mbar_wait_slow<How>(bar, parity, p);
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
// contracted dimension every 1,024.  The upper word is a constant; the lower one is the address
// in units of 16 bytes under it, so that the next operand is one addition.
template <bool MnMajor>
__device__ __forceinline__ uint32_t desc_low(uint32_t addr) {
    return ((addr & 0x3FFFF) >> 4) | ((MnMajor ? 8192u >> 4 : 1u) << 16);
}
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);

template <bool Accumulate>
__device__ __forceinline__ void mma_pair(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (Accumulate)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.eq.u32 p, 0, 0;\n\t"
            "mov.b64 x, {%1, %4};\n\tmov.b64 y, {%2, %4};\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(idesc), "r"(kDescHigh)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %5, 0;\n\t"
            "mov.b64 x, {%1, %4};\n\tmov.b64 y, {%2, %4};\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(idesc), "r"(kDescHigh), "r"(accumulate)
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
// 32 columns of this warp's 32 accumulator rows, one row a lane; the values are there after
// tmem_wait, which names the registers so that no use of them moves above it.
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
        "%30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
        : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
          "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
          "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
          "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
        :
        : "memory");
}
// 16 columns, there when it returns.
__device__ __forceinline__ void tmem_read16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
}
// A box of 32 rows by 32 columns from shared memory to `map` at column x, row y; what lies outside
// the matrix is dropped.
__device__ __forceinline__ void tma_store(const CUtensorMap* map, int x, int y, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
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

// Two fp32 values in a register pair: both are added or multiplied in one issue slot.
__device__ __forceinline__ unsigned long long pair_of(float lo, float hi) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split_pair(unsigned long long a, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a));
}
__device__ __forceinline__ unsigned long long fma_pair(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ unsigned long long add_pair(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

constexpr float kLog2e = 1.44269504088896341f;

// ---------------------------------------------------------------- the way out
// An epilogue warp's way out for 16-bit results: 32 columns of its 32 rows into a 64-byte swizzled
// box in shared memory (a lane's 16-byte pieces at piece ^ (row / 2 & 3): no two lanes of a quarter
// warp share banks), and a TMA store of the box, of which each warp has two.  Stored from registers,
// a warp's 16-byte pieces lie a row apart, 32 half sectors an instruction: the epilogue then took
// longer than the MMAs of a tile with 768 contracted elements (78 us against 62 us, 1,021 x 50,257).
template <class Fmt, int Boxes>
struct Outbox {
    unsigned char* mem;       // this warp's boxes
    const CUtensorMap* map;
    int lane, n;              // boxes filled so far
    __device__ __forceinline__ void fill(unsigned char* box, const float (&v)[32]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = v[8 * i + e];
            *reinterpret_cast<uint4*>(box + lane * 64 + ((i ^ (lane / 2 & 3)) * 16)) = pack8<Fmt>(f);
        }
    }
    __device__ __forceinline__ void put(const float (&v)[32], int x, int y) {
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(Boxes - 1) : "memory");
        __syncwarp();         // the box of `Boxes` stores ago has been read
        unsigned char* box = mem + n % Boxes * kOutBytes;
        fill(box, v);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) tma_store(map, x, y, smem_addr(box));
        ++n;
    }
    // Where rows do not start on 16 bytes: the box's rows one after another, a column a lane.
    __device__ __forceinline__ void put_plain(const float (&v)[32], typename Fmt::T* out, int x, int y, int rows,
                                              int cols) {
        using T = typename Fmt::T;
        __syncwarp();
        fill(mem, v);
        __syncwarp();
        if (x + lane < cols) {
            const int last = min(32, rows - y);
            T* to = out + (int64_t)y * cols + x + lane;
#pragma unroll 8
            for (int r = 0; r < last; ++r, to += cols)
                *to = *reinterpret_cast<const T*>(mem + r * 64 + (((lane / 8) ^ (r / 2 & 3)) * 16) + lane % 8 * 2);
        }
    }
};

// The same for 32 fp32 columns: one box of both halves' size, swizzled over 128 bytes, of split z.
// Stores before it are waited for.  An Outbox::put of two boxes behind it lets one store go on reading: the caller waits for
// this one, which reads both boxes.  `add`: onto what is there.  (Every element of dH's sums gets one addition a launch: the order of
// the pieces decides the result, nothing else.)
__device__ __forceinline__ void put_sums(unsigned char* box, const CUtensorMap* map, int lane, const float (&v)[32],
                                         int x, int y, int z, bool add) {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        *reinterpret_cast<float4*>(box + lane * 128 + ((i ^ (lane & 7)) * 16)) =
            make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
        const uint32_t src = smem_addr(box);
        if (add)
            asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                         ::"l"(map), "r"(x), "r"(y), "r"(z), "r"(src) : "memory");
        else
            asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                             map), "r"(x), "r"(y), "r"(z), "r"(src) : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
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
// 128 bytes; what lies outside reads as zeros.  `out`: written in boxes of 32 columns, swizzled
// over 64 bytes.
bool make_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_rows,
              bool bf16, bool out = false) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {(cuuint32_t)(out ? kOutCols : kStageK), (cuuint32_t)box_rows};
    const cuuint32_t ones[2] = {1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
              const_cast<void*>(p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              out ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The fp32 sums [splits][rows][cols] of dH or dW, written in boxes of 32 x 32.
bool make_sums_map(CUtensorMap* map, float* p, int64_t splits, int64_t rows, int64_t cols) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)splits};
    const cuuint64_t strides[2] = {(cuuint64_t)cols * 4, (cuuint64_t)(rows * cols) * 4};
    const cuuint32_t box[3] = {32, 32, 1};
    const cuuint32_t ones[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, p, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace tb
