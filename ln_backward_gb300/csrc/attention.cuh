// attention.cuh -- what the kernels of causal attention share: the sequences of a call, one-CTA
// tcgen05 products with the left operand in shared or tensor memory, and loads by TMA.
#pragma once

#include "heads_view.cuh"
#include "tensor_core.cuh"

namespace tb {
namespace {

constexpr int kRows = 128;                   // queries or keys of a tile: TMEM's lanes
constexpr int kBox = kRows * 64 * 2;         // 64 columns of a tile, swizzled over 128 bytes

// ---------------------------------------------------------------- PTX
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// 64 columns from x on of 128 rows from y on of one head of one batch entry; zeros outside the tensor.
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, int x, int y, int head, int batch, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(head), "r"(batch), "r"(bar)
        : "memory");
}
// Operand descriptors (see desc_low): rows of 64 columns contracted along the columns, or, kMn, along
// the rows, with the next 64 columns a box further on.
constexpr uint32_t kMn = 1;
__device__ __forceinline__ uint32_t tile_desc(uint32_t addr, bool mn) {
    return ((addr & 0x3FFFF) >> 4) | ((mn ? (uint32_t)kBox >> 4 : 1u) << 16);
}
__host__ __device__ constexpr uint32_t instruction(bool bf16, int cols, bool b_mn) {
    return (1u << 4) | ((uint32_t)bf16 << 7) | ((uint32_t)bf16 << 10) | ((uint32_t)b_mn << 16) | ((uint32_t)(cols / 8) << 17) |
           ((uint32_t)(kRows / 16) << 24);
}
// 16 contracted elements.  A in shared memory, or 16-bit pairs in tensor memory.  Add: onto what d holds; otherwise
// `add` says whether.
template <bool Add>
__device__ __forceinline__ void mma_smem(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
    if constexpr (Add)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.eq.u32 p, 0, 0;\n\t"
            "mov.b64 x, {%1, %4};\n\tmov.b64 y, {%2, %4};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(idesc), "r"(kDescHigh)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, 0, 0;\n\t"
            "mov.b64 x, {%1, %4};\n\tmov.b64 y, {%2, %4};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(idesc), "r"(kDescHigh)
            : "memory");
}
template <bool Add>
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add = 1) {
    if constexpr (Add)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.eq.u32 p, 0, 0;\n\t"
            "mov.b64 y, {%2, %4};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(idesc), "r"(kDescHigh)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.u32 p, %5, 0;\n\t"
            "mov.b64 y, {%2, %4};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(idesc), "r"(kDescHigh), "r"(add)
            : "memory");
}
// Two tiles' rows against each other over `steps` times 16 of a head's elements, by descriptors of their first boxes.
// An MMA of 128 x 128 x 16 takes 64 clocks, and one thread issues them all: no loop where the head is whole.
template <int Blocks>
__device__ __forceinline__ void product_by_rows(uint32_t d, uint32_t a, uint32_t b, int steps, uint32_t idesc) {
    mma_smem<false>(d, a, b, idesc);
    if (steps == 4 * Blocks) {
#pragma unroll
        for (int k = 1; k < 4 * Blocks; ++k) {
            const uint32_t at = (k < 4 ? 0 : kBox >> 4) + k % 4 * 2;
            mma_smem<true>(d, a + at, b + at, idesc);
        }
    } else {
        for (int k = 1; k < steps; ++k) {
            const uint32_t at = (k < 4 ? 0 : kBox >> 4) + k % 4 * 2;
            mma_smem<true>(d, a + at, b + at, idesc);
        }
    }
}
// d (+)= A B over the 128 tokens of B's rows.  A lies in tensor memory, 64 tokens (32 columns) and the others
// `apart` columns behind.
__device__ __forceinline__ void product_over_tokens(uint32_t d, uint32_t a, uint32_t apart, uint32_t b, uint32_t idesc, bool add) {
    mma_tmem<false>(d, a, b, idesc, add);
#pragma unroll
    for (int k = 1; k < kRows / 16; ++k) mma_tmem<true>(d, a + (k < 4 ? 8 * k : apart + 8 * (k - 4)), b + k * (2048 >> 4), idesc);
}
// Arrives on an mbarrier of this CTA when the MMAs issued so far are done.
__device__ __forceinline__ void mma_done(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_alloc_all(uint32_t slot) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_all(uint32_t tmem) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}
__device__ __forceinline__ unsigned long long mul_pair(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// Two values as 16-bit pairs lie in TMEM and in registers: the first in the low half.
template <class Fmt>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if constexpr (std::is_same<Fmt, BF16>::value) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 32 rows of a result from tensor memory, a row a lane, times the lane's factor and rounded, to `rows` rows
// `stride` apart: through shared memory, from which eight lanes write a row's 64 columns.  `box`: the warp's own,
// 1,024-byte aligned.
constexpr int kOutStage = 32 * 128;
template <class Fmt>
__device__ __forceinline__ void store_rows(unsigned char* box, uint32_t tmem, float factor, typename Fmt::T* out, int64_t stride,
                                           int rows, int dim, int lane) {
    for (int x = 0; x < dim; x += 64) {
        uint32_t o[2][32];
        tmem_load32(tmem + x, o[0]);
        tmem_load32(tmem + x + 32, o[1]);
        tmem_wait(o[0]);
        tmem_wait(o[1]);
        __syncwarp();
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                h[e] = pack2<Fmt>(__uint_as_float(o[g / 4][g % 4 * 8 + 2 * e]) * factor,
                                  __uint_as_float(o[g / 4][g % 4 * 8 + 2 * e + 1]) * factor);
            *reinterpret_cast<uint4*>(box + lane * 128 + ((g ^ (lane & 7)) * 16)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
        __syncwarp();
        const int c = lane & 7;              // 16 bytes of a row
        if (x + 8 * c < dim)
#pragma unroll
            for (int y = lane >> 3; y < 32; y += 4)
                if (y < rows)
                    *reinterpret_cast<uint4*>(out + y * stride + x + 8 * c) =
                        *reinterpret_cast<const uint4*>(box + y * 128 + ((c ^ (y & 7)) * 16));
    }
}

// A tile of `Blocks` boxes whose rows from `rows` on are to be zeros, which whatever lies there need not be
// times 0.  By a whole warp, before the tile is handed to the MMAs.
template <int Blocks>
__device__ __forceinline__ void clear_behind(unsigned char* tile, int rows, int lane) {
    for (int b = 0; b < Blocks; ++b)
        for (int x = rows * 8 + lane; x < kRows * 8; x += 32) *reinterpret_cast<uint4*>(tile + b * kBox + x * 16) = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
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

// Tiles of `size` tokens are numbered so that a sequence is found without adding up the lengths before it:
// sequence i's are slots floor(offsets[i] / size) + i and on, as floor((o + n) / size) - floor(o / size) + 1
// is at least ceil(n / size).  Some slots have no tile.
__host__ __device__ inline int64_t slots_of(int64_t tokens, int64_t sequences, int size) { return tokens / size + sequences; }

// The tile in a slot, by a whole warp; false: none.  `last_first`: a sequence's last tile in its first slot.
// Offsets that do not count up within the row are cut to it, and reported in the device error word.
__device__ __forceinline__ bool find_tile(const Tokens& t, int size, int slot, bool last_first, Span* s) {
    const int lane = threadIdx.x & 31;
    auto offset = [&](int i) { return (int)min(max(t.offsets[i], (int64_t)0), (int64_t)t.seq); };
    int lo = 0, hi = t.sequences;        // the sequence is the last whose first slot is not behind `slot`
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const bool before = at < hi && offset(at) / size + at <= slot;
        const int n = __popc(__ballot_sync(0xffffffffu, before));
        if (n == 0) return false;
        lo += (n - 1) * step;
        hi = min(lo + step, hi);
    }
    const int64_t a = t.offsets[lo], b = t.offsets[lo + 1];
    if ((a < 0 || b < a || b > t.seq) && lane == 0) atomicExch(t.err, (int)TB_ERR_INVALID_VALUE);
    const int first = offset(lo), len = max(offset(lo + 1) - first, 0), tiles = (len + size - 1) / size;
    const int k = slot - (first / size + lo);
    if (k < 0 || k >= tiles) return false;
    *s = Span{0, first, len, last_first ? tiles - 1 - k : k};
    return true;
}

// ---------------------------------------------------------------- host
// A tensor of heads as a caller describes it, [batch, seq, heads, head_dim], as boxes of 64 columns by 128 tokens.
inline bool make_heads_map(CUtensorMap* map, const tb_heads& h, int64_t batch, int64_t seq, int64_t dim, bool bf16) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)dim, (cuuint64_t)seq, (cuuint64_t)h.heads, (cuuint64_t)batch};
    const cuuint64_t row = (cuuint64_t)dim * 2;      // of a dimension of size 1, whose stride is anything
    const cuuint64_t strides[3] = {seq > 1 ? (cuuint64_t)h.stride_seq * 2 : row, h.heads > 1 ? (cuuint64_t)h.stride_head * 2 : row,
                                   batch > 1 ? (cuuint64_t)h.stride_batch * 2 : row};
    const cuuint32_t box[4] = {64, kRows, 1, 1};
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, h.data, dims, strides, box, ones,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What every entry point checks of a call's sizes.
constexpr int64_t kMaxTokens = 1ll << 30;    // of a batch entry: token numbers are 32-bit
constexpr int64_t kMaxHeadDim = 128;
inline tb_status check_call(int64_t batch, int64_t seq, int64_t dim, const int64_t* offsets, int64_t sequences, float scale,
                            tb_dtype dtype) {
    if (batch < 0 || seq < 0 || batch > (1 << 20) || seq > kMaxTokens) return TB_ERR_INVALID_VALUE;
    if (dim < 8 || dim % 8 || dim > kMaxHeadDim) return TB_ERR_INVALID_VALUE;
    if (!(scale > 0.f && scale <= 3.4028235e38f)) return TB_ERR_INVALID_VALUE;
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
