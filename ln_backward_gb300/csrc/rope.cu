// rope.cu -- rotary positions and the per-head RMS norm of queries and keys.
//
// tb_rope / tb_rope_bwd rotate the pairs of each head's first rotary_dim elements by
// an angle that grows with the token's position; tb_qk_norm_rope normalises each head
// by its root mean square first, in the same pass, and tb_qk_norm_rope_bwd is its
// gradient (dq, dk and the deterministic dgamma of both).
//
// Angles.  A frequency is kept as the fraction of a turn that one position adds, in
// units of 2^-64 turn.  pos * freq in wrapping 64-bit arithmetic is then the angle
// modulo one turn with no rounding at all, for any position of either sign; the upper
// 32 bits (2^-32 turn, 1.5e-9 rad) go to the sine and cosine.  A product in fp32 would
// be off by 0.004 rad at position 131,072; the same in fp64 would run at 1/64 of the
// fp32 rate here.
//
// What bounds it.  Every element is read once and written once (the gradient reads two
// and writes one), with a few FMAs each: HBM.  The angles depend on the token alone,
// so a warp forms the sines of its token once and keeps them in registers over the
// token's heads.
//
// Layout.  A head is dealt to L lanes, each holding NU "units" of two vectors of E
// elements, corresponding ones of the two halves of the rotated part or of the rest.  Both
// members of every pair are then in one lane in either layout: no shuffles but the norm's
// row sums.  32 / L heads go through a warp at a time; L is the number of units, not a power
// of two above it, so that heads of 80 or 96 elements leave few lanes idle.  Queries and keys
// get CTAs of their own, so gamma and the dgamma sums of one tensor stay in registers.  Heads
// whose sizes, strides or pointers no vector width fits take the general kernels (one element
// at a time).
//
// Measured at bf16 2 x 8,192 tokens of 32 + 8 heads of 128, norm and rotation (50 us at the
// copy bandwidth): 58.8 to 59.1 us.  What did not pay there: loads a group ahead in a persistent
// grid (71 us), a ring of cp.async copies (69 us) or of bulk copies (76 us) per warp; all
// spend on addresses and bookkeeping what they save in waiting, and the kernel is bound by
// issue slots first.  At its 80 registers the forward with the norm spills: 40 bytes a thread of
// 16-bit heads of 128, 64 to 84 of 80, 96 and 192, 104 where the lanes are not known when compiling;
// the fp32 gradient 96 bytes at 10 and 12 lanes.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "tb_common.cuh"

namespace tb {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxHeadDim = 1024;
constexpr int kBwdCtasPerSm = 4;      // bound on the gradient's grid (workspace rows)

enum { kRope = 0, kNorm = 1 };

struct Strides {
    int64_t b, s, h;
};

struct HeadsArg {
    const void* x;       // input (the forward's input in the gradient)
    const void* dy;      // gradient of the output (gradient only)
    void* y;             // output (dx in the gradient)
    Strides sx, sdy, sy;
    const float* gamma;
    float* inv_rms;      // written by the forward (may be NULL), read by the gradient
    int heads;
    int chunks;          // warps (or CTAs, general kernels) that share one token's heads
    int steps;           // head groups of one token per chunk
    int tokens;          // tokens that share a head group (above 1 where a token's heads leave room)
    int ctas;            // CTAs of this tensor
    float* partial;      // gradient: [ctas][head_dim] sums of dgamma
    float* dgamma;
};

struct Args {
    HeadsArg t[2];
    const unsigned long long* freqs;
    const int64_t* positions;
    int64_t pos_stride;
    int64_t offset;
    unsigned tokens, seq;      // batch * seq < 2^31
    int head_dim, rot;
    int lanes;           // of a head (vector kernels)
    int interleaved;
    float magnitude;     // sines and cosines are multiplied by it
    float turn;          // +1, or -1 for the transposed rotation
    float eps, inv_dim;
};

// ---------------------------------------------------------------- packed fp32
// Two fp32 values in one 64-bit register pair: the packed multiply and FMA do both in one issue
// slot, each rounded as the scalar one is.  Issue slots bound these kernels before HBM does.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ void split(F2 a, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ F2 swap(F2 a) {
    float lo, hi;
    split(a, lo, hi);
    return f2(hi, lo);
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// ---------------------------------------------------------------- one lane's part of a head
template <int Bytes> struct Raw;
template <> struct Raw<16> { using V = uint4; };
template <> struct Raw<8> { using V = uint2; };
template <> struct Raw<4> { using V = unsigned; };

template <class Fmt, int E>
struct Chunk {                    // a vector of E elements as loaded
    using T = typename Fmt::T;
    using V = typename Raw<E * (int)sizeof(T)>::V;
    V raw;
    __device__ __forceinline__ void load(const T* p) { raw = __ldcs(reinterpret_cast<const V*>(p)); }
    __device__ __forceinline__ void get(F2 (&f)[E / 2]) const {
        const T* h = reinterpret_cast<const T*>(&raw);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) f[e] = f2(Fmt::to_f32(h[2 * e]), Fmt::to_f32(h[2 * e + 1]));
    }
    __device__ __forceinline__ static void store(T* p, const F2 (&f)[E / 2]) {
        V v;
        T* h = reinterpret_cast<T*>(&v);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            float lo, hi;
            split(f[e], lo, hi);
            if constexpr (std::is_same<Fmt, BF16>::value)
                reinterpret_cast<__nv_bfloat162*>(h)[e] = __floats2bfloat162_rn(lo, hi);
            else if constexpr (std::is_same<Fmt, F16>::value)
                reinterpret_cast<__half2*>(h)[e] = __floats2half2_rn(lo, hi);
            else
                h[2 * e] = lo, h[2 * e + 1] = hi;
        }
        __stcs(reinterpret_cast<V*>(p), v);
    }
};

// cos and sin of turn * pos * freq, times the magnitude.  The 32-bit fraction of a turn
// is signed, so it converts to a float in [-1, 1] of half turns with a relative error of
// 2^-24.  16-bit outputs take the hardware's sine and cosine (absolute error below
// 2^-21 on [-pi, pi], 2^-20 with the roundings of the angle, against a rounding of 2^-8 or 2^-11 of
// the output); fp32 outputs take the library's.
template <class Fmt>
__device__ __forceinline__ void cos_sin(const Args& a, long long pos, unsigned long long freq,
                                        float* c, float* s) {
    const unsigned long long phase = (unsigned long long)pos * freq;
    const float half_turns = (float)(int)(phase >> 32) * 0x1p-31f * a.turn;
    float cv, sv;
    if constexpr (sizeof(typename Fmt::T) == 2) {
        const float x = half_turns * 3.14159265358979f;
        cv = __cosf(x);
        sv = __sinf(x);
    } else {
        sincospif(half_turns, &sv, &cv);
    }
    *c = cv * a.magnitude;
    *s = sv * a.magnitude;
}

__device__ __forceinline__ void split_token(const Args& a, unsigned token, unsigned* b, unsigned* s) {
    *b = token / a.seq;
    *s = token - *b * a.seq;
}

__device__ __forceinline__ long long position(const Args& a, unsigned b, unsigned s) {
    return (a.positions ? (long long)__ldg(a.positions + b * a.pos_stride + s) : (long long)s) +
           a.offset;
}

// What one lane holds of a head, for every head of every token.
template <int E, int NU>
struct Units {
    int first[NU], second[NU];   // element offsets of a unit's two vectors
    int freq[NU], freq2[NU];     // the frequencies of its first and second E / 2 pairs
    bool live[NU], turns[NU];
    __device__ __forceinline__ void init(const Args& a, int sub, int lanes) {
        const int units = a.head_dim / (2 * E), rot_units = a.rot / (2 * E);
#pragma unroll
        for (int j = 0; j < NU; ++j) {
            const int c = sub + j * lanes;
            live[j] = c < units;
            turns[j] = c < rot_units;
            // the second vector lies half of the rotated part (of the rest) behind the first in
            // either layout: neighbouring lanes read neighbouring vectors
            first[j] = turns[j] ? c * E : a.rot + (c - rot_units) * E;
            second[j] = first[j] + (turns[j] ? a.rot / 2 : (a.head_dim - a.rot) / 2);
            freq[j] = turns[j] ? (a.interleaved ? first[j] / 2 : first[j]) : 0;
            freq2[j] = turns[j] ? (a.interleaved ? second[j] / 2 : first[j] + E / 2) : 0;
            if (!live[j]) first[j] = second[j] = 0;
        }
    }
};

template <class Fmt, int E, int NU>
struct Head {                     // one lane's vectors of a head; dead units read as zeros
    Chunk<Fmt, E> p[NU], q[NU];
    __device__ __forceinline__ void load(const typename Fmt::T* head, const Units<E, NU>& u) {
#pragma unroll
        for (int j = 0; j < NU; ++j) {
            p[j].raw = {};
            q[j].raw = {};
            if (NU == 1 || u.live[j]) {
                p[j].load(head + u.first[j]);
                q[j].load(head + u.second[j]);
            }
        }
    }
};

// The rotation of one unit (vectors p and q) as p' = p A + partner(p) B, where the partner of p is
// q in the half layout and p with its neighbours swapped in the interleaved one; likewise for q.
// The forward's gamma is in A and B (element x of a pair counts gamma(x) x), so the norm costs a
// head no more multiplications than the rotation and its 1/rms.
template <int E>
struct Turn {
    F2 a[E], b[E];                // p's E / 2 pairs of elements, then q's
    // cos_p, cos_q: the cosines of the first and second E / 2 pairs; sines lie `sines` behind them
    __device__ __forceinline__ void set(const float* cos_p, const float* cos_q, int sines, const float (&g)[2 * E],
                                        bool turns, bool interleaved) {
        constexpr int H = E / 2;
        auto c = [&](int e) { return e < H ? cos_p[e] : cos_q[e - H]; };
        auto s = [&](int e) { return e < H ? cos_p[sines + e] : cos_q[sines + e - H]; };
#pragma unroll
        for (int e = 0; e < E; ++e) a[e] = f2(g[2 * e], g[2 * e + 1]), b[e] = f2(0.f);
        if (!turns) return;
        if (interleaved) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                a[e] = f2(c(e)) * f2(g[2 * e], g[2 * e + 1]);
                b[e] = f2(-s(e), s(e)) * f2(g[2 * e + 1], g[2 * e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < H; ++e) {
                const F2 gp = f2(g[2 * e], g[2 * e + 1]), gq = f2(g[E + 2 * e], g[E + 2 * e + 1]);
                const F2 cc = f2(c(2 * e), c(2 * e + 1));
                a[e] = gp * cc;
                b[e] = gq * f2(-s(2 * e), -s(2 * e + 1));
                a[H + e] = gq * cc;
                b[H + e] = gp * f2(s(2 * e), s(2 * e + 1));
            }
        }
    }
    __device__ __forceinline__ void apply(F2 (&p)[E / 2], F2 (&q)[E / 2], bool turns, bool interleaved) const {
        constexpr int H = E / 2;
        if (!turns) {             // behind rotary_dim nothing is added, not even 0 * inf
#pragma unroll
            for (int e = 0; e < H; ++e) p[e] = p[e] * a[e], q[e] = q[e] * a[H + e];
        } else if (interleaved) {
#pragma unroll
            for (int e = 0; e < H; ++e) {
                p[e] = fma2(swap(p[e]), b[e], p[e] * a[e]);
                q[e] = fma2(swap(q[e]), b[H + e], q[e] * a[H + e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < H; ++e) {
                const F2 x = p[e], y = q[e];
                p[e] = fma2(y, b[e], x * a[e]);
                q[e] = fma2(x, b[H + e], y * a[H + e]);
            }
        }
    }
};

// Whether heads of this many lanes fill a warp (a power of two, known when compiling).
template <int Lanes>
constexpr bool kWhole = Lanes > 0 && (Lanes & (Lanes - 1)) == 0;

// Sum over a head's lanes, in all of them.  Lanes: their number where it is known when compiling,
// else 0.
template <int Lanes>
__device__ __forceinline__ float sum_lanes(float v, int lanes, int sub) {
    if constexpr (kWhole<Lanes>) {
#pragma unroll
        for (int o = 1; o < Lanes; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    } else {
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            if (Lanes && o >= Lanes) continue;
            const float w = __shfl_down_sync(0xffffffffu, v, o);
            v = sub + o < min(lanes, 2 * o) ? v + w : v;
        }
        return __shfl_sync(0xffffffffu, v, (int)(threadIdx.x & 31) - sub);
    }
}

// An item's cosines and sines, one row of the warp's table (rotary_dim floats) for each of its
// tokens: each lane forms those of every 32nd pair, and the lanes share them.  `pos` is the position
// of the lane's own token; lane k * stride is one of token k.
template <class Fmt>
__device__ __forceinline__ void fill_table(const Args& a, long long pos, float* table, int lane, int tokens = 1,
                                           int stride = 0) {
    const int half = a.rot / 2;
    __syncwarp();                 // the previous item's values have been read
    for (int k = 0; k < tokens; ++k, table += a.rot) {
        const long long at = tokens > 1 ? __shfl_sync(0xffffffffu, pos, k * stride) : pos;
        for (int i = lane; i < half; i += 32)
            cos_sin<Fmt>(a, at, __ldg(a.freqs + i), &table[i], &table[half + i]);
    }
    __syncwarp();
}

// What a lane does in every item: which of a group's heads is its own.  Where a token has fewer heads
// than a group (keys shared by many queries), a group takes several tokens' heads.
struct Place {
    int token, head;      // offsets in the item and in the group
    bool own;             // false: the lane doubles another one and writes nothing
    __device__ __forceinline__ void init(const HeadsArg& t, int grp, bool whole) {
        token = 0;
        head = grp;
        own = whole;
        if (t.tokens > 1) {
            token = grp / t.heads;
            head = grp - token * t.heads;
            if (token >= t.tokens) token = head = 0, own = false;
        }
    }
};

// An item: a token, a share of its heads, or a few tokens; the lane's token of it.
struct Item {
    unsigned token, b, s;
    int head, end;
    bool in;              // the token exists (the last item may have fewer than its tokens)
    __device__ __forceinline__ void open(const Args& a, const HeadsArg& t, unsigned item, int per_step,
                                         int token_offset = 0) {
        int chunk = 0;
        token = item;
        in = true;
        if (t.chunks > 1) {
            token = item / (unsigned)t.chunks;
            chunk = (int)(item - token * t.chunks);
        } else if (t.tokens > 1) {
            token = item * t.tokens + token_offset;
            in = token < a.tokens;
            if (!in) token = a.tokens - 1;
        }
        split_token(a, token, &b, &s);
        head = chunk * t.steps * per_step;
        end = min(t.heads, head + t.steps * per_step);
    }
    template <class P>
    __device__ __forceinline__ P row(P base, const Strides& st) const {
        return base + b * st.b + s * st.s;
    }
};
__device__ __forceinline__ unsigned items_of(const Args& a, const HeadsArg& t) {
    return t.tokens > 1 ? (a.tokens + t.tokens - 1) / t.tokens : a.tokens * t.chunks;
}

// ---------------------------------------------------------------- forward
template <class Fmt, int E, int NU, int Mode, int Lanes>
__device__ __forceinline__ void heads_fwd(const Args& a, const HeadsArg& t, int cta, float* table) {
    using T = typename Fmt::T;
    constexpr int H = E / 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lanes = Lanes ? Lanes : a.lanes, per_step = 32 / lanes;
    // lanes behind the last whole head double the last one's and write nothing
    const int grp = min(lane / lanes, per_step - 1), sub = lane % lanes;
    const bool whole = kWhole<Lanes> || lane < per_step * lanes;
    table += warp * t.tokens * a.rot;
    Place place;
    place.init(t, grp, whole);
    Units<E, NU> u;
    u.init(a, sub, lanes);
    pdl_wait();
    pdl_trigger();
    const unsigned item = cta * kWarps + warp;    // one for each warp
    if (item >= items_of(a, t)) return;
    Item at;
    at.open(a, t, item, per_step, place.token);
    const long long pos = position(a, at.b, at.s);
    const T* x = at.row(static_cast<const T*>(t.x), t.sx);
    T* y = at.row(static_cast<T*>(t.y), t.sy);
    Turn<E> turn[NU];
    bool fresh = true;
    constexpr int kAhead = 2;         // head groups loaded together
    for (int h0 = at.head; h0 < at.end; h0 += kAhead * per_step) {
        Head<Fmt, E, NU> in[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (k == 0 || h0 + k * per_step < at.end)
                in[k].load(x + min(h0 + k * per_step + place.head, at.end - 1) * t.sx.h, u);
        if (fresh) {                  // (while the first heads are on their way)
            fill_table<Fmt>(a, pos, table, lane, t.tokens, t.heads * lanes);
            const float* row = table + place.token * a.rot;
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                float g[2 * E];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    g[e] = Mode == kNorm ? __ldg(t.gamma + u.first[j] + e) : 1.f;
                    g[E + e] = Mode == kNorm ? __ldg(t.gamma + u.second[j] + e) : 1.f;
                }
                turn[j].set(row + u.freq[j], row + u.freq2[j], a.rot / 2, g, u.turns[j], a.interleaved);
            }
            fresh = false;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (k > 0 && h0 + k * per_step >= at.end) break;
            const int h = h0 + k * per_step + place.head;
            const bool mine = place.own && at.in && h < at.end;
            F2 p[NU][H], q[NU][H];
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                in[k].p[j].get(p[j]);
                in[k].q[j].get(q[j]);
            }
            float r = 1.f;
            if constexpr (Mode == kNorm) {
                F2 ss = f2(0.f);
#pragma unroll
                for (int j = 0; j < NU; ++j)
#pragma unroll
                    for (int e = 0; e < H; ++e) ss = fma2(q[j][e], q[j][e], fma2(p[j][e], p[j][e], ss));
                float lo, hi;
                split(ss, lo, hi);
                r = rsqrtf(sum_lanes<Lanes>(lo + hi, lanes, sub) * a.inv_dim + a.eps);
                if (t.inv_rms && sub == 0 && mine) t.inv_rms[(int64_t)at.token * t.heads + h] = r;
            }
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                turn[j].apply(p[j], q[j], u.turns[j], a.interleaved);
                if constexpr (Mode == kNorm) {
#pragma unroll
                    for (int e = 0; e < H; ++e) p[j][e] = p[j][e] * f2(r), q[j][e] = q[j][e] * f2(r);
                }
            }
            if (mine) {
                T* row = y + h * t.sy.h;
#pragma unroll
                for (int j = 0; j < NU; ++j) {
                    if (NU > 1 && !u.live[j]) continue;
                    Chunk<Fmt, E>::store(row + u.first[j], p[j]);
                    Chunk<Fmt, E>::store(row + u.second[j], q[j]);
                }
            }
        }
    }
}

// The body is there once for the queries and once for the keys, so that a tensor's strides and
// pointers are operands in the constant bank and not loads by a computed index.
template <class Fmt, int E, int NU, int Mode, int Lanes>
__global__ void __launch_bounds__(kThreads, NU == 1 ? 3 : 2) heads_fwd_kernel(const __grid_constant__ Args a) {
    extern __shared__ __align__(16) float shared[];   // tables [kWarps][rotary_dim]
    const int cta = (int)blockIdx.x - a.t[0].ctas;
    if (cta < 0) heads_fwd<Fmt, E, NU, Mode, Lanes>(a, a.t[0], (int)blockIdx.x, shared);
    else heads_fwd<Fmt, E, NU, Mode, Lanes>(a, a.t[1], cta, shared);
}

// ---------------------------------------------------------------- gradient of the norm
// dn = the transposed rotation of dy; xhat = x * r; dxhat = dn * gamma;
// dx = r * (dxhat - xhat * mean(dxhat * xhat)); dgamma = sum of dn * xhat.
//
// 16-bit heads: the next group's vectors come by cp.async into the lane's own slots of shared memory
// while the present group is worked on, at two CTAs an SM (a lane holds 16 elements of x, dy, gamma,
// dgamma and the sines: 128 registers, none left for vectors on their way; loaded into registers and
// copied, the copies wait for the loads).  bf16 4 x 4,096 tokens of 32 + 8 heads of 128 (75 us at the
// copy bandwidth): 93 us before the CTAs were dealt by cost (84 since), with the early loads in registers
// 103, without early loads 118 at three CTAs.  fp32 heads hold half as many elements a lane, so three
// CTAs fit, and load when they need it: 32,768 tokens of 16 + 2 heads of 256 (268 us): 295 us then (282
// since), with early loads at two CTAs 356.
template <class Fmt>
constexpr bool kBwdAhead = sizeof(typename Fmt::T) == 2;

template <int Bytes>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
    const unsigned to = (unsigned)__cvta_generic_to_shared(dst);
    if constexpr (Bytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(src), "n"(Bytes) : "memory");
}
// A warp's two slots for vectors on their way: x's p and q, dy's p and q for each unit, 32 lanes side
// by side, and inv_rms.  A lane reads back what it asked for itself: its own copies' completion is all
// that it waits for.
template <class Fmt, int E, int NU>
constexpr int kSlotBytes = kBwdAhead<Fmt> ? 32 * (4 * NU * E * (int)sizeof(typename Fmt::T) + 4) : 0;

template <class Fmt, int E, int NU, int Lanes>
__device__ __forceinline__ void heads_bwd(const Args& a, const HeadsArg& t, int cta, float* sums) {
    using T = typename Fmt::T;
    constexpr int H = E / 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lanes = Lanes ? Lanes : a.lanes, per_step = 32 / lanes;
    const int grp = min(lane / lanes, per_step - 1), sub = lane % lanes;
    const bool whole = kWhole<Lanes> || lane < per_step * lanes;
    float* table = sums + kWarps * a.head_dim + warp * t.tokens * a.rot;
    Place place;
    place.init(t, grp, whole);
    const float* turn_row = table + place.token * a.rot;
    using V = typename Raw<E * (int)sizeof(T)>::V;
    constexpr int kSlot = kSlotBytes<Fmt, E, NU>;
    unsigned char* slots = reinterpret_cast<unsigned char*>(sums + (kWarps * (a.head_dim + t.tokens * a.rot) + 3) / 4 * 4) +
                           warp * 2 * kSlot;
    auto vec = [&](int slot, int v) { return reinterpret_cast<V*>(slots + slot * kSlot) + v * 32 + lane; };
    auto inv_at = [&](int slot) { return reinterpret_cast<float*>(slots + (slot + 1) * kSlot - 128) + lane; };
    Units<E, NU> u;
    u.init(a, sub, lanes);
    pdl_wait();
    pdl_trigger();
    F2 g[NU][E], acc[NU][E];
    float c[NU][E], sn[NU][E];
#pragma unroll
    for (int j = 0; j < NU; ++j)
#pragma unroll
        for (int e = 0; e < H; ++e) {
            g[j][e] = f2(__ldg(t.gamma + u.first[j] + 2 * e), __ldg(t.gamma + u.first[j] + 2 * e + 1));
            g[j][H + e] = f2(__ldg(t.gamma + u.second[j] + 2 * e), __ldg(t.gamma + u.second[j] + 2 * e + 1));
            acc[j][e] = acc[j][H + e] = f2(0.f);
        }
    const unsigned items = items_of(a, t), stride = t.ctas * kWarps;
    unsigned i = cta * kWarps + warp;
    if (i < items) {
        Item at, nxt;
        at.open(a, t, i, per_step, place.token);
        long long pos = position(a, at.b, at.s);
        const T *x = at.row(static_cast<const T*>(t.x), t.sx), *dy = at.row(static_cast<const T*>(t.dy), t.sdy);
        T* dx = at.row(static_cast<T*>(t.y), t.sy);
        const float* inv = t.inv_rms + (int64_t)at.token * t.heads;
        Head<Fmt, E, NU> hx, hdy;
        float r = 0.f;
        int slot = 0;
        auto fetch = [&](const T* px, const T* pdy, const float* pinv, int h, int to) {
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                if (NU > 1 && !u.live[j]) continue;
                constexpr int kVec = E * (int)sizeof(T);
                copy_async<kVec>(vec(to, 4 * j), px + h * t.sx.h + u.first[j]);
                copy_async<kVec>(vec(to, 4 * j + 1), px + h * t.sx.h + u.second[j]);
                copy_async<kVec>(vec(to, 4 * j + 2), pdy + h * t.sdy.h + u.first[j]);
                copy_async<kVec>(vec(to, 4 * j + 3), pdy + h * t.sdy.h + u.second[j]);
            }
            copy_async<4>(inv_at(to), pinv + h);
        };
        if constexpr (kBwdAhead<Fmt>) {
#pragma unroll
            for (int j = 0; j < NU; ++j)      // units that no copy fills count as zeros
                if (NU > 1 && !u.live[j])
                    for (int k = 0; k < 8; ++k) *vec(k / 4, 4 * j + k % 4) = {};
        }
        auto load = [&](const T* px, const T* pdy, const float* pinv, int h, Head<Fmt, E, NU>& ox,
                        Head<Fmt, E, NU>& ody, float& or_) {
            ox.load(px + h * t.sx.h, u);
            ody.load(pdy + h * t.sdy.h, u);
            or_ = __ldg(pinv + h);
        };
        if constexpr (kBwdAhead<Fmt>) {
            fetch(x, dy, inv, min(at.head + place.head, at.end - 1), 0);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        for (;;) {                        // items
            fill_table<Fmt>(a, pos, table, lane, t.tokens, t.heads * lanes);
#pragma unroll
            for (int j = 0; j < NU; ++j)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float* at = turn_row + (e < H ? u.freq[j] + e : u.freq2[j] + e - H);
                    c[j][e] = u.turns[j] ? at[0] : 1.f;
                    sn[j][e] = u.turns[j] ? at[a.rot / 2] : 0.f;
                }
            i += stride;
            const bool more = i < items;
            nxt = at;
            const T *x_n = x, *dy_n = dy;
            if (more) {
                nxt.open(a, t, i, per_step, place.token);
                pos = position(a, nxt.b, nxt.s);
                x_n = nxt.row(static_cast<const T*>(t.x), t.sx);
                dy_n = nxt.row(static_cast<const T*>(t.dy), t.sdy);
            }
            const float* inv_n = t.inv_rms + (int64_t)nxt.token * t.heads;
            for (int h0 = at.head; h0 < at.end; h0 += per_step) {
                // the next group's vectors, of the next item behind the last
                const bool same = h0 + per_step < at.end;
                const int h = h0 + place.head;
                const bool mine = place.own && at.in && h < at.end;
                if constexpr (kBwdAhead<Fmt>) {
                    if (same || more)
                        fetch(same ? x : x_n, same ? dy : dy_n, same ? inv : inv_n,
                              same ? min(h + per_step, at.end - 1) : min(nxt.head + place.head, nxt.end - 1), slot ^ 1);
                    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 1;" ::: "memory");
#pragma unroll
                    for (int j = 0; j < NU; ++j) {
                        hx.p[j].raw = *vec(slot, 4 * j);
                        hx.q[j].raw = *vec(slot, 4 * j + 1);
                        hdy.p[j].raw = *vec(slot, 4 * j + 2);
                        hdy.q[j].raw = *vec(slot, 4 * j + 3);
                    }
                    r = *inv_at(slot);
                    slot ^= 1;
                } else {
                    load(x, dy, inv, min(h, at.end - 1), hx, hdy, r);
                }
                F2 d[NU][E], xr[NU][E];
                F2 dot2 = f2(0.f);
#pragma unroll
                for (int j = 0; j < NU; ++j) {
                    F2 p[H], q[H];
                    hdy.p[j].get(p);
                    hdy.q[j].get(q);
                    if (u.turns[j]) {
                        if (a.interleaved) {
#pragma unroll
                            for (int e = 0; e < E; ++e) {
                                F2& v = e < H ? p[e % H] : q[e % H];
                                float lo, hi;
                                split(v, lo, hi);
                                v = f2(lo * c[j][e] - hi * sn[j][e], lo * sn[j][e] + hi * c[j][e]);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < H; ++e) {
                                const F2 v = p[e], w = q[e];
                                const F2 cc = f2(c[j][2 * e], c[j][2 * e + 1]), ss = f2(sn[j][2 * e], sn[j][2 * e + 1]);
                                p[e] = fma2(w, ss * f2(-1.f), v * cc);
                                q[e] = fma2(v, ss, w * cc);
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < H; ++e) d[j][e] = p[e], d[j][H + e] = q[e];
                    hx.p[j].get(p);
                    hx.q[j].get(q);
#pragma unroll
                    for (int e = 0; e < H; ++e) xr[j][e] = p[e] * f2(r), xr[j][H + e] = q[e] * f2(r);
                    if (mine) {
#pragma unroll
                        for (int e = 0; e < E; ++e) acc[j][e] = fma2(d[j][e], xr[j][e], acc[j][e]);
                    }
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        d[j][e] = d[j][e] * g[j][e];
                        dot2 = fma2(d[j][e], xr[j][e], dot2);
                    }
                }
                float lo, hi;
                split(dot2, lo, hi);
                const float m = sum_lanes<Lanes>(lo + hi, lanes, sub) * a.inv_dim;
                if (mine) {
                    T* row = dx + h * t.sy.h;
#pragma unroll
                    for (int j = 0; j < NU; ++j) {
                        F2 p[H], q[H];
#pragma unroll
                        for (int e = 0; e < H; ++e) {
                            p[e] = fma2(xr[j][e], f2(-m), d[j][e]) * f2(r);
                            q[e] = fma2(xr[j][H + e], f2(-m), d[j][H + e]) * f2(r);
                        }
                        if (NU > 1 && !u.live[j]) continue;
                        Chunk<Fmt, E>::store(row + u.first[j], p);
                        Chunk<Fmt, E>::store(row + u.second[j], q);
                    }
                }
            }
            if (!more) break;
            at = nxt;
            x = x_n;
            dy = dy_n;
            inv = inv_n;
            dx = at.row(static_cast<T*>(t.y), t.sy);
        }
    }

    // the warp's head groups, then the CTA's warps, in a fixed order
#pragma unroll
    for (int j = 0; j < NU; ++j)
#pragma unroll
        for (int e = 0; e < 2 * E; ++e) {
            float lo, hi;
            split(acc[j][e / 2], lo, hi);
            const float own = e & 1 ? hi : lo;
            float v = own;
            for (int k = 1; k < per_step; ++k) v += __shfl_sync(0xffffffffu, own, (sub + k * lanes) & 31);
            if (lane < lanes && u.live[j])
                sums[warp * a.head_dim + (e < E ? u.first[j] + e : u.second[j] + e - E)] = v;
        }
    __syncthreads();
    for (int d = threadIdx.x; d < a.head_dim; d += kThreads) {
        float v = 0.f;
        for (int w = 0; w < kWarps; ++w) v += sums[w * a.head_dim + d];
        t.partial[(int64_t)cta * a.head_dim + d] = v;
    }
}

template <class Fmt, int E, int NU, int Lanes>
__global__ void __launch_bounds__(kThreads, kBwdAhead<Fmt> ? 2 : 3) heads_bwd_kernel(const __grid_constant__ Args a) {
    extern __shared__ __align__(16) float shared[];   // sums [kWarps][head_dim], tables
    const int cta = (int)blockIdx.x - a.t[0].ctas;
    if (cta < 0) heads_bwd<Fmt, E, NU, Lanes>(a, a.t[0], (int)blockIdx.x, shared);
    else heads_bwd<Fmt, E, NU, Lanes>(a, a.t[1], cta, shared);
}

// ---------------------------------------------------------------- any sizes, strides and alignment
// One element at a time, a head a warp after another of an item's.  A lane owns whole pairs, so that
// a call in place reads both members before it writes them.
struct Pair {
    int i, k;        // element offsets; k < 0: a single element behind rotary_dim
};
__device__ __forceinline__ int pair_count(const Args& a) { return a.rot / 2 + (a.head_dim - a.rot); }
__device__ __forceinline__ Pair pair_at(const Args& a, int p) {
    const int half = a.rot / 2;
    if (p >= half) return Pair{a.rot + p - half, -1};
    return a.interleaved ? Pair{2 * p, 2 * p + 1} : Pair{p, half + p};
}

template <class Fmt, int Mode, bool Bwd>
__global__ void __launch_bounds__(kThreads) heads_general_kernel(const __grid_constant__ Args a) {
    using T = typename Fmt::T;
    extern __shared__ float sh[];     // tables [kWarps][rot], gradient: sums [kWarps][head_dim]
    const int which = (int)blockIdx.x >= a.t[0].ctas;
    const HeadsArg& t = a.t[which];
    const int cta = (int)blockIdx.x - (which ? a.t[0].ctas : 0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* cs = sh + warp * a.rot;
    float* sn = cs + a.rot / 2;
    float* sums = sh + kWarps * a.rot + warp * a.head_dim;
    pdl_wait();
    pdl_trigger();
    if constexpr (Bwd) {
        for (int d = lane; d < a.head_dim; d += 32) sums[d] = 0.f;
        __syncwarp();
    }
    const int pairs = pair_count(a);
    const unsigned items = items_of(a, t);
    for (unsigned item = cta * kWarps + warp; item < items; item += t.ctas * kWarps) {
        Item at;
        at.open(a, t, item, 1);
        const unsigned token = at.token;
        fill_table<Fmt>(a, position(a, at.b, at.s), cs, lane);
        const T* xt = at.row(static_cast<const T*>(t.x), t.sx);
        const T* dt = at.row(static_cast<const T*>(t.dy), t.sdy);
        T* yt = at.row(static_cast<T*>(t.y), t.sy);
        for (int h = at.head; h < at.end; ++h) {
            const T* x = xt + h * t.sx.h;
            T* y = yt + h * t.sy.h;
            if constexpr (!Bwd) {
                float r = 1.f;
                if constexpr (Mode == kNorm) {
                    float ss = 0.f;
                    for (int d = lane; d < a.head_dim; d += 32) {
                        const float v = Fmt::to_f32(x[d]);
                        ss += v * v;
                    }
                    r = rsqrtf(sum_lanes<32>(ss, 32, lane) * a.inv_dim + a.eps);
                    if (t.inv_rms && lane == 0) t.inv_rms[(int64_t)token * t.heads + h] = r;
                }
                for (int p = lane; p < pairs; p += 32) {
                    const Pair e = pair_at(a, p);
                    float u = Fmt::to_f32(x[e.i]);
                    if constexpr (Mode == kNorm) u *= r * __ldg(t.gamma + e.i);
                    if (e.k < 0) {
                        y[e.i] = Fmt::from_f32(u);
                        continue;
                    }
                    float v = Fmt::to_f32(x[e.k]);
                    if constexpr (Mode == kNorm) v *= r * __ldg(t.gamma + e.k);
                    y[e.i] = Fmt::from_f32(u * cs[p] - v * sn[p]);
                    y[e.k] = Fmt::from_f32(u * sn[p] + v * cs[p]);
                }
            } else {
                const T* dy = dt + h * t.sdy.h;
                const float r = __ldg(t.inv_rms + (int64_t)token * t.heads + h);
                float dot = 0.f;
                for (int p = lane; p < pairs; p += 32) {
                    const Pair e = pair_at(a, p);
                    float u = Fmt::to_f32(dy[e.i]);
                    if (e.k >= 0) {
                        const float w = Fmt::to_f32(dy[e.k]);
                        const float v = u * sn[p] + w * cs[p];
                        u = u * cs[p] - w * sn[p];
                        const float m = v * (Fmt::to_f32(x[e.k]) * r);
                        sums[e.k] += m;
                        dot += m * __ldg(t.gamma + e.k);
                    }
                    const float m = u * (Fmt::to_f32(x[e.i]) * r);
                    sums[e.i] += m;
                    dot += m * __ldg(t.gamma + e.i);
                }
                const float m = sum_lanes<32>(dot, 32, lane) * a.inv_dim * r;
                for (int p = lane; p < pairs; p += 32) {
                    const Pair e = pair_at(a, p);
                    float u = Fmt::to_f32(dy[e.i]), v = 0.f, xk = 0.f;
                    const float xi = Fmt::to_f32(x[e.i]);
                    if (e.k >= 0) {
                        const float w = Fmt::to_f32(dy[e.k]);
                        xk = Fmt::to_f32(x[e.k]);
                        v = u * sn[p] + w * cs[p];
                        u = u * cs[p] - w * sn[p];
                    }
                    y[e.i] = Fmt::from_f32(r * (u * __ldg(t.gamma + e.i) - xi * m));
                    if (e.k >= 0) y[e.k] = Fmt::from_f32(r * (v * __ldg(t.gamma + e.k) - xk * m));
                }
            }
        }
    }
    if constexpr (Bwd) {
        __syncthreads();
        for (int d = threadIdx.x; d < a.head_dim; d += kThreads) {
            float v = 0.f;
            for (int w = 0; w < kWarps; ++w) v += sh[kWarps * a.rot + w * a.head_dim + d];
            t.partial[(int64_t)cta * a.head_dim + d] = v;
        }
    }
}

// ---------------------------------------------------------------- dgamma
// Adds the CTAs' partial rows in a fixed order: 32 columns a CTA, eight row lanes.
__global__ void __launch_bounds__(kThreads) dgamma_kernel(const __grid_constant__ Args a) {
    __shared__ float part[kWarps][32];
    const HeadsArg& t = a.t[blockIdx.y];
    const int d = blockIdx.x * 32 + (threadIdx.x & 31), row0 = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    float v = 0.f;
    if (t.dgamma && d < a.head_dim) {
#pragma unroll 4
        for (int r = row0; r < t.ctas; r += kWarps) v += t.partial[(int64_t)r * a.head_dim + d];
    }
    part[row0][threadIdx.x & 31] = v;
    __syncthreads();
    if (row0 == 0 && t.dgamma && d < a.head_dim) {
        float s = 0.f;
        for (int w = 0; w < kWarps; ++w) s += part[w][threadIdx.x];
        t.dgamma[d] = s;
    }
}

// ---------------------------------------------------------------- host: strided buffers
struct View {
    const char* p;
    int64_t n[3];        // batch, seq, heads
    int64_t s[3];        // strides in elements (0 where the size is 1)
};

View view_of(const tb_heads* t, int64_t batch, int64_t seq) {
    View v{static_cast<const char*>(t->data), {batch, seq, t->heads},
           {t->stride_batch, t->stride_seq, t->stride_head}};
    for (int i = 0; i < 3; ++i)
        if (v.n[i] <= 1) v.s[i] = 0;
    return v;
}

// Elements from the first to behind the last one; false when that leaves 2^60.
bool extent(const View& v, int64_t dim, int64_t* out) {
    __int128 e = dim;
    for (int i = 0; i < 3; ++i) e += (__int128)(v.n[i] - 1) * v.s[i];
    if (e > ((__int128)1 << 60)) return false;
    *out = (int64_t)e;
    return true;
}

// Whether no two (batch, seq, head) rows of `dim` elements share one, decided by
// nesting: each stride reaches over everything that the smaller strides span.  `order`
// receives the sizes above 1, by falling stride.
bool nested(const View& v, int64_t dim, int (&order)[3], int* count) {
    int n = 0;
    for (int i = 0; i < 3; ++i)
        if (v.n[i] > 1) order[n++] = i;
    std::sort(order, order + n, [&](int x, int y) { return v.s[x] > v.s[y]; });
    *count = n;
    int64_t inner = dim;
    for (int i = n - 1; i >= 0; --i) {
        if (v.s[order[i]] < inner) return false;
        inner += (v.n[order[i]] - 1) * v.s[order[i]];
    }
    return true;
}

bool meet(const View& a, const View& b, const int64_t (&s)[3], const int* order, int count, int at,
          int64_t delta, int64_t dim) {
    if (at == count) return delta > -dim && delta < dim;
    const int i = order[at];
    const int64_t step = s[i];
    // (row of b) - (row of a) = k with -(a.n - 1) <= k <= b.n - 1; what the inner strides
    // add is below one step in size
    int64_t k = -delta / step;
    for (int64_t c = k - 1; c <= k + 1; ++c)
        if (c >= -(a.n[i] - 1) && c <= b.n[i] - 1 &&
            meet(a, b, s, order, count, at + 1, delta + c * step, dim))
            return true;
    return false;
}

// Whether an output view shares an element with another view.  Exact where both walk
// memory by the same strides (slices of one buffer); otherwise any common address range
// counts as shared.
bool shares(const View& out, const View& other, int64_t dim, size_t es) {
    int64_t ea = 0, eb = 0;
    if (!extent(out, dim, &ea) || !extent(other, dim, &eb)) return true;
    if (!overlap(range_of(out.p, ea, es), range_of(other.p, eb, es))) return false;
    View both = out;
    for (int i = 0; i < 3; ++i) {
        if (out.n[i] > 1 && other.n[i] > 1 && out.s[i] != other.s[i]) return true;
        both.s[i] = out.n[i] > 1 ? out.s[i] : other.s[i];
        both.n[i] = std::max(out.n[i], other.n[i]);
    }
    int order[3], count = 0;
    if (!nested(both, dim, order, &count)) return true;
    const int64_t delta = (int64_t)(reinterpret_cast<uintptr_t>(other.p) -
                                    reinterpret_cast<uintptr_t>(out.p)) / (int64_t)es;
    return meet(out, other, both.s, order, count, 0, delta, dim);
}

// The very same rows: a call in place.
bool same(const View& a, const View& b) {
    return a.p == b.p && a.n[0] == b.n[0] && a.n[1] == b.n[1] && a.n[2] == b.n[2] &&
           a.s[0] == b.s[0] && a.s[1] == b.s[1] && a.s[2] == b.s[2];
}

tb_status check_view(const tb_heads* t, int64_t batch, int64_t seq, int64_t dim, size_t es, View* v) {
    if (t->heads < 0 || t->stride_batch < 0 || t->stride_seq < 0 || t->stride_head < 0)
        return TB_ERR_INVALID_VALUE;
    *v = view_of(t, batch, seq);
    if (batch == 0 || seq == 0 || t->heads == 0) return TB_OK;
    if (!t->data) return TB_ERR_INVALID_VALUE;
    int64_t e = 0;
    if (t->heads > (1 << 20) || !extent(*v, dim, &e)) return TB_ERR_INVALID_VALUE;
    return aligned_to(t->data, es) ? TB_OK : TB_ERR_MISALIGNED;
}

struct Call {
    int64_t batch, seq, dim;
    tb_dtype dtype;
    bool bwd_norm, norm;
    int n;                       // tensors (1 or 2)
    View in[2], dy[2], out[2];
};

tb_status check_angles(const tb_rope_angles* r, int64_t dim, int64_t batch, int64_t seq) {
    if (!r) return TB_ERR_INVALID_VALUE;
    if (r->rotary_dim < 0 || r->rotary_dim > dim || r->rotary_dim % 2) return TB_ERR_INVALID_VALUE;
    if (r->layout != TB_ROPE_HALF && r->layout != TB_ROPE_INTERLEAVED) return TB_ERR_INVALID_VALUE;
    if (!std::isfinite(r->magnitude)) return TB_ERR_INVALID_VALUE;
    if (r->positions_stride < 0) return TB_ERR_INVALID_VALUE;
    if (batch > 0 && seq > 0 && r->positions_stride > 0 && r->positions_stride < seq && batch > 1)
        return TB_ERR_INVALID_VALUE;
    if (batch > 1 && r->positions_stride > (1ll << 60) / batch) return TB_ERR_INVALID_VALUE;
    if (r->rotary_dim > 0 && !r->freqs) return TB_ERR_INVALID_VALUE;
    if (!aligned_to(r->freqs, 8) || !aligned_to(r->positions, 8)) return TB_ERR_MISALIGNED;
    return TB_OK;
}

// Whether a view's rows can be read by vectors of E elements.
bool fits(const View& v, int E, size_t es) {
    if (!aligned_to(v.p, E * es)) return false;
    for (int i = 0; i < 3; ++i)
        if (v.s[i] % E) return false;
    return true;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Head groups of one token that a warp takes: all, so that it forms the token's sines once,
// unless that would leave warps of the resident grid without work.
//
// Forward: one item a warp, and the hardware deals the CTAs out as SMs come free, which a grid of
// resident CTAs cannot (the SMs of the two dies are not equally fast): bf16 4 x 4,096 tokens of 64
// heads of 128 rotated in 83.2 us, 84.6 with two items a warp, 91.9 with four.  The gradient keeps
// its dgamma sums in registers, so its grid is the resident one.
template <class Fmt, int E, int NU, int Lanes>
tb_status launch_lanes(Args a, const Call& c, int sms, cudaStream_t st) {
    const int per_step = 32 / a.lanes;
    const void* kernel =
        c.bwd_norm ? reinterpret_cast<const void*>(&heads_bwd_kernel<Fmt, E, NU, Lanes>)
        : c.norm   ? reinterpret_cast<const void*>(&heads_fwd_kernel<Fmt, E, NU, kNorm, Lanes>)
                   : reinterpret_cast<const void*>(&heads_fwd_kernel<Fmt, E, NU, kRope, Lanes>);
    int rows = 1;                     // of a warp's table of sines
    for (int i = 0; i < c.n; ++i) rows = std::max(rows, per_step / a.t[i].heads);
    size_t smem = sizeof(float) * kWarps * a.rot * rows;
    if (c.bwd_norm) smem = (smem + sizeof(float) * kWarps * a.head_dim + 15) / 16 * 16 + kWarps * 2 * kSlotBytes<Fmt, E, NU>;
    const int resident = resident_ctas_per_sm(kernel, kThreads, smem);
    if (resident == 0) return TB_ERR_CUDA;
    const int64_t grid_ctas = (int64_t)sms * std::min(resident, kBwdCtasPerSm);
    // What a token of each tensor costs, in head groups: its groups, half of one for an item's
    // addresses and 0.3 for every 32 pairs whose sines are formed.  The gradient's CTAs are dealt by
    // it.  By the groups alone, the keys' CTAs were the last to end: 4 x 4,096 tokens, 32 query heads
    // of 128, bf16, with 8 / 4 / 1 key heads took 98 / 113 / 149 us, so they take 84 / 77 / 73.
    double cost[2] = {0, 0};
    const double sines = 0.3 * (double)ceil_div(a.rot / 2, 32);
    for (int i = 0; i < c.n; ++i) {
        const int shared = std::max(1, per_step / a.t[i].heads);
        cost[i] = ((double)ceil_div(a.t[i].heads, per_step) + 0.5) / shared + sines;
    }
    for (int i = 0; i < c.n; ++i) {
        HeadsArg& t = a.t[i];
        const int64_t steps = ceil_div(t.heads, per_step);
        t.tokens = std::max(1, per_step / t.heads);
        // the tensor's share of the grid, by its head groups
        const int64_t share = std::max<int64_t>(1, (int64_t)((double)grid_ctas * cost[i] / (cost[0] + cost[1])));
        t.chunks = (int)std::min(steps, ceil_div(share * kWarps, a.tokens));
        t.steps = (int)ceil_div(steps, t.chunks);
        t.chunks = (int)ceil_div(steps, t.steps);
        const int64_t ctas = ceil_div(t.tokens > 1 ? ceil_div(a.tokens, t.tokens) : (int64_t)a.tokens * t.chunks, kWarps);
        t.ctas = (int)(c.bwd_norm ? std::min(share, ctas) : ctas);
    }
    if (c.n == 1) a.t[1].ctas = 0;
    if (c.bwd_norm) a.t[1].partial = a.t[0].partial + (int64_t)a.t[0].ctas * a.head_dim;
    const dim3 grid((unsigned)(a.t[0].ctas + a.t[1].ctas));
    cudaError_t e;
    if (c.bwd_norm) e = launch_pdl(heads_bwd_kernel<Fmt, E, NU, Lanes>, grid, dim3(kThreads), smem, st, a);
    else if (c.norm) e = launch_pdl(heads_fwd_kernel<Fmt, E, NU, kNorm, Lanes>, grid, dim3(kThreads), smem, st, a);
    else e = launch_pdl(heads_fwd_kernel<Fmt, E, NU, kRope, Lanes>, grid, dim3(kThreads), smem, st, a);
    if (e != cudaSuccess) return TB_ERR_CUDA;
    if (c.bwd_norm &&
        launch_pdl(dgamma_kernel, dim3((unsigned)ceil_div(a.head_dim, 32), (unsigned)c.n),
                   dim3(kThreads), 0, st, a) != cudaSuccess)
        return TB_ERR_CUDA;
    return launch_status();
}

// Heads of 64, 128 and 256 elements in 16-byte vectors know their number of lanes when compiled, and
// so do those of 80, 96 and 192.
template <class Fmt, int E, int NU>
tb_status launch_vec(Args a, const Call& c, int sms, cudaStream_t st) {
    a.lanes = (int)ceil_div(a.head_dim / (2 * E), NU);
    if constexpr (E * sizeof(typename Fmt::T) == 16) {
        constexpr int k80 = sizeof(typename Fmt::T) == 2 ? 5 : 10, k96 = sizeof(typename Fmt::T) == 2 ? 6 : 24;
        if (a.lanes == k80) return launch_lanes<Fmt, E, NU, k80>(a, c, sms, st);
        if (a.lanes == k96) return launch_lanes<Fmt, E, NU, k96>(a, c, sms, st);
        if (a.lanes == 12) return launch_lanes<Fmt, E, NU, 12>(a, c, sms, st);
        if (a.lanes == 4) return launch_lanes<Fmt, E, NU, 4>(a, c, sms, st);
        if (a.lanes == 8) return launch_lanes<Fmt, E, NU, 8>(a, c, sms, st);
        if (a.lanes == 16) return launch_lanes<Fmt, E, NU, 16>(a, c, sms, st);
        if (a.lanes == 32) return launch_lanes<Fmt, E, NU, 32>(a, c, sms, st);
    }
    return launch_lanes<Fmt, E, NU, 0>(a, c, sms, st);
}

template <class Fmt>
tb_status launch_general(Args a, const Call& c, int sms, cudaStream_t st) {
    const void* kernel =
        c.bwd_norm ? reinterpret_cast<const void*>(&heads_general_kernel<Fmt, kNorm, true>)
        : c.norm   ? reinterpret_cast<const void*>(&heads_general_kernel<Fmt, kNorm, false>)
                   : reinterpret_cast<const void*>(&heads_general_kernel<Fmt, kRope, false>);
    const size_t smem = sizeof(float) * kWarps * (a.rot + (c.bwd_norm ? a.head_dim : 0));
    const int per_sm = std::min(resident_ctas_per_sm(kernel, kThreads, smem), kBwdCtasPerSm);
    if (per_sm == 0) return TB_ERR_CUDA;
    int64_t all = 0;
    for (int i = 0; i < c.n; ++i) all += a.t[i].heads;
    for (int i = 0; i < c.n; ++i) {
        HeadsArg& t = a.t[i];
        t.tokens = 1;
        const int64_t share = std::max<int64_t>(1, (int64_t)sms * per_sm * t.heads / all);
        t.chunks = (int)std::min<int64_t>(t.heads, ceil_div(share * kWarps, a.tokens));
        t.steps = (int)ceil_div(t.heads, t.chunks);
        t.chunks = (int)ceil_div(t.heads, t.steps);
        const int64_t ctas = ceil_div((int64_t)a.tokens * t.chunks, kWarps);
        t.ctas = (int)(c.bwd_norm ? std::min(share, ctas) : ctas);
    }
    if (c.n == 1) a.t[1].ctas = 0;
    if (c.bwd_norm) a.t[1].partial = a.t[0].partial + (int64_t)a.t[0].ctas * a.head_dim;
    const dim3 grid((unsigned)(a.t[0].ctas + a.t[1].ctas));
    cudaError_t e;
    if (c.bwd_norm) e = launch_pdl(heads_general_kernel<Fmt, kNorm, true>, grid, dim3(kThreads), smem, st, a);
    else if (c.norm) e = launch_pdl(heads_general_kernel<Fmt, kNorm, false>, grid, dim3(kThreads), smem, st, a);
    else e = launch_pdl(heads_general_kernel<Fmt, kRope, false>, grid, dim3(kThreads), smem, st, a);
    if (e != cudaSuccess) return TB_ERR_CUDA;
    if (c.bwd_norm &&
        launch_pdl(dgamma_kernel, dim3((unsigned)ceil_div(a.head_dim, 32), (unsigned)c.n),
                   dim3(kThreads), 0, st, a) != cudaSuccess)
        return TB_ERR_CUDA;
    return launch_status();
}

// The widest vectors that the sizes, strides and pointers allow: 16 bytes, 8, then two
// elements; a head goes to at most 32 lanes of one unit (two for the narrowest).
template <class Fmt>
tb_status dispatch(const Args& a, const Call& c, int sms, cudaStream_t st) {
    constexpr size_t es = sizeof(typename Fmt::T);
    auto ok = [&](int E, int nu) {
        if (a.head_dim % (2 * E) || a.rot % (2 * E) || a.head_dim / (2 * E) > 32 * nu) return false;
        for (int i = 0; i < c.n; ++i) {
            if (!fits(c.in[i], E, es) || !fits(c.out[i], E, es)) return false;
            if (c.bwd_norm && !fits(c.dy[i], E, es)) return false;
        }
        return true;
    };
    if constexpr (es == 2) {
        if (ok(8, 1)) return launch_vec<Fmt, 8, 1>(a, c, sms, st);
        if (ok(4, 1)) return launch_vec<Fmt, 4, 1>(a, c, sms, st);
    } else {
        if (ok(4, 1)) return launch_vec<Fmt, 4, 1>(a, c, sms, st);
    }
    if (ok(2, 1)) return launch_vec<Fmt, 2, 1>(a, c, sms, st);
    if (ok(2, 2)) return launch_vec<Fmt, 2, 2>(a, c, sms, st);
    return launch_general<Fmt>(a, c, sms, st);
}

tb_status start(const Args& a, const Call& c, void* stream) {
    int dev = 0;
    DeviceInfo info{};
    if (!current_device_info(&dev, &info)) return TB_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (c.dtype) {
        case TB_F32: return dispatch<F32>(a, c, info.sm_count, st);
        case TB_BF16: return dispatch<BF16>(a, c, info.sm_count, st);
        default: return dispatch<F16>(a, c, info.sm_count, st);
    }
}

Strides strides_of(const View& v) { return Strides{v.s[0], v.s[1], v.s[2]}; }

// Shared by the four entry points.  `in`, `dy`, `out`: queries and keys (keys may be
// NULL); gamma, inv_rms, dgamma, workspace as the entry point has them.
struct Entry {
    const tb_heads* in[2];
    const tb_heads* dy[2];
    const tb_heads* out[2];
    const float* gamma[2];
    float* inv_rms[2];
    float* dgamma[2];
    void* workspace;
    size_t workspace_bytes;
    float eps;
    bool norm, bwd_norm;
    float turn;
};

bool small_ok(const void* p, bool optional, tb_status* why) {
    if (!p) {
        *why = TB_ERR_INVALID_VALUE;
        return optional;
    }
    *why = TB_ERR_MISALIGNED;
    return aligned_to(p, 4);
}

tb_status run(const Entry& e, int64_t batch, int64_t seq, int64_t dim, const tb_rope_angles* r,
              tb_dtype dtype, void* stream) {
    if (batch < 0 || seq < 0 || dim < 1 || dim > kMaxHeadDim) return TB_ERR_INVALID_VALUE;
    if (!dtype_valid(dtype)) return TB_ERR_UNSUPPORTED_DTYPE;
    if (!e.in[0] || !e.out[0] || !e.in[1] != !e.out[1]) return TB_ERR_INVALID_VALUE;
    if (e.bwd_norm && (!e.dy[0] || !e.dy[1] != !e.in[1])) return TB_ERR_INVALID_VALUE;
    if (e.norm && !(e.eps >= 0.f && std::isfinite(e.eps))) return TB_ERR_INVALID_VALUE;
    tb_status why = check_angles(r, dim, batch, seq);
    if (why != TB_OK) return why;
    const size_t es = dtype_size(dtype);
    if (batch > 0 && seq > INT32_MAX / batch) return TB_ERR_INVALID_VALUE;
    const int64_t tokens = batch * seq;

    Call c{};
    c.batch = batch, c.seq = seq, c.dim = dim, c.dtype = dtype;
    c.norm = e.norm, c.bwd_norm = e.bwd_norm;
    c.n = e.in[1] ? 2 : 1;
    bool any = false;
    for (int i = 0; i < c.n; ++i) {
        if ((why = check_view(e.in[i], batch, seq, dim, es, &c.in[i])) != TB_OK) return why;
        if ((why = check_view(e.out[i], batch, seq, dim, es, &c.out[i])) != TB_OK) return why;
        if (e.out[i]->heads != e.in[i]->heads) return TB_ERR_INVALID_VALUE;
        if (e.bwd_norm) {
            if ((why = check_view(e.dy[i], batch, seq, dim, es, &c.dy[i])) != TB_OK) return why;
            if (e.dy[i]->heads != e.in[i]->heads) return TB_ERR_INVALID_VALUE;
        }
        if (tokens > 0 && e.in[i]->heads > (INT64_MAX >> 16) / tokens) return TB_ERR_INVALID_VALUE;
        any = any || (tokens > 0 && e.in[i]->heads > 0);
        if (e.norm || e.bwd_norm) {
            if (!small_ok(e.gamma[i], false, &why)) return why;
            const bool needs = e.bwd_norm && tokens > 0 && e.in[i]->heads > 0;
            if (!small_ok(e.inv_rms[i], !needs, &why)) return why;
            if (e.bwd_norm && !small_ok(e.dgamma[i], false, &why)) return why;
        }
    }

    // buffers that the call writes, against all others
    Range small_out[4], read[8];
    int n_small = 0, n_read = 0;
    for (int i = 0; i < c.n; ++i) {
        const int64_t stats = tokens * e.in[i]->heads;
        if (e.norm && e.inv_rms[i]) small_out[n_small++] = range_of(e.inv_rms[i], stats, 4);
        if (e.bwd_norm) {
            small_out[n_small++] = range_of(e.dgamma[i], dim, 4);
            read[n_read++] = range_of(e.inv_rms[i], stats, 4);
        }
        if (e.norm || e.bwd_norm) read[n_read++] = range_of(e.gamma[i], dim, 4);
    }
    read[n_read++] = range_of(r->freqs, r->rotary_dim / 2, 8);
    if (r->positions && tokens > 0)
        read[n_read++] = range_of(r->positions, (batch - 1) * r->positions_stride + seq, 8);
    size_t ws_need = 0;
    if (e.bwd_norm && any) {
        why = tb_qk_norm_rope_bwd_workspace_size(batch, seq, e.in[0]->heads,
                                                 c.n > 1 ? e.in[1]->heads : 0, dim, dtype, &ws_need);
        if (why != TB_OK) return why;
        if (!e.workspace || e.workspace_bytes < ws_need) return TB_ERR_WORKSPACE;
        if (!aligned_to(e.workspace, 16)) return TB_ERR_MISALIGNED;
        small_out[n_small++] = range_of(e.workspace, (int64_t)ws_need, 1);
    }
    for (int i = 0; i < n_small; ++i) {
        for (int j = i + 1; j < n_small; ++j)
            if (overlap(small_out[i], small_out[j])) return TB_ERR_ALIAS;
        for (int j = 0; j < n_read; ++j)
            if (overlap(small_out[i], read[j])) return TB_ERR_ALIAS;
    }
    for (int i = 0; i < c.n && tokens > 0; ++i) {
        if (e.out[i]->heads == 0) continue;
        int order[3], count = 0;
        if (!nested(c.out[i], dim, order, &count)) return TB_ERR_ALIAS;
        int64_t ext = 0;
        extent(c.out[i], dim, &ext);
        const Range out = range_of(c.out[i].p, ext, es);
        for (int j = 0; j < n_read; ++j)
            if (overlap(out, read[j])) return TB_ERR_ALIAS;
        for (int j = 0; j < n_small; ++j) {
            if (overlap(out, small_out[j])) return TB_ERR_ALIAS;
        }
        for (int j = 0; j < c.n; ++j) {
            if (e.in[j]->heads == 0) continue;
            if (!(i == j && same(c.out[i], c.in[j])) && shares(c.out[i], c.in[j], dim, es))
                return TB_ERR_ALIAS;
            if (e.bwd_norm && !(i == j && same(c.out[i], c.dy[j])) &&
                shares(c.out[i], c.dy[j], dim, es))
                return TB_ERR_ALIAS;
            if (j != i && shares(c.out[i], c.out[j], dim, es)) return TB_ERR_ALIAS;
        }
    }
    for (int i = 0; i < c.n && tokens > 0; ++i) {   // small outputs against the big inputs
        if (e.in[i]->heads == 0) continue;
        int64_t ext = 0;
        for (int j = 0; j < n_small; ++j) {
            extent(c.in[i], dim, &ext);
            if (overlap(small_out[j], range_of(c.in[i].p, ext, es))) return TB_ERR_ALIAS;
            if (e.bwd_norm) {
                extent(c.dy[i], dim, &ext);
                if (overlap(small_out[j], range_of(c.dy[i].p, ext, es))) return TB_ERR_ALIAS;
            }
        }
    }

    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (e.bwd_norm)   // no row of a tensor: its sums are empty
        for (int i = 0; i < c.n; ++i)
            if ((tokens == 0 || e.in[i]->heads == 0) &&
                cudaMemsetAsync(e.dgamma[i], 0, dim * sizeof(float), st) != cudaSuccess)
                return TB_ERR_CUDA;
    if (!any) return TB_OK;

    Args a{};
    int used = 0;
    for (int i = 0; i < c.n; ++i) {
        if (e.in[i]->heads == 0) continue;
        HeadsArg& t = a.t[used];
        t.x = c.in[i].p;
        t.y = const_cast<char*>(c.out[i].p);
        t.sx = strides_of(c.in[i]);
        t.sy = strides_of(c.out[i]);
        if (e.bwd_norm) {
            t.dy = c.dy[i].p;
            t.sdy = strides_of(c.dy[i]);
            t.dgamma = e.dgamma[i];
            t.partial = static_cast<float*>(e.workspace);
        }
        t.gamma = e.gamma[i];
        t.inv_rms = e.inv_rms[i];
        t.heads = (int)e.in[i]->heads;
        c.in[used] = c.in[i], c.out[used] = c.out[i], c.dy[used] = c.dy[i];
        ++used;
    }
    c.n = used;
    a.freqs = reinterpret_cast<const unsigned long long*>(r->freqs);
    a.positions = r->positions;
    a.pos_stride = batch > 1 ? r->positions_stride : 0;
    a.offset = r->offset;
    a.tokens = (unsigned)tokens;
    a.seq = (unsigned)seq;
    a.head_dim = (int)dim;
    a.rot = r->rotary_dim;
    a.interleaved = r->layout == TB_ROPE_INTERLEAVED;
    a.magnitude = r->magnitude;
    a.turn = e.turn;
    a.eps = e.eps;
    a.inv_dim = 1.0f / (float)dim;
    return start(a, c, stream);
}

}  // namespace
}  // namespace tb

extern "C" tb_status tb_rope_freqs(int rotary_dim, double base, const tb_rope_scaling* scaling,
                                   uint64_t* freqs, float* magnitude) {
    if (rotary_dim < 0 || rotary_dim % 2 || rotary_dim > tb::kMaxHeadDim || !(base > 0) ||
        !std::isfinite(base) || !magnitude || (rotary_dim > 0 && !freqs))
        return TB_ERR_INVALID_VALUE;
    tb_rope_scaling s{};
    if (scaling) s = *scaling;
    const bool by_parts = s.kind == TB_ROPE_SCALE_YARN || s.kind == TB_ROPE_SCALE_WAVELENGTH;
    if (s.kind < TB_ROPE_SCALE_NONE || s.kind > TB_ROPE_SCALE_WAVELENGTH) return TB_ERR_INVALID_VALUE;
    if (s.kind != TB_ROPE_SCALE_NONE && !(s.factor >= 1.0 && std::isfinite(s.factor)))
        return TB_ERR_INVALID_VALUE;
    if (by_parts && !(s.original_context > 0 && std::isfinite(s.original_context) && s.fast > s.slow &&
                      s.slow > 0 && std::isfinite(s.fast)))
        return TB_ERR_INVALID_VALUE;
    if (s.kind == TB_ROPE_SCALE_YARN && !(base > 1)) return TB_ERR_INVALID_VALUE;
    const double pi = 3.14159265358979323846;
    const int half = rotary_dim / 2;
    if (s.kind == TB_ROPE_SCALE_NTK) {
        // the base is raised so that the slowest frequency falls by the factor
        if (rotary_dim > 2) base *= pow(s.factor, (double)rotary_dim / (rotary_dim - 2));
    }
    double low = 0, high = 1;
    if (s.kind == TB_ROPE_SCALE_YARN && half > 0) {
        // the pair whose frequency makes n turns over the original context
        auto pair_of = [&](double n) {
            return rotary_dim * log(s.original_context / (n * 2 * pi)) / (2 * log(base));
        };
        low = fmax(floor(pair_of(s.fast)), 0.0);
        high = fmin(ceil(pair_of(s.slow)), (double)(rotary_dim - 1));
        if (low == high) high += 0.001;
        // all pairs on one side of the blend: none makes as many turns as `slow` (all are
        // divided), or none as few as `fast` (all keep their frequency)
        if (low > high && high < 0) low = high - 1;
        else if (low > high) high = low + 1;
    }
    for (int i = 0; i < half; ++i) {
        double w = pow(base, -2.0 * i / rotary_dim);
        if (s.kind == TB_ROPE_SCALE_LINEAR) w /= s.factor;
        if (s.kind == TB_ROPE_SCALE_YARN) {
            const double ramp = fmin(fmax((i - low) / (high - low), 0.0), 1.0);
            w = w / s.factor * ramp + w * (1 - ramp);
        }
        if (s.kind == TB_ROPE_SCALE_WAVELENGTH) {
            // turns over the original context: many keep their frequency, few are
            // stretched, between them a linear blend
            const double turns = s.original_context * w / (2 * pi);
            const double keep = fmin(fmax((turns - s.slow) / (s.fast - s.slow), 0.0), 1.0);
            w = (1 - keep) * w / s.factor + keep * w;
        }
        double turn = w / (2 * pi);
        turn -= floor(turn);
        const double scaled = nearbyint(ldexp(turn, 64));
        freqs[i] = scaled >= 18446744073709551616.0 ? 0 : (uint64_t)scaled;
    }
    *magnitude = s.kind == TB_ROPE_SCALE_YARN ? (float)(0.1 * log(s.factor) + 1.0) : 1.0f;
    return TB_OK;
}

extern "C" tb_status tb_rope(const tb_heads* q, const tb_heads* k, const tb_heads* q_out,
                             const tb_heads* k_out, int64_t batch, int64_t seq, int64_t head_dim,
                             const tb_rope_angles* angles, tb_dtype dtype, void* stream) {
    tb::Entry e{};
    e.in[0] = q, e.in[1] = k, e.out[0] = q_out, e.out[1] = k_out;
    e.turn = 1.f;
    return tb::run(e, batch, seq, head_dim, angles, dtype, stream);
}

extern "C" tb_status tb_rope_bwd(const tb_heads* dq_out, const tb_heads* dk_out, const tb_heads* dq,
                                 const tb_heads* dk, int64_t batch, int64_t seq, int64_t head_dim,
                                 const tb_rope_angles* angles, tb_dtype dtype, void* stream) {
    tb::Entry e{};
    e.in[0] = dq_out, e.in[1] = dk_out, e.out[0] = dq, e.out[1] = dk;
    e.turn = -1.f;
    return tb::run(e, batch, seq, head_dim, angles, dtype, stream);
}

extern "C" tb_status tb_qk_norm_rope(const tb_heads* q, const tb_heads* k, const float* gamma_q,
                                     const float* gamma_k, float eps, const tb_heads* q_out,
                                     const tb_heads* k_out, float* inv_rms_q, float* inv_rms_k,
                                     int64_t batch, int64_t seq, int64_t head_dim,
                                     const tb_rope_angles* angles, tb_dtype dtype, void* stream) {
    tb::Entry e{};
    e.in[0] = q, e.in[1] = k, e.out[0] = q_out, e.out[1] = k_out;
    e.gamma[0] = gamma_q, e.gamma[1] = gamma_k;
    e.inv_rms[0] = inv_rms_q, e.inv_rms[1] = inv_rms_k;
    e.eps = eps;
    e.norm = true;
    e.turn = 1.f;
    return tb::run(e, batch, seq, head_dim, angles, dtype, stream);
}

extern "C" tb_status tb_qk_norm_rope_bwd_workspace_size(int64_t batch, int64_t seq, int64_t heads_q,
                                                        int64_t heads_k, int64_t head_dim,
                                                        tb_dtype dtype, size_t* bytes) {
    if (!bytes || batch < 0 || seq < 0 || heads_q < 0 || heads_k < 0 || head_dim < 1 ||
        head_dim > tb::kMaxHeadDim)
        return TB_ERR_INVALID_VALUE;
    if (!tb::dtype_valid(dtype)) return TB_ERR_UNSUPPORTED_DTYPE;
    *bytes = 0;
    if (batch == 0 || seq == 0 || heads_q + heads_k == 0) return TB_OK;
    int dev = 0;
    tb::DeviceInfo info{};
    if (!tb::current_device_info(&dev, &info)) return TB_ERR_CUDA;
    // one partial row per CTA; each tensor has one CTA at least
    *bytes = sizeof(float) * (size_t)head_dim * ((size_t)info.sm_count * tb::kBwdCtasPerSm + 2);
    return TB_OK;
}

extern "C" tb_status tb_qk_norm_rope_bwd(const tb_heads* dq_out, const tb_heads* dk_out,
                                         const tb_heads* q, const tb_heads* k,
                                         const float* inv_rms_q, const float* inv_rms_k,
                                         const float* gamma_q, const float* gamma_k,
                                         const tb_heads* dq, const tb_heads* dk, float* dgamma_q,
                                         float* dgamma_k, int64_t batch, int64_t seq,
                                         int64_t head_dim, const tb_rope_angles* angles,
                                         tb_dtype dtype, void* workspace, size_t workspace_bytes,
                                         void* stream) {
    tb::Entry e{};
    e.in[0] = q, e.in[1] = k, e.out[0] = dq, e.out[1] = dk, e.dy[0] = dq_out, e.dy[1] = dk_out;
    e.gamma[0] = gamma_q, e.gamma[1] = gamma_k;
    e.inv_rms[0] = const_cast<float*>(inv_rms_q), e.inv_rms[1] = const_cast<float*>(inv_rms_k);
    e.dgamma[0] = dgamma_q, e.dgamma[1] = dgamma_k;
    e.workspace = workspace;
    e.workspace_bytes = workspace_bytes;
    e.bwd_norm = true;
    e.turn = -1.f;
    return tb::run(e, batch, seq, head_dim, angles, dtype, stream);
}
