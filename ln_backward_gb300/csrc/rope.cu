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
// elements: the two halves' corresponding vectors in the half layout, two neighbouring
// vectors in the interleaved one and behind rotary_dim.  Both members of every pair are
// then in one lane: no shuffles but the norm's row sums.  32 / L heads go through a warp
// at a time; L is the number of units, not a power of two above it, so that heads of 80
// or 96 elements leave few lanes idle.  Queries and keys get CTAs of their own, so gamma
// and the dgamma sums of one tensor stay in registers.  A warp of the persistent grid
// loads its next heads, of the next token too, before it works on the present ones.
// Heads whose sizes, strides or pointers no vector width fits take the general kernels
// (one element at a time).
#include <math.h>

#include <algorithm>

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

// ---------------------------------------------------------------- vectors
template <int Bytes> struct Raw;
template <> struct Raw<16> { using V = uint4; };
template <> struct Raw<8> { using V = uint2; };
template <> struct Raw<4> { using V = unsigned; };

template <class Fmt, int E>
struct Chunk {
    using T = typename Fmt::T;
    using V = typename Raw<E * (int)sizeof(T)>::V;
    V raw;
    __device__ __forceinline__ void load(const T* p) { raw = __ldcs(reinterpret_cast<const V*>(p)); }
    __device__ __forceinline__ void get(float (&f)[E]) const {
        const T* h = reinterpret_cast<const T*>(&raw);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = Fmt::to_f32(h[e]);
    }
    __device__ __forceinline__ static void store(T* p, const float (&f)[E]) {
        V v;
        T* h = reinterpret_cast<T*>(&v);
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] = Fmt::from_f32(f[e]);
        __stcs(reinterpret_cast<V*>(p), v);
    }
};

// cos and sin of turn * pos * freq, times the magnitude.  The 32-bit fraction of a turn
// is signed, so it converts to a float in [-1, 1] of half turns with a relative error of
// 2^-24.  16-bit outputs take the hardware's sine and cosine (absolute error below
// 2^-21 on [-pi, pi], against a rounding of 2^-9 or 2^-12 of the output); fp32 outputs
// take the library's.
template <class Fmt>
__device__ __forceinline__ void cos_sin(const Args& a, long long pos, unsigned long long freq,
                                        float* c, float* s) {
    const unsigned long long phase = (unsigned long long)pos * freq;
    const float half_turns = (float)(int)(phase >> 32) * 0x1p-31f * a.turn;
    if constexpr (sizeof(typename Fmt::T) == 2) {
        const float x = half_turns * 3.14159265358979f;
        *c = __cosf(x);
        *s = __sinf(x);
    } else {
        sincospif(half_turns, s, c);
    }
    *c *= a.magnitude;
    *s *= a.magnitude;
}

// Rotates one unit: E pairs, whose frequencies are consecutive.
template <int E>
__device__ __forceinline__ void rotate(float (&u)[E], float (&v)[E], const float (&c)[E],
                                       const float (&s)[E], int interleaved) {
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            const float a0 = u[2 * e], b0 = u[2 * e + 1];
            u[2 * e] = a0 * c[e] - b0 * s[e];
            u[2 * e + 1] = a0 * s[e] + b0 * c[e];
            const float a1 = v[2 * e], b1 = v[2 * e + 1];
            v[2 * e] = a1 * c[E / 2 + e] - b1 * s[E / 2 + e];
            v[2 * e + 1] = a1 * s[E / 2 + e] + b1 * c[E / 2 + e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float p = u[e], q = v[e];
            u[e] = p * c[e] - q * s[e];
            v[e] = p * s[e] + q * c[e];
        }
    }
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
    int freq[NU];                // its first frequency
    bool live[NU], turns[NU];
    __device__ __forceinline__ void init(const Args& a, int sub) {
        const int units = a.head_dim / (2 * E), rot_units = a.rot / (2 * E);
#pragma unroll
        for (int j = 0; j < NU; ++j) {
            const int c = sub + j * a.lanes;
            live[j] = sub < a.lanes && c < units;
            turns[j] = live[j] && c < rot_units;
            const bool half = turns[j] && !a.interleaved;
            first[j] = half ? c * E : 2 * c * E;
            second[j] = half ? a.rot / 2 + c * E : 2 * c * E + E;
            freq[j] = c * E;
        }
    }
};

template <class Fmt, int E, int NU>
__device__ __forceinline__ void angles(const Args& a, const Units<E, NU>& u, long long pos,
                                       float (&c)[NU][E], float (&s)[NU][E]) {
#pragma unroll
    for (int j = 0; j < NU; ++j) {
        if (u.turns[j]) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                cos_sin<Fmt>(a, pos, __ldg(a.freqs + u.freq[j] + e), &c[j][e], &s[j][e]);
        } else {   // behind rotary_dim: unchanged
#pragma unroll
            for (int e = 0; e < E; ++e) c[j][e] = 1.f, s[j][e] = 0.f;
        }
    }
}

// Sum over a head's `lanes` lanes, in all of them.
__device__ __forceinline__ float sum_lanes(float v, int lanes, int sub) {
    if ((lanes & (lanes - 1)) == 0) {
        for (int o = 1; o < lanes; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    for (int o = 16; o; o >>= 1) {
        const float w = __shfl_down_sync(0xffffffffu, v, o);
        if (sub + o < min(lanes, 2 * o)) v += w;
    }
    return __shfl_sync(0xffffffffu, v, (int)(threadIdx.x & 31) - sub);
}

template <int E, int NU>
__device__ __forceinline__ void load_gamma(const float* gamma, const Units<E, NU>& u,
                                           float (&g)[NU][2 * E]) {
#pragma unroll
    for (int j = 0; j < NU; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e) {
            g[j][e] = u.live[j] ? __ldg(gamma + u.first[j] + e) : 0.f;
            g[j][E + e] = u.live[j] ? __ldg(gamma + u.second[j] + e) : 0.f;
        }
}

// Where a warp is: a head group of one token.
template <class T>
struct Cursor {
    unsigned item, token;
    int h0, h_end;
    const T *x, *dy;
    T* y;
    __device__ __forceinline__ void open(const Args& a, const HeadsArg& t, int per_step, long long* pos) {
        int chunk = 0;
        token = item;
        if (t.chunks > 1) {
            token = item / (unsigned)t.chunks;
            chunk = (int)(item - token * t.chunks);
        }
        unsigned b, s;
        split_token(a, token, &b, &s);
        x = static_cast<const T*>(t.x) + b * t.sx.b + s * t.sx.s;
        dy = static_cast<const T*>(t.dy) + b * t.sdy.b + s * t.sdy.s;
        y = static_cast<T*>(t.y) + b * t.sy.b + s * t.sy.s;
        h0 = chunk * t.steps * per_step;
        h_end = min(t.heads, h0 + t.steps * per_step);
        *pos = position(a, b, s);
    }
};

template <class Fmt, int E, int NU>
struct Head {                      // one lane's vectors of a head
    Chunk<Fmt, E> p[NU], q[NU];
    __device__ __forceinline__ void load(const typename Fmt::T* head, const Units<E, NU>& u, bool mine) {
#pragma unroll
        for (int j = 0; j < NU; ++j) {
            p[j].raw = {};
            q[j].raw = {};
            if (mine && u.live[j]) {
                p[j].load(head + u.first[j]);
                q[j].load(head + u.second[j]);
            }
        }
    }
};

// ---------------------------------------------------------------- forward
template <class Fmt, int E, int NU, int Mode>
__global__ void __launch_bounds__(kThreads, NU == 1 ? 3 : 2) heads_fwd_kernel(const __grid_constant__ Args a) {
    using T = typename Fmt::T;
    const int which = (int)blockIdx.x >= a.t[0].ctas;
    const HeadsArg& t = a.t[which];
    const int cta = (int)blockIdx.x - (which ? a.t[0].ctas : 0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per_step = 32 / a.lanes, grp = lane / a.lanes, sub = lane - grp * a.lanes;
    Units<E, NU> u;
    u.init(a, grp < per_step ? sub : a.lanes);
    pdl_wait();
    pdl_trigger();
    const unsigned items = a.tokens * t.chunks;
    Cursor<T> cur;
    cur.item = cta * kWarps + warp;
    if (cur.item >= items) return;
    long long pos;
    cur.open(a, t, per_step, &pos);
    Head<Fmt, E, NU> in;
    in.load(cur.x + (cur.h0 + grp) * t.sx.h, u, cur.h0 + grp < cur.h_end);
    float g[NU][2 * E], c[NU][E], sn[NU][E];
    if constexpr (Mode == kNorm) load_gamma<E, NU>(t.gamma, u, g);
    bool fresh = true, more = true;
    while (more) {
        Cursor<T> nxt = cur;
        long long pos_nxt = pos;
        bool fresh_nxt = false;
        nxt.h0 += per_step;
        if (nxt.h0 >= nxt.h_end) {
            nxt.item += t.ctas * kWarps;
            more = nxt.item < items;
            fresh_nxt = true;
            if (more) nxt.open(a, t, per_step, &pos_nxt);
        }
        Head<Fmt, E, NU> ahead;
        ahead.load(nxt.x + (nxt.h0 + grp) * t.sx.h, u, more && nxt.h0 + grp < nxt.h_end);
        if (fresh) angles<Fmt, E, NU>(a, u, pos, c, sn);

        const int h = cur.h0 + grp;
        const bool mine = h < cur.h_end && grp < per_step;
        float r = 1.f;
        if constexpr (Mode == kNorm) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                float v[E], w[E];
                in.p[j].get(v);
                in.q[j].get(w);
#pragma unroll
                for (int e = 0; e < E; ++e) ss += v[e] * v[e] + w[e] * w[e];
            }
            r = rsqrtf(sum_lanes(ss, a.lanes, sub) * a.inv_dim + a.eps);
            if (t.inv_rms && sub == 0 && mine) t.inv_rms[(int64_t)cur.token * t.heads + h] = r;
        }
        if (mine) {
            T* y = cur.y + h * t.sy.h;
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                float v[E], w[E];
                in.p[j].get(v);
                in.q[j].get(w);
                if constexpr (Mode == kNorm) {
#pragma unroll
                    for (int e = 0; e < E; ++e) v[e] *= r * g[j][e], w[e] *= r * g[j][E + e];
                }
                if (u.turns[j]) rotate<E>(v, w, c[j], sn[j], a.interleaved);
                if (u.live[j]) {
                    Chunk<Fmt, E>::store(y + u.first[j], v);
                    Chunk<Fmt, E>::store(y + u.second[j], w);
                }
            }
        }
        in = ahead;
        cur = nxt;
        pos = pos_nxt;
        fresh = fresh_nxt;
    }
}

// ---------------------------------------------------------------- gradient of the norm
// dn = the transposed rotation of dy; xhat = x * r; dxhat = dn * gamma;
// dx = r * (dxhat - xhat * mean(dxhat * xhat)); dgamma = sum of dn * xhat.
template <class Fmt, int E, int NU>
__global__ void __launch_bounds__(kThreads, 2) heads_bwd_kernel(const __grid_constant__ Args a) {
    using T = typename Fmt::T;
    extern __shared__ float sums[];   // [kWarps][head_dim]
    const int which = (int)blockIdx.x >= a.t[0].ctas;
    const HeadsArg& t = a.t[which];
    const int cta = (int)blockIdx.x - (which ? a.t[0].ctas : 0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per_step = 32 / a.lanes, grp = lane / a.lanes, sub = lane - grp * a.lanes;
    Units<E, NU> u;
    u.init(a, grp < per_step ? sub : a.lanes);
    pdl_wait();
    pdl_trigger();
    float g[NU][2 * E], acc[NU][2 * E], c[NU][E], sn[NU][E];
#pragma unroll
    for (int j = 0; j < NU; ++j)
#pragma unroll
        for (int e = 0; e < 2 * E; ++e) acc[j][e] = 0.f;

    const unsigned items = a.tokens * t.chunks;
    Cursor<T> cur;
    cur.item = cta * kWarps + warp;
    bool more = cur.item < items;
    if (more) {
        long long pos;
        cur.open(a, t, per_step, &pos);
        Head<Fmt, E, NU> x, dy;
        float r = 0.f;
        auto load = [&](const Cursor<T>& at, bool any, Head<Fmt, E, NU>& hx, Head<Fmt, E, NU>& hdy, float& hr) {
            const int h = at.h0 + grp;
            const bool mine = any && h < at.h_end && grp < per_step;
            hx.load(at.x + h * t.sx.h, u, mine);
            hdy.load(at.dy + h * t.sdy.h, u, mine);
            hr = mine ? __ldg(t.inv_rms + (int64_t)at.token * t.heads + h) : 0.f;
        };
        load(cur, true, x, dy, r);
        load_gamma<E, NU>(t.gamma, u, g);
        bool fresh = true;
        while (more) {
            Cursor<T> nxt = cur;
            long long pos_nxt = pos;
            bool fresh_nxt = false;
            nxt.h0 += per_step;
            if (nxt.h0 >= nxt.h_end) {
                nxt.item += t.ctas * kWarps;
                more = nxt.item < items;
                fresh_nxt = true;
                if (more) nxt.open(a, t, per_step, &pos_nxt);
            }
            Head<Fmt, E, NU> x_ahead, dy_ahead;
            float r_ahead;
            load(nxt, more, x_ahead, dy_ahead, r_ahead);
            if (fresh) angles<Fmt, E, NU>(a, u, pos, c, sn);

            float dot = 0.f;
            float d0[NU][E], d1[NU][E];
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                dy.p[j].get(d0[j]);
                dy.q[j].get(d1[j]);
                if (u.turns[j]) rotate<E>(d0[j], d1[j], c[j], sn[j], a.interleaved);
                float v[E], w[E];
                x.p[j].get(v);
                x.q[j].get(w);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float m0 = d0[j][e] * (v[e] * r), m1 = d1[j][e] * (w[e] * r);
                    acc[j][e] += m0;
                    acc[j][E + e] += m1;
                    dot += m0 * g[j][e] + m1 * g[j][E + e];
                }
            }
            const float m = sum_lanes(dot, a.lanes, sub) * a.inv_dim * r;   // mean * r
            const int h = cur.h0 + grp;
            if (h < cur.h_end && grp < per_step) {
                T* dx = cur.y + h * t.sy.h;
#pragma unroll
                for (int j = 0; j < NU; ++j) {
                    float v[E], w[E];
                    x.p[j].get(v);
                    x.q[j].get(w);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        v[e] = r * (d0[j][e] * g[j][e] - v[e] * m);
                        w[e] = r * (d1[j][e] * g[j][E + e] - w[e] * m);
                    }
                    if (u.live[j]) {
                        Chunk<Fmt, E>::store(dx + u.first[j], v);
                        Chunk<Fmt, E>::store(dx + u.second[j], w);
                    }
                }
            }
            x = x_ahead;
            dy = dy_ahead;
            r = r_ahead;
            cur = nxt;
            pos = pos_nxt;
            fresh = fresh_nxt;
        }
    }

    // the warp's head groups, then the CTA's warps, in a fixed order
#pragma unroll
    for (int j = 0; j < NU; ++j)
#pragma unroll
        for (int e = 0; e < 2 * E; ++e) {
            float v = acc[j][e];
            for (int k = 1; k < per_step; ++k) v += __shfl_sync(0xffffffffu, acc[j][e], (sub + k * a.lanes) & 31);
            if (grp == 0 && u.live[j])
                sums[warp * a.head_dim + (e < E ? u.first[j] + e : u.second[j] + e - E)] = v;
        }
    __syncthreads();
    for (int d = threadIdx.x; d < a.head_dim; d += kThreads) {
        float v = 0.f;
        for (int w = 0; w < kWarps; ++w) v += sums[w * a.head_dim + d];
        t.partial[(int64_t)cta * a.head_dim + d] = v;
    }
}

// ---------------------------------------------------------------- any sizes, strides and alignment
// One CTA per token (or per chunk of a token's heads), one warp per head; the token's
// sines are formed once, in shared memory.  A lane owns whole pairs, so that a call in
// place reads both members before it writes them.
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
    extern __shared__ float sh[];     // cos [rot/2], sin [rot/2], gradient: sums [kWarps][head_dim]
    float* cs = sh;
    float* sn = sh + a.rot / 2;
    const int which = (int)blockIdx.x >= a.t[0].ctas;
    const HeadsArg& t = a.t[which];
    const int cta = (int)blockIdx.x - (which ? a.t[0].ctas : 0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* sums = sh + a.rot + warp * a.head_dim;
    pdl_wait();
    pdl_trigger();
    if constexpr (Bwd) {
        for (int d = lane; d < a.head_dim; d += 32) sums[d] = 0.f;
        __syncwarp();
    }
    const int pairs = pair_count(a);
    const unsigned items = a.tokens * t.chunks;
    for (unsigned item = cta; item < items; item += t.ctas) {
        const unsigned token = item / (unsigned)t.chunks;
        const int chunk = (int)(item - token * t.chunks);
        unsigned b, s;
        split_token(a, token, &b, &s);
        const long long pos = position(a, b, s);
        __syncthreads();   // the previous token's sines have been read
        for (int i = threadIdx.x; i < a.rot / 2; i += kThreads)
            cos_sin<Fmt>(a, pos, __ldg(a.freqs + i), &cs[i], &sn[i]);
        __syncthreads();
        const T* xt = static_cast<const T*>(t.x) + b * t.sx.b + s * t.sx.s;
        const T* dt = Bwd ? static_cast<const T*>(t.dy) + b * t.sdy.b + s * t.sdy.s : nullptr;
        T* yt = static_cast<T*>(t.y) + b * t.sy.b + s * t.sy.s;
        const int h_end = min(t.heads, (chunk + 1) * t.steps);
        for (int h = chunk * t.steps + warp; h < h_end; h += kWarps) {
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
                    r = rsqrtf(sum_lanes(ss, 32, lane) * a.inv_dim + a.eps);
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
                const float m = sum_lanes(dot, 32, lane) * a.inv_dim * r;
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
            for (int w = 0; w < kWarps; ++w) v += sh[a.rot + w * a.head_dim + d];
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
template <class Fmt, int E, int NU>
tb_status launch_vec(Args a, const Call& c, int sms, cudaStream_t st) {
    const int units = a.head_dim / (2 * E);
    a.lanes = (int)ceil_div(units, NU);
    const int per_step = 32 / a.lanes;
    const void* kernel =
        c.bwd_norm ? reinterpret_cast<const void*>(&heads_bwd_kernel<Fmt, E, NU>)
        : c.norm   ? reinterpret_cast<const void*>(&heads_fwd_kernel<Fmt, E, NU, kNorm>)
                   : reinterpret_cast<const void*>(&heads_fwd_kernel<Fmt, E, NU, kRope>);
    const size_t smem = c.bwd_norm ? sizeof(float) * kWarps * a.head_dim : 0;
    const int resident = resident_ctas_per_sm(kernel, kThreads, smem);
    if (resident == 0) return TB_ERR_CUDA;
    const int64_t grid_ctas = (int64_t)sms * (c.bwd_norm ? std::min(resident, kBwdCtasPerSm) : resident);
    int64_t all_steps = 0;
    for (int i = 0; i < c.n; ++i) all_steps += ceil_div(a.t[i].heads, per_step);
    for (int i = 0; i < c.n; ++i) {
        HeadsArg& t = a.t[i];
        const int64_t steps = ceil_div(t.heads, per_step);
        // the tensor's share of the grid, by its head groups
        const int64_t share = std::max<int64_t>(1, grid_ctas * steps / all_steps);
        t.chunks = (int)std::min(steps, ceil_div(share * kWarps, a.tokens));
        t.steps = (int)ceil_div(steps, t.chunks);
        t.chunks = (int)ceil_div(steps, t.steps);
        t.ctas = (int)std::min(share, ceil_div(a.tokens * t.chunks, kWarps));
    }
    if (c.n == 1) a.t[1].ctas = 0;
    if (c.bwd_norm) a.t[1].partial = a.t[0].partial + (int64_t)a.t[0].ctas * a.head_dim;
    const dim3 grid((unsigned)(a.t[0].ctas + a.t[1].ctas));
    cudaError_t e;
    if (c.bwd_norm) e = launch_pdl(heads_bwd_kernel<Fmt, E, NU>, grid, dim3(kThreads), smem, st, a);
    else if (c.norm) e = launch_pdl(heads_fwd_kernel<Fmt, E, NU, kNorm>, grid, dim3(kThreads), smem, st, a);
    else e = launch_pdl(heads_fwd_kernel<Fmt, E, NU, kRope>, grid, dim3(kThreads), smem, st, a);
    if (e != cudaSuccess) return TB_ERR_CUDA;
    if (c.bwd_norm &&
        launch_pdl(dgamma_kernel, dim3((unsigned)ceil_div(a.head_dim, 32), (unsigned)c.n),
                   dim3(kThreads), 0, st, a) != cudaSuccess)
        return TB_ERR_CUDA;
    return launch_status();
}

template <class Fmt>
tb_status launch_general(Args a, const Call& c, int sms, cudaStream_t st) {
    const void* kernel =
        c.bwd_norm ? reinterpret_cast<const void*>(&heads_general_kernel<Fmt, kNorm, true>)
        : c.norm   ? reinterpret_cast<const void*>(&heads_general_kernel<Fmt, kNorm, false>)
                   : reinterpret_cast<const void*>(&heads_general_kernel<Fmt, kRope, false>);
    const size_t smem = sizeof(float) * (a.rot + (c.bwd_norm ? (size_t)kWarps * a.head_dim : 0));
    const int per_sm = std::min(resident_ctas_per_sm(kernel, kThreads, smem), kBwdCtasPerSm);
    if (per_sm == 0) return TB_ERR_CUDA;
    int64_t all = 0;
    for (int i = 0; i < c.n; ++i) all += a.t[i].heads;
    for (int i = 0; i < c.n; ++i) {
        HeadsArg& t = a.t[i];
        // chunks of whole rounds of the CTA's warps
        const int64_t rounds = ceil_div(t.heads, kWarps);
        t.chunks = (int)std::min(rounds, std::max<int64_t>(1, ceil_div(2 * sms, a.tokens)));
        t.steps = (int)(ceil_div(rounds, t.chunks) * kWarps);
        t.chunks = (int)ceil_div(t.heads, t.steps);
        int64_t ctas = a.tokens * t.chunks;
        if (c.bwd_norm)
            ctas = std::min(ctas, std::max<int64_t>(1, (int64_t)sms * per_sm * t.heads / all));
        t.ctas = (int)std::min<int64_t>(ctas, INT32_MAX / 4);
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
