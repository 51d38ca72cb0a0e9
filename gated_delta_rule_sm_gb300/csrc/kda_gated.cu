// kda_gated.cu -- the gated linear recurrence: its scan over long sequences, the scan's backward pass and the
// single-token step.  Per channel
//     log a_t = -exp(a_log) sigmoid(g_t),   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t,   y_t = h_t.
//
// One pass over the data: 8 bytes an element forward and 20 backward in bf16 (the gradients are fp32).  The tokens
// are cut into tiles, a CTA takes one tile of 64 channels (32 where two channels cannot be read at once) and keeps
// it in registers: a warp takes consecutive tokens, a lane neighbouring channels.  The recurrence is affine, so that
// a run of tokens is a pair (P, h): state -> P state + h, and runs are joined in three steps: a thread's tokens, the
// warps of a CTA, the tiles.  The last is a chain along the tokens inside the one launch: a tile publishes its pair
// as soon as it has it, then looks back over its predecessors to the nearest one whose leaving state is known, and
// applies the pairs between in order.  Tiles are taken from a counter, so that whatever a tile waits for was begun
// before it; the waits are bounded.  A state is the same chain of the same operations wherever the look-back began, so
// results do not depend on timing.
// The backward pass runs the same chain from the last token to the first, on m_t = a_t (dy_t + m_{t+1}), the
// gradient of h_{t-1}; the states it needs enter every 64th token from the forward's record and are carried on inside
// a tile.
// Precision: everything in fp32.  1 - a comes from a series in log a, so that decays next to 1, the long memories,
// are right to a rounding, and sqrt(1 - a^2) = sqrt(e (2 - e)) with e = 1 - a loses nothing there either.
#include <math.h>
#include <string.h>

#include <type_traits>

#include "kda.h"
#include "kda_common.cuh"
#include "kda_internal.h"
#include "kda_sm100.cuh"

namespace kda {

using namespace sm100;

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kFwdTok = 16, kFwdTile = kWarps * kFwdTok;     // tokens of a thread and of a CTA, forward
constexpr int kBwdTok = 8, kBwdTile = kWarps * kBwdTok;      // backward; the forward's record has a state every kBwdTile tokens
constexpr float kLog2e = 1.4426950408889634f;

struct GatedArgs {
    int T, TT, C, rows, tiles, cols, planned;
    int64_t xs, gs, is;                  // elements between neighbouring tokens
    const void *x, *g, *i, *dy;
    const float *a_log, *s0, *dsT;
    const int32_t* cu;
    void* y;
    float *sT, *rec;                     // rec [ceil(TT / kBwdTile), C]: the state that enters each kBwdTile tokens
    float *dx, *dg, *di, *da_log, *ds0;
    // workspace (planned)
    int *ticket, *ok, *flags, *first;    // flags [tiles, cols]; first [tiles]: the first row that begins at or after the tile's first token
    float *agg, *inc;                    // agg [tiles, C] pairs, inc [tiles, C] leaving states; by order in the chain
    float* part;                         // [tiles, C] da_log's parts
    int* status;
};

__device__ __forceinline__ int row_begin(const GatedArgs& a, int n) { return a.cu ? a.cu[n] : n * a.T; }

// ------------------------------------------------------------------ one or two channels at once

template <int VEC> using Val = std::conditional_t<VEC == 2, float2, float>;
__device__ __forceinline__ float vfma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float2 vfma(float2 a, float2 b, float2 c) { return fma2(a, b, c); }
__device__ __forceinline__ float vmul(float a, float b) { return a * b; }
__device__ __forceinline__ float2 vmul(float2 a, float2 b) { return mul2(a, b); }
template <typename V> __device__ __forceinline__ V vdup(float x) {
    if constexpr (std::is_same_v<V, float2>) return make_float2(x, x);
    else return x;
}
// P s + h, and h where P is 0: where a row begins P is 0, and whatever the row before left is not read as a number.
__device__ __forceinline__ float join(float P, float s, float h) { return P == 0.f ? h : fmaf(P, s, h); }
__device__ __forceinline__ float2 join(float2 P, float2 s, float2 h) { return make_float2(join(P.x, s.x, h.x), join(P.y, s.y, h.y)); }
template <typename F> __device__ __forceinline__ float vmap(F&& f, float a) { return f(a); }
template <typename F> __device__ __forceinline__ float2 vmap(F&& f, float2 a) { return make_float2(f(a.x), f(a.y)); }
template <typename V> __device__ __forceinline__ V vload(const float* p) { return *reinterpret_cast<const V*>(p); }
template <typename V> __device__ __forceinline__ V vload_l2(const float* p) { return __ldcg(reinterpret_cast<const V*>(p)); }
template <typename V> __device__ __forceinline__ void vstore(float* p, V v) { *reinterpret_cast<V*>(p) = v; }
template <typename V> __device__ __forceinline__ void vstore_stream(float* p, V v) { __stcs(reinterpret_cast<V*>(p), v); }

// A thread's channels of one token as they lie in memory.
template <typename E, int VEC> struct Raw;
template <> struct Raw<__nv_bfloat16, 2> {
    uint32_t u;
    __device__ __forceinline__ void load(const void* p, size_t i) {
        u = __ldcs(reinterpret_cast<const unsigned int*>(static_cast<const __nv_bfloat16*>(p) + i));
    }
    __device__ __forceinline__ void zero() { u = 0; }
    __device__ __forceinline__ float2 get() const { return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)); }
    static __device__ __forceinline__ void store(void* p, size_t i, float2 v) {
        __stcs(reinterpret_cast<unsigned int*>(static_cast<__nv_bfloat16*>(p) + i), pack_bf16(v.x, v.y));
    }
};
template <> struct Raw<__nv_bfloat16, 1> {
    unsigned short u;
    __device__ __forceinline__ void load(const void* p, size_t i) { u = static_cast<const unsigned short*>(p)[i]; }
    __device__ __forceinline__ void zero() { u = 0; }
    __device__ __forceinline__ float get() const { return __uint_as_float((uint32_t)u << 16); }
    static __device__ __forceinline__ void store(void* p, size_t i, float v) { static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v); }
};
template <> struct Raw<float, 1> {
    float u;
    __device__ __forceinline__ void load(const void* p, size_t i) { u = __ldcs(static_cast<const float*>(p) + i); }
    __device__ __forceinline__ void zero() { u = 0.f; }
    __device__ __forceinline__ float get() const { return u; }
    static __device__ __forceinline__ void store(void* p, size_t i, float v) { __stcs(static_cast<float*>(p) + i, v); }
};

// ------------------------------------------------------------------ the gates

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rsq(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float min_nan(float x, float y) {     // NaN if either is
    float z;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
    return z;
}

// e^-z, which stops at 2^60: the product of two sums 1 + e^-z stays finite, and one reciprocal serves both gates.  From
// there, z = -41.6, a sigmoid stays at 2^-60, 9e-19, which no sum it enters can tell from zero.
template <typename V> __device__ __forceinline__ V exp_neg(V z) {
    return vmap([](float t) { return min_nan(ex2(t), 0x1p60f); }, vmul(z, vdup<V>(-kLog2e)));
}

// The rate of a channel, -exp(a_log); wide: some rate of the warp is above 1/4.
template <typename V> struct Rate {
    V n, log2;
    bool wide;
};
template <typename V> __device__ __forceinline__ Rate<V> rate_of(const float* a_log, int c, bool in) {
    Rate<V> r;
    const V a = in ? vload<V>(a_log + c) : vdup<V>(-1e30f);
    r.n = vmap([](float t) { return -expf(t); }, a);
    r.log2 = vmul(a, vdup<V>(kLog2e));
    bool over = false;
    vmap([&](float t) { over |= !(t >= -0.25f); return 0.f; }, r.n);
    r.wide = __any_sync(__activemask(), over);
    return r;
}
// log a from the gate and its sigmoid.  Rates up to 1/4 multiply the sigmoid.  Above, a gate that is all but closed may still
// count, and the rate may be past fp32: there log2 of the product is formed, a_log - log(1 + e^-g), and what it gives
// stops at 1e30, where the decay is 0 and products with it stay finite.
__device__ __forceinline__ float wide_log(float g, float log2_rate) {
    const float t = g * -kLog2e;
    float l;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(l) : "f"(1.f + ex2(t)));
    return -min_nan(ex2(log2_rate - (t > 30.f ? t : l)), 1e30f);
}
__device__ __forceinline__ float log_decay(float g, float sig, const Rate<float>& r) {
    return r.wide && !(r.n >= -0.25f) ? wide_log(g, r.log2) : sig * r.n;
}
__device__ __forceinline__ float2 log_decay(float2 g, float2 sig, const Rate<float2>& r) {
    float2 l = mul2(sig, r.n);
    if (r.wide) {
        if (!(r.n.x >= -0.25f)) l.x = wide_log(g.x, r.log2.x);
        if (!(r.n.y >= -0.25f)) l.y = wide_log(g.y, r.log2.y);
    }
    return l;
}

// 1 - e^l for l <= 0: the series to l^7 / 5040 down to -1/4 (its rest is below 2^-28 of the value), the exponential below
// that, which only a wide rate can reach.
template <typename V> __device__ __forceinline__ V one_minus_exp(V l, bool wide) {
    V p = vfma(l, vdup<V>(1.f / 5040.f), vdup<V>(1.f / 720.f));
    p = vfma(p, l, vdup<V>(1.f / 120.f));
    p = vfma(p, l, vdup<V>(1.f / 24.f));
    p = vfma(p, l, vdup<V>(1.f / 6.f));
    p = vfma(p, l, vdup<V>(0.5f));
    p = vfma(p, l, vdup<V>(1.f));
    V e = vmul(vmul(l, vdup<V>(-1.f)), p);
    if (wide) {
        auto far = [](float t, float near) { return t < -0.25f ? 1.f - ex2(t * kLog2e) : near; };
        if constexpr (std::is_same_v<V, float2>) e = make_float2(far(l.x, e.x), far(l.y, e.y));
        else e = far(l, e);
    }
    return e;
}

// e = 1 - a, 1 / sqrt(1 - a^2) (0 where a is 1: there the input's factor is 0 and so is the limit of the gradients'
// a^2 log a / sqrt(1 - a^2)), and w = 1 - a^2
template <typename V> struct Decay {
    V e, rb, w;
};
template <typename V> __device__ __forceinline__ Decay<V> decay_of(V g, V sig, const Rate<V>& r) {
    Decay<V> d;
    d.e = one_minus_exp(log_decay(g, sig, r), r.wide);
    d.w = vmul(d.e, vfma(d.e, vdup<V>(-1.f), vdup<V>(2.f)));
    d.rb = vmap([](float t) { return t > 1e-36f ? rsq(t) : 0.f; }, d.w);
    return d;
}
template <typename V> __device__ __forceinline__ V keep_of(V e) { return vfma(e, vdup<V>(-1.f), vdup<V>(1.f)); }

// ------------------------------------------------------------------ rows inside a tile

// Which rows begin at and end with a token of the tile, -1: none.  All threads; the answer: whether any does.
template <int TILE> struct Edges {
    int first[TILE], last[TILE];
};
template <int TILE> __device__ __forceinline__ bool find_edges(const GatedArgs& a, int t0, int tile, Edges<TILE>& s) {
    if (threadIdx.x < TILE) s.first[threadIdx.x] = s.last[threadIdx.x] = -1;
    __syncthreads();
    bool any = false;
    const int t1 = min(t0 + TILE, a.TT);
    for (int m = (a.cu ? a.first[tile] : (t0 + a.T - 1) / a.T) + threadIdx.x; m <= a.rows; m += kThreads) {
        const int at = row_begin(a, m);
        if (at > t1) break;
        if (m < a.rows && at < t1 && row_begin(a, m + 1) > at) {
            s.first[at - t0] = m;
            any = true;
        }
        if (m > 0 && at > t0 && row_begin(a, m - 1) < at) {
            s.last[at - 1 - t0] = m - 1;
            any = true;
        }
    }
    return __syncthreads_or(any);
}

// ------------------------------------------------------------------ the chain of tiles

__device__ __forceinline__ int load_acquire(const int* p) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void store_release(int* p, int v) {
    asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

enum Flag { kNothing = 0, kPair = 1, kState = 2 };

// Called by one warp.  (The lanes' stores come before lane 0's release: __syncwarp orders them, the fence carries them to
// the other CTAs.)
__device__ __forceinline__ void publish(const GatedArgs& a, int o, int col, Flag f) {
    __threadfence();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) store_release(a.flags + (size_t)o * a.cols + col, f);
}

// The state that enters the o-th tile of the chain: from the nearest tile before it that has published its leaving state
// on, the pairs of those between.  The first tile of a chain, and every tile in which a row begins, publishes a
// state, so there is one.  One warp; at most about a second, then the error is recorded and the state is 0.
template <typename V> __device__ __forceinline__ V look_back(const GatedArgs& a, int o, int col, int c, bool in) {
    const int lane = threadIdx.x & 31;
    int from = -1;
    for (int back = o - 1, tries = 0; from < 0;) {
        const int j = back - lane;
        const int f = j >= 0 ? load_acquire(a.flags + (size_t)j * a.cols + col) : (int)kState;
        const unsigned none = __ballot_sync(0xffffffffu, f == kNothing), state = __ballot_sync(0xffffffffu, f == kState);
        const unsigned before = state ? (state & (0u - state)) - 1u : 0xffffffffu;
        if (none & before) {
            if (++tries > (1 << 20)) {
                if (lane == 0) record_error(a.status, KDA_ERR_TIMEOUT);
                return vdup<V>(0.f);
            }
            __nanosleep(64);
        } else if (state) {
            from = max(back - (__ffs(state) - 1), 0);
        } else {
            back -= 32;
        }
    }
    __syncwarp();
    if (!in) return vdup<V>(0.f);
    V s = vload_l2<V>(a.inc + (size_t)from * a.C + c);
    constexpr int AHEAD = 8;
    for (int j = from + 1; j < o; j += AHEAD) {
        V P[AHEAD], h[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (j + k < o) {
                const float* p = a.agg + 2 * ((size_t)(j + k) * a.C + c);
                P[k] = vload_l2<V>(p);
                h[k] = vload_l2<V>(p + sizeof(V) / 4);
            }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (j + k < o) s = join(P[k], s, h[k]);
    }
    return s;
}

// The tile's pair or leaving state for its successors, and the state that enters it.  closed: a row begins in the tile, so
// that what leaves it does not depend on what enters.  needs: some token depends on what enters.
template <typename V>
__device__ __forceinline__ V join_chain(const GatedArgs& a, int o, int col, int c, bool in, V P, V h, bool closed, bool needs) {
    if (!a.planned) return vdup<V>(0.f);
    float* leaving = a.inc + (size_t)o * a.C + c;
    if (closed) {
        if (in) vstore(leaving, h);
        publish(a, o, col, kState);
        return needs ? look_back<V>(a, o, col, c, in) : vdup<V>(0.f);
    }
    if (in) {
        float* p = a.agg + 2 * ((size_t)o * a.C + c);
        vstore(p, P);
        vstore(p + sizeof(V) / 4, h);
    }
    publish(a, o, col, kPair);
    const V s = look_back<V>(a, o, col, c, in);
    if (in) vstore(leaving, join(P, s, h));
    publish(a, o, col, kState);
    return s;
}

// The tile and the columns of this CTA, in the order in which tiles are begun.
__device__ __forceinline__ int take_ticket(const GatedArgs& a, int* slot) {
    if (!a.planned) return blockIdx.x;
    if (threadIdx.x == 0) *slot = atomicAdd(a.ticket, 1);
    __syncthreads();
    return *slot;
}

// Clears the counter and the flags, checks the offsets, finds each tile's first row, and passes the states of rows without
// tokens through (of all rows where the offsets break the contract).
__global__ void __launch_bounds__(kThreads) gated_plan_kernel(GatedArgs a, int tile_tokens, const float* from, float* to) {
    bool bad = false;
    if (a.cu) {
        for (int n = threadIdx.x; n < a.rows; n += kThreads) bad |= a.cu[n + 1] < a.cu[n];
        if (threadIdx.x == 0) bad |= a.cu[0] != 0 || a.cu[a.rows] != a.TT;
        bad = __syncthreads_or(bad);
    }
    const int id = blockIdx.x * kThreads + threadIdx.x, all = gridDim.x * kThreads;
    if (id == 0) {
        *a.ticket = 0;
        *a.ok = !bad;
        if (bad) record_error(a.status, KDA_ERR_INVALID_ARG);
    }
    for (int64_t k = id; k < (int64_t)a.tiles * a.cols; k += all) a.flags[k] = kNothing;
    if (!a.cu) return;
    for (int k = id; !bad && k < a.tiles; k += all) {
        int lo = 0, hi = a.rows;          // (cu[rows] = TT is past every tile's first token)
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (a.cu[mid] >= k * tile_tokens) hi = mid; else lo = mid + 1;
        }
        a.first[k] = lo;
    }
    if (to)
        for (int n = blockIdx.x; n < a.rows; n += gridDim.x)
            if (bad || a.cu[n + 1] == a.cu[n])
                for (int c = threadIdx.x; c < a.C; c += kThreads)
                    to[(size_t)n * a.C + c] = from ? from[(size_t)n * a.C + c] : 0.f;
}

// ------------------------------------------------------------------ forward

template <typename E, int VEC>
__global__ void __launch_bounds__(kThreads, 2) gated_fwd_kernel(const __grid_constant__ GatedArgs a) {
    using V = Val<VEC>;
    using R = Raw<E, VEC>;
    __shared__ Edges<kFwdTile> edges;
    __shared__ V sp[kWarps][32], sh[kWarps][32], senter[32];
    __shared__ int slot;
    const int idx = take_ticket(a, &slot), tile = idx / a.cols, col = idx - tile * a.cols;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = (col * 32 + lane) * VEC;
    const bool in = c < a.C;
    const int t0 = tile * kFwdTile, tb = t0 + warp * kFwdTok;
    const int n = in ? max(0, min(kFwdTok, a.TT - tb)) : 0;
    R rx[kFwdTok], rg[kFwdTok], ri[kFwdTok];
#pragma unroll
    for (int k = 0; k < kFwdTok; ++k)
        if (k < n) {
            rx[k].load(a.x, (size_t)(tb + k) * a.xs + c);
            rg[k].load(a.g, (size_t)(tb + k) * a.gs + c);
            ri[k].load(a.i, (size_t)(tb + k) * a.is + c);
        } else {
            rx[k].zero();
            rg[k].zero();
            ri[k].zero();
        }
    if (a.planned && !*a.ok) return;
    const bool split = find_edges(a, t0, tile, edges);
    const Rate<V> rate = rate_of<V>(a.a_log, c, in);
    auto begins_at = [&](int k) { return split ? edges.first[warp * kFwdTok + k] : -1; };
    // a token as h -> ka h + kb; where a row begins the state is the row's own, and ka is 0
    V ka[kFwdTok], kb[kFwdTok], P = vdup<V>(1.f), h = vdup<V>(0.f);
#pragma unroll
    for (int k = 0; k < kFwdTok; ++k) {
        const V da = vfma(exp_neg(rg[k].get()), vdup<V>(1.f), vdup<V>(1.f)), db = vfma(exp_neg(ri[k].get()), vdup<V>(1.f), vdup<V>(1.f));
        const V r = vmap([](float t) { return rcp(t); }, vmul(da, db));
        const Decay<V> d = decay_of(rg[k].get(), vmul(r, db), rate);
        ka[k] = keep_of(d.e);
        kb[k] = vmul(vmul(vmul(d.w, d.rb), vmul(r, da)), rx[k].get());
        if (k >= n) {
            ka[k] = vdup<V>(1.f);
            kb[k] = vdup<V>(0.f);
        } else if (begins_at(k) >= 0) {
            if (a.s0) kb[k] = vfma(ka[k], vload<V>(a.s0 + (size_t)begins_at(k) * a.C + c), kb[k]);
            P = h = ka[k] = vdup<V>(0.f);
        }
        P = vmul(P, ka[k]);
        h = vfma(ka[k], h, kb[k]);
    }
    sp[warp][lane] = P;
    sh[warp][lane] = h;
    bool begins = false;
    if (split)
        for (int k = lane; k < kFwdTile; k += 32) begins |= edges.first[k] >= 0;
    begins = __any_sync(0xffffffffu, begins);
    __syncthreads();
    if (warp == 0) {
        P = vdup<V>(1.f);
        h = vdup<V>(0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            P = join(sp[w][lane], P, vdup<V>(0.f));
            h = join(sp[w][lane], h, sh[w][lane]);
        }
        senter[lane] = join_chain<V>(a, tile, col, c, in, P, h, begins, edges.first[0] < 0);
    }
    __syncthreads();
    h = senter[lane];
    for (int w = 0; w < warp; ++w) h = join(sp[w][lane], h, sh[w][lane]);
    if (a.rec && n > 0 && warp * kFwdTok % kBwdTile == 0) vstore(a.rec + (size_t)(tb / kBwdTile) * a.C + c, h);
#pragma unroll
    for (int k = 0; k < kFwdTok; ++k)
        if (k < n) {
            h = begins_at(k) >= 0 ? kb[k] : vfma(ka[k], h, kb[k]);
            if (a.y) R::store(a.y, (size_t)(tb + k) * a.C + c, h);
            if (split && a.sT && edges.last[warp * kFwdTok + k] >= 0)
                vstore(a.sT + (size_t)edges.last[warp * kFwdTok + k] * a.C + c, h);
        }
}

// ------------------------------------------------------------------ backward

template <typename E, int VEC>
__global__ void __launch_bounds__(kThreads, 2) gated_bwd_kernel(const __grid_constant__ GatedArgs a) {
    using V = Val<VEC>;
    using R = Raw<E, VEC>;
    constexpr int N = kBwdTok;
    __shared__ Edges<kBwdTile> edges;
    __shared__ V sp[kWarps][32], sh[kWarps][32], sq[kWarps][32], sm[kWarps][32], senter[32];
    __shared__ int slot;
    const int idx = take_ticket(a, &slot), o = idx / a.cols, col = idx - o * a.cols, tile = a.tiles - 1 - o;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = (col * 32 + lane) * VEC;
    const bool in = c < a.C;
    const int t0 = tile * kBwdTile, tb = t0 + warp * N;
    const int n = in ? max(0, min(N, a.TT - tb)) : 0;
    R rx[N], rg[N], ri[N], rd[N];
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (k < n) {
            rx[k].load(a.x, (size_t)(tb + k) * a.xs + c);
            rg[k].load(a.g, (size_t)(tb + k) * a.gs + c);
            ri[k].load(a.i, (size_t)(tb + k) * a.is + c);
            rd[k].load(a.dy, (size_t)(tb + k) * a.C + c);
        } else {
            rx[k].zero();
            rg[k].zero();
            ri[k].zero();
            rd[k].zero();
        }
    if (a.planned && !*a.ok) return;
    const bool split = find_edges(a, t0, tile, edges);
    auto begins_at = [&](int k) { return split ? edges.first[warp * N + k] : -1; };
    auto ends_at = [&](int k) { return split ? edges.last[warp * N + k] : -1; };
    const Rate<V> rate = rate_of<V>(a.a_log, c, in);
    // the forward's runs, from the first token on
    V eg[N], ei[N], e[N], rb[N], P = vdup<V>(1.f), h = vdup<V>(0.f);
    const V one = vdup<V>(1.f);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        eg[k] = exp_neg(rg[k].get());
        ei[k] = exp_neg(ri[k].get());
        const V da = vfma(eg[k], one, one), db = vfma(ei[k], one, one), r = vmap([](float t) { return rcp(t); }, vmul(da, db));
        const Decay<V> d = decay_of(rg[k].get(), vmul(r, db), rate);
        e[k] = d.e;
        rb[k] = d.rb;
        if (k >= n) {
            e[k] = vdup<V>(0.f);
            rb[k] = vdup<V>(0.f);
        } else if (begins_at(k) >= 0) {
            P = vdup<V>(0.f);
            h = a.s0 ? vload<V>(a.s0 + (size_t)begins_at(k) * a.C + c) : vdup<V>(0.f);
        }
        const V ka = keep_of(e[k]);
        P = vmul(P, ka);
        h = vfma(ka, h, vmul(vmul(vmul(d.w, rb[k]), vmul(r, da)), rx[k].get()));
    }
    sp[warp][lane] = P;
    sh[warp][lane] = h;
    // the gradient's, from the last
    P = one;
    V m = vdup<V>(0.f);
#pragma unroll
    for (int k = N - 1; k >= 0; --k) {
        if (k < n && ends_at(k) >= 0) {
            P = vdup<V>(0.f);
            m = a.dsT ? vload<V>(a.dsT + (size_t)ends_at(k) * a.C + c) : vdup<V>(0.f);
        }
        const V ka = keep_of(e[k]);
        P = vmul(P, ka);
        m = vmul(ka, vfma(rd[k].get(), one, m));
    }
    sq[warp][lane] = P;
    sm[warp][lane] = m;
    bool ends = false;
    if (split)
        for (int k = lane; k < kBwdTile; k += 32) ends |= edges.last[k] >= 0;
    ends = __any_sync(0xffffffffu, ends);
    __syncthreads();
    if (warp == 0) {
        P = one;
        m = vdup<V>(0.f);
#pragma unroll
        for (int w = kWarps - 1; w >= 0; --w) {
            P = join(sq[w][lane], P, vdup<V>(0.f));
            m = join(sq[w][lane], m, sm[w][lane]);
        }
        senter[lane] = join_chain<V>(a, o, col, c, in, P, m, ends, edges.last[min(kBwdTile, a.TT - t0) - 1] < 0);
    }
    // meanwhile the states before the tokens
    auto input = [&](int k) {      // sqrt(1 - a^2) sigmoid(i) x
        const V da = vfma(eg[k], one, one), db = vfma(ei[k], one, one), r = vmap([](float t) { return rcp(t); }, vmul(da, db));
        const V w = vmul(e[k], vfma(e[k], vdup<V>(-1.f), vdup<V>(2.f)));
        return vmul(vmul(vmul(w, rb[k]), vmul(r, da)), rx[k].get());
    };
    h = in ? vload<V>(a.rec + (size_t)tile * a.C + c) : vdup<V>(0.f);
    for (int w = 0; w < warp; ++w) h = join(sp[w][lane], h, sh[w][lane]);
    V before[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (k < n && begins_at(k) >= 0) h = a.s0 ? vload<V>(a.s0 + (size_t)begins_at(k) * a.C + c) : vdup<V>(0.f);
        before[k] = h;
        h = vfma(keep_of(e[k]), h, input(k));
    }
    __syncthreads();
    m = senter[lane];
    for (int w = kWarps - 1; w > warp; --w) m = join(sq[w][lane], m, sm[w][lane]);
    V dlog = vdup<V>(0.f);
#pragma unroll
    for (int k = N - 1; k >= 0; --k)
        if (k < n) {
            if (ends_at(k) >= 0) m = a.dsT ? vload<V>(a.dsT + (size_t)ends_at(k) * a.C + c) : vdup<V>(0.f);
            const V da = vfma(eg[k], one, one), db = vfma(ei[k], one, one), r = vmap([](float t) { return rcp(t); }, vmul(da, db));
            const V sg = vmul(r, db), si = vmul(r, da), ka = keep_of(e[k]);
            const V w = vmul(e[k], vfma(e[k], vdup<V>(-1.f), vdup<V>(2.f)));
            const V dh = vfma(rd[k].get(), one, m);                  // the gradient of h_t
            m = vmul(ka, dh);
            if (begins_at(k) >= 0 && a.ds0) vstore(a.ds0 + (size_t)begins_at(k) * a.C + c, m);
            const V u = vmul(si, rx[k].get()), du = vmul(dh, vmul(w, rb[k]));
            // of log a: a (h_{t-1} - u a / sqrt(1 - a^2)) times that of h_t; then times log a for a_log, and 1 - sigmoid(g) for g
            const V dl = vmul(vmul(m, vfma(vmul(u, vdup<V>(-1.f)), vmul(ka, rb[k]), before[k])), log_decay(rg[k].get(), sg, rate));
            dlog = vfma(dl, one, dlog);
            const size_t at = (size_t)(tb + k) * a.C + c;
            vstore_stream(a.dx + at, vmul(du, si));
            vstore_stream(a.dg + at, vmul(dl, vmul(eg[k], sg)));
            vstore_stream(a.di + at, vmul(vmul(du, u), vmul(ei[k], si)));
        }
    __syncthreads();
    sp[warp][lane] = dlog;
    __syncthreads();
    if (warp == 0 && in) {
        dlog = sp[0][lane];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) dlog = vfma(sp[w][lane], one, dlog);
        vstore(a.part + (size_t)tile * a.C + c, dlog);
    }
}

// da_log: the tiles' parts in a fixed order, 32 channels to a CTA.
__global__ void __launch_bounds__(kThreads) gated_reduce_kernel(const __grid_constant__ GatedArgs a) {
    __shared__ float s[kWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane;
    float t = 0.f;
    if (c < a.C && (!a.planned || *a.ok))
        for (int k = warp; k < a.tiles; k += kWarps) t += a.part[(size_t)k * a.C + c];
    s[warp][lane] = t;
    __syncthreads();
    if (warp || c >= a.C) return;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) t += s[w][lane];
    a.da_log[c] = t;
}

// ------------------------------------------------------------------ one token

struct StepArgs {
    int B, C, num_slots;
    int64_t xs, gs, is;
    const void *x, *g, *i;
    const float* a_log;
    const int32_t* slots;
    const float* s_in;
    float* s_out;
    void* y;
    int* status;
};
constexpr int kStepThreads = 128;

template <typename E, int VEC>
__global__ void __launch_bounds__(kStepThreads) gated_step_kernel(const __grid_constant__ StepArgs a) {
    using V = Val<VEC>;
    using R = Raw<E, VEC>;
    const int b = blockIdx.x, c = (blockIdx.y * kStepThreads + threadIdx.x) * VEC;
    if (c >= a.C) return;
    int slot = a.slots ? a.slots[b] : b;
    if (slot >= a.num_slots) {
        if (c == 0) record_error(a.status, KDA_ERR_INVALID_ARG);
        slot = -1;
    }
    if (slot < 0) {
        R::store(a.y, (size_t)b * a.C + c, vdup<V>(0.f));
        return;
    }
    R rx, rg, ri;
    rx.load(a.x, (size_t)b * a.xs + c);
    rg.load(a.g, (size_t)b * a.gs + c);
    ri.load(a.i, (size_t)b * a.is + c);
    const V old = vload<V>(a.s_in + (size_t)slot * a.C + c);
    const Rate<V> rate = rate_of<V>(a.a_log, c, true);
    const V one = vdup<V>(1.f), da = vfma(exp_neg(rg.get()), one, one), db = vfma(exp_neg(ri.get()), one, one);
    const V r = vmap([](float t) { return rcp(t); }, vmul(da, db));
    const Decay<V> d = decay_of(rg.get(), vmul(r, db), rate);
    const V h = vfma(keep_of(d.e), old, vmul(vmul(vmul(d.w, d.rb), vmul(r, da)), rx.get()));
    vstore(a.s_out + (size_t)slot * a.C + c, h);
    R::store(a.y, (size_t)b * a.C + c, h);
}

// ------------------------------------------------------------------ host

struct Shape {
    int B, T, TT, C, rows, dtype, es;
    int64_t xs, gs, is;
};

kda_status gated_check(const kda_gated_dims* d, bool varlen, Shape* s) {
    if (!d || d->B < 1 || d->T < 1 || d->C < 1) return KDA_ERR_INVALID_ARG;
    if (d->dtype != KDA_BF16 && d->dtype != KDA_FP32) return KDA_ERR_INVALID_ARG;
    if (varlen && (d->B != 1 || d->num_seqs < 1)) return KDA_ERR_INVALID_ARG;
    for (int64_t st : {d->x_stride, d->g_stride, d->i_stride})
        if (st != 0 && st < d->C) return KDA_ERR_INVALID_ARG;
    if ((int64_t)d->B * d->T > (1LL << 30) || (varlen && d->num_seqs > (1 << 24))) return KDA_ERR_UNSUPPORTED;
    s->B = d->B; s->T = d->T; s->TT = d->B * d->T; s->C = d->C; s->rows = varlen ? d->num_seqs : d->B;
    s->dtype = d->dtype; s->es = d->dtype == KDA_BF16 ? 2 : 4;
    s->xs = d->x_stride ? d->x_stride : d->C;
    s->gs = d->g_stride ? d->g_stride : d->C;
    s->is = d->i_stride ? d->i_stride : d->C;
    for (int64_t st : {s->xs, s->gs, s->is})
        if (s->TT > 1 && st > (1LL << 40) / s->TT) return KDA_ERR_UNSUPPORTED;
    // (tiles x columns and the workspace's indices)
    if ((int64_t)((s->TT + kBwdTile - 1) / kBwdTile) * ((s->C + 31) / 32) > (1LL << 30)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }
size_t gated_record_bytes(const Shape& s) { return (size_t)((s.TT + kBwdTile - 1) / kBwdTile) * s.C * 4; }

// Workspace of one pass over tiles of `tile` tokens; fills the views where ws is given.
size_t gated_layout(const Shape& s, int tile, bool reduce, char* ws, GatedArgs* a) {
    const size_t tiles = (s.TT + tile - 1) / tile, most = (s.C + 31) / 32;
    size_t o = 0;
    auto take = [&](size_t n) {
        char* p = ws ? ws + o : nullptr;
        o += up(n);
        return p;
    };
    char* head = take(8);
    char* flags = take(tiles * most * 4);
    char* first = take(tiles * 4);
    char* agg = take(tiles * s.C * 8);
    char* inc = take(tiles * s.C * 4);
    char* part = reduce ? take(tiles * s.C * 4) : nullptr;
    if (a) {
        a->ticket = reinterpret_cast<int*>(head);
        a->ok = a->ticket + 1;
        a->flags = reinterpret_cast<int*>(flags);
        a->first = reinterpret_cast<int*>(first);
        a->agg = reinterpret_cast<float*>(agg);
        a->inc = reinterpret_cast<float*>(inc);
        a->part = reinterpret_cast<float*>(part);
    }
    return o;
}

bool pairs_ok(const Shape& s, std::initializer_list<const void*> acts, std::initializer_list<const void*> floats) {
    if (s.dtype != KDA_BF16 || s.C % 2 || s.xs % 2 || s.gs % 2 || s.is % 2) return false;
    for (const void* p : acts)
        if (reinterpret_cast<uintptr_t>(p) % 4) return false;
    for (const void* p : floats)
        if (reinterpret_cast<uintptr_t>(p) % 8) return false;
    return true;
}

GatedArgs gated_args(const Shape& s, const void* x, const void* g, const void* i, const float* a_log, const int32_t* cu, const float* s0) {
    GatedArgs a;
    memset(&a, 0, sizeof(a));
    a.T = s.T; a.TT = s.TT; a.C = s.C; a.rows = s.rows; a.xs = s.xs; a.gs = s.gs; a.is = s.is;
    a.x = x; a.g = g; a.i = i; a.a_log = a_log; a.cu = cu; a.s0 = s0;
    return a;
}

// The plan where the call has more than one tile or packed documents; from, to: the states that pass through.
cudaError_t gated_begin(GatedArgs& a, int tile, int vec, const float* from, float* to, cudaStream_t st) {
    a.tiles = (a.TT + tile - 1) / tile;
    a.cols = (a.C + 32 * vec - 1) / (32 * vec);
    a.planned = a.tiles > 1 || a.cu;
    if (!a.planned) return cudaSuccess;
    const int64_t work = (int64_t)a.tiles * a.cols / kThreads + 1, most = a.cu ? (work > a.rows ? work : a.rows) : work;
    timing_pre(st, K_GATED_PLAN);
    gated_plan_kernel<<<(int)(most < 152 ? most : 152), kThreads, 0, st>>>(a, tile, from, to);
    timing_post(st);
    return cudaGetLastError();
}

cudaError_t gated_forward(GatedArgs a, int dtype, bool pairs, cudaStream_t st) {
    cudaError_t e = gated_begin(a, kFwdTile, pairs ? 2 : 1, a.s0, a.sT, st);
    if (e != cudaSuccess) return e;
    const int ctas = a.tiles * a.cols;
    timing_pre(st, K_GATED_SCAN);
    if (pairs) gated_fwd_kernel<__nv_bfloat16, 2><<<ctas, kThreads, 0, st>>>(a);
    else if (dtype == KDA_BF16) gated_fwd_kernel<__nv_bfloat16, 1><<<ctas, kThreads, 0, st>>>(a);
    else gated_fwd_kernel<float, 1><<<ctas, kThreads, 0, st>>>(a);
    timing_post(st);
    return cudaGetLastError();
}

size_t span_bytes(const Shape& s, int64_t stride) { return ((size_t)(s.TT - 1) * stride + s.C) * s.es; }

}  // namespace

}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_gated_scan_fwd_workspace_size(const kda_gated_dims* dims) {
    Shape s;
    if (!dims || gated_check(dims, false, &s) != KDA_OK) return 0;
    return gated_layout(s, kFwdTile, false, nullptr, nullptr);
}

size_t kda_gated_scan_bwd_workspace_size(const kda_gated_dims* dims) {
    Shape s;
    if (!dims || gated_check(dims, false, &s) != KDA_OK) return 0;
    const size_t f = gated_layout(s, kFwdTile, false, nullptr, nullptr), b = gated_layout(s, kBwdTile, true, nullptr, nullptr);
    return up(gated_record_bytes(s)) + (f > b ? f : b);
}

size_t kda_gated_scan_saved_size(const kda_gated_dims* dims) {
    Shape s;
    if (!dims || gated_check(dims, false, &s) != KDA_OK) return 0;
    return gated_record_bytes(s);
}

kda_status kda_gated_scan_fwd(const kda_gated_dims* dims, const void* x, const void* g_raw, const void* i_raw, const float* a_log,
                              const int32_t* cu_seqlens, const int32_t* cu_seqlens_host, const float* initial_state, void* y,
                              float* final_state, void* saved, size_t saved_bytes, void* workspace, size_t workspace_bytes,
                              cudaStream_t stream) {
    Shape s;
    kda_status st = gated_check(dims, cu_seqlens != nullptr, &s);
    if (st != KDA_OK) return st;
    if (!x || !g_raw || !i_raw || !a_log || !y) return KDA_ERR_INVALID_ARG;
    st = check_offsets_host(s.rows, s.TT, cu_seqlens, cu_seqlens_host);
    if (st != KDA_OK) return st;
    const size_t rec = saved ? gated_record_bytes(s) : 0;
    if (saved && (saved_bytes < rec || reinterpret_cast<uintptr_t>(saved) % 256)) return KDA_ERR_WORKSPACE;
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < gated_layout(s, kFwdTile, false, nullptr, nullptr))
        return KDA_ERR_WORKSPACE;
    // a thread has read an element of x before it writes y's there, and a row's first tile its state before its last tile
    // writes one; the tiles otherwise run in no order
    const size_t nx = span_bytes(s, s.xs), ng = span_bytes(s, s.gs), ni = span_bytes(s, s.is), ny = (size_t)s.TT * s.C * s.es;
    const size_t ns = (size_t)s.rows * s.C * 4;
    const bool y_on_x = y == x && s.xs == s.C;
    if ((!y_on_x && ranges_meet(y, ny, x, nx)) || ranges_meet(y, ny, g_raw, ng) || ranges_meet(y, ny, i_raw, ni) ||
        ranges_meet(y, ny, initial_state, ns) || ranges_meet(y, ny, final_state, ns) || ranges_meet(y, ny, saved, rec))
        return KDA_ERR_INVALID_ARG;
    for (void* out : {static_cast<void*>(final_state), saved}) {
        const size_t n = out == saved ? rec : ns;
        if (ranges_meet(out, n, x, nx) || ranges_meet(out, n, g_raw, ng) || ranges_meet(out, n, i_raw, ni) ||
            (out != initial_state && ranges_meet(out, n, initial_state, ns)) || (out == saved && out == initial_state && out))
            return KDA_ERR_INVALID_ARG;
    }
    if (ranges_meet(final_state, ns, saved, rec)) return KDA_ERR_INVALID_ARG;
    GatedArgs a = gated_args(s, x, g_raw, i_raw, a_log, cu_seqlens, initial_state);
    a.y = y; a.sT = final_state; a.rec = static_cast<float*>(saved);
    gated_layout(s, kFwdTile, false, static_cast<char*>(workspace), &a);
    st = status_ptr(&a.status);
    if (st != KDA_OK) return st;
    const bool pairs = pairs_ok(s, {x, g_raw, i_raw, y}, {a_log, initial_state, final_state});
    return gated_forward(a, s.dtype, pairs, stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_gated_scan_bwd(const kda_gated_dims* dims, const void* x, const void* g_raw, const void* i_raw, const float* a_log,
                              const int32_t* cu_seqlens, const int32_t* cu_seqlens_host, const float* initial_state, const void* dy,
                              const float* dfinal_state, float* dx, float* dg_raw, float* di_raw, float* da_log,
                              float* dinitial_state, const void* saved, size_t saved_bytes, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
    Shape s;
    kda_status st = gated_check(dims, cu_seqlens != nullptr, &s);
    if (st != KDA_OK) return st;
    if (!x || !g_raw || !i_raw || !a_log || !dy || !dx || !dg_raw || !di_raw || !da_log) return KDA_ERR_INVALID_ARG;
    st = check_offsets_host(s.rows, s.TT, cu_seqlens, cu_seqlens_host);
    if (st != KDA_OK) return st;
    const size_t rec = gated_record_bytes(s);
    if (saved && (saved_bytes < rec || reinterpret_cast<uintptr_t>(saved) % 256)) return KDA_ERR_WORKSPACE;
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < kda_gated_scan_bwd_workspace_size(dims))
        return KDA_ERR_WORKSPACE;
    const size_t nf = (size_t)s.TT * s.C * 4, ns = (size_t)s.rows * s.C * 4;
    struct Span {
        const void* p;
        size_t n;
    };
    const Span in[] = {{x, span_bytes(s, s.xs)}, {g_raw, span_bytes(s, s.gs)}, {i_raw, span_bytes(s, s.is)}, {dy, (size_t)s.TT * s.C * s.es},
                       {a_log, (size_t)s.C * 4}, {initial_state, ns}, {dfinal_state, ns}, {saved, rec}};
    const Span out[] = {{dx, nf}, {dg_raw, nf}, {di_raw, nf}, {da_log, (size_t)s.C * 4}, {dinitial_state, ns}};
    for (int k = 0; k < 5; ++k) {
        for (const Span& q : in)
            if (ranges_meet(out[k].p, out[k].n, q.p, q.n)) return KDA_ERR_INVALID_ARG;
        for (int j = 0; j < k; ++j)
            if (ranges_meet(out[k].p, out[k].n, out[j].p, out[j].n)) return KDA_ERR_INVALID_ARG;
    }
    GatedArgs a = gated_args(s, x, g_raw, i_raw, a_log, cu_seqlens, initial_state);
    st = status_ptr(&a.status);
    if (st != KDA_OK) return st;
    char* ws = static_cast<char*>(workspace);
    const bool pairs = pairs_ok(s, {x, g_raw, i_raw, dy}, {a_log, initial_state, dfinal_state, dx, dg_raw, di_raw, dinitial_state});
    a.rec = static_cast<float*>(const_cast<void*>(saved));
    if (!saved) {      // the states again: a forward that writes only its record
        a.rec = reinterpret_cast<float*>(ws);
        gated_layout(s, kFwdTile, false, ws + up(rec), &a);
        if (gated_forward(a, s.dtype, pairs, stream) != cudaSuccess) return KDA_ERR_CUDA;
    }
    gated_layout(s, kBwdTile, true, ws + up(rec), &a);
    a.dy = dy; a.dsT = dfinal_state; a.dx = dx; a.dg = dg_raw; a.di = di_raw; a.da_log = da_log; a.ds0 = dinitial_state;
    if (gated_begin(a, kBwdTile, pairs ? 2 : 1, dfinal_state, dinitial_state, stream) != cudaSuccess) return KDA_ERR_CUDA;
    const int ctas = a.tiles * a.cols;
    timing_pre(stream, K_GATED_BWD);
    if (pairs) gated_bwd_kernel<__nv_bfloat16, 2><<<ctas, kThreads, 0, stream>>>(a);
    else if (s.dtype == KDA_BF16) gated_bwd_kernel<__nv_bfloat16, 1><<<ctas, kThreads, 0, stream>>>(a);
    else gated_bwd_kernel<float, 1><<<ctas, kThreads, 0, stream>>>(a);
    timing_post(stream);
    if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
    timing_pre(stream, K_GATED_REDUCE);
    gated_reduce_kernel<<<(s.C + 31) / 32, kThreads, 0, stream>>>(a);
    timing_post(stream);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_gated_step(const kda_gated_dims* dims, const void* x, const void* g_raw, const void* i_raw, const float* a_log,
                          const int32_t* slots, int num_slots, const float* state_in, float* state_out, void* y, cudaStream_t stream) {
    Shape s;
    if (!dims || dims->T != 1) return KDA_ERR_INVALID_ARG;
    kda_status st = gated_check(dims, false, &s);
    if (st != KDA_OK) return st;
    if (!x || !g_raw || !i_raw || !a_log || !y || !state_in || !state_out) return KDA_ERR_INVALID_ARG;
    if (num_slots < 1 || (!slots && num_slots < s.B)) return KDA_ERR_INVALID_ARG;
    StepArgs a;
    memset(&a, 0, sizeof(a));
    a.B = s.B; a.C = s.C; a.num_slots = num_slots; a.xs = s.xs; a.gs = s.gs; a.is = s.is;
    a.x = x; a.g = g_raw; a.i = i_raw; a.a_log = a_log; a.slots = slots; a.s_in = state_in; a.s_out = state_out; a.y = y;
    const bool pairs = pairs_ok(s, {x, g_raw, i_raw, y}, {a_log, state_in, state_out});
    const int per = kStepThreads * (pairs ? 2 : 1), cols = (s.C + per - 1) / per;
    if (cols > 65535) return KDA_ERR_UNSUPPORTED;
    st = status_ptr(&a.status);
    if (st != KDA_OK) return st;
    const dim3 grid(s.B, cols);
    timing_pre(stream, K_GATED_STEP);
    if (pairs) gated_step_kernel<__nv_bfloat16, 2><<<grid, kStepThreads, 0, stream>>>(a);
    else if (s.dtype == KDA_BF16) gated_step_kernel<__nv_bfloat16, 1><<<grid, kStepThreads, 0, stream>>>(a);
    else gated_step_kernel<float, 1><<<grid, kStepThreads, 0, stream>>>(a);
    timing_post(stream);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
