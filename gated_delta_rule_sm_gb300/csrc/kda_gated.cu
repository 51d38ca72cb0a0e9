// kda_gated.cu -- the gated linear recurrence: its scan over long sequences, the scan's backward pass and the
// single-token step.  Per channel
//     log a_t = -exp(a_log) sigmoid(g_t),   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t,   y_t = h_t.
//
// One pass over the data: 8 bytes an element forward and 20 backward in bf16 (the gradients are fp32).  The tokens are cut
// into tiles of 64 tokens and 64 channels (32 where two channels cannot be read at once).  A CTA copies a tile's rows to
// shared memory (cp.async, 16 bytes at a time where they are aligned); each of eight warps takes eight consecutive tokens, a
// lane a pair of neighbouring channels.  The recurrence is affine, so that a run of tokens is a pair (P, h): state -> P state
// + h, and runs are joined in three steps: a thread's tokens, the warps of a CTA, the tiles.  The last is a chain along the
// tokens inside the one launch, which a ninth warp follows: it tells the tile's pair, looks back over the tiles before it
// to the nearest one whose leaving state is told, and applies the pairs between in order.  Pairs and states are words that
// say themselves whether they are there.  Tiles are taken from a counter, so that whatever a tile waits for was begun
// before it; the waits are bounded.  A state is the same chain of the same operations wherever the look-back began, so
// results do not depend on timing.
// The backward pass runs the same chain from the last token to the first, on m_t = a_t (dy_t + m_{t+1}), the
// gradient of h_{t-1}; the states it needs enter every 64th token from the forward's record and are carried on inside
// a tile.
// Measured, 16384 tokens x 4096 channels in bf16: forward 134 us with 12 documents and 131 us with 4 rows (537 MB: 4.1
// TB/s), backward 264 us (1.34 GB: 5.1 TB/s; a copy reaches 6.7).  Bound by both sides of a tile's life: the instructions
// (some 90 for two channels of a token forward, 180 backward, 60% of the issue slots) and the waits between its phases.
// Calls of that size with the plan (10 us): 142 and 282 us; every tile with row edges (256 documents of 64 tokens) 190 and 371 us; rates
// above 1/4 everywhere 201 and 417 us; fp32 200 and 368 us (1.07 GB and 1.9).
// Without the chain's waits the forward took 117 us.  The tile's size is at its best: eight warps and 4 CTAs of an SM forward,
// 3 backward; before the copies went ahead (149 and 262 us), 16 warps and tiles of 128 tokens took 164 and 323, 4 warps and tiles of
// 32 tokens 163 and 276, and a fifth CTA (the inputs kept in shared memory, 40 registers) as long as four.
// Precision: everything in fp32, the gates through the approximate exponential, reciprocal and square root (2^-22 or so each; the fp32
// gradients are 2.9e-7 of the norm off where a form with library functions is 2.2e-7).  1 - a comes from a series in
// log a, so that decays next to 1, the long memories, are right to a rounding, and sqrt(1 - a^2) = sqrt(e (2 - e)) with e = 1 - a loses
// nothing there either; decays next to 0, of fast rates, are right to a rounding of themselves.
#include <math.h>
#include <string.h>

#include <type_traits>

#include "kda.h"
#include "kda_common.cuh"
#include "kda_gated.h"
#include "kda_internal.h"
#include "kda_sm100.cuh"

namespace kda {

using namespace sm100;

namespace {

constexpr int kThreads = kGatedThreads, kWarps = kGatedWarps, kAll = kThreads + 32;
constexpr int kTok = kGatedTok, kTile = kGatedTile;
using Spot = GatedSpot;
using Edges = GatedEdges;
static_assert(kThreads == 4 * kTile, "a thread asks for a row of one of four arrays");
constexpr int kFwdCtas = 4, kBwdCtas = 3;           // CTAs of an SM: as many as registers and shared memory allow
constexpr float kLog2e = 1.4426950408889634f;

struct GatedArgs {
    int T, TT, C, rows, tiles, cols, planned, aligned;   // aligned: 16-byte copies of the token arrays
    int64_t xs, gs, is;                  // elements between neighbouring tokens
    const void *x, *g, *i, *dy;
    const float *a_log, *s0, *dsT;
    const int32_t* cu;
    void* y;
    float *sT, *rec;                     // rec [tiles, C]: the state that enters each tile
    float *dx, *dg, *di, *da_log, *ds0;
    // workspace (planned)
    int *ticket, *ok, *first;            // first [tiles]: the first row that begins at or after the tile's first token
    float *agg, *inc;                    // agg [tiles, C] pairs, inc [tiles, C] leaving states; by order in the chain; kUnset before they are known
    int64_t unset;                       // 16-byte pieces of agg and inc together
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
__device__ __forceinline__ float sqr(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float min_nan(float x, float y) {     // NaN if either is
    float z;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
    return z;
}

// e^-z for the gradients, which need 1 less the sigmoid as well; it stops at 2^60: the product of two sums 1 + e^-z stays
// finite, and one reciprocal serves both gates.  From there, z = -41.6, the sigmoid stays at 2^-60, 9e-19.  Next to x and 1 - sigmoid,
// which is 1, that is zero; log a is not formed from it (decay_log).
constexpr float kGateStop = 0x1p60f;
template <typename V> __device__ __forceinline__ V exp_neg(V z) {
    return vmap([](float t) { return min_nan(ex2(t), kGateStop); }, vmul(z, vdup<V>(-kLog2e)));
}

// The rate of a channel, -exp(a_log); wide: some rate of the warp is above 1/4.
template <typename V> struct Rate {
    V n, log2;
    bool wide;
};
template <typename V> __device__ __forceinline__ Rate<V> rate_of(V a) {
    Rate<V> r;
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
template <bool WIDE> __device__ __forceinline__ float log_decay(float g, float sig, const Rate<float>& r) {
    return WIDE && r.wide && !(r.n >= -0.25f) ? wide_log(g, r.log2) : sig * r.n;
}
template <bool WIDE> __device__ __forceinline__ float2 log_decay(float2 g, float2 sig, const Rate<float2>& r) {
    float2 l = mul2(sig, r.n);
    if (WIDE && r.wide) {
        if (!(r.n.x >= -0.25f)) l.x = wide_log(g.x, r.log2.x);
        if (!(r.n.y >= -0.25f)) l.y = wide_log(g.y, r.log2.y);
    }
    return l;
}

// A decay a = e^l, l <= 0, and e = 1 - a, each right to a rounding of itself.  Down to -1/4 e is l times a polynomial of degree 4 for
// (1 - e^l) / l (interpolated at the Chebyshev points of [-1/4, 0] in 64 bits; off by 5e-9 of the value with its coefficients in
// fp32), and a is 1 - e; below, which only a wide rate can reach, a is the exponential, and e is 1 - a.
template <typename V> struct Decay {
    V a, e;
};
template <typename V> __device__ __forceinline__ Decay<V> exp_decay(V l, bool wide) {
    V p = vfma(l, vdup<V>(-0.007513606455177069f), vdup<V>(-0.04149065539240837f));
    p = vfma(p, l, vdup<V>(-0.16665108501911163f));
    p = vfma(p, l, vdup<V>(-0.4999995231628418f));
    p = vfma(p, l, vdup<V>(-1.f));
    Decay<V> d;
    d.e = vmul(l, p);
    d.a = vfma(d.e, vdup<V>(-1.f), vdup<V>(1.f));
    if (wide) {
        auto far = [](float t, float& a, float& e) {
            if (t < -0.25f) {
                a = ex2(t * kLog2e);
                e = 1.f - a;
            }
        };
        if constexpr (std::is_same_v<V, float2>) {
            far(l.x, d.a.x, d.e.x);
            far(l.y, d.a.y, d.e.y);
        } else {
            far(l, d.a, d.e);
        }
    }
    return d;
}
// Both in one word, which the backward pass keeps: e, or, where a is below a half, a with its sign set (-0 where a is 0).  (Only where a
// rate may be wide; the backward calls with row edges or wide rates everywhere took 352 and 397 us with e alone, 371 and 417 so.)
template <bool WIDE> __device__ __forceinline__ float pack(const Decay<float>& d) { return WIDE && d.a < 0.5f ? -d.a : d.e; }
template <bool WIDE> __device__ __forceinline__ float2 pack(const Decay<float2>& d) {
    return make_float2(WIDE && d.a.x < 0.5f ? -d.a.x : d.e.x, WIDE && d.a.y < 0.5f ? -d.a.y : d.e.y);
}
template <bool WIDE> __device__ __forceinline__ bool holds_a(float w) { return WIDE && __float_as_int(w) < 0; }
template <bool WIDE> __device__ __forceinline__ float keep_of(float w) { return holds_a<WIDE>(w) ? -w : 1.f - w; }
template <bool WIDE> __device__ __forceinline__ float2 keep_of(float2 w) {
    const float2 a = fma2(w, make_float2(-1.f, -1.f), make_float2(1.f, 1.f));
    return make_float2(holds_a<WIDE>(w.x) ? -w.x : a.x, holds_a<WIDE>(w.y) ? -w.y : a.y);
}
template <bool WIDE, typename V> __device__ __forceinline__ V loss_of(V w) {
    return vmap([](float t) { return holds_a<WIDE>(t) ? 1.f + t : t; }, w);
}

// 1 / sqrt(1 - a^2) from w = 1 - a^2 = e (2 - e).  Where a is 1 to fp32 it stops at 1e18: w, and with it -log a, is then below 1e-36, so that
// the input's factor w / sqrt(w) and the gradients' log a / sqrt(w) are below 1e-18, as their limit is.
template <typename V> __device__ __forceinline__ V square_of(V e) { return vmul(e, vfma(e, vdup<V>(-1.f), vdup<V>(2.f))); }
template <typename V> __device__ __forceinline__ V root_of(V w) {
    return vmap([](float t) { return rsq(fmaxf(t, 1e-36f)); }, w);
}

// Both gates of a token: their sigmoids, and 1 less them (e^-z times them, exact where they are close to 1).
template <typename V> struct Gates {
    V eg, ei, sg, si;
};
template <typename V> __device__ __forceinline__ Gates<V> gates_of(V g, V i) {
    Gates<V> k;
    k.eg = exp_neg(g);
    k.ei = exp_neg(i);
    const V one = vdup<V>(1.f), da = vfma(k.eg, one, one), db = vfma(k.ei, one, one);
    const V r = vmap([](float t) { return rcp(t); }, vmul(da, db));
    k.sg = vmul(r, db);
    k.si = vmul(r, da);
    return k;
}

// log a of a token whose e = 1 - a is known, for the gradients, which divide it by sqrt(1 - a^2).  Where the gate's e^-g stopped the sigmoid is too
// large by up to any factor, and the quotient would be of the order of 1 where its limit is 0; e is of the true sigmoid, and
// log a is -e there to less than a rounding (e < 2^-61).
template <bool WIDE> __device__ __forceinline__ float decay_log(float g, float e, const Gates<float>& z, const Rate<float>& r) {
    return WIDE && r.wide && !(r.n >= -0.25f) ? wide_log(g, r.log2) : z.eg == kGateStop ? -e : z.sg * r.n;
}
template <bool WIDE> __device__ __forceinline__ float2 decay_log(float2 g, float2 e, const Gates<float2>& z, const Rate<float2>& r) {
    float2 l = log_decay<WIDE>(g, z.sg, r);
    if (z.eg.x == kGateStop && (!WIDE || r.n.x >= -0.25f)) l.x = -e.x;
    if (z.eg.y == kGateStop && (!WIDE || r.n.y >= -0.25f)) l.y = -e.y;
    return l;
}

// What the state needs of them: a reciprocal each, which takes an infinite e^-z as it is.
template <typename V> __device__ __forceinline__ V sigmoid(V z) {
    const V one = vdup<V>(1.f), e = vmap([](float t) { return ex2(t); }, vmul(z, vdup<V>(-kLog2e)));
    return vmap([](float t) { return rcp(t); }, vfma(e, one, one));
}
// The decay of a token and its input sqrt(1 - a^2) sigmoid(i) x.
template <bool WIDE, typename V> __device__ __forceinline__ Decay<V> decay_of(V g, V i, V x, const Rate<V>& rate, V& b) {
    const Decay<V> d = exp_decay(log_decay<WIDE>(g, sigmoid(g), rate), WIDE && rate.wide);
    b = vmul(vmap([](float t) { return sqr(t); }, square_of(d.e)), vmul(sigmoid(i), x));
    return d;
}

// ------------------------------------------------------------------ rows inside a tile

__device__ __forceinline__ void tile_sync();

// The first row that begins at or after token t0 of a tile, and where.
struct RowHint {
    int row, begin;
};
__device__ __forceinline__ bool has_edges(const GatedArgs& a, int t0, const RowHint& h) { return h.begin <= t0 + kTile; }
__device__ __forceinline__ void find_edges(const GatedArgs& a, int t0, const RowHint& hint, Edges& s) {
    if (threadIdx.x < kTile) s.first[threadIdx.x] = s.last[threadIdx.x] = -1;
    tile_sync();
    const int t1 = min(t0 + kTile, a.TT);
    for (int m = hint.row + threadIdx.x; m <= a.rows; m += kThreads) {
        const int at = row_begin(a, m);
        if (at > t1) break;
        if (m < a.rows && at < t1 && row_begin(a, m + 1) > at) s.first[at - t0] = m;
        if (m > 0 && at > t0 && row_begin(a, m - 1) < at) s.last[at - 1 - t0] = m - 1;
    }
    tile_sync();
}

// ------------------------------------------------------------------ the chain of tiles

// What a tile tells its successors are single words, each of which says itself whether it is there: kUnset is a NaN that no operation
// gives.  So nothing has to be ordered, and what is read is the value itself: a flag beside it would cost the writer a wait for its
// stores and the reader a second trip to the L2.
constexpr uint32_t kUnset = 0xffffffffu;
__device__ __forceinline__ float told(float v) { return __float_as_uint(v) == kUnset ? __uint_as_float(0x7fffffffu) : v; }
__device__ __forceinline__ bool known(float v) { return __float_as_uint(v) != kUnset; }
__device__ __forceinline__ bool known(float2 v) { return known(v.x) && known(v.y); }
__device__ __forceinline__ void tell(float* p, float v) { asm volatile("st.relaxed.gpu.global.f32 [%0], %1;" ::"l"(p), "f"(told(v)) : "memory"); }
__device__ __forceinline__ void tell(float* p, float2 v) {
    asm volatile("st.relaxed.gpu.global.v2.f32 [%0], {%1, %2};" ::"l"(p), "f"(told(v.x)), "f"(told(v.y)) : "memory");
}
__device__ __forceinline__ void tell(float* p, float a, float b) { tell(p, make_float2(a, b)); }
__device__ __forceinline__ void tell(float* p, float2 a, float2 b) {
    asm volatile("st.relaxed.gpu.global.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(told(a.x)), "f"(told(a.y)), "f"(told(b.x)), "f"(told(b.y)) : "memory");
}
__device__ __forceinline__ void ask(const float* p, float& v) { asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory"); }
__device__ __forceinline__ void ask(const float* p, float2& v) {
    asm volatile("ld.relaxed.gpu.global.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
}
__device__ __forceinline__ void ask(const float* p, float& a, float& b) {
    float2 v;
    ask(p, v);
    a = v.x;
    b = v.y;
}
__device__ __forceinline__ void ask(const float* p, float2& a, float2& b) {
    asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(a.x), "=f"(a.y), "=f"(b.x), "=f"(b.y) : "l"(p) : "memory");
}

// The state that enters the o-th tile of the chain, of this lane's channels: from the nearest tile before it that has told its
// leaving state on, the pairs of those between, in order.  The first tile of a chain, and every tile in which a row begins,
// tells a state, so there is one.  At most about a second, then the error is recorded and the state is 0.
template <typename V> __device__ __forceinline__ V look_back(const GatedArgs& a, int o, int c) {
    constexpr int W = 4;                 // tiles looked at together (1, 2: the same time; 8: 158 us for 137, the L2 is asked too often)
    const float *inc = a.inc + c, *agg = a.agg + 2 * (size_t)c;
    int near = o - 1;                    // the pairs of the tiles above it are there
    V s = vdup<V>(0.f);
    for (int tries = 0;;) {
        V state[W], P[W], h[W];
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const size_t j = max(near - k, 0);
            ask(inc + j * a.C, state[k]);
            ask(agg + 2 * j * a.C, P[k], h[k]);
        }
        // the nearest state, if every pair before it is there
        int at = -1;
        bool open = true;
#pragma unroll
        for (int k = 0; k < W; ++k)
            if (open) {
                if (known(state[k])) {
                    at = k;
                    open = false;
                } else {
                    open = known(P[k]) && known(h[k]);
                }
            }
        if (at >= 0) {
#pragma unroll
            for (int k = W - 1; k >= 0; --k)
                if (k == at) s = state[k];
                else if (k < at) s = vfma(P[k], s, h[k]);
            break;
        }
        if (open && near - W >= 0) {
            near -= W;
        } else if (++tries > (1 << 20)) {
            record_error(a.status, KDA_ERR_TIMEOUT);
            return vdup<V>(0.f);
        }
    }
    // the pairs that were passed on the way
    for (int j = near + 1; j < o; ++j) {
        V P, h;
        ask(agg + 2 * (size_t)j * a.C, P, h);
        s = vfma(P, s, h);
    }
    return s;
}

// The chain's warp.  closed: a row begins in the tile, so that what leaves it does not depend on what enters; needs: some token
// depends on what enters; give(the state that enters).
template <typename V, typename F>
__device__ __forceinline__ void join_chain(const GatedArgs& a, int o, int c, bool in, V P, V h, bool closed, bool needs, F&& give) {
    if (!a.planned || !in) return give(vdup<V>(0.f));
    float* leaving = a.inc + (size_t)o * a.C + c;
    if (closed) tell(leaving, h);
    else tell(a.agg + 2 * ((size_t)o * a.C + c), P, h);
    const V s = needs || !closed ? look_back<V>(a, o, c) : vdup<V>(0.f);
    if (!closed) tell(leaving, vfma(P, s, h));
    give(s);
}

// Barriers of a tile: 4, backward, which tile it is, is known (the eight warps wait); 1, its runs are in shared memory (the chain's warp
// waits); 2, the entering state is (the others wait); 3, the eight warps among themselves.
__device__ __forceinline__ void runs_ready() {
    __syncwarp();
    asm volatile("bar.arrive 1, %0;" ::"n"(kAll) : "memory");
}
__device__ __forceinline__ void runs_wait() { asm volatile("bar.sync 1, %0;" ::"n"(kAll) : "memory"); }
__device__ __forceinline__ void state_ready() {
    __syncwarp();
    asm volatile("bar.arrive 2, %0;" ::"n"(kAll) : "memory");
}
__device__ __forceinline__ void state_wait() { asm volatile("bar.sync 2, %0;" ::"n"(kAll) : "memory"); }
template <bool TELLS> __device__ __forceinline__ void tile_known() {
    __syncwarp();
    if constexpr (TELLS) asm volatile("bar.arrive 4, %0;" ::"n"(kAll) : "memory");
    else asm volatile("bar.sync 4, %0;" ::"n"(kAll) : "memory");
}
__device__ __forceinline__ void tile_sync() { asm volatile("bar.sync 3, %0;" ::"n"(kThreads) : "memory"); }

// Tiles in the order in which they are begun.  A tile that was taken and not begun holds up all that wait for it.  Forward a CTA
// takes its next one when it has told the runs of the one it has, and copies it while it waits for the entering state
// (taken with that state known, 149 us for 141; a whole tile ahead, 188).  Backward the copies have to stay until the gradients are
// formed, and the next tile is taken when the entering state is known.
__device__ __forceinline__ int take_ticket(const GatedArgs& a, int before) {
    return a.planned ? atomicAdd(a.ticket, 1) : before < 0 ? (int)blockIdx.x : before + (int)gridDim.x;
}

// Clears the counter and what the tiles will tell, checks the offsets, finds each tile's first row, and passes the states of rows without
// tokens through (of all rows where the offsets break the contract).
__global__ void __launch_bounds__(kThreads) gated_plan_kernel(GatedArgs a, const float* from, float* to) {
    cudaTriggerProgrammaticLaunchCompletion();       // the pass may be launched; it waits for this kernel's end
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
    for (int64_t k = id; k < a.unset; k += all) reinterpret_cast<uint4*>(a.agg)[k] = make_uint4(kUnset, kUnset, kUnset, kUnset);
    if (!a.cu) return;
    for (int k = id; !bad && k < a.tiles; k += all) {
        int lo = 0, hi = a.rows;          // (cu[rows] = TT is past every tile's first token)
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (a.cu[mid] >= k * kTile) hi = mid; else lo = mid + 1;
        }
        a.first[k] = lo;
    }
    if (to)
        for (int n = blockIdx.x; n < a.rows; n += gridDim.x)
            if (bad || a.cu[n + 1] == a.cu[n])
                for (int c = threadIdx.x; c < a.C; c += kThreads)
                    to[(size_t)n * a.C + c] = from ? from[(size_t)n * a.C + c] : 0.f;
}

template <int VEC> __device__ __forceinline__ Spot spot_of(const GatedArgs& a, int tile, int col) {
    return gated_spot<VEC>(a.TT, a.C, tile, col, threadIdx.x);
}
// A [tokens, C] array's elements of the tile, a token's 32 lanes side by side as the threads will read them.
template <typename E, int VEC> using Plane = Raw<E, VEC>[kTok][kThreads];
template <int BYTES> __device__ __forceinline__ void copy_async(void* dst, const void* src) {
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_landed() {
    asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;" ::: "memory");
    tile_sync();
}
// Whole tiles of arrays that allow it move 16 bytes at a time; otherwise a thread brings its own elements.  (The tile's base is one for
// the CTA; an offset from it fits 32 bits.)
template <typename E, int VEC>
__device__ __forceinline__ void load_plane(const void* p, int64_t stride, const Spot& s, bool whole, bool aligned, Plane<E, VEC>& to) {
    const E* base = static_cast<const E*>(p) + s.t0 * stride;
    const uint32_t step = (uint32_t)stride;
    if (sizeof(Raw<E, VEC>) == 4 && whole && aligned) {
        constexpr int PER = 128 / 16;        // pieces of a token's 32 lanes
#pragma unroll
        for (int i = 0; i < kTile * PER / kThreads; ++i) {
            const int id = i * kThreads + threadIdx.x, token = id / PER, piece = id % PER;
            copy_async<16>(&to[token % kTok][token / kTok * 32 + piece * 4], base + (token * step + s.col * 32 * VEC + piece * (int)(16 / sizeof(E))));
        }
        return;
    }
    const uint32_t at = s.warp * kTok * step + s.c;
#pragma unroll
    for (int k = 0; k < kTok; ++k) {
        Raw<E, VEC>& r = to[k][threadIdx.x];
        if (k >= s.n) r.zero();
        else if constexpr (sizeof(Raw<E, VEC>) == 4) copy_async<4>(&r, base + (at + k * step));
        else r.load(base, at + k * step);
    }
}

// Asks the L2 for a row of a tile that some CTA will take soon: by then its copies find it there.
template <typename E, int VEC>
__device__ __forceinline__ void prefetch_row(const GatedArgs& a, const void* p, int64_t stride, int tile, int col, int row) {
    const int t = tile * kTile + row;
    if (t < a.TT)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const E*>(p) + t * stride + col * 32 * VEC));
}

// Whether every thread of the CTA has all its tokens and channels.
template <int VEC> __device__ __forceinline__ bool whole_tile(const GatedArgs& a, const Spot& s) {
    return s.t0 + kTile <= a.TT && (s.col + 1) * 32 * VEC <= a.C;
}

// ------------------------------------------------------------------ forward

// A tile as the one who takes it announces it (the first thread, backward the ninth warp): its place in the chain (past the last: none), itself, its columns; and, backwards, one that
// comes as many tickets later as there are CTAs.
struct TileWord {
    int o, tile, col, soon_o, soon_col;
};
struct TileWords {
    TileWord at[2];
    int closed, needs;
};
template <typename E, int VEC> struct FwdShared {
    using V = Val<VEC>;
    Plane<E, VEC> x, g, i;
    Edges edges;
    V sp[kWarps][32], sh[kWarps][32], senter[32];
    TileWords w;
};

// EDGE: the tile has rows that begin or end in it, tokens or channels past the last, or a rate above 1/4.
template <typename E, int VEC, bool EDGE, typename N>
__device__ __forceinline__ void forward_tile(const GatedArgs& a, const Spot& s, FwdShared<E, VEC>& m_, bool split, const Rate<Val<VEC>>& rate, N&& next) {
    using V = Val<VEC>;
    const Edges& edges = m_.edges;
    auto &sp = m_.sp, &sh = m_.sh;
    auto &mx = m_.x, &mg = m_.g, &mi = m_.i;
    const int tid = threadIdx.x;
    auto begins_at = [&](int k) { return EDGE && split ? edges.first[s.warp * kTok + k] : -1; };
    // a token as h -> ka h + kb; where a row begins the state is the row's own, and ka is 0 (also for lanes past the last channel, which
    // ask for no state: a branch of the whole warp took 1 % less than one of its lanes)
    V ka[kTok], kb[kTok], P, h;
#pragma unroll
    for (int k = 0; k < kTok; ++k) {
        ka[k] = decay_of<EDGE>(mg[k][tid].get(), mi[k][tid].get(), mx[k][tid].get(), rate, kb[k]).a;
        if (EDGE && k >= s.n) {
            ka[k] = vdup<V>(1.f);
            kb[k] = vdup<V>(0.f);
        }
        const bool begins = begins_at(k) >= 0;
        if (EDGE && begins) {
            if (a.s0 && edges.begins(s, k) >= 0) kb[k] = vfma(ka[k], vload<V>(a.s0 + (size_t)begins_at(k) * a.C + s.c), kb[k]);
            ka[k] = vdup<V>(0.f);
        }
        if (k == 0 || (EDGE && begins)) {
            P = ka[k];
            h = kb[k];
        } else {
            P = vmul(P, ka[k]);
            h = vfma(ka[k], h, kb[k]);
        }
    }
    sp[s.warp][s.lane] = P;
    sh[s.warp][s.lane] = h;
    if (s.warp == 0) {
        bool begins = false;
        if (EDGE && split)
            for (int k = s.lane; k < kTile; k += 32) begins |= edges.first[k] >= 0;
        if (EDGE) begins = __any_sync(0xffffffffu, begins);
        m_.w.closed = begins;
        m_.w.needs = !EDGE || !split || edges.first[0] < 0;
    }
    runs_ready();
    next();
    // meanwhile the runs of the warps before this one
    auto over = [](V P, V s, V h) { return EDGE ? join(P, s, h) : vfma(P, s, h); };
    P = vdup<V>(1.f);
    h = vdup<V>(0.f);
    for (int w = 0; w < s.warp; ++w) {
        const V p = sp[w][s.lane];
        P = over(p, P, vdup<V>(0.f));
        h = over(p, h, sh[w][s.lane]);
    }
    state_wait();
    h = over(P, m_.senter[s.lane], h);
    E* y = static_cast<E*>(a.y) + (size_t)s.t0 * a.C;
    const uint32_t at = s.warp * kTok * (uint32_t)a.C + s.c;
#pragma unroll
    for (int k = 0; k < kTok; ++k)
        if (!EDGE || k < s.n) {
            h = EDGE && begins_at(k) >= 0 ? kb[k] : vfma(ka[k], h, kb[k]);
            if (a.y) Raw<E, VEC>::store(y, at + k * (uint32_t)a.C, h);
            if (EDGE && split && a.sT && edges.ends(s, k) >= 0) vstore(a.sT + (size_t)edges.ends(s, k) * a.C + s.c, h);
        }
}

// The loop of both passes.  load(spot) issues a tile's copies, work(spot, hint, rate, next) does it and, forward, calls next() when its
// copies have been read, soon(tile, columns)
// asks the L2 for a later one (backwards alone: it brought 301 to 287 us there, but 154 to 159 forward).  The ninth warp joins
// the chain: the runs of the warps from the first (or, backwards, from the last) on.
template <bool BACK, int VEC, typename L, typename N, typename W>
__device__ __forceinline__ void walk_tiles(const GatedArgs& a, TileWords& w, Val<VEC> (&sp)[kWarps][32], Val<VEC> (&sh)[kWarps][32],
                                           Val<VEC> (&senter)[32], L&& load, N&& soon, W&& work) {
    using V = Val<VEC>;
    const uint32_t total = (uint32_t)a.tiles * a.cols;
    // (offsets that break the contract: the plan has found no tile's first row, and nothing is read by them)
    const bool go = !a.planned || *a.ok;
    if (!go) return;
    const int lane = threadIdx.x & 31;
    int before = -1;
    auto take = [&](int it) {            // (by one thread)
        const uint32_t ticket = take_ticket(a, before);
        before = (int)ticket;
        TileWord n;
        n.o = ticket < total ? (int)(ticket / (uint32_t)a.cols) : a.tiles;
        n.col = (int)(ticket - (uint32_t)n.o * a.cols);
        n.tile = BACK ? a.tiles - 1 - n.o : n.o;
        if constexpr (BACK) {
            const uint32_t later = ticket + gridDim.x;
            n.soon_o = later < total ? (int)(later / (uint32_t)a.cols) : a.tiles;
            n.soon_col = (int)(later - (uint32_t)n.soon_o * a.cols);
        }
        w.at[it & 1] = n;
    };
    if (threadIdx.x >= kThreads) {
        for (int it = 0;; ++it) {
            if constexpr (BACK) {
                if (lane == 0) take(it);
                tile_known<true>();
                if (w.at[it & 1].o >= a.tiles) return;
            }
            runs_wait();
            const int o = w.at[it & 1].o, c = (w.at[it & 1].col * 32 + lane) * VEC;
            if (!BACK && o >= a.tiles) return;
            V P = sp[BACK ? kWarps - 1 : 0][lane], h = sh[BACK ? kWarps - 1 : 0][lane];
#pragma unroll
            for (int k = 1; k < kWarps; ++k) {
                const V p = sp[BACK ? kWarps - 1 - k : k][lane], q = sh[BACK ? kWarps - 1 - k : k][lane];
                P = join(p, P, vdup<V>(0.f));
                h = join(p, h, q);
            }
            V enters;
            join_chain<V>(a, o, c, c < a.C, P, h, w.closed, w.needs, [&](V v) { enters = v; });
            senter[lane] = enters;
            state_ready();
            if (!BACK && a.rec && c < a.C) vstore(a.rec + (size_t)o * a.C + c, enters);
        }
    }
    if constexpr (!BACK) {
        if (threadIdx.x == 0) take(0);
        tile_sync();
        if (w.at[0].o < a.tiles) load(spot_of<VEC>(a, w.at[0].tile, w.at[0].col));
    }
    for (int it = 0;; ++it) {
        if constexpr (BACK) tile_known<false>();
        const TileWord now = w.at[it & 1];
        if (now.o >= a.tiles) {
            if (!BACK) runs_ready();
            return;
        }
        const Spot s = spot_of<VEC>(a, now.tile, now.col);
        if constexpr (BACK) {
            load(s);
            if (now.soon_o < a.tiles) soon(a.tiles - 1 - now.soon_o, now.soon_col);
        }
        RowHint hint;
        hint.row = a.cu ? a.first[s.tile] : (int)(((uint32_t)s.t0 + a.T - 1) / (uint32_t)a.T);
        hint.begin = row_begin(a, hint.row);
        const Rate<V> rate = rate_of(s.in ? vload<V>(a.a_log + s.c) : vdup<V>(-1e30f));
        copies_landed();
        work(s, hint, rate, [&]() {
            // the next tile, whose copies go where this one's were
            if (threadIdx.x == 0) take(it + 1);
            tile_sync();
            const TileWord next = w.at[(it + 1) & 1];
            if (next.o < a.tiles) load(spot_of<VEC>(a, next.tile, next.col));
        });
    }
}

template <typename E, int VEC>
__global__ void __launch_bounds__(kAll, kFwdCtas) gated_fwd_kernel(const __grid_constant__ GatedArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    FwdShared<E, VEC>& m = *reinterpret_cast<FwdShared<E, VEC>*>(smem);
    cudaGridDependencySynchronize();
    walk_tiles<false, VEC>(
        a, m.w, m.sp, m.sh, m.senter,
        [&](const Spot& s) {
            const bool whole = whole_tile<VEC>(a, s);
            load_plane<E, VEC>(a.x, a.xs, s, whole, a.aligned, m.x);
            load_plane<E, VEC>(a.g, a.gs, s, whole, a.aligned, m.g);
            load_plane<E, VEC>(a.i, a.is, s, whole, a.aligned, m.i);
        },
        [](int, int) {},
        [&](const Spot& s, const RowHint& hint, const Rate<Val<VEC>>& rate, auto&& next) {
            const bool split = has_edges(a, s.t0, hint);
            if (split) find_edges(a, s.t0, hint, m.edges);
            if (whole_tile<VEC>(a, s) && !split && !rate.wide) forward_tile<E, VEC, false>(a, s, m, split, rate, next);
            else forward_tile<E, VEC, true>(a, s, m, split, rate, next);
        });
}

// ------------------------------------------------------------------ backward

// The gates are formed twice, before and after the chain: keeping them in between would halve the number of CTAs.
template <typename E, int VEC> struct BwdShared {
    using V = Val<VEC>;
    Plane<E, VEC> x, g, i, dy;
    Edges edges;
    V sp[kWarps][32], sh[kWarps][32], sq[kWarps][32], sm[kWarps][32], senter[32];
    V d[kTok][kThreads], b[kTok][kThreads];       // the decays; the inputs, then the states before the tokens
    TileWords w;
};

template <typename E, int VEC, bool EDGE>
__device__ __forceinline__ void backward_tile(const GatedArgs& a, const Spot& s, BwdShared<E, VEC>& m_, bool split, const Rate<Val<VEC>>& rate) {
    using V = Val<VEC>;
    const int tid = threadIdx.x, warp = s.warp, lane = s.lane, c = s.c;
    auto &mx = m_.x, &mg = m_.g, &mi = m_.i, &md = m_.dy;
    auto begins_at = [&](int k) { return EDGE && split ? m_.edges.begins(s, k) : -1; };
    auto ends_at = [&](int k) { return EDGE && split ? m_.edges.ends(s, k) : -1; };
    auto row_of = [&](const float* p, int row) { return p ? vload<V>(p + (size_t)row * a.C + c) : vdup<V>(0.f); };
    auto over = [](V P, V s, V h) { return EDGE ? join(P, s, h) : vfma(P, s, h); };
    const V one = vdup<V>(1.f), entering = s.in ? vload<V>(a.rec + (size_t)s.tile * a.C + c) : vdup<V>(0.f);
    // the forward's runs, from the first token on
    V P = one, h = vdup<V>(0.f);
#pragma unroll 8
    for (int k = 0; k < kTok; ++k) {
        V b;
        Decay<V> d = decay_of<EDGE>(mg[k][tid].get(), mi[k][tid].get(), mx[k][tid].get(), rate, b);
        if (EDGE && k >= s.n) d = {one, b = vdup<V>(0.f)};
        const V ka = d.a;
        if (EDGE && begins_at(k) >= 0) {
            P = vdup<V>(0.f);
            h = row_of(a.s0, begins_at(k));
        }
        P = vmul(P, ka);
        h = vfma(ka, h, b);
        m_.d[k][tid] = pack<EDGE>(d);
        m_.b[k][tid] = b;
    }
    m_.sp[warp][lane] = P;
    m_.sh[warp][lane] = h;
    // the gradient's, from the last
    P = one;
    V m = vdup<V>(0.f);
#pragma unroll 8
    for (int k = kTok - 1; k >= 0; --k) {
        if (EDGE && ends_at(k) >= 0) {
            P = vdup<V>(0.f);
            m = row_of(a.dsT, ends_at(k));
        }
        const V ka = keep_of<EDGE>(m_.d[k][tid]);
        P = vmul(P, ka);
        m = vmul(ka, vfma(md[k][tid].get(), one, m));
    }
    m_.sq[warp][lane] = P;
    m_.sm[warp][lane] = m;
    if (warp == 0) {
        bool ends = false;
        if (EDGE && split)
            for (int k = lane; k < kTile; k += 32) ends |= m_.edges.last[k] >= 0;
        if (EDGE) ends = __any_sync(0xffffffffu, ends);
        m_.w.closed = ends;
        m_.w.needs = !EDGE || !split || m_.edges.last[min(kTile, a.TT - s.t0) - 1] < 0;
    }
    runs_ready();
    tile_sync();
    // meanwhile the states before the tokens
    h = entering;
    for (int w = 0; w < warp; ++w) h = over(m_.sp[w][lane], h, m_.sh[w][lane]);
#pragma unroll 8
    for (int k = 0; k < kTok; ++k) {
        if (EDGE && begins_at(k) >= 0) h = row_of(a.s0, begins_at(k));
        const V b = m_.b[k][tid];
        m_.b[k][tid] = h;
        h = vfma(keep_of<EDGE>(m_.d[k][tid]), h, b);
    }
    state_wait();
    m = m_.senter[lane];
    for (int w = kWarps - 1; w > warp; --w) m = over(m_.sq[w][lane], m, m_.sm[w][lane]);
    V dlog = vdup<V>(0.f);
    const size_t base = (size_t)s.t0 * a.C;
    float *dx = a.dx + base, *dg = a.dg + base, *di = a.di + base;
    const uint32_t at = warp * kTok * (uint32_t)a.C + c;
#pragma unroll 8
    for (int k = kTok - 1; k >= 0; --k)
        if (!EDGE || k < s.n) {
            if (EDGE && ends_at(k) >= 0) m = row_of(a.dsT, ends_at(k));
            const V g = mg[k][tid].get();
            const Gates<V> z = gates_of(g, mi[k][tid].get());
            const V d = m_.d[k][tid], e = loss_of<EDGE>(d), w = square_of(e), root = root_of(w), ka = keep_of<EDGE>(d);
            const V dh = vfma(md[k][tid].get(), one, m);                  // the gradient of h_t
            m = vmul(ka, dh);
            if (EDGE && begins_at(k) >= 0 && a.ds0) vstore(a.ds0 + (size_t)begins_at(k) * a.C + c, m);
            const V u = vmul(z.si, mx[k][tid].get()), du = vmul(dh, vmul(w, root));
            // of log a: a (h_{t-1} - u a / sqrt(1 - a^2)) times that of h_t; then times log a for a_log, and 1 - sigmoid(g) for g
            const V dl = vmul(vmul(m, vfma(vmul(u, vdup<V>(-1.f)), vmul(ka, root), m_.b[k][tid])), decay_log<EDGE>(g, e, z, rate));
            dlog = vfma(dl, one, dlog);
            const uint32_t to = at + k * (uint32_t)a.C;
            vstore_stream(dx + to, vmul(du, z.si));
            vstore_stream(dg + to, vmul(dl, vmul(z.eg, z.sg)));
            vstore_stream(di + to, vmul(vmul(du, u), vmul(z.ei, z.si)));
        }
    tile_sync();
    m_.sp[warp][lane] = dlog;
    tile_sync();
    if (warp == 0 && s.in) {
        dlog = m_.sp[0][lane];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) dlog = vfma(m_.sp[w][lane], one, dlog);
        vstore(a.part + (size_t)s.tile * a.C + c, dlog);
    }
}

template <typename E, int VEC>
__global__ void __launch_bounds__(kAll, kBwdCtas) gated_bwd_kernel(const __grid_constant__ GatedArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    BwdShared<E, VEC>& m = *reinterpret_cast<BwdShared<E, VEC>*>(smem);
    cudaGridDependencySynchronize();
    walk_tiles<true, VEC>(
        a, m.w, m.sq, m.sm, m.senter,
        [&](const Spot& s) {
            const bool whole = whole_tile<VEC>(a, s);
            load_plane<E, VEC>(a.x, a.xs, s, whole, a.aligned, m.x);
            load_plane<E, VEC>(a.g, a.gs, s, whole, a.aligned, m.g);
            load_plane<E, VEC>(a.i, a.is, s, whole, a.aligned, m.i);
            load_plane<E, VEC>(a.dy, a.C, s, whole, a.aligned, m.dy);
        },
        [&](int tile, int col) {
            const int row = threadIdx.x % kTile;
            if (threadIdx.x < kTile) prefetch_row<E, VEC>(a, a.x, a.xs, tile, col, row);
            else if (threadIdx.x < 2 * kTile) prefetch_row<E, VEC>(a, a.g, a.gs, tile, col, row);
            else if (threadIdx.x < 3 * kTile) prefetch_row<E, VEC>(a, a.i, a.is, tile, col, row);
            else prefetch_row<E, VEC>(a, a.dy, a.C, tile, col, row);
        },
        [&](const Spot& s, const RowHint& hint, const Rate<Val<VEC>>& rate, auto&&) {
            const bool split = has_edges(a, s.t0, hint);
            if (split) find_edges(a, s.t0, hint, m.edges);
            if (whole_tile<VEC>(a, s) && !split && !rate.wide) backward_tile<E, VEC, false>(a, s, m, split, rate);
            else backward_tile<E, VEC, true>(a, s, m, split, rate);
        });
}

// da_log: the tiles' parts in a fixed order, 32 channels to a CTA.
constexpr int kReduceWarps = 32;
__global__ void __launch_bounds__(kReduceWarps * 32) gated_reduce_kernel(const __grid_constant__ GatedArgs a) {
    __shared__ float s[kReduceWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane;
    cudaGridDependencySynchronize();
    float t = 0.f;
    if (c < a.C && (!a.planned || *a.ok))
        for (int k = warp; k < a.tiles; k += kReduceWarps) t += a.part[(size_t)k * a.C + c];
    s[warp][lane] = t;
    __syncthreads();
    if (warp || c >= a.C) return;
#pragma unroll
    for (int w = 1; w < kReduceWarps; ++w) t += s[w][lane];
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
    const Rate<V> rate = rate_of(vload<V>(a.a_log + c));
    V add;
    const V h = vfma(decay_of<true>(rg.get(), ri.get(), rx.get(), rate, add).a, old, add);
    vstore(a.s_out + (size_t)slot * a.C + c, h);
    R::store(a.y, (size_t)b * a.C + c, h);
}

// ------------------------------------------------------------------ host

struct Shape {
    int B, T, TT, C, rows, dtype, es;
    int64_t xs, gs, is;
};

constexpr int64_t kMostStride = 1 << 25;      // an offset inside a tile fits 32 bits

kda_status gated_check(const kda_gated_dims* d, bool varlen, Shape* s) {
    if (!d || d->B < 1 || d->T < 1 || d->C < 1) return KDA_ERR_INVALID_ARG;
    if (d->dtype != KDA_BF16 && d->dtype != KDA_FP32) return KDA_ERR_INVALID_ARG;
    if (varlen && (d->B != 1 || d->num_seqs < 1)) return KDA_ERR_INVALID_ARG;
    for (int64_t st : {d->x_stride, d->g_stride, d->i_stride})
        if (st != 0 && st < d->C) return KDA_ERR_INVALID_ARG;
    if ((int64_t)d->B * d->T > (1LL << 30) || d->C > kMostStride || (varlen && d->num_seqs > (1 << 24))) return KDA_ERR_UNSUPPORTED;
    s->B = d->B; s->T = d->T; s->TT = d->B * d->T; s->C = d->C; s->rows = varlen ? d->num_seqs : d->B;
    s->dtype = d->dtype; s->es = d->dtype == KDA_BF16 ? 2 : 4;
    s->xs = d->x_stride ? d->x_stride : d->C;
    s->gs = d->g_stride ? d->g_stride : d->C;
    s->is = d->i_stride ? d->i_stride : d->C;
    for (int64_t st : {s->xs, s->gs, s->is})
        if (s->TT > 1 && (st > (1LL << 40) / s->TT || st > kMostStride)) return KDA_ERR_UNSUPPORTED;
    // (tiles x columns and the workspace's indices)
    if ((int64_t)((s->TT + kTile - 1) / kTile) * ((s->C + 31) / 32) > (1LL << 30)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }
size_t gated_record_bytes(const Shape& s) { return (size_t)((s.TT + kTile - 1) / kTile) * s.C * 4; }

// Workspace of one pass; fills the views where ws is given.
size_t gated_layout(const Shape& s, bool reduce, char* ws, GatedArgs* a) {
    const size_t tiles = (s.TT + kTile - 1) / kTile;
    size_t o = 0;
    auto take = [&](size_t n) {
        char* p = ws ? ws + o : nullptr;
        o += up(n);
        return p;
    };
    char* head = take(8);
    char* first = take(tiles * 4);
    char* agg = take(tiles * s.C * 8);
    char* inc = take(tiles * s.C * 4);
    char* part = reduce ? take(tiles * s.C * 4) : nullptr;
    if (a) {
        a->ticket = reinterpret_cast<int*>(head);
        a->ok = a->ticket + 1;
        a->first = reinterpret_cast<int*>(first);
        a->agg = reinterpret_cast<float*>(agg);
        a->inc = reinterpret_cast<float*>(inc);
        a->unset = (int64_t)((up(tiles * s.C * 8) + up(tiles * s.C * 4)) / 16);      // (inc follows agg)
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

bool rows16(const Shape& s, std::initializer_list<const void*> acts) {
    for (const void* p : acts)
        if (reinterpret_cast<uintptr_t>(p) % 16) return false;
    for (int64_t st : {s.xs, s.gs, s.is, (int64_t)s.C})
        if (st * s.es % 16) return false;
    return true;
}

GatedArgs gated_args(const Shape& s, const void* x, const void* g, const void* i, const float* a_log, const int32_t* cu, const float* s0) {
    GatedArgs a;
    memset(&a, 0, sizeof(a));
    a.T = s.T; a.TT = s.TT; a.C = s.C; a.rows = s.rows; a.xs = s.xs; a.gs = s.gs; a.is = s.is;
    a.x = x; a.g = g; a.i = i; a.a_log = a_log; a.cu = cu; a.s0 = s0;
    return a;
}

// early: while the launch before it in the stream still runs (the kernels begin with a wait for that one's end).
cudaError_t gated_launch(void (*kernel)(GatedArgs), int ctas, int threads, size_t shared, bool early, const GatedArgs& a, cudaStream_t st) {
    if (shared) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    c.gridDim = dim3(ctas);
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = shared;
    c.stream = st;
    c.attrs = &at;
    c.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&c, kernel, a);
}

// The plan where the call has more than one tile or packed documents; from, to: the states that pass through.
cudaError_t gated_begin(GatedArgs& a, int vec, const float* from, float* to, cudaStream_t st) {
    a.tiles = (a.TT + kTile - 1) / kTile;
    a.cols = (a.C + 32 * vec - 1) / (32 * vec);
    a.planned = a.tiles > 1 || a.cu;
    if (!a.planned) return cudaSuccess;
    const int64_t work = a.unset / (4 * kThreads) + 1, most = a.cu ? (work > a.rows ? work : a.rows) : work;
    timing_pre(st, K_GATED_PLAN);
    gated_plan_kernel<<<(int)(most < 608 ? most : 608), kThreads, 0, st>>>(a, from, to);
    timing_post(st);
    return cudaGetLastError();
}

cudaError_t gated_forward(GatedArgs a, int dtype, bool pairs, cudaStream_t st) {
    cudaError_t e = gated_begin(a, pairs ? 2 : 1, a.s0, a.sT, st);
    if (e != cudaSuccess) return e;
    timing_pre(st, K_GATED_SCAN);
    const int ctas = a.tiles * a.cols, most = 152 * kFwdCtas;
    e = gated_launch(pairs ? gated_fwd_kernel<__nv_bfloat16, 2> : dtype == KDA_BF16 ? gated_fwd_kernel<__nv_bfloat16, 1> : gated_fwd_kernel<float, 1>,
                     ctas < most ? ctas : most, kAll, pairs ? sizeof(FwdShared<__nv_bfloat16, 2>) : dtype == KDA_BF16 ? sizeof(FwdShared<__nv_bfloat16, 1>) : sizeof(FwdShared<float, 1>),
                     a.planned, a, st);
    timing_post(st);
    return e;
}

struct Span {
    const void* p;
    size_t n;
};
// Whether a result lies over the rates or the offsets.
bool over_tables(const void* out, size_t n, const Shape& s, const float* a_log, const int32_t* cu) {
    return ranges_meet(out, n, a_log, (size_t)s.C * 4) || ranges_meet(out, n, cu, ((size_t)s.rows + 1) * 4);
}
size_t span_bytes(const Shape& s, int64_t stride) { return ((size_t)(s.TT - 1) * stride + s.C) * s.es; }

}  // namespace

}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_gated_scan_fwd_workspace_size(const kda_gated_dims* dims) {
    Shape s;
    if (!dims || gated_check(dims, false, &s) != KDA_OK) return 0;
    return gated_layout(s, false, nullptr, nullptr);
}

size_t kda_gated_scan_bwd_workspace_size(const kda_gated_dims* dims) {
    Shape s;
    if (!dims || gated_check(dims, false, &s) != KDA_OK) return 0;
    const size_t f = gated_layout(s, false, nullptr, nullptr), b = gated_layout(s, true, nullptr, nullptr);
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
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < gated_layout(s, false, nullptr, nullptr))
        return KDA_ERR_WORKSPACE;
    // a thread has read an element of x before it writes y's there, and a row's first tile its state before its last tile
    // writes one; the tiles otherwise run in no order
    const size_t nx = span_bytes(s, s.xs), ng = span_bytes(s, s.gs), ni = span_bytes(s, s.is), ny = (size_t)s.TT * s.C * s.es;
    const size_t ns = (size_t)s.rows * s.C * 4;
    const bool y_on_x = y == x && s.xs == s.C;
    if ((!y_on_x && ranges_meet(y, ny, x, nx)) || ranges_meet(y, ny, g_raw, ng) || ranges_meet(y, ny, i_raw, ni) ||
        ranges_meet(y, ny, initial_state, ns) || ranges_meet(y, ny, final_state, ns) || ranges_meet(y, ny, saved, rec) ||
        over_tables(y, ny, s, a_log, cu_seqlens))
        return KDA_ERR_INVALID_ARG;
    for (void* out : {static_cast<void*>(final_state), saved}) {
        const size_t n = out == saved ? rec : ns;
        if (ranges_meet(out, n, x, nx) || ranges_meet(out, n, g_raw, ng) || ranges_meet(out, n, i_raw, ni) ||
            (out != initial_state && ranges_meet(out, n, initial_state, ns)) || (out == saved && out == initial_state && out) ||
            over_tables(out, n, s, a_log, cu_seqlens))
            return KDA_ERR_INVALID_ARG;
    }
    if (ranges_meet(final_state, ns, saved, rec)) return KDA_ERR_INVALID_ARG;
    GatedArgs a = gated_args(s, x, g_raw, i_raw, a_log, cu_seqlens, initial_state);
    a.aligned = rows16(s, {x, g_raw, i_raw});
    a.y = y; a.sT = final_state; a.rec = static_cast<float*>(saved);
    gated_layout(s, false, static_cast<char*>(workspace), &a);
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
    const Span in[] = {{x, span_bytes(s, s.xs)}, {g_raw, span_bytes(s, s.gs)}, {i_raw, span_bytes(s, s.is)}, {dy, (size_t)s.TT * s.C * s.es},
                       {a_log, (size_t)s.C * 4}, {initial_state, ns}, {dfinal_state, ns}, {saved, rec}};
    const Span offsets = {cu_seqlens, ((size_t)s.rows + 1) * 4};
    const Span out[] = {{dx, nf}, {dg_raw, nf}, {di_raw, nf}, {da_log, (size_t)s.C * 4}, {dinitial_state, ns}};
    for (int k = 0; k < 5; ++k) {
        for (const Span& q : in)
            if (ranges_meet(out[k].p, out[k].n, q.p, q.n)) return KDA_ERR_INVALID_ARG;
        if (ranges_meet(out[k].p, out[k].n, offsets.p, offsets.n)) return KDA_ERR_INVALID_ARG;
        for (int j = 0; j < k; ++j)
            if (ranges_meet(out[k].p, out[k].n, out[j].p, out[j].n)) return KDA_ERR_INVALID_ARG;
    }
    GatedArgs a = gated_args(s, x, g_raw, i_raw, a_log, cu_seqlens, initial_state);
    st = status_ptr(&a.status);
    if (st != KDA_OK) return st;
    a.aligned = rows16(s, {x, g_raw, i_raw, dy});
    char* ws = static_cast<char*>(workspace);
    const bool pairs = pairs_ok(s, {x, g_raw, i_raw, dy}, {a_log, initial_state, dfinal_state, dx, dg_raw, di_raw, dinitial_state});
    a.rec = static_cast<float*>(const_cast<void*>(saved));
    if (!saved) {      // the states again: a forward that writes only its record
        a.rec = reinterpret_cast<float*>(ws);
        gated_layout(s, false, ws + up(rec), &a);
        if (gated_forward(a, s.dtype, pairs, stream) != cudaSuccess) return KDA_ERR_CUDA;
    }
    gated_layout(s, true, ws + up(rec), &a);
    a.dy = dy; a.dsT = dfinal_state; a.dx = dx; a.dg = dg_raw; a.di = di_raw; a.da_log = da_log; a.ds0 = dinitial_state;
    if (gated_begin(a, pairs ? 2 : 1, dfinal_state, dinitial_state, stream) != cudaSuccess) return KDA_ERR_CUDA;
    timing_pre(stream, K_GATED_BWD);
    const int ctas = a.tiles * a.cols, most = 152 * kBwdCtas;
    cudaError_t e = gated_launch(pairs ? gated_bwd_kernel<__nv_bfloat16, 2> : s.dtype == KDA_BF16 ? gated_bwd_kernel<__nv_bfloat16, 1> : gated_bwd_kernel<float, 1>,
                                 ctas < most ? ctas : most, kAll, pairs ? sizeof(BwdShared<__nv_bfloat16, 2>) : s.dtype == KDA_BF16 ? sizeof(BwdShared<__nv_bfloat16, 1>) : sizeof(BwdShared<float, 1>),
                                 a.planned, a, stream);
    timing_post(stream);
    if (e != cudaSuccess) return KDA_ERR_CUDA;
    timing_pre(stream, K_GATED_REDUCE);
    e = gated_launch(gated_reduce_kernel, (s.C + 31) / 32, kReduceWarps * 32, 0, true, a, stream);
    timing_post(stream);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_gated_step(const kda_gated_dims* dims, const void* x, const void* g_raw, const void* i_raw, const float* a_log,
                          const int32_t* slots, int num_slots, const float* state_in, float* state_out, void* y, cudaStream_t stream) {
    Shape s;
    if (!dims || dims->T != 1) return KDA_ERR_INVALID_ARG;
    kda_status st = gated_check(dims, false, &s);
    if (st != KDA_OK) return st;
    if (!x || !g_raw || !i_raw || !a_log || !y || !state_in || !state_out) return KDA_ERR_INVALID_ARG;
    if (num_slots < 1 || (!slots && num_slots < s.B)) return KDA_ERR_INVALID_ARG;
    // a thread has read its elements before it writes them
    const size_t ny = (size_t)s.B * s.C * s.es, np = (size_t)num_slots * s.C * 4;
    const Span in[] = {{x, span_bytes(s, s.xs)}, {g_raw, span_bytes(s, s.gs)}, {i_raw, span_bytes(s, s.is)}, {a_log, (size_t)s.C * 4},
                       {slots, (size_t)s.B * 4}, {state_in, np}};
    for (const Span& q : in)
        if ((ranges_meet(y, ny, q.p, q.n) && !(q.p == x && y == x && s.xs == s.C)) ||
            (ranges_meet(state_out, np, q.p, q.n) && !(q.p == state_in && state_out == state_in)))
            return KDA_ERR_INVALID_ARG;
    if (ranges_meet(y, ny, state_out, np)) return KDA_ERR_INVALID_ARG;
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
