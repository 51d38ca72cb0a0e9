// kda_ssm.cu -- selective state space scan: arguments, schedule and the fp32 token-by-token kernel.
//
//     S_t = exp(D_t a) S_{t-1} + D_t B_t x_t^T,   y_t = S_t^T C_t + d x_t,   D_t = softplus(dt_raw_t + dt_bias)
// The end state of a span of tokens is affine in its entering state with the scalar factor exp(sum D a),
// so rows are cut into segments: one pass forms each segment's end state from zero (all segments at
// once), a join walks each row's segments (fp32, elementwise), and a second pass forms the outputs from
// the entering states.  Rows of one segment, and calls with enough rows x heads to fill the GPU, take the
// output pass alone.
#include <math.h>
#include <string.h>

#include "kda.h"
#include "kda_sm100.cuh"
#include "kda_ssm.h"

namespace kda {

using namespace sm100;

kda_status ssm_check(const kda_ssm_dims* d, bool varlen, const void* x, const void* dt_raw, const void* b,
                     const void* c, const float* a_log, const float* dt_bias, SsmShape* s) {
    if (!d) return KDA_ERR_INVALID_ARG;
    if (d->B < 1 || d->T < 1 || d->H < 1 || d->G < 1 || d->H % d->G || d->N < 1 || d->P < 1) return KDA_ERR_INVALID_ARG;
    if (d->dtype != KDA_BF16 && d->dtype != KDA_FP32) return KDA_ERR_INVALID_ARG;
    if (!x || !dt_raw || !b || !c || !a_log || !dt_bias) return KDA_ERR_INVALID_ARG;
    const int64_t xw = (int64_t)d->H * d->P, bw = (int64_t)d->G * d->N;
    if ((d->x_stride && d->x_stride < xw) || (d->b_stride && d->b_stride < bw) || (d->c_stride && d->c_stride < bw) ||
        (d->dt_stride && d->dt_stride < d->H))
        return KDA_ERR_INVALID_ARG;
    if (varlen && (d->B != 1 || d->num_seqs < 1)) return KDA_ERR_INVALID_ARG;
    if (d->N > 256 || d->P > 256) return KDA_ERR_UNSUPPORTED;
    if (varlen && d->num_seqs > (1 << 24)) return KDA_ERR_UNSUPPORTED;
    const long long TT = (long long)d->B * d->T;
    if (TT > (1LL << 30) || xw > (1 << 30) || bw > (1 << 30)) return KDA_ERR_UNSUPPORTED;
    s->B = d->B; s->T = d->T; s->TT = (int)TT; s->H = d->H; s->G = d->G; s->N = d->N; s->P = d->P;
    s->dtype = d->dtype; s->rows = varlen ? d->num_seqs : d->B;
    s->xs = d->x_stride ? d->x_stride : xw;
    s->bs = d->b_stride ? d->b_stride : bw;
    s->cs = d->c_stride ? d->c_stride : bw;
    s->ds = d->dt_stride ? d->dt_stride : d->H;
    int64_t most = s->xs > s->bs ? s->xs : s->bs;
    if (s->cs > most) most = s->cs;
    if (s->ds > most) most = s->ds;
    if (most > (1LL << 40) / TT) return KDA_ERR_UNSUPPORTED;
    if ((long long)s->rows * d->H > (1LL << 30)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

namespace {

// ------------------------------------------------------------------ schedule

// A schedule's cost, in times that the output pass takes for q tokens of a segment.  A segment costs its tokens
// and `start`; the states-only pass `state` of the output pass again; the join and the launches `join`.  CTAs
// run in waves of equal segments, or (documents, of any lengths) as SMs fall free: then the last one may start
// when the others are done.
//   tensor cores: 3.8 us for 128 tokens; start two chunks, states 0.5 (109 and 218 us on a row of 65536
//   tokens, 32 heads), join and launches 15 us;
//   fp32: 3.3 us for 32 tokens; start 0.5, states 0.6, join and launches 6.6 us (3.5 units in place of 2: 128 tokens
//   uncut, 16.3 us and not 12.6).
constexpr int kSsmSms = 152;
struct Costs {
    int64_t units;       // CTAs per segment over all heads, counted in CTAs that have an SM to themselves
    int q;               // tokens of a unit of time, and what a segment's length is a multiple of
    double start, state, join;
};
double segment_cost(const Costs& k, double work, double longest, bool even, bool one_pass) {
    const double out = even ? work : work / kSsmSms + longest / 2 > longest ? work / kSsmSms + longest / 2 : longest;
    return one_pass ? out : (1 + k.state) * out + k.join;
}

struct Schedule {
    int L, per_row, nseg;
    bool single, plan;
    size_t off_seg, off_row, off_decay, off_states, total;
};

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

Schedule make_schedule(const SsmShape& s, bool varlen, const Costs& k) {
    const int64_t units = k.units, q = k.q;
    Schedule w;
    memset(&w, 0, sizeof(w));
    int64_t best = 0;                       // length of a segment in q; 0: rows are not cut
    if (!varlen) {
        const int64_t chunks = (s.T + q - 1) / q, ctas = s.rows * units;
        double least = segment_cost(k, (ctas + kSsmSms - 1) / kSsmSms * (chunks + k.start), 0, true, true);
        for (int64_t segs = 2; segs <= chunks && (segs - 1) * ctas < 4 * kSsmSms; ++segs) {
            const int64_t len = (chunks + segs - 1) / segs, n = (chunks + len - 1) / len;
            const double c = segment_cost(k, (n * ctas + kSsmSms - 1) / kSsmSms * (len + k.start), 0, true, false);
            if (n > 1 && c < least) {
                least = c;
                best = len;
            }
        }
    } else {
        // The lengths are on the device: take the longest of a random cut of the tokens, (1 + ln rows) / rows
        const double chunks = (double)s.TT / q, share = (1.0 + log((double)s.rows)) / s.rows;
        const double longest = chunks * (share < 1 ? share : 1) + k.start;
        double least = segment_cost(k, (chunks + (k.start + 0.5) * s.rows) * units, longest, false, true);
        for (int64_t len = 4; len < longest; len += len < 16 ? 4 : len / 4) {
            const double ctas = s.rows + chunks / len;
            const double c = segment_cost(k, (chunks + (k.start + 0.5) * ctas) * units, len + k.start, false, false);
            if (c < least) {
                least = c;
                best = len;
            }
        }
    }
    w.single = best == 0;
    const int64_t longest = varlen ? s.TT : s.T;
    w.L = (int)((w.single ? (longest + q - 1) / q : best) * q);
    w.per_row = varlen ? 0 : (s.T + w.L - 1) / w.L;
    w.nseg = varlen ? (w.single ? s.rows : s.rows + s.TT / w.L) : s.rows * w.per_row;
    size_t o = 0;
    w.plan = varlen && (!w.single || s.rows > kSsmOwnRows);
    if (varlen) {      // (wanted of the caller whether or not this schedule has a planner)
        w.off_seg = o; o = up256(o + sizeof(SsmSeg) * (size_t)w.nseg);
        w.off_row = o; o = up256(o + sizeof(int32_t) * ((size_t)s.rows + 1));
    }
    if (!w.single) {
        w.off_decay = o; o = up256(o + sizeof(float) * (size_t)w.nseg * s.H);
        w.off_states = o; o = up256(o + sizeof(float) * (size_t)w.nseg * s.H * s.N * s.P);
    }
    w.total = o;
    return w;
}

// Whether the results lie apart from what other CTAs still read.  In place are right: y over x of the same layout (a
// CTA reads a token's columns before it writes them, and no other CTA uses them but as zeros), the end states over
// the entering ones (a thread writes the elements that it read, or the join has read them all before).
bool results_apart(const SsmShape& s, const void* x, const void* dt, const void* b, const void* c, const void* S0,
                   const void* y, const void* ST) {
    const size_t es = s.dtype == KDA_BF16 ? 2 : 4, state = (size_t)s.rows * s.H * s.N * s.P * 4;
    auto span = [&](int64_t stride, int64_t width) { return ((size_t)(s.TT - 1) * stride + width) * es; };
    const int64_t xw = (int64_t)s.H * s.P, bw = (int64_t)s.G * s.N;
    const size_t nx = span(s.xs, xw), nb = span(s.bs, bw), nc = span(s.cs, bw), nd = span(s.ds, s.H), ny = span(xw, xw);
    const bool over_x = y == x && s.xs == xw, over_S0 = ST == S0;
    if (ranges_meet(y, ny, b, nb) || ranges_meet(y, ny, c, nc) || ranges_meet(y, ny, dt, nd) || ranges_meet(y, ny, S0, state) ||
        ranges_meet(y, ny, ST, state) || (!over_x && ranges_meet(y, ny, x, nx)))
        return false;
    return !ranges_meet(ST, state, x, nx) && !ranges_meet(ST, state, b, nb) && !ranges_meet(ST, state, c, nc) &&
           !ranges_meet(ST, state, dt, nd) && (over_S0 || !ranges_meet(ST, state, S0, state));
}

// Two CTAs of the fp32 kernel share an SM, each 64 columns of P.
int simt_parts(int P) { return (P + 63) / 64; }
Costs simt_costs(const SsmShape& s) { return {((int64_t)s.H * simt_parts(s.P) + 1) / 2, 32, 0.5, 0.6, 2.0}; }
Costs tc_costs(const SsmShape& s) { return {ssm_tc_units(s.H, s.G, s.P), 128, 2.0, 0.5, 4.0}; }

// Segments of every row in order: ceil(len / L) of them, one empty segment for an empty row (its state
// passes through).  Offsets that break the contract are recorded and give every row one empty segment.
__global__ void __launch_bounds__(1024) ssm_plan_kernel(SsmArgs a, SsmSeg* seg, int32_t* row_seg) {
    __shared__ int part[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    bool bad = tid == 0 && (a.cu[0] != 0 || a.cu[a.rows] != a.TT);
    for (int n = tid; n < a.rows; n += 1024) bad |= a.cu[n + 1] < a.cu[n];
    bad = __syncthreads_or(bad);
    if (bad && tid == 0) record_error(a.status, KDA_ERR_INVALID_ARG);
    int carry = 0;
    for (int n0 = 0; n0 < a.rows; n0 += 1024) {
        const int n = n0 + tid;
        int b0 = 0, len = 0, cnt = 0;
        if (n < a.rows) {
            if (!bad) {
                b0 = a.cu[n];
                len = a.cu[n + 1] - b0;
            }
            cnt = len > 0 ? (len - 1) / a.L + 1 : 1;
        }
        int inc = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        __syncthreads();
        if (lane == 31) part[warp] = inc;
        __syncthreads();
        if (warp == 0) {
            int v = part[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            part[lane] = v;
        }
        __syncthreads();
        const int first = carry + inc - cnt + (warp ? part[warp - 1] : 0);
        carry += part[31];
        if (n < a.rows) {
            row_seg[n] = first;
            for (int k = 0; k < cnt; ++k) {
                SsmSeg s;
                s.n = n;
                s.k = k;
                s.t0 = b0 + k * a.L;
                s.t1 = (int)min((long long)b0 + len, (long long)s.t0 + a.L);
                if (first + k < a.nseg) seg[first + k] = s;
            }
        }
    }
    if (tid == 0) row_seg[a.rows] = carry;
    for (int i = carry + tid; i < a.nseg; i += 1024) {
        SsmSeg s;
        s.n = -1;
        s.t0 = s.t1 = s.k = 0;
        seg[i] = s;
    }
}

// Entering states of a row's segments: S <- decay_k S + loc_k, in place of loc_k.  Elementwise over the
// state, bound by memory: a thread walks VEC elements along the row's segments, kJoinAhead of them in flight.
constexpr int kJoinAhead = 16;
template <int VEC>
__global__ void __launch_bounds__(128) ssm_join_kernel(SsmArgs a) {
    const int np = a.N * a.P;
    const int e = (blockIdx.y * 128 + threadIdx.x) * VEC;
    const int n = blockIdx.x / a.H, h = blockIdx.x - n * a.H;
    if (e >= np) return;
    int first;
    const int segs = ssm_row_segments(a, n, &first);
    float S[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) S[v] = a.S0 ? a.S0[((size_t)n * a.H + h) * np + e + v] : 0.f;
    const size_t step = (size_t)a.H * np;
    float* p = a.states + ((size_t)first * a.H + h) * np + e;
    // the last segment's end state comes from the output pass
    for (int k0 = 0; k0 < segs; k0 += kJoinAhead, p += kJoinAhead * step) {
        float loc[kJoinAhead][VEC], d[kJoinAhead];
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k) {
            const bool in = k0 + k + 1 < segs;
            d[k] = in ? a.decay[(size_t)(first + k0 + k) * a.H + h] : 0.f;
            if constexpr (VEC == 4) {
                const float4 f = in ? *reinterpret_cast<const float4*>(p + k * step) : make_float4(0.f, 0.f, 0.f, 0.f);
                loc[k][0] = f.x; loc[k][1] = f.y; loc[k][2] = f.z; loc[k][3] = f.w;
            } else {
                loc[k][0] = in ? p[k * step] : 0.f;
            }
        }
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k) {
            if (k0 + k >= segs) break;
            if constexpr (VEC == 4) *reinterpret_cast<float4*>(p + k * step) = make_float4(S[0], S[1], S[2], S[3]);
            else p[k * step] = S[0];
#pragma unroll
            for (int v = 0; v < VEC; ++v) S[v] = fmaf(d[k], S[v], loc[k][v]);
        }
    }
}

// ------------------------------------------------------------------ fp32 kernel
//
// A CTA takes one (segment, head, 64 columns of P); a warp eight columns, eight lanes for two of them, a lane
// N / 8 state values of each in registers (groups of four n, eight lanes apart, so that the 16-byte reads of B and
// C from shared memory are free of conflicts).  Per token and state value: one multiply and two fused
// multiply-adds, two columns to an instruction; the eight lanes' partial outputs of eight tokens are summed
// together (seven shuffles for eight tokens and a column).  Bound by the shared memory's reads of B and C: a warp's
// 16-byte read takes four cycles although its lanes want 128 bytes in all.  So a lane has two columns, not one: 4096
// tokens x 32 heads of 128 x 64 take 266 us, with one column 500 us.  Few CTAs are bound by latency, some 150
// cycles a token: 2 x 1021 tokens x 6 heads of 48 x 40 take 25 us, 37 us with one column and the element type asked
// at every load.
constexpr int kSimtCols = 64;
constexpr int simt_tokens(int NJ) { return NJ <= 4 ? 32 : 16; }      // staged in shared memory at once

template <typename E> __device__ __forceinline__ float as_f32(E v);
template <> __device__ __forceinline__ float as_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float as_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <int NJ, bool OUT, typename E>
__global__ void __launch_bounds__(256, NJ <= 4 ? 2 : 1) ssm_simt_kernel(SsmArgs a) {
    constexpr int NP = 32 * NJ, TOK = simt_tokens(NJ);
    __shared__ __align__(16) float sb[TOK][NP], sc[OUT ? TOK : 1][NP];
    __shared__ __align__(8) float2 sx[TOK][kSimtCols / 2];      // y takes x's place
    __shared__ __align__(8) float2 sad[TOK];                    // a token's decay and step
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slice = lane & 7, pp = warp * 4 + (lane >> 3);     // pair of columns
    const int h = blockIdx.y, p0 = blockIdx.z * kSimtCols, p = p0 + 2 * pp;
    __shared__ SsmSeg found;
    const SsmSeg sg = ssm_segment(a, blockIdx.x, &found);
    if (sg.n < 0) return;
    if (!OUT) {   // the last segment's end state comes from the output pass
        int first;
        const int segs = ssm_row_segments(a, sg.n, &first);
        if ((int)blockIdx.x == first + segs - 1) return;
    }
    const bool in0 = p < a.P, in1 = p + 1 < a.P, works = p0 + 8 * warp < a.P;      // (the warp has columns)
    const int g = h / (a.H / a.G);
    const float ea = ssm_rate(a.a_log[h]), bias = a.dt_bias[h];
    const float dsk = OUT && a.d_skip ? a.d_skip[h] : 0.f;
    float2 S[NJ][4];
    const float* from = OUT ? ssm_entering(a, sg, blockIdx.x, h) : nullptr;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int n = (j * 8 + slice) * 4 + e;
            const bool in = from && n < a.N;
            S[j][e] = make_float2(in && in0 ? from[(size_t)n * a.P + p] : 0.f, in && in1 ? from[(size_t)n * a.P + p + 1] : 0.f);
        }
    float lsum = 0.f;
    // a block of tokens is loaded into registers while the one before it is worked on; a thread has one column of b
    // and c (NP divides 256 or is it), and one of x
    constexpr int TB = 256 / NP, PB = TOK / TB, TX = 256 / kSimtCols, PX = TOK / TX;
    const int bn = tid % NP, bt = tid / NP, xc = tid % kSimtCols, xt = tid / kSimtCols;
    const bool bin = bn < a.N, xin = p0 + xc < a.P;
    const E* pb = static_cast<const E*>(a.b) + (size_t)(sg.t0 + bt) * a.bs + (size_t)g * a.N + bn;
    const E* pcc = static_cast<const E*>(a.c) + (size_t)(sg.t0 + bt) * a.cs + (size_t)g * a.N + bn;
    const E* px = static_cast<const E*>(a.x) + (size_t)(sg.t0 + xt) * a.xs + (size_t)h * a.P + p0 + xc;
    const E* pd = static_cast<const E*>(a.dt) + (size_t)(sg.t0 + tid) * a.ds + h;
    E* py = static_cast<E*>(a.y) + ((size_t)(sg.t0 + xt) * a.H + h) * a.P + p0 + xc;
    E rb[PB], rc[OUT ? PB : 1], rx[PX], rdt = E(0.f);
    auto fetch = [&](int nt) {
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            const bool in = bin && bt + i * TB < nt;
            rb[i] = in ? pb[i * TB * a.bs] : E(0.f);
            if (OUT) rc[i] = in ? pcc[i * TB * a.cs] : E(0.f);
        }
#pragma unroll
        for (int i = 0; i < PX; ++i) rx[i] = xin && xt + i * TX < nt ? px[i * TX * a.xs] : E(0.f);
        if (tid < nt) rdt = *pd;
        pb += TOK * a.bs;
        pcc += TOK * a.cs;
        px += TOK * a.xs;
        pd += TOK * a.ds;
    };
    if (sg.t0 < sg.t1) fetch(min(TOK, sg.t1 - sg.t0));
    for (int t0 = sg.t0; t0 < sg.t1; t0 += TOK) {
        const int nt = min(TOK, sg.t1 - t0);
        float* fx = reinterpret_cast<float*>(sx);
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            sb[bt + i * TB][bn] = as_f32<E>(rb[i]);
            if (OUT) sc[bt + i * TB][bn] = as_f32<E>(rc[i]);
        }
#pragma unroll
        for (int i = 0; i < PX; ++i) fx[(xt + i * TX) * kSimtCols + xc] = as_f32<E>(rx[i]);
        if (tid < TOK) {
            const float dt = tid < nt ? softplusf(as_f32<E>(rdt) + bias) : 0.f;
            sad[tid] = make_float2(expf(-ea * dt), dt);   // a token past the end keeps the state
            if (!OUT) lsum += dt;
        }
        __syncthreads();
        if (t0 + TOK < sg.t1) fetch(min(TOK, sg.t1 - t0 - TOK));
#pragma unroll 1
        for (int t8 = 0; t8 < nt && works; t8 += 8) {
            float2 y[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int t = t8 + u;
                const float2 ad = sad[t], al = dup(ad.x), ux = mul2(dup(ad.y), sx[t][pp]);
                float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const float4 b4 = *reinterpret_cast<const float4*>(&sb[t][(j * 8 + slice) * 4]);
                    S[j][0] = fma2(al, S[j][0], mul2(ux, dup(b4.x)));
                    S[j][1] = fma2(al, S[j][1], mul2(ux, dup(b4.y)));
                    S[j][2] = fma2(al, S[j][2], mul2(ux, dup(b4.z)));
                    S[j][3] = fma2(al, S[j][3], mul2(ux, dup(b4.w)));
                    if (OUT) {
                        const float4 c4 = *reinterpret_cast<const float4*>(&sc[t][(j * 8 + slice) * 4]);
                        acc = fma2(S[j][0], dup(c4.x), acc);
                        acc = fma2(S[j][1], dup(c4.y), acc);
                        acc = fma2(S[j][2], dup(c4.z), acc);
                        acc = fma2(S[j][3], dup(c4.w), acc);
                    }
                }
                y[u] = acc;
            }
            if (OUT) {   // lane `slice` ends with the sums of token t8 + slice
#pragma unroll
                for (int w = 4; w >= 1; w >>= 1) {
                    const bool up = slice & w;
#pragma unroll
                    for (int i = 0; i < w; ++i) {
                        const float2 send = up ? y[i] : y[i + w], keep = up ? y[i + w] : y[i];
                        y[i] = make_float2(keep.x + __shfl_xor_sync(0xffffffffu, send.x, w), keep.y + __shfl_xor_sync(0xffffffffu, send.y, w));
                    }
                }
                __syncwarp();      // the warp has read its columns' x
                sx[t8 + slice][pp] = fma2(dup(dsk), sx[t8 + slice][pp], y[0]);
            }
        }
        __syncthreads();
        if (OUT) {
#pragma unroll
            for (int i = 0; i < PX; ++i)
                if (xin && xt + i * TX < nt) py[(size_t)i * TX * a.H * a.P] = E(fx[(xt + i * TX) * kSimtCols + xc]);
            py += (size_t)TOK * a.H * a.P;
            __syncthreads();      // the next block's x goes there
        }
    }
    float* to = OUT ? ssm_leaving(a, sg, blockIdx.x, h) : a.states + ((size_t)blockIdx.x * a.H + h) * a.N * a.P;
    if (to)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int n = (j * 8 + slice) * 4 + e;
                if (n < a.N && in0) to[(size_t)n * a.P + p] = S[j][e].x;
                if (n < a.N && in1) to[(size_t)n * a.P + p + 1] = S[j][e].y;
            }
    if (!OUT && blockIdx.z == 0 && warp == 0) {
        lsum = warp_sum(lsum);
        if (lane == 0) a.decay[(size_t)blockIdx.x * a.H + h] = expf(-ea * lsum);
    }
}

}  // namespace

cudaError_t launch_ssm_simt(const SsmArgs& a, bool out, cudaStream_t st) {
    const dim3 grid(a.nseg, a.H, (a.P + kSimtCols - 1) / kSimtCols);
    timing_pre(st, out ? K_SSM_OUT : K_SSM_STATE);
#define KDA_SSM_SIMT(NJ)                                                                         \
    do {                                                                                         \
        if (a.dtype == KDA_BF16) {                                                               \
            if (out) ssm_simt_kernel<NJ, true, __nv_bfloat16><<<grid, 256, 0, st>>>(a);          \
            else ssm_simt_kernel<NJ, false, __nv_bfloat16><<<grid, 256, 0, st>>>(a);             \
        } else {                                                                                 \
            if (out) ssm_simt_kernel<NJ, true, float><<<grid, 256, 0, st>>>(a);                  \
            else ssm_simt_kernel<NJ, false, float><<<grid, 256, 0, st>>>(a);                     \
        }                                                                                        \
    } while (0)
    if (a.N <= 32) KDA_SSM_SIMT(1);
    else if (a.N <= 64) KDA_SSM_SIMT(2);
    else if (a.N <= 128) KDA_SSM_SIMT(4);
    else KDA_SSM_SIMT(8);
#undef KDA_SSM_SIMT
    timing_post(st);
    return cudaGetLastError();
}

}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_ssm_fwd_workspace_size(const kda_ssm_dims* dims) {
    SsmShape s;
    const int some = 0;   // the checks want pointers
    const float* f = reinterpret_cast<const float*>(&some);
    if (!dims) return 0;
    // with num_seqs the larger of the packed and the row layout
    size_t most = 0;
    bool valid = false;
    for (int varlen = 0; varlen < 2; ++varlen) {
        if (varlen && !(dims->num_seqs > 0 && dims->B == 1)) continue;
        if (ssm_check(dims, varlen != 0, f, f, f, f, f, f, &s) != KDA_OK) continue;
        valid = true;
        // which kernels run also depends on the pointers' alignment
        for (const Costs& k : {simt_costs(s), tc_costs(s)}) {
            const size_t t = make_schedule(s, varlen != 0, k).total;
            if (t > most) most = t;
        }
    }
    return valid ? (most ? most : 256) : 0;
}

kda_status kda_ssm_fwd(const kda_ssm_dims* dims, const void* x, const void* dt_raw, const void* b, const void* c,
                       const float* a_log, const float* dt_bias, const float* d_skip, const int32_t* cu_seqlens,
                       const int32_t* cu_seqlens_host, const float* initial_state, void* y, float* final_state,
                       void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    SsmShape s;
    kda_status st = ssm_check(dims, cu_seqlens != nullptr, x, dt_raw, b, c, a_log, dt_bias, &s);
    if (st != KDA_OK) return st;
    if (!y) return KDA_ERR_INVALID_ARG;
    st = check_offsets_host(s.rows, s.TT, cu_seqlens, cu_seqlens_host);
    if (st != KDA_OK) return st;
    // A few tokens to a row.  The tensor-core kernel takes 10.6 to 13 us for a chunk, however few its tokens are; one
    // wave of the fp32 kernel's CTAs 4.5 to 12.8 us up to 16 tokens, and with N up to 64 and an SM to each CTA 8.7 us
    // for 37 tokens, 11.2 us for 64 (N 128, 32 heads: 13.4 and 17.8 us)
    const int64_t ctas = (int64_t)s.rows * s.H * simt_parts(s.P);
    const bool few = (s.TT <= 16 * (int64_t)s.rows && ctas <= 2 * kSsmSms) ||
                     (s.TT <= 48 * (int64_t)s.rows && ctas <= kSsmSms && s.N <= 64);
    const bool tc = !few && ssm_tc_ok(s, x, b, c, y);
    const Schedule w = make_schedule(s, cu_seqlens != nullptr, tc ? tc_costs(s) : simt_costs(s));
    if (workspace_bytes < w.total || (w.total && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256)))
        return KDA_ERR_WORKSPACE;
    if (w.nseg > (1 << 30) / s.H || s.H > 65535) return KDA_ERR_UNSUPPORTED;
    if (!results_apart(s, x, dt_raw, b, c, initial_state, y, final_state)) return KDA_ERR_INVALID_ARG;
    char* ws = static_cast<char*>(workspace);
    SsmArgs a;
    memset(&a, 0, sizeof(a));
    a.T = s.T; a.TT = s.TT; a.H = s.H; a.G = s.G; a.N = s.N; a.P = s.P; a.dtype = s.dtype; a.rows = s.rows;
    a.xs = s.xs; a.bs = s.bs; a.cs = s.cs; a.ds = s.ds;
    a.x = x; a.dt = dt_raw; a.b = b; a.c = c; a.a_log = a_log; a.dt_bias = dt_bias; a.d_skip = d_skip;
    a.S0 = initial_state; a.cu = cu_seqlens; a.y = y; a.ST = final_state;
    a.L = w.L; a.per_row = w.per_row; a.nseg = w.nseg; a.single = w.single;
    st = status_ptr(&a.status);
    if (st != KDA_OK) return st;
    if (w.plan) {
        SsmSeg* seg = reinterpret_cast<SsmSeg*>(ws + w.off_seg);
        int32_t* row = reinterpret_cast<int32_t*>(ws + w.off_row);
        a.seg = seg;
        a.row_seg = row;
        timing_pre(stream, K_SSM_PLAN);
        ssm_plan_kernel<<<1, 1024, 0, stream>>>(a, seg, row);
        timing_post(stream);
        if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
    }
    if (!w.single) {
        a.decay = reinterpret_cast<float*>(ws + w.off_decay);
        a.states = reinterpret_cast<float*>(ws + w.off_states);
        if ((tc ? launch_ssm_tc(a, false, stream) : launch_ssm_simt(a, false, stream)) != cudaSuccess) return KDA_ERR_CUDA;
        timing_pre(stream, K_SSM_JOIN);
        const int np = s.N * s.P;
        if (np % 4 == 0) ssm_join_kernel<4><<<dim3(s.rows * s.H, (np + 511) / 512), 128, 0, stream>>>(a);
        else ssm_join_kernel<1><<<dim3(s.rows * s.H, (np + 127) / 128), 128, 0, stream>>>(a);
        timing_post(stream);
        if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
    }
    return (tc ? launch_ssm_tc(a, true, stream) : launch_ssm_simt(a, true, stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
