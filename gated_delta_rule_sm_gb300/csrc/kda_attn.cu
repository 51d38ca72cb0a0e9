// kda_attn.cu -- keys and values into the pages of a cache, and attention over them: the entries, the plan of the
// work, the join of what several CTAs share, and the fp32 kernel.
#include <math.h>
#include <string.h>

#include <type_traits>

#include "kda.h"
#include "kda_attn.h"
#include "kda_common.cuh"
#include "kda_internal.h"
#include "kda_sm100.cuh"

namespace kda {

using namespace sm100;

namespace {

// ------------------------------------------------------------------ append

// A warp takes a token, its lanes the 16-byte pieces (elements where those are not aligned) of its keys and values.  Bound by
// latency: the CTA meets at the offsets' check (the first of its stalls), and the address of a token comes from small loads one after the
// other (its row, the row's length, the page), while the loads of its data are under way.  Measured: 8192 tokens, 8 heads of 128
// in bf16 (67 MB), 16 us with the launch, 128 single tokens 4.1.  Eight pieces of a lane at once, which a token of 2 KB does not
// have, cost registers and so 2 us; the check before the loads 1; warps of two tokens saved nothing, of four cost 2.
constexpr int kAppendWarps = 8;
struct AppendArgs {
    AttnArgs a;
    const void *k, *v;
    int64_t ks, vs;      // elements between tokens
    void* pool;
};

// The row of packed token t: the last one that begins at or before it, by 32 offsets at a time.
__device__ __forceinline__ int row_of_token(const int32_t* cu, int rows, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = rows;                      // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32, at = lo + lane * step;
        const unsigned hit = __ballot_sync(0xffffffffu, lane * step < n && cu[at] <= t);
        const int k = 31 - __clz(hit | 1u);
        n = min(step, n - k * step);
        lo += k * step;
    }
    return lo;
}

template <typename W>
__global__ void __launch_bounds__(kAppendWarps * 32) append_kernel(const __grid_constant__ AppendArgs p) {
    const AttnArgs& a = p.a;
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    const bool live = t < a.tokens;
    const int es = a.dtype == KDA_BF16 ? 2 : 4, per = a.D * es / (int)sizeof(W), all = live ? a.Hkv * per : 0;      // pieces of a head, of a token
    const W *k = reinterpret_cast<const W*>(static_cast<const char*>(p.k) + t * p.ks * es),
            *v = reinterpret_cast<const W*>(static_cast<const char*>(p.v) + t * p.vs * es);
    constexpr int AHEAD = 4;
    W rk[AHEAD], rv[AHEAD];
    auto load = [&](int i0) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int at = i0 + i * 32 + lane;
            if (at < all) {
                rk[i] = k[at];
                rv[i] = v[at];
            }
        }
    };
    load(0);
    if (a.cu) {
        bool bad = threadIdx.x == 0 && (a.cu[0] != 0 || a.cu[a.rows] != a.tokens);
        for (int n = threadIdx.x; n < a.rows; n += kAppendWarps * 32) bad |= a.cu[n + 1] < a.cu[n];
        if (__syncthreads_or(bad)) {
            if (blockIdx.x == 0 && threadIdx.x == 0) record_error(a.status, KDA_ERR_INVALID_ARG);
            return;
        }
    }
    if (!live) return;
    const int r = a.cu ? row_of_token(a.cu, a.rows, t) : t / a.per_row;
    const AttnRow w = attn_row(a, r, lane == 0);
    const int pos = w.len - w.n + (t - w.first);
    if (w.seq < 0 || pos < 0) return;
    const int page = a.table[(size_t)w.seq * a.max_pages + pos / a.pt];
    if (page < 0 || page >= a.pages) {
        if (lane == 0) record_error(a.status, KDA_ERR_INVALID_ARG);
        return;
    }
    const size_t head = (size_t)a.pt * per;                        // pieces of a head's keys in a page
    W* to = static_cast<W*>(p.pool) + (size_t)page * 2 * a.Hkv * head + (size_t)(pos % a.pt) * per;
    for (int i0 = 0; i0 < all; i0 += AHEAD * 32) {
        if (i0) load(i0);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int at = i0 + i * 32 + lane;
            if (at < all) {
                const int h = at / per;
                W* q = to + h * head + (at - h * per);
                q[0] = rk[i];
                q[a.Hkv * head] = rv[i];
            }
        }
    }
}

// ------------------------------------------------------------------ plan

// Units of every row, then the cost of every unit, each as a running sum, by one CTA: 4 us, and the attention is launched meanwhile.
constexpr int kPlanThreads = 1024;
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* tmp, int64_t* total) {     // what comes before this thread
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += up;
    }
    __syncthreads();
    if (lane == 31) tmp[warp] = s;
    __syncthreads();
    if (warp == 0) {
        int64_t w = tmp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += up;
        }
        tmp[lane] = w;
    }
    __syncthreads();
    *total = tmp[31];
    return s - x + (warp ? tmp[warp - 1] : 0);
}

__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const __grid_constant__ AttnArgs a) {
    __shared__ int64_t tmp[32];
    const int tid = threadIdx.x;
    cudaTriggerProgrammaticLaunchCompletion();       // the attention may be launched; it waits for this kernel's end
    bool bad = false;
    if (a.cu) {
        for (int n = tid; n < a.rows; n += kPlanThreads) bad |= a.cu[n + 1] < a.cu[n];
        if (tid == 0) bad |= a.cu[0] != 0 || a.cu[a.rows] != a.tokens;
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) {
            record_error(a.status, KDA_ERR_INVALID_ARG);
            *a.units = -1;
        }
        return;
    }
    int64_t units = 0, total;
    for (int r0 = 0; r0 < a.rows; r0 += kPlanThreads) {
        const int r = r0 + tid;
        const int64_t blocks = r < a.rows ? attn_blocks(a, a.cu ? a.cu[r + 1] - a.cu[r] : a.per_row) : 0;
        const int64_t at = units + block_scan(blocks, tmp, &total);
        // (a row has few blocks next to the work that each is)
        for (int b = 0; b < blocks; ++b) {
            a.unit_row[at + b] = r;
            a.unit_row[a.units_most + at + b] = b;
        }
        units += total;
    }
    __syncthreads();
    int64_t tiles = 0;
    for (int u0 = 0; u0 < units; u0 += kPlanThreads) {
        const int u = u0 + tid;
        int64_t n = 0;
        if (u < units) {
            const int b = a.unit_row[a.units_most + u];
            n = attn_span(a, attn_row(a, a.unit_row[u], b == 0), b).tiles + a.extra;
        }
        const int64_t at = tiles + block_scan(n, tmp, &total);
        if (u < units) a.start[u] = at;
        tiles += total;
    }
    if (tid == 0) {
        a.start[units] = tiles;
        *a.units = (int)units;
    }
}

// ------------------------------------------------------------------ join

// A CTA takes some rows of one item (a unit for one key head) that several CTAs share.  With few parts a warp takes a
// row and reads them and their maxima at once; with many (a few rows over a long cache) the warps split the parts of a row,
// four of each warp's on the way at once, since it is their latency that counts (61 -> 43 us for one row over 32768 tokens).
// The attention's CTAs say which items they share, and the join is launched while they run: 3 us after a step, 14 us after
// a chunk of 8192 tokens.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32, kJoinFew = 4;
struct JoinSum {
    float o[8], sum;
};
// Parts c0 + at, c0 + at + step, ... of row i, weighted from `base`; ALL: these are all there are, four at most, and base is their
// largest maximum, found here.
template <bool ALL>
__device__ __forceinline__ JoinSum join_parts(const AttnArgs& a, int c0, int c1, int at, int step, int i, float& base) {
    const int lane = threadIdx.x & 31;
    const size_t size = attn_part_floats(a), top = (size_t)a.block * a.D + i;
    JoinSum s;
    s.sum = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s.o[k] = 0.f;
    constexpr int AHEAD = kJoinFew;
    for (int c = c0 + at; c <= c1; c += AHEAD * step) {
        float f[AHEAD], add[AHEAD], v[AHEAD][8];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const int now = c + j * step;
            const float* p = a.part + (size_t)(2 * now + (now == c0)) * size;
            f[j] = now <= c1 ? p[top] : -INFINITY;
            add[j] = now <= c1 ? p[top + a.block] : 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) v[j][k] = now <= c1 && k * 32 + lane < a.D ? p[(size_t)i * a.D + k * 32 + lane] : 0.f;
        }
        if constexpr (ALL) {
            base = -INFINITY;
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) base = fmaxf(base, f[j]);
            if (base == -INFINITY) base = 0.f;
        }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const float w = f[j] == -INFINITY ? 0.f : exp2f(f[j] - base);
            s.sum = fmaf(w, add[j], s.sum);
#pragma unroll
            for (int k = 0; k < 8; ++k) s.o[k] = fmaf(w, v[j][k], s.o[k]);
        }
    }
    return s;
}
__device__ __forceinline__ void join_write(const AttnArgs& a, size_t at, const JoinSum& s, float base) {
    const int lane = threadIdx.x & 31;
    const float inv = s.sum > 0.f ? 1.f / s.sum : s.sum == 0.f ? 0.f : s.sum;      // (NaN stays)
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k * 32 + lane < a.D) store_act(a.out, at * a.D + k * 32 + lane, s.o[k] * inv, a.dtype);
    if (a.lse && lane == 0) a.lse[at] = s.sum == 0.f ? -INFINITY : (base + log2f(s.sum)) * 0.6931471805599453f;
}
// blockIdx.x: the CTA of the attention that began the item.
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ AttnArgs a, int rows_each) {
    __shared__ float so[kJoinWarps][256], ss[kJoinWarps];
    cudaGridDependencySynchronize();
    const AttnShared it = a.shared[blockIdx.x];
    const int i0 = blockIdx.y * rows_each, i1 = min(it.rows, i0 + rows_each), c0 = blockIdx.x, c1 = it.last;
    if (i0 >= i1) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool few = rows_each > 1 || c1 - c0 < kJoinFew;      // a warp to a row
    const bool all = c1 - c0 < kJoinFew;
    for (int i = few ? i0 + warp : i0; i < i1; i += few ? kJoinWarps : 1) {
        const uint32_t row = (uint32_t)it.first_row + i, token = row / (uint32_t)a.G;
        const size_t at = (size_t)(it.token + (int)token) * a.Hq + it.head + (row - token * a.G);
        if (all) {
            float base;
            const JoinSum s = join_parts<true>(a, c0, c1, 0, 1, i, base);
            join_write(a, at, s, base);
            continue;
        }
        float top = -INFINITY;
        for (int c = c0 + lane; c <= c1; c += 32)
            top = fmaxf(top, a.part[(size_t)(2 * c + (c == c0)) * attn_part_floats(a) + (size_t)a.block * a.D + i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float base = top == -INFINITY ? 0.f : top;
        JoinSum s = join_parts<false>(a, c0, c1, few ? 0 : warp, few ? 1 : kJoinWarps, i, base);
        if (few) {
            join_write(a, at, s, base);
            continue;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) so[warp][k * 32 + lane] = s.o[k];
        if (lane == 0) ss[warp] = s.sum;
        __syncthreads();
        if (warp == 0) {
            for (int v = 1; v < kJoinWarps; ++v) {
                s.sum += ss[v];
#pragma unroll
                for (int k = 0; k < 8; ++k) s.o[k] += so[v][k * 32 + lane];
            }
            join_write(a, at, s, base);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ fp32

// 64 packed rows against 64 keys at a time, 256 threads of 4 x 4 scores each; Q, K and the weights lie transposed in
// shared memory, so that a step of a product is two 16-byte reads for 16 multiplications.  A thread keeps 4 rows of D / 16
// columns of the output.  Bound by fp32 arithmetic with full blocks; a block of few rows leaves most warps idle.  Measured:
// 301 tokens of three requests over 700, 6 heads of 40, 28.6 us with the plan and the join, mostly latency: the cut gives a CTA a few tiles.
constexpr int kSimtRows = 64, kSimtKeys = 64, kSimtThreads = 256, kSimtPad = 68;

template <typename E> __device__ __forceinline__ float4 load4(const char* p, int d, int D, bool vec) {
    const E* e = reinterpret_cast<const E*>(p) + d;
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (vec) {
        if constexpr (sizeof(E) == 4) f = *reinterpret_cast<const float4*>(e);
        else {
            const uint2 u = *reinterpret_cast<const uint2*>(e);
            f = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                            __uint_as_float(u.y & 0xffff0000u));
        }
    } else {
        if (d < D) f.x = (float)e[0];
        if (d + 1 < D) f.y = (float)e[1];
        if (d + 2 < D) f.z = (float)e[2];
        if (d + 3 < D) f.w = (float)e[3];
    }
    return f;
}

// DC: columns of the output a thread keeps, in groups of four: D <= 64 DC.
template <typename E, int DC>
__global__ void __launch_bounds__(kSimtThreads, DC > 2 ? 1 : 2) attn_simt_kernel(const __grid_constant__ AttnArgs a) {
    extern __shared__ __align__(16) float sh[];
    const int D4 = (a.D + 3) / 4 * 4;
    float* sq = sh;                                  // [D4][kSimtPad] q by channel
    float* sk = sq + (size_t)D4 * kSimtPad;          // [D4][kSimtPad] keys by channel
    float* sv = sk + (size_t)D4 * kSimtPad;          // [kSimtKeys][64 DC] values
    float* sp = sv + kSimtKeys * 64 * DC;            // [kSimtKeys][kSimtPad] weights by key
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, warp = tid >> 5;
    __shared__ int64_t own[kAttnDirectRows + 1];
    const AttnUnits units = attn_units(a, own);
    if (units.units <= 0) return;
    const AttnCut cut(a, units.cost(a));
    const int cta = blockIdx.x;
    if (cta >= cut.ctas) return;
    const bool vq = a.D % 4 == 0 && a.qs % 4 == 0 && reinterpret_cast<uintptr_t>(a.q) % (4 * sizeof(E)) == 0;
    const bool vk = a.D % 4 == 0 && reinterpret_cast<uintptr_t>(a.pool) % (4 * sizeof(E)) == 0;
    const size_t values = (size_t)a.Hkv * a.pt * a.D * sizeof(E);      // from a page's keys to its values
    const float c = a.scale * 1.4426950408889634f;
    for (AttnWalk p(a, units, cut, cta); p.more(); p.next(a, units)) {
        const AttnRow w = p.w;
        const AttnSpan s = p.s;
        const int n = p.rows(a);
        __syncthreads();
        for (int i = tid; i < kSimtRows * (D4 / 4); i += kSimtThreads) {
            const int r = i % kSimtRows, d = i / kSimtRows * 4;
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < n) {
                const AttnWalk::Place from = p.place(a, r);
                const char* q = static_cast<const char*>(a.q) + (from.token * a.qs + from.head * a.D) * (int64_t)sizeof(E);
                f = load4<E>(q, d, a.D, vq);
            }
            sq[d * kSimtPad + r] = f.x;
            sq[(d + 1) * kSimtPad + r] = f.y;
            sq[(d + 2) * kSimtPad + r] = f.z;
            sq[(d + 3) * kSimtPad + r] = f.w;
        }
        float o[DC][4][4], top[4], sum[4];
        int pos[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            top[i] = -INFINITY;
            sum[i] = 0.f;
            pos[i] = 4 * ty + i < n ? p.position(a, 4 * ty + i) : -1;
#pragma unroll
            for (int k = 0; k < DC; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[k][i][j] = 0.f;
        }
        const bool busy = warp * 8 < n;          // the warp's rows: 8
        for (int t = p.t0; t < p.t1; ++t) {
            const int k0 = (s.tile0 + t) * kSimtKeys;
            __syncthreads();
            for (int i = tid; i < kSimtKeys * (D4 / 4); i += kSimtThreads) {
                const int k = i % kSimtKeys, d = i / kSimtKeys * 4, key = k0 + k;
                float4 f = make_float4(0.f, 0.f, 0.f, 0.f), g = f;
                if (key >= s.begin && key < s.end) {
                    const char* page = attn_page(a, w.seq, key, p.head, sizeof(E));
                    if (page) {
                        f = load4<E>(page, d, a.D, vk);
                        g = load4<E>(page + values, d, a.D, vk);
                    }
                }
                sk[d * kSimtPad + k] = f.x;
                sk[(d + 1) * kSimtPad + k] = f.y;
                sk[(d + 2) * kSimtPad + k] = f.z;
                sk[(d + 3) * kSimtPad + k] = f.w;
                *reinterpret_cast<float4*>(sv + k * 64 * DC + d) = g;
            }
            __syncthreads();
            if (!busy) continue;
            float z[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) z[i][j] = 0.f;
            for (int d = 0; d < a.D; ++d) {
                const float4 q = *reinterpret_cast<const float4*>(sq + d * kSimtPad + 4 * ty);
                const float4 k = *reinterpret_cast<const float4*>(sk + d * kSimtPad + 4 * tx);
                const float qv[4] = {q.x, q.y, q.z, q.w}, kv[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) z[i][j] = fmaf(qv[i], kv[j], z[i][j]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float m = top[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = k0 + 4 * tx + j;
                    z[i][j] *= c;
                    if (key > pos[i] || (a.window && key <= pos[i] - a.window)) z[i][j] = -INFINITY;
                    m = fmaxf(m, z[i][j]);
                }
#pragma unroll
                for (int b = 8; b > 0; b >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, b));
                const float base = m == -INFINITY ? 0.f : m, f = exp2f(top[i] - base);
                top[i] = m;
                float add = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    z[i][j] = exp2f(z[i][j] - base);
                    add += z[i][j];
                }
#pragma unroll
                for (int b = 8; b > 0; b >>= 1) add += __shfl_xor_sync(0xffffffffu, add, b);
                sum[i] = fmaf(sum[i], f, add);
#pragma unroll
                for (int k = 0; k < DC; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[k][i][j] *= f;
            }
            // the weights of a row are used by the warp that made them
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<float4*>(sp + (4 * tx + j) * kSimtPad + 4 * ty) = make_float4(z[0][j], z[1][j], z[2][j], z[3][j]);
            __syncwarp();
            const int live = min(kSimtKeys, s.end - k0);
            for (int k = 0; k < live; ++k) {
                const float4 q = *reinterpret_cast<const float4*>(sp + k * kSimtPad + 4 * ty);
                const float pv[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int b = 0; b < DC; ++b) {
                    const float4 v = *reinterpret_cast<const float4*>(sv + k * 64 * DC + b * 64 + 4 * tx);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        o[b][i][0] = fmaf(pv[i], v.x, o[b][i][0]);
                        o[b][i][1] = fmaf(pv[i], v.y, o[b][i][1]);
                        o[b][i][2] = fmaf(pv[i], v.z, o[b][i][2]);
                        o[b][i][3] = fmaf(pv[i], v.w, o[b][i][3]);
                    }
                }
            }
        }
        if (tid == 0) p.tell_join(a, cut, cta);
        float* part = a.part + p.slot(cta) * attn_part_floats(a);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * ty + i;
            if (r >= n) continue;
            const AttnWalk::Place to_row = p.place(a, r);
            const size_t at = (size_t)to_row.token * a.Hq + to_row.head;
            const float inv = sum[i] > 0.f ? 1.f / sum[i] : sum[i] == 0.f ? 0.f : sum[i];
#pragma unroll
            for (int b = 0; b < DC; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int d = b * 64 + 4 * tx + j;
                    if (d >= a.D) continue;
                    if (p.whole()) store_act(a.out, at * a.D + d, o[b][i][j] * inv, a.dtype);
                    else part[(size_t)r * a.D + d] = o[b][i][j];
                }
            if (tx == 0) {
                if (!p.whole()) {
                    part[(size_t)a.block * a.D + r] = top[i];
                    part[(size_t)a.block * (a.D + 1) + r] = sum[i];
                } else if (a.lse) {
                    a.lse[at] = sum[i] == 0.f ? -INFINITY : (top[i] + log2f(sum[i])) * 0.6931471805599453f;
                }
            }
        }
    }
}

template <typename E, int DC> cudaError_t simt_launch(const AttnArgs& a, cudaStream_t st) {
    const size_t D4 = (a.D + 3) / 4 * 4, bytes = 4 * (2 * D4 * kSimtPad + (size_t)kSimtKeys * 64 * DC + kSimtKeys * kSimtPad);
    // (the same for every D of the instance: calls of several threads may come between this and the launch)
    const cudaError_t e = cudaFuncSetAttribute(attn_simt_kernel<E, DC>, cudaFuncAttributeMaxDynamicSharedMemorySize, 222 * 1024);
    if (e != cudaSuccess) return e;
    return attn_launch(attn_simt_kernel<E, DC>, a.ctas, kSimtThreads, bytes, !a.direct, st, a);
}

// ------------------------------------------------------------------ host

size_t up(size_t n) { return (n + 255) / 256 * 256; }

kda_status attn_check(const kda_attention_dims* d, bool varlen, bool append, AttnArgs* a) {
    if (!d || d->rows < 1 || d->tokens < 1 || d->Hkv < 1 || d->D < 1) return KDA_ERR_INVALID_ARG;
    if (d->dtype != KDA_BF16 && d->dtype != KDA_FP32) return KDA_ERR_INVALID_ARG;
    if (d->num_pages < 1 || d->page_tokens < 1 || d->table_rows < 1 || d->max_pages < 1 || d->window < 0) return KDA_ERR_INVALID_ARG;
    if (!append && (d->Hq < 1 || d->Hq % d->Hkv)) return KDA_ERR_INVALID_ARG;
    if (!varlen && d->tokens % d->rows) return KDA_ERR_INVALID_ARG;
    if (d->D > 256) return KDA_ERR_UNSUPPORTED;
    const int64_t kv = (int64_t)d->Hkv * d->D, q = (int64_t)d->Hq * d->D;
    if (append ? (d->k_stride != 0 && d->k_stride < kv) || (d->v_stride != 0 && d->v_stride < kv) : d->q_stride != 0 && d->q_stride < q)
        return KDA_ERR_INVALID_ARG;
    const int64_t most = 1LL << 30;
    if (d->tokens > most || d->rows > (1 << 24) || kv > (1 << 24) || q > (1 << 24) || (int64_t)d->num_pages > most ||
        (int64_t)d->max_pages * d->page_tokens > most || (int64_t)d->table_rows * d->max_pages > (1LL << 40))
        return KDA_ERR_UNSUPPORTED;
    if (2 * kv * d->page_tokens > (1LL << 40) / d->num_pages) return KDA_ERR_UNSUPPORTED;
    if (!append && (int64_t)d->tokens * d->Hq > (1LL << 31) - 1) return KDA_ERR_UNSUPPORTED;
    for (int64_t s : {d->q_stride, d->k_stride, d->v_stride})
        if (s > (1LL << 40) / d->tokens) return KDA_ERR_UNSUPPORTED;
    memset(a, 0, sizeof(*a));
    a->rows = d->rows; a->tokens = d->tokens; a->per_row = varlen ? 0 : d->tokens / d->rows;
    a->Hq = d->Hq; a->Hkv = d->Hkv; a->G = append ? 1 : d->Hq / d->Hkv; a->D = d->D; a->dtype = d->dtype;
    a->pages = d->num_pages; a->pt = d->page_tokens; a->table_rows = d->table_rows; a->max_pages = d->max_pages;
    a->window = d->window < most ? d->window : 0;      // (no position reaches it, and differences of positions stay in 32 bits)
    a->qs = d->q_stride ? d->q_stride : q;
    return KDA_OK;
}

// The cut for a kernel of `block` packed rows, `tile` keys and at most `ctas` CTAs.
void attn_cut(AttnArgs* a, int block, int tile, int extra, int ctas) {
    a->block = block;
    a->tile = tile;
    a->extra = extra;
    a->ctas = ctas;
    const int64_t most = ((int64_t)a->tokens * a->G + block - 1) / block + a->rows;      // a row's last block may be short
    a->units_most = (int)(most < (1LL << 30) ? most : (1LL << 30));
}
size_t attn_layout(char* ws, AttnArgs* a) {
    size_t o = 0;
    auto take = [&](size_t n) {
        char* p = ws ? ws + o : nullptr;
        o += up(n);
        return p;
    };
    a->units = reinterpret_cast<int*>(take(4));
    a->start = reinterpret_cast<int64_t*>(take(8 * ((size_t)a->units_most + 1)));
    a->unit_row = reinterpret_cast<int*>(take(8 * (size_t)a->units_most));
    a->shared = reinterpret_cast<AttnShared*>(take(sizeof(AttnShared) * (size_t)a->ctas));
    a->part = reinterpret_cast<float*>(take((size_t)2 * a->ctas * a->block * (a->D + 2) * 4));
    return o;
}

// Which kernel a call takes, and its cut.  aligned: the pool's base allows 16-byte copies.  The choice is the call's, by its rows'
// average, so that the same row may get the weights' one bf16 term (tc) in one call and two (mma) in another.
// mma reads a row's keys once for 16 packed rows, tc for 256: mma where a row has 16 on average at most (4 query heads to a key
// head, D = 128, attention and join: 16 packed rows of 8 requests over 8192 keys 71 us by mma, 68 by tc; of 64 over 2048 115
// and 115; with D = 64 single tokens of the 8 requests 48 and 53, of the 64 77 and 95), tc above it (32 packed rows: 93 us by mma, 70 by
// tc; 198 and 118).
// Above D = 128 mma has chunks as well, 16 packed rows to a read of the keys: 8192 tokens after 8192, 32 heads on 8 of 256, 34 ms.
// Their two or one CTAs of an SM share its registers and shared memory; extra: an item's beginning and end in key tiles, fitted to the
// CTAs' own times (tc: 8.2 us for an item, 1.53 us for a tile; cuts with 1 in place of 4 left some CTAs at twice the mean of
// short causal items, 774 for 1103 TFLOP/s).
void attn_choose(AttnArgs* a, bool aligned) {
    const int64_t packed = (int64_t)a->tokens * a->G;
    if (a->dtype == KDA_BF16 && a->D % 8 == 0 && aligned && a->D <= 128 && packed > kAttnMmaRows * (int64_t)a->rows &&
        (int64_t)a->pages * 2 * a->Hkv < (1 << 30)) {      // (a tensor map's coordinate)
        a->kernel = kAttnTc;
        attn_cut(a, kAttnTcRows, kAttnTcKeys, 5, 152);
    } else if (a->dtype == KDA_BF16 && a->D % 8 == 0 && aligned) {
        a->kernel = kAttnMma;
        attn_cut(a, kAttnMmaRows, kAttnMmaKeys, 2, a->D > 128 ? 152 : 304);
    } else {
        a->kernel = kAttnSimt;
        attn_cut(a, kSimtRows, kSimtKeys, 1, a->D > 128 ? 152 : 304);
    }
    a->direct = a->per_row && (int64_t)a->per_row * a->G <= a->block && a->rows <= kAttnDirectRows;
}

struct Span {
    const void* p;
    size_t n;
};
// Whether a result lies over what names the rows and their pages.
bool over_tables(const Span& r, const AttnArgs& a, const int32_t* table, const int32_t* lengths, const int32_t* seqs, const int32_t* cu) {
    return ranges_meet(r.p, r.n, table, (size_t)a.table_rows * a.max_pages * 4) || ranges_meet(r.p, r.n, lengths, (size_t)a.table_rows * 4) ||
           ranges_meet(r.p, r.n, seqs, (size_t)a.rows * 4) || ranges_meet(r.p, r.n, cu, ((size_t)a.rows + 1) * 4);
}

}  // namespace

cudaError_t launch_attn_simt(const AttnArgs& a, cudaStream_t st) {
#define KDA_ATTN_SIMT(DC) return a.dtype == KDA_BF16 ? simt_launch<__nv_bfloat16, DC>(a, st) : simt_launch<float, DC>(a, st)
    if (a.D <= 64) KDA_ATTN_SIMT(1);
    if (a.D <= 128) KDA_ATTN_SIMT(2);
    KDA_ATTN_SIMT(4);
#undef KDA_ATTN_SIMT
}

}  // namespace kda

using namespace kda;

extern "C" {

kda_status kda_pages_append(const kda_attention_dims* dims, void* pool, const int32_t* table, const int32_t* lengths,
                            const int32_t* seqs, const int32_t* cu_seqlens, const int32_t* cu_seqlens_host, const void* k,
                            const void* v, cudaStream_t stream) {
    AppendArgs p;
    memset(&p, 0, sizeof(p));
    kda_status st = attn_check(dims, cu_seqlens != nullptr, true, &p.a);
    if (st != KDA_OK) return st;
    if (!pool || !table || !lengths || !k || !v) return KDA_ERR_INVALID_ARG;
    if (!seqs && p.a.rows > p.a.table_rows) return KDA_ERR_INVALID_ARG;
    st = check_offsets_host(p.a.rows, p.a.tokens, cu_seqlens, cu_seqlens_host);
    if (st != KDA_OK) return st;
    const int64_t kv = (int64_t)p.a.Hkv * p.a.D, es = p.a.dtype == KDA_BF16 ? 2 : 4;
    p.k = k; p.v = v; p.pool = pool;
    p.ks = dims->k_stride ? dims->k_stride : kv;
    p.vs = dims->v_stride ? dims->v_stride : kv;
    const size_t np = (size_t)p.a.pages * 2 * kv * p.a.pt * es;
    if (ranges_meet(pool, np, k, ((size_t)(p.a.tokens - 1) * p.ks + kv) * es) || ranges_meet(pool, np, v, ((size_t)(p.a.tokens - 1) * p.vs + kv) * es))
        return KDA_ERR_INVALID_ARG;
    if (over_tables({pool, np}, p.a, table, lengths, seqs, cu_seqlens)) return KDA_ERR_INVALID_ARG;
    p.a.table = table; p.a.lengths = lengths; p.a.seqs = seqs; p.a.cu = cu_seqlens;
    st = status_ptr(&p.a.status);
    if (st != KDA_OK) return st;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(pool) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
                           (uintptr_t)(p.ks * es) | (uintptr_t)(p.vs * es) | (uintptr_t)(p.a.D * es);
    const int grid = (p.a.tokens + kAppendWarps - 1) / kAppendWarps;
    timing_pre(stream, K_PAGES_APPEND);
    if (bits % 16 == 0) append_kernel<uint4><<<grid, kAppendWarps * 32, 0, stream>>>(p);
    else if (es == 4) append_kernel<uint32_t><<<grid, kAppendWarps * 32, 0, stream>>>(p);
    else append_kernel<uint16_t><<<grid, kAppendWarps * 32, 0, stream>>>(p);
    timing_post(stream);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_pages_attention_workspace_size(const kda_attention_dims* dims) {
    AttnArgs a;
    if (!dims || attn_check(dims, true, false, &a) != KDA_OK) return 0;
    size_t most = 0;
    for (bool aligned : {false, true}) {
        attn_choose(&a, aligned);
        const size_t n = attn_layout(nullptr, &a);
        if (n > most) most = n;
    }
    return most;
}

kda_status kda_pages_attention(const kda_attention_dims* dims, const void* q, const void* pool, const int32_t* table,
                               const int32_t* lengths, const int32_t* seqs, const int32_t* cu_seqlens,
                               const int32_t* cu_seqlens_host, float scale, void* out, float* lse, void* workspace,
                               size_t workspace_bytes, cudaStream_t stream) {
    AttnArgs a;
    kda_status st = attn_check(dims, cu_seqlens != nullptr, false, &a);
    if (st != KDA_OK) return st;
    if (!q || !pool || !table || !lengths || !out || !isfinite(scale)) return KDA_ERR_INVALID_ARG;
    if (!seqs && a.rows > a.table_rows) return KDA_ERR_INVALID_ARG;
    st = check_offsets_host(a.rows, a.tokens, cu_seqlens, cu_seqlens_host);
    if (st != KDA_OK) return st;
    const size_t es = a.dtype == KDA_BF16 ? 2 : 4, no = (size_t)a.tokens * a.Hq * a.D * es, nl = (size_t)a.tokens * a.Hq * 4;
    const size_t nq = ((size_t)(a.tokens - 1) * a.qs + (size_t)a.Hq * a.D) * es, np = (size_t)a.pages * 2 * a.Hkv * a.pt * a.D * es;
    if (ranges_meet(out, no, q, nq) || ranges_meet(out, no, pool, np) || ranges_meet(lse, nl, q, nq) || ranges_meet(lse, nl, pool, np) ||
        ranges_meet(out, no, lse, nl))
        return KDA_ERR_INVALID_ARG;
    for (const Span& r : {Span{out, no}, Span{lse, nl}})
        if (over_tables(r, a, table, lengths, seqs, cu_seqlens)) return KDA_ERR_INVALID_ARG;
    attn_choose(&a, reinterpret_cast<uintptr_t>(pool) % 16 == 0);
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < attn_layout(nullptr, &a)) return KDA_ERR_WORKSPACE;
    attn_layout(static_cast<char*>(workspace), &a);
    a.q = q; a.pool = pool; a.table = table; a.lengths = lengths; a.seqs = seqs; a.cu = cu_seqlens; a.scale = scale; a.out = out; a.lse = lse;
    if ((int64_t)a.units_most * a.Hkv > (1LL << 30)) return KDA_ERR_UNSUPPORTED;
    st = status_ptr(&a.status);
    if (st != KDA_OK) return st;
    if (!a.direct) {
        timing_pre(stream, K_ATTN_PLAN);
        attn_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
        timing_post(stream);
        if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
    }
    timing_pre(stream, K_ATTN);
    const cudaError_t e = a.kernel == kAttnTc ? launch_attn_tc(a, stream) : a.kernel == kAttnMma ? launch_attn_mma(a, stream) : launch_attn_simt(a, stream);
    timing_post(stream);
    if (e != cudaSuccess) return KDA_ERR_CUDA;
    // rows of a block that may exist; a CTA for each where they are few, else a warp (two rows of a warp: 2 us more for small chunks)
    const int64_t longest = (cu_seqlens ? a.tokens : a.per_row) * (int64_t)a.G;
    const int rows = (int)(longest < a.block ? longest : a.block), each = a.block <= 32 ? 1 : kJoinWarps;
    timing_pre(stream, K_ATTN_JOIN);
    // (launched while the attention still runs; it waits for its end itself)
    if (a.ctas > 1)
        st = attn_launch(attn_join_kernel, dim3(a.ctas - 1, (rows + each - 1) / each), kJoinThreads, 0, true, stream, a, each) == cudaSuccess
                 ? KDA_OK : KDA_ERR_CUDA;
    timing_post(stream);
    return st;
}

}  // extern "C"
