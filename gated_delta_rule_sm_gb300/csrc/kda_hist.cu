// kda_hist.cu -- the short convolution with a carried history: prompts that go on from the last W - 1
// inputs of what came before, and single tokens on a pool of histories.
//
//     a[t, c] = bias[c] + sum_{i < W} weight[c, i] x[t - (W - 1) + i, c],    y = a * sigmoid(a)
// with x at negative times taken from the history.  Bound by memory: x read once, y written once.  A
// thread owns four channels over a tile of tokens and keeps the last W inputs in a ring of registers; its loads
// run up to eight tokens ahead.  Measured on 16384 tokens x 4096 channels, W 4: bf16 53 us (5.0 TB/s), fp32 90
// us (5.9 TB/s); with eight channels a thread 61 and 104 us (fewer warps: waiting for loads), with tiles that
// leave a last wave of CTAs part empty 59 us, with histories in place 59 us (a second launch).  One token of 128 rows x 12288 channels: 9 us of kernel, 11 us
// with two rows to a CTA in place of four.
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

constexpr int kHistMaxW = 8;
constexpr int kHistLeast = 8, kHistMost = 80;   // tokens per CTA
// tokens whose loads a thread has in flight: a multiple of W, so that the window's place in its registers is
// the same in every batch
constexpr int hist_ahead(int W) { return 8 / W * W; }
constexpr int kHistThreads = 128;

struct HistArgs {
    int TT, T, C, W, dtype, rows, tile, tiles, num_slots, wide;   // wide: the weights allow 16-byte loads
    int64_t xs;            // elements between tokens of x
    const void* x;
    const float* w;        // [C, W]
    const float* b;        // [C] or nullptr
    const int32_t* cu;     // [rows + 1] or nullptr
    const int32_t* slots;
    const void* h_in;      // [rows or num_slots, W - 1, C] or nullptr
    void* h_out;           // likewise
    void* y;               // [TT, C]
    int* status;
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A thread's channels of one token.
constexpr int kCh = 4, kPairs = kCh / 2;
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> {
    uint2 u;
    __device__ __forceinline__ void load(const void* p, size_t i) {
        u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + i);
    }
    __device__ __forceinline__ void zero() { u = make_uint2(0, 0); }
    __device__ __forceinline__ void store(void* p, size_t i) const {
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + i) = u;
    }
    __device__ __forceinline__ void get(float2* v) const {
        v[0] = make_float2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
        v[1] = make_float2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
    }
    __device__ __forceinline__ void put(const float2* v) { u = make_uint2(pack_bf16(v[0].x, v[0].y), pack_bf16(v[1].x, v[1].y)); }
};
template <> struct Raw<float> {
    float4 a;
    __device__ __forceinline__ void load(const void* p, size_t i) {
        a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    }
    __device__ __forceinline__ void zero() { a = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void store(void* p, size_t i) const { *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = a; }
    __device__ __forceinline__ void get(float2* v) const {
        v[0] = make_float2(a.x, a.y);
        v[1] = make_float2(a.z, a.w);
    }
    __device__ __forceinline__ void put(const float2* v) { a = make_float4(v[0].x, v[0].y, v[1].x, v[1].y); }
};

// A thread's taps are kCh W consecutive floats; kept as pairs of channels.
template <int W>
__device__ __forceinline__ void load_weights(const HistArgs& a, int c0, float2 (*w)[W], float2* bias) {
    const float* src = a.w + (size_t)c0 * W;
    float f[kCh * W];
    if (a.wide) {
#pragma unroll
        for (int i = 0; i < kCh * W; i += 4) *reinterpret_cast<float4*>(f + i) = __ldg(reinterpret_cast<const float4*>(src + i));
    } else {
#pragma unroll
        for (int i = 0; i < kCh * W; ++i) f[i] = src[i];
    }
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
        bias[k] = a.b ? make_float2(a.b[c0 + 2 * k], a.b[c0 + 2 * k + 1]) : make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < W; ++i) w[k][i] = make_float2(f[2 * k * W + i], f[(2 * k + 1) * W + i]);
    }
}

// silu(bias + w . window); the window is a ring of W inputs, the oldest at place `first`.
// a / (1 + e^-a) takes one reciprocal for two values (the special function unit is half as busy), so the exponential
// stops at 2^60, which keeps the product of two sums finite.  From there, a = -41.6, the sigmoid is taken as 0: a times
// it is above -3.7e-17.  (A reciprocal each and no limit: 51.1 us for 53.2 in bf16 with W 4, but 61.3 for 55.2 in fp32
// with W 8, 8192 tokens.)
template <int W, typename R>
__device__ __forceinline__ void conv_out(const float2 (*w)[W], const float2* bias, const float2 (*win)[kPairs], int first, R& out) {
    float2 y[kPairs];
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
        y[k] = bias[k];
#pragma unroll
        for (int i = 0; i < W; ++i) y[k] = fma2(w[k][i], win[(first + i) % W][k], y[k]);
        const float2 x = mul2(y[k], dup(-1.4426950408889634f));
        const float2 d = fma2(make_float2(fminf(exp2_fast(x.x), 0x1p60f), fminf(exp2_fast(x.y), 0x1p60f)), dup(1.f), dup(1.f));
        const float r = rcp_fast(d.x * d.y);
        y[k] = mul2(y[k], mul2(dup(r), make_float2(d.x < 0x1p60f ? d.y : 0.f, d.y < 0x1p60f ? d.x : 0.f)));
    }
    out.put(y);
}

// Whether the offsets keep the contract; the same answer in every thread.  A CTA reads them all: they are
// few next to its tokens, and no separate pass has to run first.
__device__ __forceinline__ bool offsets_ok(const HistArgs& a) {
    bool bad = false;
    for (int n = threadIdx.x; n < a.rows; n += kHistThreads) bad |= a.cu[n + 1] < a.cu[n];
    if (threadIdx.x == 0) bad |= a.cu[0] != 0 || a.cu[a.rows] != a.TT;
    return !__syncthreads_or(bad);
}

__device__ __forceinline__ int row_begin(const HistArgs& a, int n) { return a.cu ? a.cu[n] : n * a.T; }

// CTAs below `tiles` take a.tile tokens each; the others write the final history of one row each.  Where that goes
// over the initial history, which the first tokens' CTAs read, they are a launch of their own after the tokens'
// (tiles 0): there a thread reads and writes only its own channels of one row, the oldest input first, and its
// reads are never behind its writes.
template <int W, typename E>
__global__ void __launch_bounds__(kHistThreads, W > 4 ? 3 : sizeof(E) == 2 ? 6 : 4) conv_prompt_kernel(HistArgs a) {
    if (a.cu && !offsets_ok(a)) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) record_error(a.status, KDA_ERR_INVALID_ARG);
        return;
    }
    const int c0 = (blockIdx.y * kHistThreads + threadIdx.x) * kCh;
    if (c0 >= a.C) return;
    Raw<E> raw;
    if ((int)blockIdx.x >= a.tiles) {
        const int n = blockIdx.x - a.tiles;
        const int s0 = row_begin(a, n), s1 = row_begin(a, n + 1);
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            const int t = s1 - (W - 1) + i;       // before s0: row i + (s1 - s0) of the old history
            if (t >= s0) raw.load(a.x, (size_t)t * a.xs + c0);
            else if (a.h_in) raw.load(a.h_in, ((size_t)n * (W - 1) + i + (s1 - s0)) * a.C + c0);
            else raw.zero();
            raw.store(a.h_out, ((size_t)n * (W - 1) + i) * a.C + c0);
        }
        return;
    }
    constexpr int AHEAD = hist_ahead(W);
    float2 w[kPairs][W], bias[kPairs], win[W][kPairs];
    load_weights<W>(a, c0, w, bias);
    const int t0 = blockIdx.x * a.tile, t1 = min(t0 + a.tile, a.TT);
    int n, s0, s1;
    if (a.cu) {
        int lo = 0, hi = a.rows - 1;   // last n with cu[n] <= t0
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.cu[mid] <= t0) lo = mid; else hi = mid - 1;
        }
        n = lo;
    } else {
        n = t0 / a.T;
    }
    s0 = row_begin(a, n);
    s1 = row_begin(a, n + 1);
    auto fill = [&](int t) {   // the W - 1 inputs before token t of row n
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            const int tau = t - (W - 1) + i;
            if (tau >= s0) raw.load(a.x, (size_t)tau * a.xs + c0);
            else if (a.h_in) raw.load(a.h_in, ((size_t)n * (W - 1) + (tau - s0 + W - 1)) * a.C + c0);
            else raw.zero();
            raw.get(win[i]);
        }
    };
    fill(t0);
    for (int t = t0; t < t1;) {
        if (t == s1) {
            while (t >= s1) {   // empty rows in between
                ++n;
                s0 = s1;
                s1 = row_begin(a, n + 1);
            }
            fill(t);
        }
        // tokens up to the row's or the tile's end, each one's load AHEAD tokens before its use
        const int end = min(t1, s1);
        Raw<E> in[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (t + i < end) in[i].load(a.x, (size_t)(t + i) * a.xs + c0);
        // fill() leaves the inputs before t at places 0 .. W - 2: token t + i goes to place (W - 1 + i) % W
        auto put = [&](int i) {
            in[i].get(win[(W - 1 + i) % W]);
            if (t + i + AHEAD < end) in[i].load(a.x, (size_t)(t + i + AHEAD) * a.xs + c0);
            Raw<E> out;
            conv_out<W>(w, bias, win, i % W, out);
            out.store(a.y, (size_t)(t + i) * a.C + c0);
        };
        for (; t + AHEAD <= end; t += AHEAD)
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) put(i);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (t + i >= end) break;
            put(i);
        }
        t = end;
    }
}

// kHistRows rows of the batch with one set of weights (16 bytes of weights per channel beside 16 bytes of
// inputs, outputs and histories per channel and row), all rows' loads in flight at once.
constexpr int kHistRows = 4;
template <int W, typename E>
__global__ void __launch_bounds__(kHistThreads) conv_step_kernel(HistArgs a) {
    const int c0 = (blockIdx.y * kHistThreads + threadIdx.x) * kCh;
    if (c0 >= a.C) return;
    Raw<E> raw[kHistRows][W];
    int slot[kHistRows];
#pragma unroll
    for (int k = 0; k < kHistRows; ++k) {
        const int r = blockIdx.x * kHistRows + k;
        slot[k] = r >= a.rows ? -1 : a.slots ? a.slots[r] : r;
        if (slot[k] >= a.num_slots) {
            if (c0 == 0) record_error(a.status, KDA_ERR_INVALID_ARG);
            slot[k] = -1;
        }
    }
#pragma unroll
    for (int k = 0; k < kHistRows; ++k) {
        const int r = blockIdx.x * kHistRows + k;
        if (slot[k] < 0) continue;
        const size_t hb = (size_t)slot[k] * (W - 1) * a.C + c0;
#pragma unroll
        for (int i = 0; i < W - 1; ++i) raw[k][i].load(a.h_in, hb + (size_t)i * a.C);
        raw[k][W - 1].load(a.x, (size_t)r * a.xs + c0);
    }
    float2 w[kPairs][W], bias[kPairs], win[W][kPairs];
    load_weights<W>(a, c0, w, bias);
#pragma unroll
    for (int k = 0; k < kHistRows; ++k) {
        const int r = blockIdx.x * kHistRows + k;
        if (r >= a.rows) break;
        Raw<E> out;
        if (slot[k] < 0) {
            out.zero();
            out.store(a.y, (size_t)r * a.C + c0);
            continue;
        }
#pragma unroll
        for (int i = 0; i < W; ++i) raw[k][i].get(win[i]);
        conv_out<W>(w, bias, win, 0, out);
        out.store(a.y, (size_t)r * a.C + c0);
        const size_t hb = (size_t)slot[k] * (W - 1) * a.C + c0;
#pragma unroll
        for (int i = 0; i < W - 1; ++i) raw[k][i + 1].store(a.h_out, hb + (size_t)i * a.C);
    }
}

kda_status hist_check(int B, int T, int C, int W, int dtype, const void* x, int64_t xs, const float* weight,
                      const void* h_in, const void* h_out, const void* y) {
    if (B < 1 || T < 1 || C < 1 || W < 1) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_BF16 && dtype != KDA_FP32) return KDA_ERR_INVALID_ARG;
    if (!x || !weight || !y || (xs != 0 && xs < C)) return KDA_ERR_INVALID_ARG;
    if (W > kHistMaxW || C % 8 || xs % 8) return KDA_ERR_UNSUPPORTED;
    if ((long long)B * T > (1LL << 30) || (long long)B * T * (xs ? xs : C) > (1LL << 40)) return KDA_ERR_UNSUPPORTED;
    for (const void* p : {x, h_in, h_out, y})
        if (reinterpret_cast<uintptr_t>(p) % 16) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

}  // namespace

// f of the kernel's width and element type as constants.
template <typename F>
static cudaError_t hist_dispatch(int W, int dtype, F&& f) {
#define KDA_HIST_CASE(w) \
    case w: return dtype == KDA_BF16 ? f(std::integral_constant<int, w>(), __nv_bfloat16()) : f(std::integral_constant<int, w>(), float());
    switch (W) {
        KDA_HIST_CASE(1)
        KDA_HIST_CASE(2)
        KDA_HIST_CASE(3)
        KDA_HIST_CASE(4)
        KDA_HIST_CASE(5)
        KDA_HIST_CASE(6)
        KDA_HIST_CASE(7)
        KDA_HIST_CASE(8)
    }
#undef KDA_HIST_CASE
    return cudaErrorInvalidValue;
}

// CTAs of a kernel that the GPU holds at once.
template <int W, typename E>
static int prompt_slots() {
    static const int n = [] {
        int per = 0;
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, conv_prompt_kernel<W, E>, kHistThreads, 0) == cudaSuccess && per > 0
                   ? per * 152 : 152;
    }();
    return n;
}

}  // namespace kda

using namespace kda;

extern "C" {

kda_status kda_short_conv_prompt(int B, int T, int C, int W, kda_dtype dtype, const void* x, int64_t x_stride,
                                 const float* weight, const float* bias, const int32_t* cu_seqlens,
                                 const int32_t* cu_seqlens_host, int num_seqs, const void* initial_history, void* y,
                                 void* final_history, cudaStream_t stream) {
    kda_status st = hist_check(B, T, C, W, dtype, x, x_stride, weight, initial_history, final_history, y);
    if (st != KDA_OK) return st;
    if (cu_seqlens && (B != 1 || num_seqs < 1)) return KDA_ERR_INVALID_ARG;
    if (cu_seqlens && num_seqs > (1 << 24)) return KDA_ERR_UNSUPPORTED;
    HistArgs a;
    memset(&a, 0, sizeof(a));
    a.TT = B * T; a.T = T; a.C = C; a.W = W; a.dtype = dtype; a.rows = cu_seqlens ? num_seqs : B;
    st = check_offsets_host(a.rows, a.TT, cu_seqlens, cu_seqlens_host);
    if (st != KDA_OK) return st;
    a.xs = x_stride ? x_stride : C;
    a.wide = reinterpret_cast<uintptr_t>(weight) % 16 == 0;
    a.x = x; a.w = weight; a.b = bias; a.cu = cu_seqlens; a.h_in = initial_history; a.h_out = final_history; a.y = y;
    // other CTAs read what one writes: the results get memory of their own, but for histories in place
    const size_t es = dtype == KDA_BF16 ? 2 : 4, nx = ((size_t)(a.TT - 1) * a.xs + C) * es, ny = (size_t)a.TT * C * es;
    const size_t nh = (size_t)a.rows * (W - 1) * C * es;
    const bool in_place = nh && final_history == initial_history;
    if (ranges_meet(y, ny, x, nx) || ranges_meet(y, ny, initial_history, nh) || ranges_meet(y, ny, final_history, nh) ||
        ranges_meet(final_history, nh, x, nx) || (!in_place && ranges_meet(final_history, nh, initial_history, nh)))
        return KDA_ERR_INVALID_ARG;
    st = status_ptr(&a.status);
    if (st != KDA_OK) return st;
    timing_pre(stream, K_CONV_PROMPT);
    const cudaError_t e = hist_dispatch(W, dtype, [&](auto w, auto type) {
        using E = decltype(type);
        // the fewest whole waves of CTAs with no more than kHistMost tokens each
        const int cols = (C / kCh + kHistThreads - 1) / kHistThreads;
        const int64_t slots = prompt_slots<w.value, E>(), work = (int64_t)a.TT * cols;
        const int64_t ctas = (work + slots * kHistMost - 1) / (slots * kHistMost) * slots;
        a.tile = (int)((work + ctas - 1) / ctas);
        if (a.tile < kHistLeast) a.tile = kHistLeast;
        a.tiles = (a.TT + a.tile - 1) / a.tile;
        const int ends = final_history && w.value > 1 ? a.rows : 0;
        conv_prompt_kernel<w.value, E><<<dim3(a.tiles + (in_place ? 0 : ends), cols), kHistThreads, 0, stream>>>(a);
        if (in_place) {
            a.tiles = 0;
            conv_prompt_kernel<w.value, E><<<dim3(ends, cols), kHistThreads, 0, stream>>>(a);
        }
        return cudaGetLastError();
    });
    timing_post(stream);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_short_conv_step(int B, int C, int W, kda_dtype dtype, const void* x, int64_t x_stride,
                               const float* weight, const float* bias, const int32_t* slots, int num_slots,
                               const void* history_in, void* history_out, void* y, cudaStream_t stream) {
    kda_status st = hist_check(B, 1, C, W, dtype, x, x_stride, weight, history_in, history_out, y);
    if (st != KDA_OK) return st;
    if (num_slots < 1 || (!slots && num_slots < B)) return KDA_ERR_INVALID_ARG;
    if (W > 1 && (!history_in || !history_out)) return KDA_ERR_INVALID_ARG;
    HistArgs a;
    memset(&a, 0, sizeof(a));
    a.C = C; a.W = W; a.dtype = dtype; a.rows = B; a.num_slots = num_slots; a.xs = x_stride ? x_stride : C;
    a.wide = reinterpret_cast<uintptr_t>(weight) % 16 == 0;
    a.x = x; a.w = weight; a.b = bias; a.slots = slots; a.h_in = history_in; a.h_out = history_out; a.y = y;
    st = status_ptr(&a.status);
    if (st != KDA_OK) return st;
    const dim3 grid((B + kHistRows - 1) / kHistRows, (C / kCh + kHistThreads - 1) / kHistThreads);
    timing_pre(stream, K_CONV_STEP);
    const cudaError_t e = hist_dispatch(W, dtype, [&](auto w, auto type) {
        conv_step_kernel<w.value, decltype(type)><<<grid, kHistThreads, 0, stream>>>(a);
        return cudaGetLastError();
    });
    timing_post(stream);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
