// kda_step.cu -- one token per row on a pool of recurrent states: the delta rule's step and the state
// space step.
//
// Both read a [rows of k or n][columns of v or p] fp32 state once and write it once, so they are bound by
// memory: 8 bytes per state element against ~100 bytes of activations per row of the state.
//   delta rule:   S' = Diag(alpha) S,  u = beta (v - S'^T k),  S'' = S' + k u^T,
//                 o = scale S''^T q = scale (S'^T q + (k.q) u)
// The second form of o needs only sums over the loaded state, so S' stays in registers between its one
// load and its one store, with one reduction over the rows (for S'^T k and S'^T q) in between.
//   state space:  S' = exp(D a) S + (D B) x^T,  y = S'^T C + d x
// has no such dependence: a row of the state is stored as soon as it is formed.
// The columns are independent, so a CTA takes one (row, head, 64-column tile): 256 threads as 16 column
// groups of four (one 16-byte access each) x 16 state rows; a pool whose base or column count does not
// allow 16-byte accesses is read a float at a time by 64 x 4 threads.
// Measured, bf16, rows scattered over the pool, a seventh of them idle: 64 rows x 32 heads of 128 x 128 (delta
// rule) 43 us, 128 rows x 32 heads of 128 x 64 (state space) 45 us, 232 MB each: 5.4 and 5.2 TB/s, 0.8 of a plain
// copy's rate.  One row: 4 us of kernel, the launch is what counts.
#include <math.h>
#include <string.h>

#include "kda.h"
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {

namespace {

constexpr int kStepThreads = 256;
constexpr int kStepTile = 64;     // state columns per CTA

struct StepArgs {
    int B, H, Hk, G, K, V, dtype, gate, num_slots;   // K x V: state rows x columns (N x P of the state space step)
    int64_t xs, bs, cs, ds;                          // row strides of x, b, c, dt_raw (state space step)
    const void *q, *k, *v, *g_raw, *beta_raw;        // c, b, x, -, dt_raw of the state space step
    const float *a_log, *dt_bias, *d_skip;
    float scale, lb;
    const int32_t* slots;
    const float* s_in;
    float* s_out;
    void* out;
    int* status;
};

// The row's slot; -1 for an idle row.
__device__ __forceinline__ int step_slot(const StepArgs& a, int b) {
    if (!a.slots) return b;
    const int s = a.slots[b];
    if (s >= a.num_slots && threadIdx.x == 0) record_error(a.status, KDA_ERR_INVALID_ARG);
    return s < 0 || s >= a.num_slots ? -1 : s;
}

template <int VEC> struct Cols { float v[VEC]; };

template <int VEC>
__device__ __forceinline__ Cols<VEC> load_cols(const float* p) {
    Cols<VEC> r;
    if constexpr (VEC == 4) {
        const float4 f = __ldcs(reinterpret_cast<const float4*>(p));
        r.v[0] = f.x; r.v[1] = f.y; r.v[2] = f.z; r.v[3] = f.w;
    } else {
        r.v[0] = *p;
    }
    return r;
}

template <int VEC>
__device__ __forceinline__ void store_cols(float* p, const Cols<VEC>& r) {
    if constexpr (VEC == 4) __stcs(reinterpret_cast<float4*>(p), make_float4(r.v[0], r.v[1], r.v[2], r.v[3]));
    else *p = r.v[0];
}

// K <= 128: a thread holds rows ty, ty + RY, ... of its VEC columns, 32 floats.
template <int VEC>
__global__ void __launch_bounds__(kStepThreads, VEC == 4 ? 4 : 3) decode_step_kernel(StepArgs a) {
    constexpr int CX = kStepTile / VEC, RY = kStepThreads / CX, PER = 128 / RY;
    constexpr int WROWS = kStepThreads / 32;          // partial sums left per column after a warp's own
    __shared__ float sk[128], sq[128], sal[128];
    __shared__ float sr[WROWS][kStepTile], sw[WROWS][kStepTile];
    __shared__ __align__(16) float su[kStepTile];
    __shared__ float red[3][4];
    const int tid = threadIdx.x, cx = tid % CX, ry = tid / CX;
    const int bh = blockIdx.x, b = bh / a.H, h = bh - b * a.H;
    const int col = blockIdx.y * kStepTile + cx * VEC;
    const bool in = col < a.V;
    const int slot = step_slot(a, b);
    if (slot < 0) {
        if (ry == 0 && in)
#pragma unroll
            for (int e = 0; e < VEC; ++e) store_act(a.out, (size_t)bh * a.V + col + e, 0.f, a.dtype);
        return;
    }
    const size_t base = ((size_t)slot * a.H + h) * a.K * a.V + col;
    Cols<VEC> S[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r = ry + i * RY;
        if (in && r < a.K) S[i] = load_cols<VEC>(a.s_in + base + (size_t)r * a.V);
        else
#pragma unroll
            for (int e = 0; e < VEC; ++e) S[i].v[e] = 0.f;
    }
    // the row's q, k (L2 norm over K) and alpha, while the state is on its way
    const size_t kb = ((size_t)b * a.Hk + h / (a.H / a.Hk)) * a.K;
    float qv = 0.f, kv = 0.f;
    if (tid < a.K) {
        qv = load_act(a.q, kb + tid, a.dtype);
        kv = load_act(a.k, kb + tid, a.dtype);
        const float z = load_act(a.g_raw, (size_t)bh * a.K + tid, a.dtype) + a.dt_bias[h * a.K + tid];
        const float ea = expf(a.a_log[h]);
        const float g = a.gate == KDA_GATE_SOFTPLUS ? -ea * softplusf(z) : a.lb * sigmoidf_acc(ea * z);
        sal[tid] = expf(g);
    }
    if (tid < 128) {
        sq[tid] = qv;
        sk[tid] = kv;
        const float qq = warp_sum(qv * qv), kk = warp_sum(kv * kv), qk = warp_sum(qv * kv);
        if ((tid & 31) == 0) {
            red[0][tid >> 5] = qq;
            red[1][tid >> 5] = kk;
            red[2][tid >> 5] = qk;
        }
    }
    __syncthreads();
    float sum[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) sum[i] = (red[i][0] + red[i][1]) + (red[i][2] + red[i][3]);
    const float rq = 1.0f / sqrtf(sum[0] + kNormEps), rk = 1.0f / sqrtf(sum[1] + kNormEps);
    float r_[VEC], w_[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) r_[e] = w_[e] = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r = ry + i * RY;
        if (r >= a.K) break;
        const float al = sal[r], kr = sk[r], qr = sq[r];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            S[i].v[e] *= al;
            r_[e] = fmaf(S[i].v[e], kr, r_[e]);
            w_[e] = fmaf(S[i].v[e], qr, w_[e]);
        }
    }
    // S'^T k and S'^T q (k, q not yet divided by their norms): first the warp's rows, then the warps
    if (CX == 16) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            r_[e] += __shfl_xor_sync(0xffffffffu, r_[e], 16);
            w_[e] += __shfl_xor_sync(0xffffffffu, w_[e], 16);
        }
    }
    constexpr int PARTS = CX == 16 ? WROWS : RY;
    const int part = CX == 16 ? tid >> 5 : ry;
    if (CX != 16 || (tid & 16) == 0)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            sr[part][cx * VEC + e] = r_[e];
            sw[part][cx * VEC + e] = w_[e];
        }
    __syncthreads();
    const int c = blockIdx.y * kStepTile + tid;
    if (tid < kStepTile && c < a.V) {
        float r = 0.f, w = 0.f;
#pragma unroll
        for (int j = 0; j < PARTS; ++j) {
            r += sr[j][tid];
            w += sw[j][tid];
        }
        const float beta = sigmoidf_acc(load_act(a.beta_raw, bh, a.dtype));
        const float u = beta * (load_act(a.v, (size_t)bh * a.V + c, a.dtype) - r * rk);
        su[tid] = u * rk;
        store_act(a.out, (size_t)bh * a.V + c, a.scale * rq * fmaf(sum[2] * rk, u, w), a.dtype);
    }
    __syncthreads();
    if (!in) return;
    float u[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) u[e] = su[cx * VEC + e];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r = ry + i * RY;
        if (r >= a.K) break;
        const float kr = sk[r];
#pragma unroll
        for (int e = 0; e < VEC; ++e) S[i].v[e] = fmaf(kr, u[e], S[i].v[e]);
        store_cols<VEC>(a.s_out + base + (size_t)r * a.V, S[i]);
    }
}

template <int VEC>
__global__ void __launch_bounds__(kStepThreads, 3) ssm_step_kernel(StepArgs a) {
    constexpr int CX = kStepTile / VEC, RY = kStepThreads / CX, BATCH = VEC == 4 ? 8 : 16;
    __shared__ float sy[RY][kStepTile + 4];
    const int tid = threadIdx.x, cx = tid % CX, ry = tid / CX;
    const int bh = blockIdx.x, b = bh / a.H, h = bh - b * a.H;
    const int col = blockIdx.y * kStepTile + cx * VEC;
    const bool in = col < a.V;
    const int slot = step_slot(a, b);
    if (slot < 0) {
        if (ry == 0 && in)
#pragma unroll
            for (int e = 0; e < VEC; ++e) store_act(a.out, (size_t)bh * a.V + col + e, 0.f, a.dtype);
        return;
    }
    const size_t base = ((size_t)slot * a.H + h) * a.K * a.V + col;
    const size_t gb = (size_t)(h / (a.H / a.G)) * a.K;
    Cols<VEC> S[BATCH];
    float bv[BATCH], cv[BATCH];
    auto load = [&](int r0) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int r = r0 + i * RY;
            if (r < a.K && in) S[i] = load_cols<VEC>(a.s_in + base + (size_t)r * a.V);
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int r = r0 + i * RY;
            if (r < a.K) {
                bv[i] = load_act(a.k, (size_t)b * a.bs + gb + r, a.dtype);
                cv[i] = load_act(a.q, (size_t)b * a.cs + gb + r, a.dtype);
            }
        }
    };
    load(ry);     // on its way while the row's scalars are formed
    const float dt = softplusf(load_act(a.beta_raw, (size_t)b * a.ds + h, a.dtype) + a.dt_bias[h]);
    const float al = expf(-expf(a.a_log[h]) * dt);
    float u[VEC], y[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        u[e] = in ? dt * load_act(a.v, (size_t)b * a.xs + (size_t)h * a.V + col + e, a.dtype) : 0.f;
        y[e] = 0.f;
    }
    for (int r0 = ry; r0 < a.K; r0 += BATCH * RY) {
        if (r0 != ry) load(r0);
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int r = r0 + i * RY;
            if (r >= a.K || !in) break;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                S[i].v[e] = fmaf(al, S[i].v[e], u[e] * bv[i]);
                y[e] = fmaf(S[i].v[e], cv[i], y[e]);
            }
            store_cols<VEC>(a.s_out + base + (size_t)r * a.V, S[i]);
        }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) sy[ry][cx * VEC + e] = y[e];
    __syncthreads();
    const int c = blockIdx.y * kStepTile + tid;
    if (tid < kStepTile && c < a.V) {
        float t = 0.f;
#pragma unroll
        for (int j = 0; j < RY; ++j) t += sy[j][tid];
        if (a.d_skip)
            t = fmaf(a.d_skip[h], load_act(a.v, (size_t)b * a.xs + (size_t)h * a.V + c, a.dtype), t);
        store_act(a.out, (size_t)bh * a.V + c, t, a.dtype);
    }
}

bool pool_vec_ok(const StepArgs& a) {
    auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    return a.V % 4 == 0 && al(a.s_in) && al(a.s_out);
}

kda_status slots_check(int B, const int32_t* slots, int num_slots, const float* s_in, float* s_out) {
    if (num_slots < 1 || (!slots && num_slots < B)) return KDA_ERR_INVALID_ARG;
    if (!s_in || !s_out) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

}  // namespace

}  // namespace kda

using namespace kda;

extern "C" {

kda_status kda_decode_step(const kda_dims* dims, const void* q, const void* k, const void* v, const void* g_raw,
                           const void* beta_raw, const float* a_log, const float* dt_bias, float scale,
                           float lower_bound, const int32_t* slots, int num_slots, const float* state_in,
                           float* state_out, void* out, cudaStream_t stream) {
    if (!dims || dims->T != 1) return KDA_ERR_INVALID_ARG;
    const kda_dims& d = *dims;
    const int Hk = d.Hk > 0 ? d.Hk : d.H;
    if (d.B < 1 || d.H < 1 || d.Hk < 0 || d.H % Hk || d.K < 16 || d.V < 16) return KDA_ERR_INVALID_ARG;
    if (d.dtype != KDA_BF16 && d.dtype != KDA_FP32) return KDA_ERR_INVALID_ARG;
    if (d.gate != KDA_GATE_LOWER_BOUNDED && d.gate != KDA_GATE_SOFTPLUS) return KDA_ERR_INVALID_ARG;
    if (!q || !k || !v || !g_raw || !beta_raw || !a_log || !dt_bias || !out) return KDA_ERR_INVALID_ARG;
    if (!(lower_bound < 0.0f) || !isfinite(lower_bound) || !isfinite(scale)) return KDA_ERR_INVALID_ARG;
    kda_status st = slots_check(d.B, slots, num_slots, state_in, state_out);
    if (st != KDA_OK) return st;
    if (d.K > 128 || d.V > 128 || d.K % 16 || d.V % 16 || (long long)d.B * d.H > (1LL << 30)) return KDA_ERR_UNSUPPORTED;
    StepArgs a;
    memset(&a, 0, sizeof(a));
    a.B = d.B; a.H = d.H; a.Hk = Hk; a.K = d.K; a.V = d.V; a.dtype = d.dtype; a.gate = d.gate;
    a.q = q; a.k = k; a.v = v; a.g_raw = g_raw; a.beta_raw = beta_raw; a.a_log = a_log; a.dt_bias = dt_bias;
    a.scale = scale; a.lb = lower_bound; a.slots = slots; a.num_slots = num_slots; a.s_in = state_in;
    a.s_out = state_out; a.out = out;
    st = status_ptr(&a.status);
    if (st != KDA_OK) return st;
    const dim3 grid(d.B * d.H, (d.V + kStepTile - 1) / kStepTile);
    timing_pre(stream, K_DECODE_STEP);
    if (pool_vec_ok(a)) decode_step_kernel<4><<<grid, kStepThreads, 0, stream>>>(a);
    else decode_step_kernel<1><<<grid, kStepThreads, 0, stream>>>(a);
    timing_post(stream);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_ssm_step(const kda_ssm_dims* dims, const void* x, const void* dt_raw, const void* b, const void* c,
                        const float* a_log, const float* dt_bias, const float* d_skip, const int32_t* slots,
                        int num_slots, const float* state_in, float* state_out, void* y, cudaStream_t stream) {
    if (!dims || dims->T != 1) return KDA_ERR_INVALID_ARG;
    SsmShape s;
    kda_status st = ssm_check(dims, false, x, dt_raw, b, c, a_log, dt_bias, &s);
    if (st != KDA_OK) return st;
    if (!y) return KDA_ERR_INVALID_ARG;
    st = slots_check(s.B, slots, num_slots, state_in, state_out);
    if (st != KDA_OK) return st;
    StepArgs a;
    memset(&a, 0, sizeof(a));
    a.B = s.B; a.H = s.H; a.G = s.G; a.K = s.N; a.V = s.P; a.dtype = s.dtype;
    a.xs = s.xs; a.bs = s.bs; a.cs = s.cs; a.ds = s.ds;
    a.q = c; a.k = b; a.v = x; a.beta_raw = dt_raw; a.a_log = a_log; a.dt_bias = dt_bias; a.d_skip = d_skip;
    a.slots = slots; a.num_slots = num_slots; a.s_in = state_in; a.s_out = state_out; a.out = y;
    st = status_ptr(&a.status);
    if (st != KDA_OK) return st;
    const dim3 grid(s.B * s.H, (s.P + kStepTile - 1) / kStepTile);
    timing_pre(stream, K_SSM_STEP);
    if (pool_vec_ok(a)) ssm_step_kernel<4><<<grid, kStepThreads, 0, stream>>>(a);
    else ssm_step_kernel<1><<<grid, kStepThreads, 0, stream>>>(a);
    timing_post(stream);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
