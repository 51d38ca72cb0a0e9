// kda_ssm.h -- what the state space scan's translation units share.
#pragma once

#include "kda_internal.h"

namespace kda {

// One CTA's span of tokens: [t0, t1) of row n, the k-th segment of that row; n < 0: none.
struct SsmSeg {
    int n, t0, t1, k;
};

struct SsmArgs {
    int T, TT, H, G, N, P, dtype, rows;
    int64_t xs, bs, cs, ds;
    const void *x, *dt, *b, *c;
    const float *a_log, *dt_bias, *d_skip, *S0;
    const int32_t* cu;       // [rows + 1] or nullptr
    void* y;
    float* ST;
    // schedule: rows cut into segments of L tokens; nseg entries at most
    int L, per_row, nseg, single;
    const SsmSeg* seg;       // packed documents: the planner's table; nullptr: document i, or the (i % per_row)-th of row i / per_row
    const int32_t* row_seg;  // [rows + 1] first segment of each row (with seg)
    float* states;           // [nseg, H, N, P] end states from zero, then the entering states (not single)
    float* decay;            // [nseg, H] product of the decays of a segment (not single)
    int* status;
};

// Documents that are not cut, and not more of them than this, need no planner: every CTA checks the offsets itself,
// two loads a thread, which saves a launch (12 documents of 16384 tokens in all: 155 -> 150 us; above, each
// CTA's reading costs more than the one planner's).  Offsets that break the contract are recorded and leave
// every row empty, so that its state passes through.  Not inlined: there its registers cost the tensor-core
// kernel's loops 7 %.
constexpr int kSsmOwnRows = 1024;
static __device__ __noinline__ void ssm_document(const SsmArgs& a, int i, SsmSeg* out) {
    bool bad = threadIdx.x == 0 && (a.cu[0] != 0 || a.cu[a.rows] != a.TT);
    for (int n = threadIdx.x; n < a.rows; n += blockDim.x) bad |= a.cu[n + 1] < a.cu[n];
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        if (bad) record_error(a.status, KDA_ERR_INVALID_ARG);
        const SsmSeg s = {i, bad ? 0 : a.cu[i], bad ? 0 : a.cu[i + 1], 0};
        *out = s;
    }
    __syncthreads();
}

// All threads of a CTA call it; tmp: in shared memory.
__device__ __forceinline__ SsmSeg ssm_segment(const SsmArgs& a, int i, SsmSeg* tmp) {
    if (a.seg) return a.seg[i];
    if (a.cu) {
        ssm_document(a, i, tmp);
        return *tmp;
    }
    SsmSeg s;
    s.n = i / a.per_row;
    s.k = i - s.n * a.per_row;
    s.t0 = s.n * a.T + s.k * a.L;
    const long long e = (long long)s.n * a.T + (long long)(s.k + 1) * a.L, last = (long long)(s.n + 1) * a.T;
    s.t1 = (int)(e < last ? e : last);
    return s;
}
// Segments of row n, and the first of them.
__device__ __forceinline__ int ssm_row_segments(const SsmArgs& a, int n, int* first) {
    if (a.cu && !a.seg) {
        *first = n;
        return 1;
    }
    if (a.seg) {
        *first = a.row_seg[n];
        return a.row_seg[n + 1] - *first;
    }
    *first = n * a.per_row;
    return a.per_row;
}

// exp(a_log), kept finite: tokens past a row's end have the step 0, and infinity times that is no number.  Any step
// above 1e-36 forgets everything at the limit as it would at infinity.
__device__ __forceinline__ float ssm_rate(float a_log) {
    const float e = expf(a_log);
    return e > 1e38f ? 1e38f : e;      // (a NaN stays one)
}

// The state a segment starts from (nullptr: zero) and where its end state goes (nullptr: nowhere).
__device__ __forceinline__ const float* ssm_entering(const SsmArgs& a, const SsmSeg& s, int seg, int h) {
    const size_t np = (size_t)a.N * a.P;
    if (a.single) return a.S0 ? a.S0 + ((size_t)s.n * a.H + h) * np : nullptr;
    return a.states + ((size_t)seg * a.H + h) * np;
}
__device__ __forceinline__ float* ssm_leaving(const SsmArgs& a, const SsmSeg& s, int seg, int h) {
    if (!a.ST) return nullptr;
    int first;
    const int n = ssm_row_segments(a, s.n, &first);
    return seg == first + n - 1 ? a.ST + ((size_t)s.n * a.H + h) * a.N * a.P : nullptr;
}

cudaError_t launch_ssm_simt(const SsmArgs& a, bool out, cudaStream_t st);

// The tensor-core kernels: whether they take these arguments, CTAs per segment, launch.
bool ssm_tc_ok(const SsmShape& s, const void* x, const void* b, const void* c, const void* y);
int ssm_tc_units(int H, int G, int P);
cudaError_t launch_ssm_tc(const SsmArgs& a, bool out, cudaStream_t st);

}  // namespace kda
