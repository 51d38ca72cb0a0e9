// kda_attn_mma.cu -- attention of a few query rows over paged keys and values: the steps of a decoder.  bf16, D a multiple
// of 8.
//
// One query row per head and token against every key of its sequence: 4 D operations for 4 D bytes of a key and its
// value, times the query heads that share them (and the tokens of a short chunk).  Bound by memory; the warps' matrix
// instructions (m16n8k16) do 16 packed rows at the price of one, which is what there is to hide behind the loads.
//
// A warp is on its own: it takes 16 of a tile's 64 keys, copies them and their values to its own ring in shared memory
// (cp.async, two stages ahead, so that an SM has 128 KB on the way), and keeps its own maxima, sums and output; the
// four warps of a CTA meet when a piece ends.  A lane looks up the page of one key, a stage before its address is needed.
// Measured: one token over 32768 keys, 32 query heads on 8 key heads, D = 128 (134 MB): 30 us of the kernel, of which the copies
// run 22 (6.2 TB/s); 4 go by before the first are issued (lengths and the page table are read one after the other, by all
// CTAs at once) and 3 for the first to arrive.  A batch of 64 such rows of up to 8192 tokens: 148 to 170 us for 0.91 GB, 5.4 to 6.2 TB/s.
// Precision: scores and sums fp32; a weight meets the values as the sum of two bf16 values, off by 2^-16 of it at most (the
// second products cost no time; the output's error is then its own rounding, 0.0017 for 0.0021).  The maximum that scores
// are taken from is raised only when it is passed by more than 8 (in log2): weights up to 2^8 lose nothing in bf16 or fp32, and the output is rescaled a few times, not each tile.
#include <math.h>

#include "kda.h"
#include "kda_attn.h"
#include "kda_common.cuh"
#include "kda_sm100.cuh"

namespace kda {

using namespace sm100;

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps, kGroup = 16;      // kGroup: keys of a warp's step
static_assert(kWarps * kGroup == kAttnMmaKeys, "a tile is a step of the four warps");
constexpr int kRows = kAttnMmaRows;
constexpr float kRaise = 8.f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4t(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// d (16 x 8, fp32) += A (16 x 16) B (16 x 8), bf16
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Byte of 16-byte piece c of row r in a tile of DP columns: the pieces of eight rows lie in different banks.
template <int DP> __device__ __forceinline__ uint32_t piece(int r, int c) { return (uint32_t)(r * DP * 2 + ((c ^ (r & 7)) << 4)); }

template <int DP> struct Lay {
    static constexpr int STAGES = DP == 64 ? 4 : 3;
    static constexpr uint32_t KV = kGroup * DP * 2;                       // keys (or values) of a stage
    static constexpr uint32_t RING = kWarps * STAGES * 2 * KV;            // the warps' rings, then, at a piece's end, their outputs
    static constexpr uint32_t Q = RING;                                   // 16 rows
    static constexpr uint32_t STAT = Q + kRows * DP * 2;                  // [2][kWarps][kRows] maxima, sums
    static constexpr uint32_t TOTAL = STAT + 2 * kWarps * kRows * 4;
    static_assert(RING >= kWarps * kRows * DP * 4, "the outputs fit into the rings");
};

template <int DP>
__global__ void __launch_bounds__(kThreads, DP == 256 ? 1 : 2) attn_mma_kernel(const __grid_constant__ AttnArgs a) {
    using L = Lay<DP>;
    constexpr int KS = DP / 16, NT = DP / 8;
    constexpr bool QREG = DP <= 128;             // Q's fragments stay in registers
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
    __shared__ int64_t own[kAttnDirectRows + 1];
    const AttnUnits units = attn_units(a, own);
    if (units.units <= 0) return;
    const AttnCut cut(a, units.cost(a));
    if (cta >= cut.ctas) return;
    const bool vq = a.qs % 8 == 0 && reinterpret_cast<uintptr_t>(a.q) % 16 == 0;
    const bool vo = reinterpret_cast<uintptr_t>(a.out) % 4 == 0;
    const size_t values = (size_t)a.Hkv * a.pt * a.D * 2;
    const float c = a.scale * 1.4426950408889634f;
    float* stat = reinterpret_cast<float*>(smem + L::STAT);
    const uint32_t ring = sbase + warp * L::STAGES * 2 * L::KV;
    // what a lane reads of a tile: row and piece of its address in the four 8 x 8 blocks
    const int krow = (lane & 7) + ((lane >> 4) << 3), kpiece = (lane >> 3) & 1;       // keys (and, transposed, nothing)
    const int vrow = lane & 15, vpiece = lane >> 4;                                    // values, and Q
    for (AttnWalk p(a, units, cut, cta); p.more(); p.next(a, units)) {
        const AttnRow w = p.w;
        const AttnSpan s = p.s;
        const int n = p.rows(a);
        const int steps = p.t1 - p.t0, first = (s.tile0 + p.t0) * kAttnMmaKeys + warp * kGroup;
        const int32_t* pages = a.table + (size_t)max(w.seq, 0) * a.max_pages;
        const char* pool = static_cast<const char*>(a.pool);

        // the page of this lane's key of step t (lanes 16 apart: the same); -1: none to read
        auto look = [&](int t) {
            const int key = first + t * kAttnMmaKeys + (lane & 15);
            if (t >= steps || key < s.begin || key >= s.end) return -1;
            const int page = pages[key / a.pt];
            if (page < 0 || page >= a.pages) {
                record_error(a.status, KDA_ERR_INVALID_ARG);
                return -1;
            }
            return page;
        };
        auto fetch = [&](int t, int page) {
            if (t < steps) {
                const int key = first + t * kAttnMmaKeys + (lane & 15);
                const int64_t at = page < 0 ? 0 : (((int64_t)page * 2 * a.Hkv + p.head) * a.pt + key % a.pt) * (a.D * 2);
                const uint32_t to = ring + (t % L::STAGES) * 2 * L::KV;
                constexpr int PER = DP / 8, ROUNDS = kGroup * PER / 32;        // pieces of a row; rows of 32 lanes' pieces
#pragma unroll
                for (int j = 0; j < ROUNDS; ++j) {
                    const int r = (j * 32 + lane) / PER, b = (j * 32 + lane) % PER;
                    const int64_t from = __shfl_sync(0xffffffffu, at, r);
                    const bool ok = __shfl_sync(0xffffffffu, page, r) >= 0 && b * 8 < a.D;
                    const char* src = pool + from + (ok ? b * 16 : 0);
                    cp_async16(to + piece<DP>(r, b), src, ok ? 16 : 0);
                    cp_async16(to + L::KV + piece<DP>(r, b), ok ? src + values : src, ok ? 16 : 0);
                }
            }
            cp_commit();
        };
        __syncthreads();          // the last piece's outputs have been read
        int page = look(0);
#pragma unroll
        for (int t = 0; t < L::STAGES - 1; ++t) {
            const int next = look(t + 1);
            fetch(t, page);
            page = next;
        }
        // Q, zeros past its rows and columns
        for (int i = tid; i < kRows * (DP / 8); i += kThreads) {
            const int r = i / (DP / 8), b = i % (DP / 8);
            uint4 f = make_uint4(0, 0, 0, 0);
            if (r < n && b * 8 < a.D) {
                const AttnWalk::Place from = p.place(a, r);
                const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + from.token * a.qs + from.head * a.D + b * 8;
                if (vq) f = *reinterpret_cast<const uint4*>(q);
                else {
                    const unsigned short* e = reinterpret_cast<const unsigned short*>(q);
                    f = make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16, e[4] | (uint32_t)e[5] << 16, e[6] | (uint32_t)e[7] << 16);
                }
            }
            *reinterpret_cast<uint4*>(smem + L::Q + piece<DP>(r, b)) = f;
        }
        __syncthreads();
        uint32_t qf[QREG ? KS : 1][4];
        if constexpr (QREG)
#pragma unroll
            for (int k = 0; k < KS; ++k) ldmatrix4(sbase + L::Q + piece<DP>(vrow, 2 * k + vpiece), qf[k]);

        float o[NT][4], base[2], sum[2];
        int pos[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = h * 8 + (lane >> 2);
            base[h] = -INFINITY;
            sum[h] = 0.f;
            pos[h] = r < n ? p.position(a, r) : -1;
        }
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[k][j] = 0.f;

        for (int t = 0; t < steps; ++t) {
            const int next = look(t + L::STAGES);
            fetch(t + L::STAGES - 1, page);       // into the stage that was read a step ago (by this warp alone)
            page = next;
            cp_wait<L::STAGES - 1>();
            __syncwarp();
            const int k0 = first + t * kAttnMmaKeys;
            if (k0 < s.end) {
                const uint32_t keys = ring + (t % L::STAGES) * 2 * L::KV, vals = keys + L::KV;
                float z[2][4];
#pragma unroll
                for (int j = 0; j < 8; ++j) z[j >> 2][j & 3] = 0.f;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t b[4];
                    ldmatrix4(keys + piece<DP>(krow, 2 * k + kpiece), b);
                    uint32_t q[4];
                    if constexpr (!QREG) ldmatrix4(sbase + L::Q + piece<DP>(vrow, 2 * k + vpiece), q);
                    const uint32_t* f = QREG ? qf[k] : q;
                    mma16816(z[0], f, b[0], b[1]);
                    mma16816(z[1], f, b[2], b[3]);
                }
                uint32_t wgt[4], low[4];
                bool raise = false;
                float top[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    top[h] = -INFINITY;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int key = k0 + (j >> 1) * 8 + 2 * (lane & 3) + (j & 1);
                        float& v = z[j >> 1][2 * h + (j & 1)];
                        v = key > pos[h] || (a.window && key <= pos[h] - a.window) ? -INFINITY : v * c;
                        top[h] = fmaxf(top[h], v);
                    }
                    top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
                    top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
                    raise |= top[h] > base[h] + kRaise;
                }
                if (__any_sync(0xffffffffu, raise))
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float now = top[h] > base[h] + kRaise ? top[h] : base[h];
                        const float f = now == -INFINITY ? 1.f : ex2(base[h] - now);
                        base[h] = now;
                        sum[h] *= f;
#pragma unroll
                        for (int k = 0; k < NT; ++k) {
                            o[k][2 * h] *= f;
                            o[k][2 * h + 1] *= f;
                        }
                    }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float from = base[h] == -INFINITY ? 0.f : base[h];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float *v = z[j] + 2 * h;
                        v[0] = ex2(v[0] - from);
                        v[1] = ex2(v[1] - from);
                        sum[h] += v[0] + v[1];
                        const uint32_t w = pack_bf16(v[0], v[1]);
                        wgt[2 * j + h] = w;
                        low[2 * j + h] = pack_bf16(v[0] - __uint_as_float(w << 16), v[1] - __uint_as_float(w & 0xffff0000u));
                    }
                }
#pragma unroll
                for (int k = 0; k < NT; k += 2) {
                    uint32_t b[4];
                    ldmatrix4t(vals + piece<DP>(vrow, k + vpiece), b);
                    mma16816(o[k], wgt, b[0], b[1]);
                    mma16816(o[k + 1], wgt, b[2], b[3]);
                    mma16816(o[k], low, b[0], b[1]);
                    mma16816(o[k + 1], low, b[2], b[3]);
                }
            }
            __syncwarp();          // all lanes have read the stage that the next step fills
        }
        cp_wait<0>();
        // the warps' outputs, taken from the largest of their maxima
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
            if ((lane & 3) == 0) {
                const int r = h * 8 + (lane >> 2);
                stat[warp * kRows + r] = base[h];
                stat[(kWarps + warp) * kRows + r] = sum[h];
            }
        }
        __syncthreads();
        float* outs = reinterpret_cast<float*>(smem);       // [kWarps][kRows][DP]
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = h * 8 + (lane >> 2);
            if (r >= n) continue;
            float top = -INFINITY;
#pragma unroll
            for (int v = 0; v < kWarps; ++v) top = fmaxf(top, stat[v * kRows + r]);
            const float f = base[h] == -INFINITY ? 0.f : ex2(base[h] - top);
#pragma unroll
            for (int k = 0; k < NT; ++k)
                *reinterpret_cast<float2*>(outs + (warp * kRows + r) * DP + k * 8 + 2 * (lane & 3)) =
                    make_float2(o[k][2 * h] * f, o[k][2 * h + 1] * f);
        }
        __syncthreads();
        if (tid == 0) p.tell_join(a, cut, cta);
        float* part = a.part + p.slot(cta) * attn_part_floats(a);
        for (int i = tid; i < n * (DP / 2); i += kThreads) {
            const int r = i / (DP / 2), d = i % (DP / 2) * 2;
            if (d >= a.D) continue;
            float top = -INFINITY, sum_r = 0.f;
#pragma unroll
            for (int v = 0; v < kWarps; ++v) top = fmaxf(top, stat[v * kRows + r]);
            float2 y = make_float2(0.f, 0.f);
#pragma unroll
            for (int v = 0; v < kWarps; ++v) {
                const float b = stat[v * kRows + r], f = b == -INFINITY ? 0.f : ex2(b - top);
                sum_r = fmaf(stat[(kWarps + v) * kRows + r], f, sum_r);
                const float2 add = *reinterpret_cast<const float2*>(outs + (v * kRows + r) * DP + d);
                y.x += add.x;
                y.y += add.y;
            }
            if (!p.whole()) {
                *reinterpret_cast<float2*>(part + (size_t)r * a.D + d) = y;
                if (d == 0) {
                    part[(size_t)a.block * a.D + r] = top;
                    part[(size_t)a.block * (a.D + 1) + r] = sum_r;
                }
                continue;
            }
            const float inv = sum_r > 0.f ? 1.f / sum_r : sum_r == 0.f ? 0.f : sum_r;
            const AttnWalk::Place to_row = p.place(a, r);
            const size_t at = (size_t)to_row.token * a.Hq + to_row.head;
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + at * a.D + d;
            if (vo) *reinterpret_cast<uint32_t*>(out) = pack_bf16(y.x * inv, y.y * inv);
            else {
                out[0] = __float2bfloat16_rn(y.x * inv);
                out[1] = __float2bfloat16_rn(y.y * inv);
            }
            if (a.lse && d == 0) a.lse[at] = sum_r == 0.f ? -INFINITY : (top + log2f(sum_r)) * 0.6931471805599453f;
        }
    }
}

template <int DP> cudaError_t go(const AttnArgs& a, cudaStream_t st) {
    const cudaError_t e = cudaFuncSetAttribute(attn_mma_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<DP>::TOTAL);
    if (e != cudaSuccess) return e;
    return attn_launch(attn_mma_kernel<DP>, a.ctas, kThreads, Lay<DP>::TOTAL, !a.direct, st, a);
}

}  // namespace

cudaError_t launch_attn_mma(const AttnArgs& a, cudaStream_t st) {
    return a.D > 128 ? go<256>(a, st) : a.D > 64 ? go<128>(a, st) : go<64>(a, st);
}

}  // namespace kda
