// kda_ssm_tc.cu -- the state space scan on the tensor cores (tcgen05, TMEM, TMA): bf16, N, P <= 128.
//
// Chunks of Q = 128 tokens.  With l the running sum of log-decays inside a chunk and D the steps,
//     G    = C B^T                                        [t, s]   one product per chunk, shared by the heads
//     M    = G o exp(l_t - l_s) D_s  (s <= t)             [t, s]
//     Y    = M X + diag(exp(l_t)) (C S) + d X             [t, p]
//     S'   = exp(l_Q) S + U^T B,  U_s = D_s exp(l_Q - l_s) x_s     (kept as S^T: rows p, columns n)
// A CTA walks the chunks of one segment for a unit of 128 columns of x: two heads of one group with
// P <= 64, or one head with P <= 128 (columns past P are zeros that TMA fills in).  Both heads of a unit share
// G, and their states form the 128 rows of one product U^T B.
//
// Operands: B, C and X tiles arrive by TMA with the 128-byte swizzle and are read by the products as they
// are, K-major for G and C S, MN-major (tokens as K) for M X and U^T B.  M and U are A operands in TMEM:
// M is written over G, 32 fp32 columns of G giving 16 + 16 packed columns for the two heads.  The state
// stays in fp32 registers; its bf16 copy in shared memory is the B operand of C S.
// Precision: M is rounded to bf16 (relative 2^-9 of each term of y, which is bf16 itself); C S takes S as
// two bf16 values, one after the other in one buffer: with one, a large entering state alone cost y up to
// 0.04 of its rms.  The state is an fp32 result, so U is kept as the sum of three bf16 values (24 bits) and X and
// B are exact: two values would leave 1.5e-6 of the state, three leave fp32 rounding.
// Decays: log2 units, every sum taken inside blocks of 32 tokens and extended by whole blocks' sums, so no
// exponent is the difference of two large numbers; a token's exponent is cut at -150 (2^-150 is 0 in
// fp32).
//
// Roles (512 threads): warps 0-7 form M, scale C S, update S and finish Y (two warpgroups: columns of G
// and of the state are split between them, Y by head); warps 8-11 form U, a row of the unit per thread,
// 32 tokens at a time into one of two TMEM buffers; warp 12 issues G, C S and M X, warp 13 the copies,
// warp 14 prepares the decays of the next chunk, warp 15 issues U^T B.
// TMEM columns: G / M 128, Y 128, U^T B 128, U 2 x 48.
// Bound: per chunk and unit 25 MFLOP (half of them the state's three-term product) against 64 KB of x and y,
// 1.95 us and 1.49 us of an SM's share at the measured rates.
#include <cudaTypedefs.h>
#include <string.h>

#include "kda.h"
#include "kda_sm100.cuh"
#include "kda_ssm.h"

namespace kda {

using namespace sm100;

namespace {

constexpr int Q = 128;
constexpr float kLog2e = 1.4426950408889634f;

// Shared memory (bytes).  HALF: a tile of 128 rows of 128 bytes (64 bf16 columns).
constexpr uint32_t HALF = 16384;
template <int NB> struct Lay {
    static constexpr uint32_t X = 0;                       // 2 stages x 2 halves
    static constexpr uint32_t B = X + 4 * HALF;            // 2 stages x NB halves
    static constexpr uint32_t C = B + 2 * NB * HALF;       // NB halves
    static constexpr uint32_t SB = C + NB * HALF;          // NB halves: S^T rounded to bf16
    static constexpr uint32_t PREP = SB + NB * HALF;       // 2 buffers x 2 slots x kPrepFloats
    static constexpr uint32_t BAR = PREP + 2 * 2 * 4 * 400;
    static constexpr uint32_t TOTAL = BAR + 256;
};
// A slot's decays: [0] lb - log2 D, [128] D 2^(sum to the chunk's end), [256] lb = running sum inside the
// block of 32 tokens, [384..387] the blocks' sums, [388] 2^(chunk's sum)
constexpr int kPrepFloats = 400;

enum Bars {
    kFull = 0,        // [2] X and B of a stage landed
    kCFull = 2,       // C landed
    kCEmpty = 3,      // C read (G and both C S complete)
    kPrepFull = 4,    // [2]
    kPrepEmpty = 6,   // [2] 12 warps
    kG = 8,           // G complete
    kY2 = 9,          // C S complete
    kM = 10,          // M written and C S scaled (8 warps)
    kMX = 11,         // M X complete
    kUFull = 12,      // [2] a quarter of U written (4 warps)
    kUEmpty = 14,     // [2] its product complete
    kD3 = 16,         // U^T B complete
    kD3Free = 17,     // read (8 warps)
    kSB = 18,         // S copied and Y read (8 warps)
    kYOut = 19,       // [2] y over the stage's X (8 warps)
    kStage = 21,      // [2] states only: the stage's last product complete
    kSBLo = 23,       // the remainder of S copied (8 warps)
    kY2Lo = 24,       // its product complete
    kTail = 25,       // X past the end cleared (8 warps)
    kBars = 26
};

// TMEM columns
constexpr uint32_t TG = 0, TY = 128, TD = 256, TU = 384, TCOLS = 512;

// Shared-memory operand descriptor, 128-byte swizzle (tiles are 1 KB aligned).
__device__ __forceinline__ uint64_t desc128(uint32_t addr, uint32_t lbo) {
    return smem_desc(addr, lbo, 1024) | (2ull << 61);
}

// D[tmem] (+)= A[tmem] * B[smem]^T, issued by one thread.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate));
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(src))
                 : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// softplus, one copy of the code for its four uses
__device__ __noinline__ float step_of(float x) { return softplusf(x); }

// Byte of 16-byte chunk j of row r in a HALF tile.
__device__ __forceinline__ uint32_t sw(int r, int j) { return (uint32_t)(r * 128 + ((j ^ (r & 7)) << 4)); }

struct Unit {
    int h[2];     // heads of the two slots (SAME: one head twice); h[1] < 0: no second head
    int g;
};

template <bool SAME>
__device__ __forceinline__ Unit unit_of(const SsmArgs& a, int u) {
    Unit r;
    const int R = a.H / a.G;
    if (SAME) {
        r.h[0] = r.h[1] = u;
        r.g = u / R;
    } else {
        const int pairs = (R + 1) / 2;
        r.g = u / pairs;
        const int k = 2 * (u - r.g * pairs);
        r.h[0] = r.g * R + k;
        r.h[1] = k + 1 < R ? r.h[0] + 1 : -1;
    }
    return r;
}

template <int NB, bool SAME, bool OUT>
__global__ void __launch_bounds__(512, 1)
ssm_tc_kernel(SsmArgs a, const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mb,
              const __grid_constant__ CUtensorMap mc, const __grid_constant__ CUtensorMap my) {
    using L = Lay<NB>;
    constexpr int NC = 64 * NB;                      // padded state columns
    extern __shared__ __align__(1024) uint8_t smem[];
    const int seg = blockIdx.x;
    const SsmSeg sg = ssm_segment(a, seg);
    if (sg.n < 0) return;
    if (!OUT) {   // the last segment's end state comes from the output pass
        int first;
        const int segs = ssm_row_segments(a, sg.n, &first);
        if (seg == first + segs - 1) return;
    }
    const Unit un = unit_of<SAME>(a, blockIdx.y);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nch = (sg.t1 - sg.t0 + Q - 1) / Q;
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::BAR);
    volatile int* fail = reinterpret_cast<volatile int*>(smem + L::BAR + 8 * kBars);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + L::BAR + 8 * kBars + 4);
    float* prep = reinterpret_cast<float*>(smem + L::PREP);

    if (tid == 0) {
        for (int i = 0; i < kBars; ++i) {
            const int cnt = i == kM || i == kD3Free || i == kSB || i == kYOut || i == kYOut + 1 ||
                            i == kSBLo || i == kTail ? 8
                          : i == kUFull || i == kUFull + 1 ? 4
                          : i == kPrepEmpty || i == kPrepEmpty + 1 ? 12 : 1;
            mbar_init(&bar[i], cnt);
        }
        *fail = 0;
        mbar_fence_init();
    }
    if (warp == 0) tmem_alloc(tslot, TCOLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;

    // Bounded wait of one thread; false once any wait of the CTA has given up.  (Kept short: it is inlined
    // some thirty times, and the loop's code has to stay in the instruction cache.)
    auto wait1 = [&](int b, uint32_t parity) {
        if (mbar_test_wait(&bar[b], parity)) return true;
        for (uint32_t i = 0; i < (1u << 22); ++i) {
            if (mbar_try_wait(&bar[b], parity)) return true;
            if ((i & 255) == 255 && *fail) return false;
        }
        *fail = 1;
        return false;
    };
    // The same with one answer for the whole warp.
    auto wait = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, wait1(b, parity)) != 0; };
    auto arrive_warp = [&](int b) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[b]);
    };
    auto chunk_len = [&](int c) { return min(Q, sg.t1 - (sg.t0 + c * Q)); };
    auto slot_prep = [&](int c, int s) { return prep + ((c & 1) * 2 + (SAME ? 0 : s)) * kPrepFloats; };

    if (warp < 8) {
        // ---------------------------------------------------------------- M, C S, state, Y
        const int wg = warp >> 2, lq = warp & 3;
        const int row = 32 * lq + lane;              // token of the chunk; row (slot, p) of the state
        const uint32_t lanes = (uint32_t)(lq * 32) << 16;
        const int srow = row >> 6, p = SAME ? row : row & 63;
        constexpr int SN = NC / 2;                   // state columns of this thread: SN wg ..
        float S[SN];
        {
            const int h = un.h[srow];
            const float* from = OUT && h >= 0 && p < a.P ? ssm_entering(a, sg, seg, h) : nullptr;
#pragma unroll
            for (int j = 0; j < SN; ++j) {
                const int n = SN * wg + j;
                S[j] = from && n < a.N ? from[(size_t)n * a.P + p] : 0.f;
            }
        }
        // S rounded to bf16, or what that rounding left, as C S's operand
        auto copy_state = [&](bool rest) {
#pragma unroll
            for (int j = 0; j < SN; j += 8) {
                const int n = SN * wg + j;
                uint4 o = pack8_bf16(S + j);
                if (rest) {
                    const uint32_t w[4] = {o.x, o.y, o.z, o.w};
                    float r[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        r[2 * e] = S[j + 2 * e] - __uint_as_float(w[e] << 16);
                        r[2 * e + 1] = S[j + 2 * e + 1] - __uint_as_float(w[e] & 0xffff0000u);
                    }
                    o = pack8_bf16(r);
                }
                *reinterpret_cast<uint4*>(smem + L::SB + (n >> 6) * HALF + sw(row, (n & 63) >> 3)) = o;
            }
            fence_async_smem();
        };
        if (OUT && nch > 0) {
            copy_state(false);
            arrive_warp(kSB);
        }
        for (int c = 0; c < nch; ++c) {
            const uint32_t par = c & 1;
            const int st = c & 1, len = chunk_len(c);
            uint8_t* xh = smem + L::X + (2 * st + wg) * HALF;
            if (!wait(kPrepFull + st, (c >> 1) & 1)) break;
            if (len < Q) {
                // rows past the end may hold another document's values: as zeros they cannot meet M's zeros
                if (!wait(kFull + st, (c >> 1) & 1)) break;
                if (row >= len)
#pragma unroll
                    for (int j = 0; j < 8; ++j) *reinterpret_cast<uint4*>(xh + row * 128 + 16 * j) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
                arrive_warp(kTail);
            }
            if (OUT) {
                const float* pr = slot_prep(c, 0);
                constexpr int PS = SAME ? 0 : kPrepFloats;
                if (!wait(kG, par)) break;
                tc_fence_after();
                // (not unrolled: fetching code that all roles' loops cannot keep in the instruction cache
                // costs more than the loop)
                bool ok = true;
#pragma unroll 1
                for (int b = 0; b < 2; ++b) {
                    const int J = wg == 0 ? 3 * b : 1 + b;
                    const uint32_t tg = tmem + TG + lanes + 32 * J;
                    uint32_t m[16];
                    if (b == 1) {     // C S of the rounded state is complete: its remainder takes the same place
                        ok = wait(kY2, par);
                        if (!ok) break;
                        copy_state(true);
                        arrive_warp(kSBLo);
                    }
                    if (J > lq) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) m[i] = 0;
                        tmem_st16(tg, m);
                        if (!SAME) tmem_st16(tg + 16, m);
                        continue;
                    }
                    float v[32];
                    tmem_ld16(tg, v);
                    tmem_ld16(tg + 16, v + 16);
                    tmem_ld_wait();
                    const int last = J == lq ? lane : 31;    // the diagonal block's columns end at the row
#pragma unroll 1
                    for (int s = 0; s < (SAME ? 1 : 2); ++s) {
                        const float* ps = pr + s * PS;
                        float l = ps[256 + row];             // from the column block's start to the row
                        for (int k = J; k < lq; ++k) l += ps[384 + k];
                        const float4* ld = reinterpret_cast<const float4*>(ps + 32 * J);
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float4 l4 = ld[i >> 2];
                            const float e0 = v[i] * ex2(l - l4.x), e1 = v[i + 1] * ex2(l - l4.y);
                            const float e2 = v[i + 2] * ex2(l - l4.z), e3 = v[i + 3] * ex2(l - l4.w);
                            m[i >> 1] = pack_bf16(i <= last ? e0 : 0.f, i + 1 <= last ? e1 : 0.f);
                            m[(i >> 1) + 1] = pack_bf16(i + 2 <= last ? e2 : 0.f, i + 3 <= last ? e3 : 0.f);
                        }
                        tmem_st16(tg + 16 * s, m);
                    }
                }
                if (!ok) break;
                // C S of this warpgroup's columns, scaled by exp(l_t)
                if (!wait(kY2Lo, par)) break;
                tc_fence_after();
                {
                    float l = pr[wg * PS + 256 + row];
                    for (int k = 0; k < lq; ++k) l += pr[wg * PS + 384 + k];
                    const float el = ex2(l);
                    const uint32_t ty = tmem + TY + lanes + 64 * wg;
#pragma unroll 1
                    for (int j = 0; j < 64; j += 32) {
                        float v[32];
                        tmem_ld16(ty + j, v);
                        tmem_ld16(ty + j + 16, v + 16);
                        tmem_ld_wait();
                        uint32_t r[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i] * el);
                        tmem_st16(ty + j, r);
                        tmem_st16(ty + j + 16, r + 16);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                arrive_warp(kM);
            }
            if (!wait(kD3, par)) break;
            tc_fence_after();
            {
                const float eq = slot_prep(c, srow)[388];
                const uint32_t td = tmem + TD + lanes + SN * wg;
#pragma unroll
                for (int j = 0; j < SN; j += 16) {
                    float v[16];
                    tmem_ld16(td + j, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) S[j + i] = fmaf(eq, S[j + i], v[i]);
                }
            }
            tc_fence_before();
            arrive_warp(kD3Free);
            if (OUT) {
                copy_state(false);
                if (!wait(kMX, par)) break;
                tc_fence_after();
                const int h = un.h[wg];
                const float dsk = a.d_skip && h >= 0 ? a.d_skip[h] : 0.f;
                const uint32_t ty = tmem + TY + lanes + 64 * wg;
#pragma unroll 1
                for (int j = 0; j < 8; j += 4) {
                    float v[32];
                    tmem_ld16(ty + 8 * j, v);
                    tmem_ld16(ty + 8 * j + 16, v + 16);
                    tmem_ld_wait();
                    if (j) {
                        tc_fence_before();
                        arrive_warp(kSB);     // S is copied and Y read: C S of the next chunk may start
                    }
                    // y over x, which nothing else reads any more
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint4* at = reinterpret_cast<uint4*>(xh + sw(row, j + k));
                        const uint4 u = *at;
                        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
                        float y[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            y[2 * e] = fmaf(dsk, __uint_as_float(w[e] << 16), v[8 * k + 2 * e]);
                            y[2 * e + 1] = fmaf(dsk, __uint_as_float(w[e] & 0xffff0000u), v[8 * k + 2 * e + 1]);
                        }
                        *at = pack8_bf16(y);
                    }
                }
                if (len == Q) {
                    fence_async_smem();       // the copy warp stores the tile
                } else if (row < len && h >= 0) {
                    const int p0 = SAME ? 64 * wg : 0;
                    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) +
                                       ((size_t)(sg.t0 + c * Q + row) * a.H + h) * a.P + p0;
#pragma unroll 1
                    for (int k = 0; k < 8 && p0 + 8 * k < a.P; ++k)
                        *reinterpret_cast<uint4*>(y + 8 * k) = *reinterpret_cast<const uint4*>(xh + sw(row, k));
                }
                arrive_warp(kYOut + st);
            }
            arrive_warp(kPrepEmpty + st);
        }
        if (*fail == 0) {
            const int h = un.h[srow];
            float* to = h < 0 || p >= a.P ? nullptr
                      : OUT ? ssm_leaving(a, sg, seg, h) : a.states + ((size_t)seg * a.H + h) * a.N * a.P;
            if (to)
#pragma unroll
                for (int j = 0; j < SN; ++j) {
                    const int n = SN * wg + j;
                    if (n < a.N) to[(size_t)n * a.P + p] = S[j];
                }
        }
    } else if (warp < 12) {
        // ---------------------------------------------------------------- U, transposed: row (slot, p), 32 tokens a quarter
        const int lq = warp & 3, row = 32 * lq + lane;
        const uint32_t lanes = (uint32_t)(lq * 32) << 16;
        for (int c = 0; c < nch; ++c) {
            const int st = c & 1, len = chunk_len(c);
            if (!wait(kFull + st, (c >> 1) & 1) || !wait(kPrepFull + st, (c >> 1) & 1)) break;
            const float* w = slot_prep(c, row >> 6) + 128;
            const uint8_t* xh = smem + L::X + (2 * st + (row >> 6)) * HALF;
            if (len < Q) {
                // B past the end: zeros for the same reason as X there
                if (row >= len)
#pragma unroll
                    for (int j = 0; j < 8 * NB; ++j)
                        *reinterpret_cast<uint4*>(smem + L::B + (NB * st + (j >> 3)) * HALF + row * 128 + 16 * (j & 7)) =
                            make_uint4(0, 0, 0, 0);
                fence_async_smem();
            }
            bool ok = len == Q || wait(kTail, 0);
#pragma unroll 1
            for (int q = 0; q < 4 && ok; ++q) {
                const int b = q & 1, k = 2 * c + (q >> 1);
                if (k > 0 && !wait(kUEmpty + b, (k - 1) & 1)) { ok = false; break; }
                tc_fence_after();
                uint32_t hi[16], mid[16], lo[16];
                const uint32_t pb = 2 * (row & 63);
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 w4 = *reinterpret_cast<const float4*>(w + 32 * q + i);
                    const float wv[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const int t = i + e;      // (32 q is a multiple of 8: the swizzle is the same)
                        const uint32_t x0 = *reinterpret_cast<const uint16_t*>(xh + q * 4096 + t * 128 + (pb ^ ((t & 7) << 4)));
                        const uint32_t x1 = *reinterpret_cast<const uint16_t*>(xh + q * 4096 + (t + 1) * 128 + (pb ^ (((t + 1) & 7) << 4)));
                        float u0 = __uint_as_float(x0 << 16) * wv[e], u1 = __uint_as_float(x1 << 16) * wv[e + 1];
                        const int o = (i + e) >> 1;
                        hi[o] = pack_bf16(u0, u1);
                        u0 -= __uint_as_float(hi[o] << 16);
                        u1 -= __uint_as_float(hi[o] & 0xffff0000u);
                        mid[o] = pack_bf16(u0, u1);
                        u0 -= __uint_as_float(mid[o] << 16);
                        u1 -= __uint_as_float(mid[o] & 0xffff0000u);
                        lo[o] = pack_bf16(u0, u1);
                    }
                }
                const uint32_t tu = tmem + TU + 48 * b + lanes;
                tmem_st16(tu, hi);
                tmem_st16(tu + 16, mid);
                tmem_st16(tu + 32, lo);
                tmem_st_wait();
                tc_fence_before();
                arrive_warp(kUFull + b);
            }
            if (!ok) break;
            arrive_warp(kPrepEmpty + st);
        }
    } else if (warp == 12) {
        // ---------------------------------------------------------------- G, C S, M X
        if (OUT && lane == 0) {
            constexpr uint32_t idG = idesc_bf16(128, 128, 0, 0), idX = idesc_bf16(128, SAME ? 128 : 64, 0, 1);
            const uint32_t sc = smem_u32(smem + L::C), ss = smem_u32(smem + L::SB);
            for (int c = 0; c < nch; ++c) {
                const int st = c & 1;
                const uint32_t sbt = smem_u32(smem + L::B + NB * st * HALF), sx = smem_u32(smem + L::X + 2 * st * HALF);
                if (!wait1(kCFull, c & 1) || !wait1(kFull + st, (c >> 1) & 1)) break;
                if (c > 0 && !wait1(kMX, (c - 1) & 1)) break;    // M, over which G goes, has been read
                tc_fence_after();
#pragma unroll 1
                for (int kk = 0; kk < 4 * NB; ++kk) {
                    const uint32_t o = (kk >> 2) * HALF + (kk & 3) * 32;
                    mma_bf16(tmem + TG, desc128(sc + o, 16), desc128(sbt + o, 16), idG, kk > 0);
                }
                mma_commit(&bar[kG]);
                bool ok = true;
#pragma unroll 1
                for (int part = 0; part < 2 && ok; ++part) {     // S rounded, then the remainder
                    ok = wait1(part ? kSBLo : kSB, c & 1);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int kk = 0; kk < 4 * NB; ++kk) {
                        const uint32_t o = (kk >> 2) * HALF + (kk & 3) * 32;
                        mma_bf16(tmem + TY, desc128(sc + o, 16), desc128(ss + o, 16), idG, part + kk > 0);
                    }
                    mma_commit(&bar[part ? kY2Lo : kY2]);
                }
                if (!ok) break;
                mma_commit(&bar[kCEmpty]);
                if (!wait1(kM, c & 1)) break;
                tc_fence_after();
#pragma unroll 1
                for (int i = 0; i < (SAME ? 8 : 16); ++i) {
                    const int s = i >> 3, kk = i & 7;
                    mma_bf16_ts(tmem + TY + 64 * s, tmem + TG + 32 * (kk >> 1) + 16 * s + 8 * (kk & 1),
                                desc128(sx + s * HALF + kk * 2048, HALF), idX, 1);
                }
                mma_commit(&bar[kMX]);
            }
        }
        __syncwarp();
    } else if (warp == 13) {
        // ---------------------------------------------------------------- copies
        if (lane == 0) {
            auto load = [&](int c) {
                const int st = c & 1, t = sg.t0 + c * Q;
                mbar_expect_tx(&bar[kFull + st], (2 + NB) * HALF);
                uint8_t* xs = smem + L::X + 2 * st * HALF;
                tma_load_3d(xs, &mx, 0, un.h[0], t, &bar[kFull + st]);
                // no second head: head index H is out of range, the tile is filled with zeros
                tma_load_3d(xs + HALF, &mx, SAME ? 64 : 0, un.h[1] < 0 ? a.H : un.h[1], t, &bar[kFull + st]);
                for (int i = 0; i < NB; ++i)
                    tma_load_3d(smem + L::B + (NB * st + i) * HALF, &mb, 64 * i, un.g, t, &bar[kFull + st]);
            };
            auto load_c = [&](int c) {
                mbar_expect_tx(&bar[kCFull], NB * HALF);
                for (int i = 0; i < NB; ++i)
                    tma_load_3d(smem + L::C + i * HALF, &mc, 64 * i, un.g, sg.t0 + c * Q, &bar[kCFull]);
            };
            if (nch > 0) {
                load(0);
                if (OUT) load_c(0);
                if (nch > 1) load(1);
            }
            for (int c = 0; c < nch; ++c) {
                const int st = c & 1;
                if (OUT) {
                    if (c + 1 < nch) {
                        if (!wait1(kCEmpty, c & 1)) break;
                        load_c(c + 1);
                    }
                    if (!wait1(kYOut + st, (c >> 1) & 1)) break;
                    if (chunk_len(c) == Q) {
                        const uint8_t* xs = smem + L::X + 2 * st * HALF;
                        const int t = sg.t0 + c * Q;
                        tma_store_3d(&my, xs, 0, un.h[0], t);
                        if (un.h[1] >= 0) tma_store_3d(&my, xs + HALF, SAME ? 64 : 0, un.h[1], t);
                        bulk_commit();
                        bulk_wait_read0();
                    }
                } else {
                    if (!wait1(kStage + st, (c >> 1) & 1)) break;
                }
                if (c + 2 < nch) load(c + 2);
            }
        }
        __syncwarp();
    } else if (warp == 14) {
        // ---------------------------------------------------------------- decays: lane = 4 tokens
        float total[2] = {0.f, 0.f};
        float ea[2], bias[2];
        uint16_t raw[2][4];       // dt_raw of the chunk to come: requested a chunk ahead
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            ea[s] = un.h[s] >= 0 ? expf(a.a_log[un.h[s]]) * kLog2e : 0.f;
            bias[s] = un.h[s] >= 0 ? a.dt_bias[un.h[s]] : 0.f;
        }
        auto fetch = [&](int c) {
            const int t0 = sg.t0 + c * Q + 4 * lane;
#pragma unroll
            for (int s = 0; s < (SAME ? 1 : 2); ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    raw[s][e] = un.h[s] >= 0 && t0 + e < sg.t1
                                    ? static_cast<const uint16_t*>(a.dt)[(size_t)(t0 + e) * a.ds + un.h[s]] : 0;
        };
        if (nch > 0) fetch(0);
        for (int c = 0; c < nch; ++c) {
            const int st = c & 1, len = chunk_len(c);
            if (c >= 2 && !wait(kPrepEmpty + st, ((c >> 1) - 1) & 1)) break;
            float x[2][4];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[s][e] = __uint_as_float((uint32_t)raw[s][e] << 16) + bias[s];
            if (c + 1 < nch) fetch(c + 1);
#pragma unroll 1
            for (int s = 0; s < (SAME ? 1 : 2); ++s) {
                const int h = s ? un.h[1] : un.h[0];
                float* pr = slot_prep(c, s);
                const float es = s ? ea[1] : ea[0];
                float D[4], la[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    D[e] = h >= 0 && 4 * lane + e < len ? step_of(s ? x[1][e] : x[0][e]) : 0.f;
                    la[e] = -es * D[e];
                    if (la[e] < -150.f) la[e] = -150.f;      // (a NaN stays one)
                }
                // a block of 32 tokens is eight lanes: running sums from its start and to its end
                const float p1 = la[0], p2 = p1 + la[1], p3 = p2 + la[2], p4 = p3 + la[3];
                const float s3 = la[3], s2 = s3 + la[2], s1 = s2 + la[1];
                float up = p4, dn = p4;
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) {
                    const float u = __shfl_up_sync(0xffffffffu, up, o, 8), d = __shfl_down_sync(0xffffffffu, dn, o, 8);
                    if ((lane & 7) >= o) up += u;
                    if ((lane & 7) + o < 8) dn += d;
                }
                const float block = __shfl_sync(0xffffffffu, up, 7, 8);
                float before = __shfl_up_sync(0xffffffffu, up, 1, 8), after = __shfl_down_sync(0xffffffffu, dn, 1, 8);
                if ((lane & 7) == 0) before = 0.f;
                if ((lane & 7) == 7) after = 0.f;
                const float b0 = __shfl_sync(0xffffffffu, block, 0), b1 = __shfl_sync(0xffffffffu, block, 8);
                const float b2 = __shfl_sync(0xffffffffu, block, 16), b3 = __shfl_sync(0xffffffffu, block, 24);
                const int blk = lane >> 3;
                after += blk == 0 ? (b1 + b2) + b3 : blk == 1 ? b2 + b3 : blk == 2 ? b3 : 0.f;
                const float pre[4] = {before + p1, before + p2, before + p3, before + p4};
                float4* o = reinterpret_cast<float4*>(pr + 4 * lane);
                o[0] = make_float4(pre[0] - __log2f(D[0]), pre[1] - __log2f(D[1]), pre[2] - __log2f(D[2]),
                                   pre[3] - __log2f(D[3]));
                o[32] = make_float4(D[0] * ex2(after + s1), D[1] * ex2(after + s2), D[2] * ex2(after + s3), D[3] * ex2(after));
                o[64] = make_float4(pre[0], pre[1], pre[2], pre[3]);
                const float sum = (b0 + b1) + (b2 + b3);
                if (lane == 0) {
                    *reinterpret_cast<float4*>(pr + 384) = make_float4(b0, b1, b2, b3);
                    pr[388] = exp2f(sum);
                }
                if (s) total[1] += sum; else total[0] += sum;
            }
            arrive_warp(kPrepFull + st);
        }
        if (!OUT && lane == 0)
#pragma unroll
            for (int s = 0; s < (SAME ? 1 : 2); ++s)
                if (un.h[s] >= 0) a.decay[(size_t)seg * a.H + un.h[s]] = exp2f(total[s]);
    } else {
        // ---------------------------------------------------------------- U^T B
        if (lane == 0) {
            constexpr uint32_t idU = idesc_bf16(128, NC, 0, 1);
            for (int c = 0; c < nch; ++c) {
                const int st = c & 1;
                const uint32_t sbt = smem_u32(smem + L::B + NB * st * HALF);
                bool ok = wait1(kFull + st, (c >> 1) & 1);
#pragma unroll 1
                for (int q = 0; q < 4 && ok; ++q) {
                    const int b = q & 1, k = 2 * c + (q >> 1);
                    if (!wait1(kUFull + b, k & 1)) { ok = false; break; }
                    if (q == 0 && c > 0 && !wait1(kD3Free, (c - 1) & 1)) { ok = false; break; }
                    tc_fence_after();
#pragma unroll 1
                    for (int i = 0; i < 6; ++i) {
                        const int j = i >= 3, term = i - 3 * j;
                        mma_bf16_ts(tmem + TD, tmem + TU + 48 * b + 16 * term + 8 * j,
                                    desc128(sbt + (2 * q + j) * 2048, HALF), idU, q + i > 0);
                    }
                    mma_commit(&bar[kUEmpty + b]);
                }
                if (!ok) break;
                mma_commit(&bar[kD3]);
                if (!OUT) mma_commit(&bar[kStage + st]);
            }
        }
        __syncwarp();
    }
    __syncthreads();
    if (*fail && tid == 0) {
        // give copies and products in flight a bounded chance to land before the memory is released
        record_error(a.status, KDA_ERR_TIMEOUT);
        for (int b = 0; b < kBars; ++b)
            if (b <= kCFull || (b >= kG && b <= kD3)) {
                mbar_wait(&bar[b], 0, 1u << 12);
                mbar_wait(&bar[b], 1, 1u << 12);
            }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, TCOLS);
}

// ------------------------------------------------------------------ launch

PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

// [TT tokens, `stride` elements apart][heads][cols] bf16 -> boxes of 128 tokens x 1 head x 64 columns in 128-byte
// swizzled rows; columns past `cols`, heads past `heads` and tokens past TT read as zeros.
bool tile_map(CUtensorMap* m, const void* base, int cols, int heads, int TT, int64_t stride) {
    auto enc = map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)heads, (cuuint64_t)TT};
    const cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, Q}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NB, bool SAME, bool OUT>
cudaError_t launch_one(const SsmArgs& a, const CUtensorMap* m, cudaStream_t st) {
    auto kern = ssm_tc_kernel<NB, SAME, OUT>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay<NB>::TOTAL);
    if (e != cudaSuccess) return e;
    kern<<<dim3(a.nseg, ssm_tc_units(a.H, a.G, a.P)), 512, Lay<NB>::TOTAL, st>>>(a, m[0], m[1], m[2], m[3]);
    return cudaGetLastError();
}

}  // namespace

int ssm_tc_units(int H, int G, int P) { return P > 64 ? H : G * ((H / G + 1) / 2); }

bool ssm_tc_ok(const SsmShape& s, const void* x, const void* b, const void* c, const void* y) {
    auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    return s.dtype == KDA_BF16 && s.N <= 128 && s.P <= 128 && s.N % 8 == 0 && s.P % 8 == 0 && s.xs % 8 == 0 &&
           s.bs % 8 == 0 && s.cs % 8 == 0 && s.xs < (1LL << 38) && s.bs < (1LL << 38) && s.cs < (1LL << 38) &&
           al(x) && al(b) && al(c) && al(y);
}

cudaError_t launch_ssm_tc(const SsmArgs& a, bool out, cudaStream_t st) {
    CUtensorMap m[4];
    if (!tile_map(&m[0], a.x, a.P, a.H, a.TT, a.xs) || !tile_map(&m[1], a.b, a.N, a.G, a.TT, a.bs) ||
        !tile_map(&m[2], a.c, a.N, a.G, a.TT, a.cs) || !tile_map(&m[3], a.y, a.P, a.H, a.TT, (int64_t)a.H * a.P))
        return cudaErrorInvalidValue;
    timing_pre(st, out ? K_SSM_OUT : K_SSM_STATE);
    cudaError_t e;
#define KDA_SSM_TC(NB, SAME) (out ? launch_one<NB, SAME, true>(a, m, st) : launch_one<NB, SAME, false>(a, m, st))
    if (a.N <= 64) e = a.P > 64 ? KDA_SSM_TC(1, true) : KDA_SSM_TC(1, false);
    else e = a.P > 64 ? KDA_SSM_TC(2, true) : KDA_SSM_TC(2, false);
#undef KDA_SSM_TC
    timing_post(st);
    return e;
}

}  // namespace kda
