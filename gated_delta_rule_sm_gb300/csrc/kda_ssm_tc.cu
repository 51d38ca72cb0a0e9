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
// M is written over G, 16 fp32 columns of G giving 8 + 8 packed columns for the two heads.  The state
// stays in fp32 registers; its two bf16 copies in shared memory are the B operands of C S.
// Precision: M is rounded to bf16 (relative 2^-9 of each term of y, which is bf16 itself: 12 documents of 16384 tokens
// are 1.72e-3 of the norm from 64 bits, 1.66e-3 of which the storage alone takes); C S takes S as
// two bf16 values, a buffer each: with one, a large entering state alone cost y up to
// 0.04 of its rms.  The state is an fp32 result, so U is kept as the sum of three bf16 values (24 bits) and X and
// B are exact: two values would leave 1.5e-6 of the state, three leave fp32 rounding.
// Decays: log2 units, every sum taken inside blocks of 32 tokens and extended by whole blocks' sums; a token's
// exponent is cut at -150 (2^-150 is 0 in fp32).  Only on M's diagonal blocks is an exponent the difference of two sums,
// of at most 32 tokens: 4800 at the cut, where it is 2^-12 off, an eighth of M's rounding.
//
// Roles (24 warps): 0-7 form M (two warpgroups, which split the columns) and finish Y (a head each); 8-11 form
// U, a quarter of a chunk at a time; 12-19 scale C S and keep the state (half a row a thread); 20 issues G,
// C S and M X, 21 the copies, 22 prepares the decays, 23 issues U^T B.  Roles meet at mbarriers only.
// The pass that only forms states has no G, M, C S or Y: its first three warpgroups all form U, in four
// TMEM buffers, with three stages of X and B.  Its U^T B is issued by warps 20 and 23, a chunk each in turn:
// one thread takes some 1000 cycles for the six products of a quarter, tensor time 400.
// TMEM columns: G / M 128, Y 128, U^T B 128, U 2 x 48.
// Bound: per chunk and unit 29 MFLOP (the state's three terms 12.6, C S 8.4) against 64 KB of x and y: 2.3 us and
// 1.5 us of an SM's share at the measured rates.  Measured on a row of 65536 tokens, 32 heads, N 128, P 64: 218
// us for the outputs, 3.8 us a chunk, and 109 us for the states, 1.9 us a chunk.  What holds the output pass is
// shared memory: 320 KB of operands and 128 KB of copies at 128 bytes a cycle and 3200 accesses of the warps, some 6600
// of a chunk's 7300 cycles.  The source asks for about 1650 of those accesses (M's factors 160, Y 512, the copies of S
// 512, U's loads 256); the other 1500 are conflicts or replays whose cause has not been found.  And the roles' loops together fill the instruction cache, which is why
// they are kept short (M unrolled over its 32 columns and two copies of copy_state: 222 us).
#include <cudaTypedefs.h>
#include <string.h>

#include <type_traits>

#include "kda.h"
#include "kda_sm100.cuh"
#include "kda_ssm.h"

namespace kda {

using namespace sm100;

namespace {

constexpr int Q = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 768;

// A slot's decays: [0] lb - log2 D, [128] D 2^(sum to the chunk's end), [256] lb = running sum inside the
// block of 32 tokens, [384] D 2^(sum to the block's end), [512..515] the blocks' sums, [516] 2^(chunk's sum)
constexpr int kPrepFloats = 528;
constexpr int kPrepBufs = 4;

// Shared memory (bytes).  HALF: a tile of 128 rows of 128 bytes (64 bf16 columns).
constexpr uint32_t HALF = 16384;
template <int NB, bool OUT> struct Lay {
    static constexpr int STAGES = OUT ? 2 : 3;
    static constexpr int BSTAGES = OUT ? 1 : 3;
    static constexpr uint32_t X = 0;                               // STAGES x 2 halves
    static constexpr uint32_t B = X + STAGES * 2 * HALF;           // BSTAGES x NB halves
    static constexpr uint32_t C = B + BSTAGES * NB * HALF;         // NB halves
    static constexpr uint32_t SB = C + (OUT ? NB * HALF : 0);      // 2 x NB halves: S^T cut to bf16, and the rest
    static constexpr uint32_t PREP = SB + (OUT ? 2 * NB * HALF : 0);   // kPrepBufs x 2 slots
    static constexpr uint32_t BAR = PREP + kPrepBufs * 2 * 4 * kPrepFloats;
    static constexpr uint32_t TOTAL = BAR + 512;
};

enum Bars {
    kFull = 0,        // [3] X of a stage landed (states only: and B)
    kStage = 3,       // [3] states only: the stage's last product complete
    kYOut = 6,        // [2] y over the stage's X (8 warps)
    kXRead = 8,       // [2] U has read the stage's X (4 warps)
    kPrepFull = 10,   // [4]
    kPrepEmpty = 14,  // [4] 20 warps
    kUFull = 18,      // [4] a quarter of U written (4 warps)
    kUEmpty = 22,     // [4] its product complete
    kBFull = 26,      // B landed
    kBEmpty = 27,     // B read (G and U^T B complete)
    kCFull = 28,      // C landed
    kCEmpty = 29,     // C read (G and C S complete)
    kG = 30,          // G complete
    kSB = 31,         // S copied (8 warps)
    kY2 = 32,         // C S complete
    kM = 33,          // [2] half the columns of M written (8 warps)
    kMX = 35,         // M X complete
    kYRead = 36,      // Y read (8 warps)
    kD3 = 37,         // [2] U^T B complete
    kD3Free = 39,     // [2] read (8 warps)
    kTail = 41,       // X and B past the end cleared (8 warps)
    kYS = 42,         // C S scaled (8 warps)
    kBars = 43
};

// TMEM columns
constexpr uint32_t TG = 0, TY = 128, TD = 256, TU = 384, TCOLS = 512;

// Low word of a shared-memory operand descriptor, 128-byte swizzle (tiles are 1 KB aligned), and the high
// word, which is one for all.  A step inside a tile adds to the low word; the sum is formed beside its one
// use so that a loop's steps do not occupy registers.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return (addr >> 4) | (lbo >> 4 << 16); }
constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);

// D[tmem] (+)= A[smem] * B[smem]^T, issued by one thread; a, b: low descriptor words, oa, ob: bytes from them.
template <int OA, int OB>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 da, db;\n\tadd.u32 x, %1, %5;\n\tadd.u32 y, %2, %6;\n\t"
        "mov.b64 da, {x, %7};\n\tmov.b64 db, {y, %7};\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(OA >> 4), "n"(OB >> 4), "r"(kDescHi));
}
// D[tmem] (+)= A[tmem] * B[smem]^T
template <int OB>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b32 y;\n\t.reg .b64 db;\n\tadd.u32 y, %2, %5;\n\tmov.b64 db, {y, %6};\n\t"
        "setp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(OB >> 4), "r"(kDescHi));
}

// Calls f with 0 .. N - 1 as constants.
template <int N, typename F, int I = 0>
__device__ __forceinline__ void steps(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>());
        steps<N, F, I + 1>(static_cast<F&&>(f));
    }
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(src))
                 : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The two values of a packed bf16 pair; what is left of a pair of fp32 values beside it.
__device__ __forceinline__ float2 bf2(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
__device__ __forceinline__ float2 rest2(float2 u, uint32_t w) { return fma2(bf2(w), dup(-1.f), u); }

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Four 8 x 8 blocks of 16-bit values, transposed; lane i gives the address of row i % 8 of block i / 8.
__device__ __forceinline__ void ldmatrix4t(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// 16 lanes x 16 columns: word w of lane l from thread 4 (l % 8) + w % 4, register 2 (w / 4) + l / 8.
__device__ __forceinline__ void tmem_st_16x16(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// softplus(x) = max(x, 0) + log1p(e^-|x|) to about 2 ulp: e^-|x| from a product split in two, log1p(e) from
// the series of 2 artanh(e / (2 + e)), whose argument is at most 1/3.
__device__ __forceinline__ float step_of(float x) {
    const float y = fmaxf(-fabsf(x), -200.f), t = y * kLog2e;
    constexpr float low = (float)(1.4426950408889634074 - (double)kLog2e);      // log2(e) less its fp32 value
    const float r = fmaf(y, kLog2e, -t) + y * low;
    float e = ex2(t);
    e = fmaf(e * 0.6931471806f, r, e);
    const float z = __fdividef(e, 2.f + e), q = z * z;
    float s = 1.f / 15.f;
    s = fmaf(s, q, 1.f / 13.f);
    s = fmaf(s, q, 1.f / 11.f);
    s = fmaf(s, q, 1.f / 9.f);
    s = fmaf(s, q, 1.f / 7.f);
    s = fmaf(s, q, 1.f / 5.f);
    s = fmaf(s, q, 1.f / 3.f);
    s = fmaf(s, q, 1.f);
    const float l = fmaf(2.f * z, s, fmaxf(x, 0.f));
    return x != x ? x : l;
}

// Shared memory by 32-bit address: fewer registers than a pointer, and nothing to keep across a loop.
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 lds4f(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float lds1f(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, const uint32_t* v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// Byte of 16-byte chunk j of row r in a HALF tile; from the address of chunk 0, chunk j is that XOR 16 j.
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

// The decays of a chunk's slot.
template <int NB, bool SAME, bool OUT>
__device__ __forceinline__ float* prep_slot(uint8_t* smem, int c, int s) {
    return reinterpret_cast<float*>(smem + Lay<NB, OUT>::PREP) + ((c & (kPrepBufs - 1)) * 2 + (SAME ? 0 : s)) * kPrepFloats;
}

template <int NB, bool SAME, bool OUT>
__global__ void __launch_bounds__(kThreads, 1)
ssm_tc_kernel(const __grid_constant__ SsmArgs a, const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mb,
              const __grid_constant__ CUtensorMap mc, const __grid_constant__ CUtensorMap my) {
    using L = Lay<NB, OUT>;
    constexpr int NC = 64 * NB;                      // padded state columns
    constexpr int NST = L::STAGES;
    constexpr uint32_t U0 = OUT ? TU : 0;            // two U buffers, or four where G, M and Y leave their columns
    constexpr int ND = OUT ? 1 : 2;                  // accumulators of U^T B
    constexpr uint32_t D0 = OUT ? TD : 192;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int seg = blockIdx.x;
    const SsmSeg sg = ssm_segment(a, seg, reinterpret_cast<SsmSeg*>(smem + L::BAR + 8 * kBars + 16));
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
    float* ptot = reinterpret_cast<float*>(smem + L::BAR + 8 * kBars + 8);    // [2 slots]

    if (tid == 0) {
#pragma unroll 1
        for (int i = 0; i < kBars; ++i) {
            int cnt = 1;
            if (i == kYOut || i == kYOut + 1 || i == kM || i == kM + 1 || i == kYRead || i == kTail || i == kSB || i == kYS || i == kD3Free ||
                i == kD3Free + 1)
                cnt = 8;
            if (i == kXRead || i == kXRead + 1 || (i >= kUFull && i < kUFull + 4)) cnt = 4;
            if (i == kBEmpty) cnt = 2;
            if (i >= kPrepEmpty && i < kPrepEmpty + 4) cnt = 20;
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

    // Bounded waits (one in good order takes microseconds; a try suspends the thread for ten at most, so that a wait gives
    // up after about a second);
    // false, and the CTA marked as failed, where one gives up: its role then leaves its loop, and
    // the roles that wait for it give up in turn.  Kept short: they are inlined some thirty times, and the
    // code of all roles' loops has to stay in the instruction cache.
    constexpr uint32_t kTries = 1u << 17;
    auto wait1 = [&](int b, uint32_t parity) {
        if (mbar_test_wait(&bar[b], parity)) return true;
#pragma unroll 1
        for (uint32_t i = 0; i < kTries; ++i)
            if (mbar_try_wait_ns(&bar[b], parity, 10000)) return true;
        *fail = 1;
        return false;
    };
    auto wait = [&](int b, uint32_t parity) {      // one answer for the whole warp
        if (__all_sync(0xffffffffu, mbar_test_wait(&bar[b], parity))) return true;
#pragma unroll 1
        for (uint32_t i = 0; i < kTries; ++i)
            if (__all_sync(0xffffffffu, mbar_try_wait_ns(&bar[b], parity, 10000))) return true;
        *fail = 1;
        return false;
    };
    auto arrive_warp = [&](int b) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[b]);
    };
    auto chunk_len = [&](int c) { return min(Q, sg.t1 - (sg.t0 + c * Q)); };
    auto slot_prep = [&](int c, int s) { return prep_slot<NB, SAME, OUT>(smem, c, s); };
    auto wait_prep = [&](int c) { return wait(kPrepFull + (c & 3), (c >> 2) & 1); };

    // The barriers' parities tell a phase from its neighbours only, so nobody may be two phases ahead of or
    // behind one it waits for: every waiter of a stage has a part in the work that its next load waits for, and a
    // U buffer's former use but one is complete by the order of the products (outputs) or by the wait for the
    // last chunk but one (states only).
    // A quarter of U, transposed: rows (slot, p) 32 (warp % 4) .., 32 tokens, as three bf16 terms in TMEM.  The
    // tile is read through transposing 8 x 8 loads, so that a thread's word holds two tokens of one row.
    auto u_quarter = [&](int c, int st, int q) {
        const int k = 4 * c + q, b = OUT ? k & 1 : 2 * (c & 1) + (q & 1), lq = warp & 3;
        if (OUT ? k >= 2 && !wait(kUEmpty + b, ((k >> 1) - 1) & 1) : q >= 2 && !wait(kUEmpty + b, 0)) return false;
        tc_fence_after();
        const float* w = slot_prep(c, lq >> 1) + 128 + 32 * q + 2 * (lane & 3);
        float2 wk[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) wk[i] = *reinterpret_cast<const float2*>(w + 8 * i);
        const uint32_t x0 = smem_u32(smem + L::X + (2 * st + (lq >> 1)) * HALF) + q * 4096 + (lane >> 4) * 1024 + (lane & 7) * 128;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {      // 16 rows
            uint32_t x[8], hi[8], mid[8], lo[8];
            const uint32_t at = x0 + ((((lq & 1) * 4 + 2 * hh + ((lane >> 3) & 1)) ^ (lane & 7)) << 4);
            ldmatrix4t(at, x);
            ldmatrix4t(at + 2048, x + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float2 u = mul2(bf2(x[i]), wk[i >> 1]);
                hi[i] = pack_bf16(u.x, u.y);
                u = rest2(u, hi[i]);
                mid[i] = pack_bf16(u.x, u.y);
                u = rest2(u, mid[i]);
                lo[i] = pack_bf16(u.x, u.y);
            }
            const uint32_t tu = tmem + U0 + 48 * b + ((uint32_t)(lq * 32 + 16 * hh) << 16);
            tmem_st_16x16(tu, hi);
            tmem_st_16x16(tu + 16, mid);
            tmem_st_16x16(tu + 32, lo);
        }
        tmem_st_wait();
        tc_fence_before();
        arrive_warp(kUFull + b);
        return true;
    };
    // What lies past the end of the row may be another document's and no number: X and B there become zeros,
    // which cannot spoil a sum by meeting M's or U's zeros.  Eight warps, one row and one half tile each thread.
    auto clear_tail = [&](int c, int st) {
        const int len = chunk_len(c), row = tid & 127, half = tid >> 7;
        if (len == Q) return true;
        if (!wait(kFull + st, (c / NST) & 1) || (OUT && !wait(kBFull, c & 1))) return false;
        if (row >= len)
#pragma unroll 1
            for (int j = 0; j < 128; j += 16) {
                const uint32_t zero[4] = {0, 0, 0, 0};
                sts128(smem_u32(smem + L::X + (2 * st + half) * HALF) + row * 128 + j, zero);
                if (half < NB) sts128(smem_u32(smem + L::B + ((OUT ? 0 : NB * st) + half) * HALF) + row * 128 + j, zero);
            }
        fence_async_smem();
        arrive_warp(kTail);
        return true;
    };

    // registers by role (the launch has 768 x 80): 256 x 72 + 128 x 64 + 256 x 104 + 128 x 64
    if (NB == 2) {
        if (warp >= 20) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        else if (warp >= 12) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        else if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    }

    if (!OUT && warp < 12) {
        // ---------------------------------------------------------------- states only: quarter k by warpgroup k % 3
        const int wg = warp >> 2;
        for (int c = 0, st = 0; c < nch; ++c, st = st + 1 == NST ? 0 : st + 1) {
            if (!wait_prep(c) || !wait(kFull + st, (c / NST) & 1)) break;
            if (c > 1 && !wait(kD3 + (c & 1), ((c >> 1) - 1) & 1)) break;    // chunk c - 2 has left the U buffers
            if (wg < 2 && !clear_tail(c, st)) break;
            if (chunk_len(c) < Q && !wait(kTail, 0)) break;
            bool ok = true;
#pragma unroll 1
            for (int q = 0; q < 4 && ok; ++q)
                if ((4 * c + q) % 3 == wg) ok = u_quarter(c, st, q);
            if (!ok) break;
            arrive_warp(kPrepEmpty + (c & 3));
        }
    } else if (warp < 8) {
        // ---------------------------------------------------------------- M
        const int wg = warp >> 2, lq = warp & 3;
        const int row = 32 * lq + lane;              // token of the chunk
        const uint32_t lanes = (uint32_t)(lq * 32) << 16;
        constexpr uint32_t PS = SAME ? 0 : 4 * kPrepFloats;
        const uint32_t ty = tmem + TY + lanes + 64 * wg;
        const int hy = wg ? un.h[1] : un.h[0];
        const float dsk = a.d_skip && hy >= 0 ? a.d_skip[hy] : 0.f;
        for (int c = 0; c < nch; ++c) {
            const uint32_t pr = smem_u32(slot_prep(c, 0));
            if (!wait_prep(c) || !clear_tail(c, c & 1)) break;
            // the row's exponents while G is formed: from its block's start (lt), and from the end of each column
            // block of this warpgroup that lies before the diagonal (lj)
            float lt[2], lj[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const float4 sum = lds4f(pr + s * PS + 4 * 512);
                lt[s] = lds1f(pr + s * PS + 4 * (256 + row));
                // blocks 0 and 3 (wg 0) or 1 and 2: what lies between the block's end and the row's block
                lj[s] = lt[s] + ((lq > 1 && !wg ? sum.y : 0.f) + (lq > 2 ? sum.z : 0.f));
            }
            if (!wait(kG, c & 1)) break;
            tc_fence_after();
            // (not unrolled: fetching code that all roles' loops cannot keep in the instruction cache
            // costs more than the loop)
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                const int J = 2 * b + (wg ^ b);
                const uint32_t tg = tmem + TG + lanes + 32 * J;
                if (J > lq) {
                    uint32_t m[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) m[i] = 0;
                    tmem_st16(tg, m);
                    tmem_st16(tg + 16, m);
                } else {
                    const bool diag = J == lq;
#pragma unroll 1
                    for (int c0 = 0; c0 < 32; c0 += 16) {
                        float v[16];
                        tmem_ld16(tg + c0, v);
                        uint32_t pc = pr + 4 * ((diag ? 0 : 384) + 32 * J + c0);
                        tmem_ld_wait();
#pragma unroll 1
                        for (int s = 0; s < (SAME ? 1 : 2); ++s, pc += PS) {
                            uint32_t m[8];
                            float4 k[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) k[i] = lds4f(pc + 16 * i);
                            if (diag) {          // an exponential each, columns up to the row
                                const float2 l = dup(s ? lt[1] : lt[0]);
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const float2 x0 = fma2(make_float2(k[i].x, k[i].y), dup(-1.f), l);
                                    const float2 x1 = fma2(make_float2(k[i].z, k[i].w), dup(-1.f), l);
                                    const float2 e0 = mul2(make_float2(v[4 * i], v[4 * i + 1]), make_float2(ex2(x0.x), ex2(x0.y)));
                                    const float2 e1 = mul2(make_float2(v[4 * i + 2], v[4 * i + 3]), make_float2(ex2(x1.x), ex2(x1.y)));
                                    const int j = c0 + 4 * i;
                                    m[2 * i] = pack_bf16(j <= lane ? e0.x : 0.f, j + 1 <= lane ? e0.y : 0.f);
                                    m[2 * i + 1] = pack_bf16(j + 2 <= lane ? e1.x : 0.f, j + 3 <= lane ? e1.y : 0.f);
                                }
                            } else {             // a factor of the column to the block's end, one of the row from there
                                const float2 rf = dup(ex2(b ? (s ? lt[1] : lt[0]) : (s ? lj[1] : lj[0])));
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const float2 e0 = mul2(make_float2(v[4 * i], v[4 * i + 1]), mul2(make_float2(k[i].x, k[i].y), rf));
                                    const float2 e1 = mul2(make_float2(v[4 * i + 2], v[4 * i + 3]), mul2(make_float2(k[i].z, k[i].w), rf));
                                    m[2 * i] = pack_bf16(e0.x, e0.y);
                                    m[2 * i + 1] = pack_bf16(e1.x, e1.y);
                                }
                            }
                            tmem_st8(tg + c0 + 8 * s, m);
                        }
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                arrive_warp(kM + b);
            }
            arrive_warp(kPrepEmpty + (c & 3));
            // Y
            const int st = c & 1, len = chunk_len(c);
            const uint32_t xrow = smem_u32(smem + L::X + (2 * st + wg) * HALF) + sw(row, 0);
            if (!wait(kXRead + st, (c >> 1) & 1) || !wait(kMX, c & 1)) break;
            tc_fence_after();
#pragma unroll 1
            for (int j = 0; j < 8; j += 2) {
                float v[16];
                uint4 u[2];
                tmem_ld16(ty + 8 * j, v);
#pragma unroll
                for (int k = 0; k < 2; ++k) u[k] = lds128(xrow ^ ((j + k) << 4));
                tmem_ld_wait();
                if (j == 6) {
                    tc_fence_before();
                    arrive_warp(kYRead);      // C S of the next chunk may start
                }
                // y over x, which nothing else reads any more
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 y = fma2(dup(dsk), bf2(w[e]), make_float2(v[8 * k + 2 * e], v[8 * k + 2 * e + 1]));
                        o[e] = pack_bf16(y.x, y.y);
                    }
                    sts128(xrow ^ ((j + k) << 4), o);
                }
            }
            if (len == Q) {
                fence_async_smem();       // the copy warp stores the tile
            } else if (row < len && hy >= 0) {
                const int p0 = SAME ? 64 * wg : 0;
                __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + ((size_t)(sg.t0 + c * Q + row) * a.H + hy) * a.P + p0;
#pragma unroll 1
                for (int k = 0; k < 8 && p0 + 8 * k < a.P; ++k) *reinterpret_cast<uint4*>(y + 8 * k) = lds128(xrow ^ (k << 4));
            }
            arrive_warp(kYOut + st);
        }
    } else if (warp < 12) {
        // ---------------------------------------------------------------- U
        for (int c = 0; c < nch; ++c) {
            const int st = c & 1;
            if (!wait_prep(c) || !wait(kFull + st, (c / NST) & 1)) break;
            if (chunk_len(c) < Q && !wait(kTail, 0)) break;
            bool ok = true;
#pragma unroll 1
            for (int q = 0; q < 4 && ok; ++q) ok = u_quarter(c, st, q);
            if (!ok) break;
            arrive_warp(kXRead + st);
            arrive_warp(kPrepEmpty + (c & 3));
        }
    } else if (warp < 20) {
        // ---------------------------------------------------------------- the state (row (slot, p), NC / 2 columns), C S and Y
        // (row: token, 64 columns)
        constexpr int SN = NC / 2;
        const int half = (warp - 12) >> 2, lq = warp & 3, row = 32 * lq + lane, srow = row >> 6, p = SAME ? row : row & 63;
        const int h = srow ? un.h[1] : un.h[0];
        float S[SN];
        {
            const float* from = OUT && h >= 0 && p < a.P ? ssm_entering(a, sg, seg, h) : nullptr;
            const int rows = from ? a.N - SN * half : 0;
            from += (size_t)(SN * half) * a.P + p;
#pragma unroll
            for (int j = 0; j < SN; ++j, from += a.P) S[j] = j < rows ? *from : 0.f;
        }
        // the thread's columns are one half tile (SN 64) or half the chunks of one (SN 32)
        const uint32_t sbrow = smem_u32(smem + L::SB + (SN == 64 ? half * HALF : 0)) + sw(row, SN == 64 ? 0 : 4 * half);
        // S cut to bf16, and what the cut left rounded to it, as C S's operands
        auto copy_state = [&]() {
#pragma unroll
            for (int j = 0; j < SN; j += 8) {
                uint32_t o[4], r[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // not before its place: the results of all of S at once would not fit the registers
                    asm volatile("" : "+f"(S[j + 2 * e]), "+f"(S[j + 2 * e + 1]));
                    const float2 v = make_float2(S[j + 2 * e], S[j + 2 * e + 1]);
                    o[e] = __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632);
                    const float2 d = rest2(v, o[e]);
                    r[e] = pack_bf16(d.x, d.y);
                }
                const uint32_t at = sbrow ^ (j << 1);
                sts128(at, o);
                sts128(at + NB * HALF, r);
            }
            fence_async_smem();
            arrive_warp(kSB);
        };
        const uint32_t ty = tmem + TY + ((uint32_t)(lq * 32) << 16) + 64 * half;
        for (int c = 0; c < nch; ++c) {
            const uint32_t par = c & 1;
            if (OUT) copy_state();      // (C S has read the last copies)
            if (!wait_prep(c)) break;
            if (OUT) {     // C S scaled by exp(l_t)
                const uint32_t pr = smem_u32(slot_prep(c, half));
                const float4 sum = lds4f(pr + 4 * 512);
                const float l = lds1f(pr + 4 * (256 + row)) + (((lq > 0 ? sum.x : 0.f) + (lq > 1 ? sum.y : 0.f)) + (lq > 2 ? sum.z : 0.f));
                const float2 el = dup(ex2(l));
                if (!wait(kY2, par)) break;
                tc_fence_after();
#pragma unroll 1
                for (int j = 0; j < 64; j += 16) {
                    float v[16];
                    uint32_t r[16];
                    tmem_ld16(ty + j, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float2 y = mul2(make_float2(v[i], v[i + 1]), el);
                        r[i] = __float_as_uint(y.x);
                        r[i + 1] = __float_as_uint(y.y);
                    }
                    tmem_st16(ty + j, r);
                }
                tmem_st_wait();
                tc_fence_before();
                arrive_warp(kYS);
            }
            if (!wait(kD3 + c % ND, (c / ND) & 1)) break;
            tc_fence_after();
            {
                const float2 eq = dup(lds1f(smem_u32(slot_prep(c, srow)) + 4 * 516));
                const uint32_t td = tmem + D0 + 128 * (c % ND) + SN * half + ((uint32_t)(lq * 32) << 16);
#pragma unroll
                for (int j = 0; j < SN; j += 16) {
                    float v[16];
                    tmem_ld16(td + j, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float2 n = fma2(eq, make_float2(S[j + i], S[j + i + 1]), make_float2(v[i], v[i + 1]));
                        S[j + i] = n.x;
                        S[j + i + 1] = n.y;
                    }
                }
            }
            tc_fence_before();
            arrive_warp(kD3Free + c % ND);
            arrive_warp(kPrepEmpty + (c & 3));
        }
        if (*fail == 0) {
            float* to = h < 0 || p >= a.P ? nullptr
                      : OUT ? ssm_leaving(a, sg, seg, h) : a.states + ((size_t)seg * a.H + h) * a.N * a.P;
            const int rows = to ? a.N - SN * half : 0;
            to += (size_t)(SN * half) * a.P + p;
#pragma unroll
            for (int j = 0; j < SN; ++j, to += a.P)
                if (j < rows) *to = S[j];
        }
    } else if (OUT && warp == 20) {
        // ---------------------------------------------------------------- G, C S, M X
        if (lane == 0) {
            constexpr uint32_t idG = idesc_bf16(128, 128, 0, 0), idX = idesc_bf16(128, SAME ? 128 : 64, 0, 1);
            const uint32_t dc = desc_lo(smem_u32(smem + L::C), 16), ds = desc_lo(smem_u32(smem + L::SB), 16);
            const uint32_t db = desc_lo(smem_u32(smem + L::B), 16);
            for (int c = 0; c < nch; ++c) {
                const int st = c & 1;
                const uint32_t dx = desc_lo(smem_u32(smem + L::X + 2 * st * HALF), HALF);
                if (!wait1(kCFull, c & 1) || !wait1(kBFull, c & 1)) break;
                if (c > 0 && !wait1(kMX, (c - 1) & 1)) break;    // M, over which G goes, has been read
                tc_fence_after();
#pragma unroll 1
                for (uint32_t i = 0; i < NB; ++i)
                    steps<4>([&](auto kk) {
                        mma_ss<kk * 32, kk * 32>(tmem + TG, dc + i * (HALF >> 4), db + i * (HALF >> 4), idG, i + kk > 0);
                    });
                mma_commit(&bar[kG]);
                mma_commit(&bar[kBEmpty]);
                if (!wait1(kSB, c & 1) || (c > 0 && !wait1(kYRead, (c - 1) & 1))) break;
                tc_fence_after();
#pragma unroll 1
                for (uint32_t i = 0; i < 2 * NB; ++i)            // S cut to bf16, then the rest
                    steps<4>([&](auto kk) {
                        mma_ss<kk * 32, kk * 32>(tmem + TY, dc + (i % NB) * (HALF >> 4), ds + i * (HALF >> 4), idG, i + kk > 0);
                    });
                mma_commit(&bar[kY2]);
                mma_commit(&bar[kCEmpty]);
                if (!wait1(kFull + st, (c / NST) & 1)) break;
                bool ok = true;
#pragma unroll 1
                for (uint32_t b = 0; b < 2 && ok; ++b) {         // tokens 64 b .. of the sum, as M's halves come
                    ok = wait1(kM + b, c & 1) && (b || wait1(kYS, c & 1));
                    if (!ok) break;
                    tc_fence_after();
                    steps<SAME ? 4 : 8>([&](auto i) {
                        constexpr int sl = i >> 2, kk = i & 3;
                        mma_ts<sl * HALF + kk * 2048>(tmem + TY + 64 * sl, tmem + TG + 64 * b + 16 * kk + 8 * sl,
                                                      dx + b * (8192 >> 4), idX, 1);
                    });
                }
                if (!ok) break;
                mma_commit(&bar[kMX]);
            }
        }
        __syncwarp();
    } else if (warp == 21) {
        // ---------------------------------------------------------------- copies
        if (lane == 0) {
            auto load_b = [&](int c, int st, uint64_t* full) {
#pragma unroll
                for (int i = 0; i < NB; ++i)
                    tma_load_3d(smem + L::B + (NB * st + i) * HALF, &mb, 64 * i, un.g, sg.t0 + c * Q, full);
            };
            auto load = [&](int c) {
                const int st = c % NST, t = sg.t0 + c * Q;
                mbar_expect_tx(&bar[kFull + st], (2 + (OUT ? 0 : NB)) * HALF);
                uint8_t* xs = smem + L::X + 2 * st * HALF;
                tma_load_3d(xs, &mx, 0, un.h[0], t, &bar[kFull + st]);
                // no second head: head index H is out of range, the tile is filled with zeros
                tma_load_3d(xs + HALF, &mx, SAME ? 64 : 0, un.h[1] < 0 ? a.H : un.h[1], t, &bar[kFull + st]);
                if (!OUT) load_b(c, st, &bar[kFull + st]);
            };
            // chunk c's iteration brings what its buffers' last users leave free, in the order they do
#pragma unroll 1
            for (int c = -NST; c < nch; ++c) {
                const bool next = c >= -1 && c + 1 < nch;
                if (OUT && next) {
                    if (c >= 0 && !wait1(kBEmpty, c & 1)) break;
                    mbar_expect_tx(&bar[kBFull], NB * HALF);
                    load_b(c + 1, 0, &bar[kBFull]);
                    if (c >= 0 && !wait1(kCEmpty, c & 1)) break;
                    mbar_expect_tx(&bar[kCFull], NB * HALF);
#pragma unroll
                    for (int i = 0; i < NB; ++i)
                        tma_load_3d(smem + L::C + i * HALF, &mc, 64 * i, un.g, sg.t0 + (c + 1) * Q, &bar[kCFull]);
                }
                if (c >= 0) {
                    const int st = c % NST;
                    if (OUT) {
                        if (!wait1(kYOut + st, (c / NST) & 1)) break;
                        if (chunk_len(c) == Q) {
                            const uint8_t* xs = smem + L::X + 2 * st * HALF;
                            const int t = sg.t0 + c * Q;
                            tma_store_3d(&my, xs, 0, un.h[0], t);
                            if (un.h[1] >= 0) tma_store_3d(&my, xs + HALF, SAME ? 64 : 0, un.h[1], t);
                            bulk_commit();
                            bulk_wait_read0();
                        }
                    } else if (!wait1(kStage + st, (c / NST) & 1)) {
                        break;
                    }
                }
                if (c + NST < nch) load(c + NST);
            }
        }
        __syncwarp();
    } else if (warp == 22) {
        // ---------------------------------------------------------------- decays: half a warp a head, a lane 8 tokens
        const int sl = SAME ? 0 : lane >> 4, l = lane & 15, blk = l >> 2;
        const int h = un.h[sl];
        const bool writes = !SAME || lane < 16;
        const float es = h >= 0 ? ssm_rate(a.a_log[h]) * kLog2e : 0.f, bias = h >= 0 ? a.dt_bias[h] : 0.f;
        float total = 0.f;
        const uint16_t* dt = static_cast<const uint16_t*>(a.dt) + (size_t)(sg.t0 + 8 * l) * a.ds + (h >= 0 ? h : 0);
        uint32_t next[8];      // dt_raw, requested a chunk ahead: under load it takes longer than a chunk's decays
        auto fetch = [&](int len) {
#pragma unroll
            for (int e = 0; e < 8; ++e) next[e] = 8 * l + e < len ? dt[e * a.ds] : 0;
        };
        if (nch > 0) fetch(chunk_len(0));
        for (int c = 0; c < nch; ++c) {
            const int len = chunk_len(c);
            float D[8], up[8], dn[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) D[e] = __uint_as_float(next[e] << 16);
            dt += Q * a.ds;
            if (c + 1 < nch) fetch(chunk_len(c + 1));
            if (c >= kPrepBufs && !wait(kPrepEmpty + (c & 3), ((c >> 2) - 1) & 1)) break;
            // running sums from the lane's start (its own token with it) and to its end (without)
            float run = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                D[e] = step_of(D[e] + bias);
                if (h < 0 || 8 * l + e >= len) D[e] = 0.f;
                float la = -es * D[e];
                if (la < -150.f) la = -150.f;      // (a NaN stays one)
                dn[e] = la;
                run += la;
                up[e] = run;
            }
            float back = 0.f;
#pragma unroll
            for (int e = 7; e >= 0; --e) {
                const float la = dn[e];
                dn[e] = back;
                back += la;
            }
            // a block of 32 tokens is four lanes
            float u = run, d = back;
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                const float x = __shfl_up_sync(0xffffffffu, u, o, 4), y = __shfl_down_sync(0xffffffffu, d, o, 4);
                if ((lane & 3) >= o) u += x;
                if ((lane & 3) + o < 4) d += y;
            }
            const float block = __shfl_sync(0xffffffffu, u, 3, 4);
            float before = __shfl_up_sync(0xffffffffu, u, 1, 4), after = __shfl_down_sync(0xffffffffu, d, 1, 4);
            if ((lane & 3) == 0) before = 0.f;
            if ((lane & 3) == 3) after = 0.f;
            const float b0 = __shfl_sync(0xffffffffu, block, 0, 16), b1 = __shfl_sync(0xffffffffu, block, 4, 16);
            const float b2 = __shfl_sync(0xffffffffu, block, 8, 16), b3 = __shfl_sync(0xffffffffu, block, 12, 16);
            const float rest = blk == 0 ? (b1 + b2) + b3 : blk == 1 ? b2 + b3 : blk == 2 ? b3 : 0.f;
            const float sum = (b0 + b1) + (b2 + b3);
            float* pr = slot_prep(c, sl);
            if (writes) {
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    float4* o = reinterpret_cast<float4*>(pr + 8 * l + e);
                    float s[4], p[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s[i] = after + dn[e + i];
                        p[i] = before + up[e + i];
                    }
                    const float* De = D + e;
                    o[32] = make_float4(De[0] * ex2(rest + s[0]), De[1] * ex2(rest + s[1]), De[2] * ex2(rest + s[2]),
                                        De[3] * ex2(rest + s[3]));
                    if (OUT) {
                        o[0] = make_float4(p[0] - __log2f(De[0]), p[1] - __log2f(De[1]), p[2] - __log2f(De[2]),
                                           p[3] - __log2f(De[3]));
                        o[64] = make_float4(p[0], p[1], p[2], p[3]);
                        o[96] = make_float4(De[0] * ex2(s[0]), De[1] * ex2(s[1]), De[2] * ex2(s[2]), De[3] * ex2(s[3]));
                    }
                }
                if (l == 0) {
                    *reinterpret_cast<float4*>(pr + 512) = make_float4(b0, b1, b2, b3);
                    pr[516] = exp2f(sum);
                }
            }
            total += sum;
            arrive_warp(kPrepFull + (c & 3));
        }
        if (!OUT && l == 0 && writes) ptot[sl] = total;
    } else if (warp == 23 || (!OUT && warp == 20)) {
        // ---------------------------------------------------------------- U^T B
        // (states only: the two warps take every other chunk, each with its accumulator and U buffers)
        if (lane == 0) {
            constexpr uint32_t idU = idesc_bf16(128, NC, 0, 1);
            for (int c = !OUT && warp == 20; c < nch; c += OUT ? 1 : 2) {
                const int st = c % NST;
                const uint32_t sbt = smem_u32(smem + L::B + (OUT ? 0 : NB * st) * HALF);
                bool ok = OUT ? wait1(kBFull, c & 1) : wait1(kFull + st, (c / NST) & 1);
#pragma unroll 1
                for (int q = 0; q < 4 && ok; ++q) {
                    const int b = OUT ? q & 1 : 2 * (c & 1) + (q & 1);
                    if (!wait1(kUFull + b, q >> 1)) { ok = false; break; }
                    if (q == 0 && c >= ND && !wait1(kD3Free + c % ND, (c / ND - 1) & 1)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t db = desc_lo(sbt + q * 4096, HALF);
                    steps<6>([&](auto i) {
                        constexpr int j = i >= 3, term = i - 3 * j;
                        mma_ts<j * 2048>(tmem + D0 + 128 * (c % ND), tmem + U0 + 48 * b + 16 * term + 8 * j, db, idU, q + i > 0);
                    });
                    mma_commit(&bar[kUEmpty + b]);
                }
                if (!ok) break;
                mma_commit(&bar[kD3 + c % ND]);
                mma_commit(&bar[OUT ? kBEmpty : kStage + st]);
            }
        }
        __syncwarp();
    }
    __syncthreads();
    if (!OUT && tid < (SAME ? 1 : 2)) {
        const int h = tid ? un.h[1] : un.h[0];
        if (h >= 0) a.decay[(size_t)seg * a.H + h] = exp2f(ptot[tid]);
    }
    if (*fail && tid == 0) {
        // give copies and products in flight a bounded chance to land before the memory is released
        record_error(a.status, KDA_ERR_TIMEOUT);
#pragma unroll 1
        for (int b = 0; b < kBars; ++b) {
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
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay<NB, OUT>::TOTAL);
    if (e != cudaSuccess) return e;
    kern<<<dim3(a.nseg, ssm_tc_units(a.H, a.G, a.P)), kThreads, Lay<NB, OUT>::TOTAL, st>>>(a, m[0], m[1], m[2], m[3]);
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
