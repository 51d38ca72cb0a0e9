// kda_attn_tc.cu -- attention of chunks of new tokens over paged keys and values on the tensor cores (tcgen05, TMEM): bf16,
// D <= 128.
//
// A CTA takes 256 packed query rows as two tiles of 128 and walks the key tiles of its piece, 128 keys each:
//     S = Q K^T  (fp32, TMEM),   P = 2^(c S - c m) in bf16 over S's columns,   O += P V  (fp32, TMEM)
// One thread owns one query row: its 128 scores come out of TMEM at once, so that maximum and sum need no exchange.
// The maximum m that scores are taken from is raised only when it is passed by more than 8 in log2; then, a few times in
// a row's life, the row's output is rescaled in TMEM, between the products that add to it.
//
// Operands: K and V lie in one ring of four 32 KB slots (K, V, K, V, ...), rows of 128 bytes in the 128-byte swizzle, put there
// by TMA in boxes of R keys, the largest power of two up to 32 that divides the page's tokens, so that a box lies in one page; a
// lane of the copying warp looks up the page of one box and issues its copy.  With D = 128 and R >= 8 a box holds both halves of its
// keys' columns, 8 keys at a time (WIDE): half as many copies.  Boxes without a key to read, and missing pages, lie out of
// the map's range, which gives zeros.  A box that a row's end (or its window's begin) cuts would bring values that are nobody's, and
// zero times those need not be zero: its values are copied row by row with cp.async, zeros for the others.  K is read
// K-major, V MN-major (keys as K), P from TMEM.
//
// Roles (12 warps): 0-3 and 4-7 the softmax of the two tiles, 8 issues the products, 10 copies keys, 9 values, and
// 9 and 11 Q.  The products come in the order P V and next S of one tile, P V and next S of the other, so that one's run
// while the other's exponentials do.  (A thread for each tile's products, in no order between them, let both tiles fall into
// step: products, then exponentials, 4430 cycles a step.)  P of a tile lies where its next S goes, hence the next S is issued when P
// V is complete.  P is handed over in halves of 64 keys.
// Registers: a softmax thread holds 128 scores, the others little: 208 and 88 (256 x 208 + 128 x 88 = 384 x 168).
// TMEM columns: S (and P) 2 x 128, O 2 x 128.
// Issuing is the products' own bottleneck if it is not looked after: the whole warp runs the loop converged and one lane
// issues, so that descriptors stay in uniform registers (1434 TFLOP/s for 1232 with a single thread's branch), and each tile has
// its copy of the code, so that counters stay in registers (1232 for 1108).
// Bound: per pair of tiles and 128 keys (D = 128) 16.8 MFLOP, 2050 cycles of the tensor core at its dense rate, 256 KB of
// operands and copies through shared memory, 2048 cycles, and beside them 32768 exponentials.  A step takes 3000 cycles: after P V
// of a tile the tensor core waits for its next S to be issued, since TMEM has no room for P beside S and two O.
// Measured, D = 128, 32 query heads, calls with the plan and the join (TFLOP/s; 2012 is what a large library product reaches): 16384
// causal tokens 1480, 8192 tokens after 8192 1535 (with a window of 2048: 948), 8192 tokens over 8 requests with 8192 before each
// 1380; D = 64, 8192 after 8192: 946.  There O takes half its columns, and P still lies over S: the products are half as long, the wait
// of a tile's next S for its P V is not.
#include <math.h>

#include <type_traits>

#include "kda.h"
#include "kda_attn.h"
#include "kda_common.cuh"
#include "kda_sm100.cuh"
#include "kda_tma.h"

namespace kda {

using namespace sm100;

namespace {

constexpr int kThreads = 384, KT = kAttnTcKeys;
constexpr float kRaise = 8.f;
constexpr uint32_t HALF = 16384;       // 128 rows of 128 bytes (64 bf16 columns)

// Shared memory: NB halves of 64 columns of D.
template <int NB> struct Lay {
    static constexpr uint32_t TILE = NB * HALF;
    static constexpr int SLOTS = 4;
    static constexpr uint32_t Q = 0;                          // two tiles
    static constexpr uint32_t KV = 2 * TILE;                  // the ring
    static constexpr uint32_t BAR = KV + SLOTS * TILE;
    static constexpr uint32_t TOTAL = BAR + 256;
};

enum Bars {
    kFull = 0,       // [4] a slot's copies landed
    kEmpty = 4,      // [4] its products complete
    kQFull = 8,      // Q landed (2 warps)
    kQEmpty = 9,     // the piece's products with Q complete
    kS = 10,         // [2] S complete
    kO = 12,         // [2] P V complete
    kP = 14,         // [2][2] half the keys of P written, and O rescaled before (4 warps)
    kOFree = 18,     // [2] the piece's O read (4 warps)
    kBars = 20
};

constexpr uint32_t TS = 0, TO = 256, TCOLS = 512;       // + 128 tile

// (as in the state space scan: low descriptor words with the offsets added beside their use, 128-byte swizzle; sbo: bytes
// between groups of eight rows)
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return (addr >> 4) | (lbo >> 4 << 16); }
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo) { return (sbo >> 4) | (1u << 14) | (2u << 29); }
template <int OA, int OB>
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 x, y;\n\t.reg .b64 da, db;\n\tadd.u32 x, %1, %5;\n\tadd.u32 y, %2, %6;\n\t"
        "mov.b64 da, {x, %7};\n\tmov.b64 db, {y, %8};\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %9, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(OA >> 4), "n"(OB >> 4), "r"(desc_hi(1024)), "r"(hi), "r"(leader));
}
template <int OB>
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 y;\n\t.reg .b64 db;\n\tadd.u32 y, %2, %5;\n\tmov.b64 db, {y, %6};\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(OB >> 4), "r"(hi), "r"(leader));
}
__device__ __forceinline__ void commit(uint32_t leader, uint64_t* mbar) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_u32(mbar)), "r"(leader) : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
    return r;
}
template <int N, typename F, int I = 0>
__device__ __forceinline__ void steps(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>());
        steps<N, F, I + 1>(static_cast<F&&>(f));
    }
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float x, float y, float z) {      // (a NaN counts as nothing, as in fmaxf)
    float m;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
    return m;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return fma2(a, dup(1.f), b); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void tma_load_3d_to(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* mbar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(mbar))
        : "memory");
}

__device__ __forceinline__ void tma_load_5d_to(uint32_t dst, const CUtensorMap* map, int c3, int c4, uint64_t* mbar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(c3), "r"(c4), "r"(smem_u32(mbar))
        : "memory");
}

// Byte of 16-byte piece c (of NB x 8) of row r in a tile of Q, or of keys: halves of 128 rows, or (WIDE) groups of eight rows
// with both halves each.
__device__ __forceinline__ uint32_t piece(int r, int c) { return (c >> 3) * HALF + (uint32_t)(r * 128 + (((c & 7) ^ (r & 7)) << 4)); }

// Values that a load from TMEM has left are used after its wait: the wait alone names no register.
template <int N> __device__ __forceinline__ void landed(float* v) {
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < N; ++j) asm volatile("" : "+f"(v[j]));
}

template <bool WIDE> __device__ __forceinline__ uint32_t key_piece(int r, int c) {
    return WIDE ? (uint32_t)((r >> 3) * 2048 + (c >> 3) * 1024 + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4)) : piece(r, c);
}

template <int NB, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1) attn_tc_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap map, int box_log2) {
    using L = Lay<NB>;
    constexpr int DP = 64 * NB;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int64_t own[kAttnDirectRows + 1];
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::BAR);
    volatile int* fail = reinterpret_cast<volatile int*>(smem + L::BAR + 8 * kBars);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + L::BAR + 8 * kBars + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
    const AttnUnits units = attn_units(a, own);
    if (units.units <= 0) return;
    const AttnCut cut(a, units.cost(a));
    if (cta >= cut.ctas) return;
    if (tid == 0) {
        for (int i = 0; i < kBars; ++i) mbar_init(&bar[i], i >= kP ? 4 : i == kQFull ? 2 : 1);
        *fail = 0;
        mbar_fence_init();
    }
    if (warp == 0) tmem_alloc(tslot, TCOLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;

    // Bounded waits: false, and the CTA marked as failed, after about a second; the role then leaves its loops, and those that
    // wait for it give up in turn.
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

    // Phases: every wait names the use of its barrier that it waits for (the n-th completes parity n & 1), and nobody is two uses
    // behind or ahead: a slot's next use waits for both tiles' products with it, S and P of a tile alternate, O's last phase of
    // a piece is followed by another only after its readers gave O free.
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        // ---------------------------------------------------------------- softmax
        const int tile = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16, ts = tmem + TS + 128 * tile + lanes, to = tmem + TO + 128 * tile + lanes;
        // the scale in log2 units, its sign apart; a scale of 0 leaves every score that is not masked at 0
        const bool negative = a.scale < 0.f;
        const float c = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-30f);
        uint32_t n = 0;                              // key tiles so far
        for (AttnWalk p(a, units, cut, cta); p.more(); p.next(a, units)) {
            const int rows = p.rows(a) - 128 * tile;
            if (rows <= 0) continue;                 // (the other roles leave this tile out as well)
            // (a row past the last sees what that one does, so that it asks for no masks of its own; nothing of it is kept)
            const int pos = p.position(a, 128 * tile + min(row, rows - 1));
            // positions of the warp's rows, for tiles that need no mask
            const int low = __reduce_min_sync(0xffffffffu, pos), high = __reduce_max_sync(0xffffffffu, pos);
            float base = -INFINITY;                  // what scores are taken from (a score, not yet times c)
            float2 sum = make_float2(0.f, 0.f), also = make_float2(0.f, 0.f);
            bool ok = true;
            for (int t = p.t0; t < p.t1; ++t, ++n) {
                const int k0 = (p.s.tile0 + t) * KT;
                if (!wait(kS + tile, n & 1)) { ok = false; break; }
                tc_fence_after();
                float v[KT];
#pragma unroll
                for (int j = 0; j < KT; j += 16) tmem_ld16(ts + j, v + j);
                landed<KT>(v);
                if (negative)
#pragma unroll
                    for (int j = 0; j < KT; ++j) v[j] = -v[j];
                if (k0 + KT - 1 > low || (a.window && k0 <= high - a.window)) {
                    const int last = pos - k0, first = a.window ? last - a.window : -1;      // keys first < j <= last
#pragma unroll
                    for (int j = 0; j < KT; ++j)
                        if (j > last || j <= first) v[j] = -INFINITY;
                }
                float m[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) m[i] = v[i];
#pragma unroll
                for (int j = 8; j + 16 <= KT; j += 16)
#pragma unroll
                    for (int i = 0; i < 8; ++i) m[i] = max3(m[i], v[j + i], v[j + 8 + i]);
#pragma unroll
                for (int i = 0; i < 8; ++i) m[i] = fmaxf(m[i], v[KT - 8 + i]);
                const float top = fmaxf(max3(max3(m[0], m[1], m[2]), m[3], m[4]), max3(m[5], m[6], m[7]));
                const bool raise = top * c > base * c + kRaise;
                if (__any_sync(0xffffffffu, raise)) {
                    const float now = raise ? top : base, f = now == -INFINITY ? 1.f : ex2((base - now) * c);
                    base = now;
                    sum = mul2(sum, dup(f));
                    also = mul2(also, dup(f));
                    if (t > p.t0) {
                        // (S of this tile came after P V of the last one: O is at rest)
#pragma unroll 1
                        for (int j = 0; j < DP; j += 16) {
                            float o[16];
                            tmem_ld16(to + j, o);
                            landed<16>(o);
                            uint32_t w[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[i] * f);
                            tmem_st16(to + j, w);
                        }
                    }
                }
                const float from = base == -INFINITY ? 0.f : -base * c;
#pragma unroll
                for (int j = 0; j < KT; j += 32) {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 z = fma2(make_float2(v[j + 2 * i], v[j + 2 * i + 1]), dup(c), dup(from));
                        z.x = ex2(z.x);
                        z.y = ex2(z.y);
                        if (i & 1) also = add2(also, z);
                        else sum = add2(sum, z);
                        w[i] = pack_bf16(z.x, z.y);
                    }
                    tmem_st16(ts + j / 2, w);
                    if (j % 64 == 32) {
                        tmem_st_wait();
                        tc_fence_before();
                        arrive_warp(kP + 2 * tile + j / 64);
                    }
                }
            }
            if (!ok || !wait(kO + tile, (n - 1) & 1)) break;
            tc_fence_after();
            const float l = (sum.x + sum.y) + (also.x + also.y);
            const bool whole = p.whole(), live = row < rows;
            const AttnWalk::Place to_row = p.place(a, live ? 128 * tile + row : 0);
            const size_t at = (size_t)to_row.token * a.Hq + to_row.head;
            const float inv = whole ? l > 0.f ? 1.f / l : l == 0.f ? 0.f : l : 1.f;
            if (tid == 0) p.tell_join(a, cut, cta);
            float* part = a.part + p.slot(cta) * attn_part_floats(a);
            const int prow = 128 * tile + row;
            const bool vec = reinterpret_cast<uintptr_t>(a.out) % 16 == 0;
#pragma unroll 1
            for (int j = 0; j < DP; j += 16) {
                float o[16];
                tmem_ld16(to + j, o);
                landed<16>(o);
                if (!live) continue;
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= inv;
#pragma unroll
                for (int i = 0; i < 16; i += 8) {
                    if (j + i >= a.D) continue;
                    if (whole) {
                        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.out) + at * a.D + j + i;
                        if (vec) *reinterpret_cast<uint4*>(y) = pack8_bf16(o + i);
                        else
#pragma unroll
                            for (int e = 0; e < 8; ++e) y[e] = __float2bfloat16_rn(o[i + e]);
                    } else {
                        float4* y = reinterpret_cast<float4*>(part + (size_t)prow * a.D + j + i);
                        y[0] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                        y[1] = make_float4(o[i + 4], o[i + 5], o[i + 6], o[i + 7]);
                    }
                }
            }
            tc_fence_before();
            arrive_warp(kOFree + tile);
            if (live) {
                const float at_log2 = base == -INFINITY ? -INFINITY : base * c;
                if (!whole) {
                    part[(size_t)a.block * a.D + prow] = at_log2;
                    part[(size_t)a.block * (a.D + 1) + prow] = l;
                } else if (a.lse) {
                    a.lse[at] = l == 0.f ? -INFINITY : (at_log2 + log2f(l)) * 0.6931471805599453f;
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 8) {
            // ------------------------------------------------------------ products
            {
                // (the whole warp runs the loop and one lane issues: what the products take stays in uniform registers)
                const uint32_t leader = elect_one();
                const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), sm = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
                constexpr uint32_t idS = idesc_bf16(128, KT, 0, 0), idO = idesc_bf16(128, DP, 0, 1), hi = desc_hi(WIDE ? 2048 : 1024);
                constexpr int STEP = WIDE ? 4096 : 2048;       // bytes of 16 keys' values in a half
                uint32_t n[2] = {0, 0}, mine[2] = {0, 0}, g = 0, pieces = 0;     // key tiles and pieces of each query tile, and of both
                auto keys = [&](uint32_t at, int v) { return wait1(kFull + (2 * at + v) % L::SLOTS, (2 * at + v) / L::SLOTS & 1); };
                auto scores = [&](int tile, uint32_t at) {
                    const uint32_t sq = desc_lo((sm + L::Q + tile * L::TILE), 16), ts = tm + TS + 128 * tile;
                    const uint32_t sk = desc_lo((sm + L::KV + 2 * at % L::SLOTS * L::TILE), 16);
                    tc_fence_after();
                    steps<4 * NB>([&](auto k) {
                        constexpr int o = (k >> 2) * HALF + (k & 3) * 32;
                        mma_ss<o, WIDE ? (k >> 2) * 1024 + (k & 3) * 32 : o>(leader, ts, sq, sk, hi, idS, k > 0);
                    });
                    commit(leader, &bar[kS + tile]);
                };
                bool ok = true;
                for (AttnWalk p(a, units, cut, cta); ok && p.more(); p.next(a, units), ++pieces) {
                    const int tiles = p.rows(a) > 128 ? 2 : 1, last = tiles - 1;
                    ok = wait1(kQFull, pieces & 1) && keys(g, 0);
                    steps<2>([&](auto tile) {
                        if (!ok || tile >= tiles) return;
                        ok = n[tile] == 0 || wait1(kO + tile, (n[tile] - 1) & 1);      // P of the last piece has been read
                        if (ok) scores(tile, g);
                    });
                    if (!ok) break;
                    commit(leader, &bar[kEmpty + 2 * g % L::SLOTS]);
                    if (p.t1 - p.t0 == 1) commit(leader, &bar[kQEmpty]);
                    for (int t = p.t0; ok && t < p.t1; ++t, ++g) {
                        const bool next = t + 1 < p.t1;
                        const uint32_t vs = (2 * g + 1) % L::SLOTS, sv = desc_lo((sm + L::KV + vs * L::TILE), WIDE ? 1024 : HALF);
                        ok = keys(g, 1);
                        // (a copy of the code for each tile: its counters stay in registers)
                        steps<2>([&](auto tile) {
                            if (!ok || tile >= tiles) return;
                            const uint32_t ts = tm + TS + 128 * tile, to = tm + TO + 128 * tile;
                            ok = wait1(kP + 2 * tile, n[tile] & 1) && (t > p.t0 || mine[tile] == 0 || wait1(kOFree + tile, (mine[tile] - 1) & 1));
                            if (!ok) return;
                            tc_fence_after();
                            steps<KT / 32>([&](auto k) { mma_ts<k * STEP>(leader, to, ts + 8 * k, sv, hi, idO, t > p.t0 || k > 0); });
                            ok = wait1(kP + 2 * tile + 1, n[tile] & 1);
                            if (!ok) return;
                            tc_fence_after();
                            steps<KT / 32>([&](auto k) { mma_ts<(k + KT / 32) * STEP>(leader, to, ts + 8 * (k + KT / 32), sv, hi, idO, 1); });
                            commit(leader, &bar[kO + tile]);
                            if (tile == last) commit(leader, &bar[kEmpty + vs]);
                            if (next) {
                                ok = (tile || keys(g + 1, 0)) && wait1(kO + tile, n[tile] & 1);
                                if (!ok) return;
                                scores(tile, g + 1);
                                if (tile == last) {
                                    commit(leader, &bar[kEmpty + (2 * g + 2) % L::SLOTS]);
                                    if (t + 2 == p.t1) commit(leader, &bar[kQEmpty]);
                                }
                            }
                            ++n[tile];
                        });
                    }
                    if (!ok) break;
                    steps<2>([&](auto tile) { mine[tile] += tile < tiles; });
                }
            }
            __syncwarp();
        } else {
            // ------------------------------------------------------------ Q: a tile each of warps 9 and 11
            constexpr int PER = DP / 8, EACH = 32 / PER;      // pieces of a row, rows of one round of the lanes
            const int c = lane % PER, sub = lane / PER;
            const bool column = c * 8 < a.D, vq = a.qs % 8 == 0 && reinterpret_cast<uintptr_t>(a.q) % 16 == 0;
            const int each_token = EACH / a.G, each_head = EACH % a.G;
            uint32_t pieces = 0;
            auto queries = [&](const AttnWalk& p, int tile) {
                if (pieces && !wait(kQEmpty, (pieces - 1) & 1)) return false;
                ++pieces;
                const int rows = p.rows(a) - 128 * tile;
                if (rows > 0) {
                    const uint32_t sq = smem_u32(smem + L::Q + tile * L::TILE);
                    // (rows one after the other: no division but the first)
                    AttnWalk::Place at = p.place(a, 128 * tile + sub);
                    at.head -= p.head * a.G;
#pragma unroll 4
                    for (int r = sub; r < 128; r += EACH) {
                        const bool in = r < rows && column;
                        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
                        if (in) q += at.token * a.qs + (p.head * a.G + at.head) * a.D + c * 8;
                        const uint32_t to = sq + piece(r, c);
                        if (vq) {
                            cp_async16(to, q, in ? 16 : 0);
                        } else {
                            uint4 f = make_uint4(0, 0, 0, 0);
                            if (in) {
                                const unsigned short* e = reinterpret_cast<const unsigned short*>(q);
                                f = make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16, e[4] | (uint32_t)e[5] << 16, e[6] | (uint32_t)e[7] << 16);
                            }
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(f.x), "r"(f.y), "r"(f.z), "r"(f.w) : "memory");
                        }
                        at.token += each_token;
                        at.head += each_head;
                        if (at.head >= a.G) {
                            at.head -= a.G;
                            ++at.token;
                        }
                    }
                }
                cp_commit();
                cp_wait<0>();
                fence_async_smem();
                arrive_warp(kQFull);
                return true;
            };
            // ------------------------------------------------------------ keys (warp 10) and values (warp 9)
            constexpr int PARTS = WIDE ? 1 : NB;              // copies of a box's keys
            const int kv = warp == 9, R = 1 << box_log2, boxes = (KT >> box_log2) * PARTS, nowhere = a.pages * 2 * a.Hkv;
            uint32_t g = 0;                                   // key tiles
            bool ok = true;
            for (AttnWalk p(a, units, cut, cta); ok && p.more(); p.next(a, units)) {
                if (warp != 10) ok = queries(p, warp == 9);
                if (warp == 11) continue;
                const int32_t* pages = a.table + (size_t)max(p.w.seq, 0) * a.max_pages;
                // the map's third coordinate of the keys (values: + Hkv) of the box that begins at `key`
                auto look = [&](int key) {
                    if (key + R <= p.s.begin || key >= p.s.end) return nowhere;
                    const int page = pages[key / a.pt];
                    if (page >= 0 && page < a.pages) return page * 2 * a.Hkv + p.head;
                    record_error(a.status, KDA_ERR_INVALID_ARG);
                    return nowhere;
                };
                auto cut_box = [&](int key) { return (key < p.s.begin && key + R > p.s.begin) || (key < p.s.end && key + R > p.s.end); };
                const int mine = (lane / PARTS) << box_log2;       // this lane's first box: its keys in a tile
                int next = look((p.s.tile0 + p.t0) * KT + mine);
                for (int t = p.t0; ok && t < p.t1; ++t, ++g) {
                    const int k0 = (p.s.tile0 + t) * KT, first = next;
                    if (t + 1 < p.t1) next = look(k0 + KT + mine);
                    const uint32_t n = 2 * g + kv, slot = n % L::SLOTS;
                    if (n >= L::SLOTS && !wait(kEmpty + slot, (n / L::SLOTS - 1) & 1)) { ok = false; break; }
                    const uint32_t to = smem_u32(smem + L::KV + slot * L::TILE);
                    int by_row = 0;
                    if (kv && R > 1) {
                        // (the box of the window's begin and that of the end; one box may be both)
                        int done = -1;
#pragma unroll 1
                        for (int edge : {p.s.begin, p.s.end}) {
                            const int key = edge & ~(R - 1);
                            if (key == edge || key < k0 || key >= k0 + KT || key == done) continue;
                            done = key;
                            ++by_row;
                            const int z = look(key);
                            const char* from = static_cast<const char*>(a.pool) + ((int64_t)(z + a.Hkv) * a.pt + key % a.pt) * (a.D * 2);
#pragma unroll 1
                            for (int i = lane; i < R * 8 * NB; i += 32) {
                                const int r = i / (8 * NB), b = i % (8 * NB);
                                const bool in = z != nowhere && key + r >= p.s.begin && key + r < p.s.end && b * 8 < a.D;
                                cp_async16(to + key_piece<WIDE>(key - k0 + r, b), in ? from + (int64_t)r * a.D * 2 + b * 16 : a.pool, in ? 16 : 0);
                            }
                        }
                        if (by_row) {
                            cp_commit();
                            cp_wait<0>();
                            fence_async_smem();
                            __syncwarp();
                        }
                    }
                    if (lane == 0) mbar_expect_tx(&bar[kFull + slot], ((KT >> box_log2) - by_row) * NB * R * 128);
                    __syncwarp();
#pragma unroll 1
                    for (int i = lane; i < boxes; i += 32) {
                        const int at = (i / PARTS) << box_log2, key = k0 + at;
                        const int z = (i < 32 ? first : look(key));
                        if (kv && R > 1 && cut_box(key)) continue;
                        const int page = z == nowhere ? nowhere : z + kv * a.Hkv, in_page = key % a.pt;
                        if constexpr (WIDE) tma_load_5d_to(to + at * 256, &map, in_page >> 3, page, &bar[kFull + slot]);
                        else tma_load_3d_to(to + (i % NB) * HALF + at * 128, &map, (i % NB) * 64, in_page, page, &bar[kFull + slot]);
                    }
                    __syncwarp();
                }
            }
            cp_wait<0>();
        }
    }
    __syncthreads();
    if (*fail && tid == 0) {
        // give products in flight a bounded chance to land before the memory is released
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

template <int NB, bool WIDE> cudaError_t go(const AttnArgs& a, int box_log2, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel<NB, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<NB>::TOTAL);
    if (e != cudaSuccess) return e;
    auto enc = map_encoder();
    if (!enc) return cudaErrorNotSupported;
    // a pool as [pages x (keys, values) x heads][page tokens][D]; WIDE: [..][page tokens / 8][halves of D][8][64]
    CUtensorMap map;
    const cuuint64_t D = a.D, pt = a.pt, all = (cuuint64_t)a.pages * 2 * a.Hkv;
    const cuuint32_t R = 1u << box_log2, es[5] = {1, 1, 1, 1, 1};
    const cuuint64_t dims3[3] = {D, pt, all}, strides3[2] = {D * 2, pt * D * 2};
    const cuuint32_t box3[3] = {64, R, 1};
    const cuuint64_t dims5[5] = {64, 8, 2, pt / 8, all}, strides5[4] = {256, 128, 2048, pt * 256};
    const cuuint32_t box5[5] = {64, 8, 2, R / 8, 1};
    if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, WIDE ? 5 : 3, const_cast<void*>(a.pool), WIDE ? dims5 : dims3, WIDE ? strides5 : strides3,
            WIDE ? box5 : box3, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    return attn_launch(attn_tc_kernel<NB, WIDE>, a.ctas, kThreads, Lay<NB>::TOTAL, !a.direct, st, a, map, box_log2);
}

}  // namespace

cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t st) {
    int box_log2 = 0;
    while (box_log2 < 5 && a.pt % (2 << box_log2) == 0) ++box_log2;
    if (a.D == 128 && box_log2 >= 3) return go<2, true>(a, box_log2, st);
    return a.D > 64 ? go<2, false>(a, box_log2, st) : go<1, false>(a, box_log2, st);
}

}  // namespace kda
