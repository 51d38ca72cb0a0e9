// kda_attn.h -- what the attention kernels over paged keys and values share: the problem, how it is cut into pieces,
// and what a piece leaves behind.
//
// The query heads of one key head and the new tokens of a row are one axis of packed query rows, token by token
// (packed row = token * G + head in the group), so that a tile of keys serves all of them.  A unit is a block of
// `block` packed rows of one row of the call with every key tile that one of them sees, at least one; an item is a unit
// for one key head.  An item costs its key tiles and, before them, `extra` tiles for its beginning and end.  All items' costs,
// laid end to end, are cut into equal spans, one to a CTA: a CTA finishes the items whose tiles lie in its span, and
// leaves the sums of those that it shares with other CTAs for the join.
#pragma once

#include "kda_internal.h"

namespace kda {

enum AttnKernel { kAttnSimt, kAttnMma, kAttnTc };

// What a CTA tells the join of the item that it begins and does not finish (rows 0: there is none): the first token's index and query head,
// the first of its packed rows, how many there are, and the last CTA with a part of it.
struct AttnShared {
    int token, head, first_row, rows, last;
};

struct AttnArgs {
    int rows, tokens, per_row;           // per_row: tokens of a row without cu
    int Hq, Hkv, G, D, dtype;
    int pages, pt, table_rows, max_pages, window;
    int64_t qs;                          // elements between tokens of q
    float scale;
    int kernel, direct;                  // AttnKernel; every row one unit
    const void *q, *pool;
    const int32_t *table, *lengths, *seqs, *cu;
    void* out;
    float* lse;
    // the cut
    int block, tile, extra;              // packed rows of a unit, keys of a tile, an item's cost beside its tiles
    int ctas;                            // most spans; with fewer tiles than that a tile each
    int units_most;
    int* units;                          // [1] units of the call, -1: nothing to do (workspace)
    int64_t* start;                      // [units + 1] cost of one key head before each unit (workspace)
    int* unit_row;                       // [units] row of the call, [units_most + units] block in it (workspace)
    AttnShared* shared;                  // [ctas] (workspace)
    float* part;                         // [2 ctas] sums of shared items: block x D, then block maxima, then block sums
    int* status;
};

struct AttnRow {
    int seq, len, n, first;              // table row (-1: idle), its tokens, new ones, the first one's index
};

// Row r of the call; what is wrong with it is recorded by one thread where `report`.
__device__ __forceinline__ AttnRow attn_row(const AttnArgs& a, int r, bool report) {
    AttnRow w;
    w.first = a.cu ? a.cu[r] : r * a.per_row;
    w.n = a.cu ? a.cu[r + 1] - w.first : a.per_row;
    w.seq = a.seqs ? a.seqs[r] : r;
    w.len = 0;
    bool bad = w.seq >= a.table_rows;
    if (!bad && w.seq >= 0) {
        w.len = max(a.lengths[w.seq], 0);
        bad = w.len > (int64_t)a.max_pages * a.pt;
    }
    if (bad) {
        if (report) record_error(a.status, KDA_ERR_INVALID_ARG);
        w.seq = -1;
        w.len = 0;
    }
    return w;
}

// Keys [begin, end) that the packed rows of a block see, and the tiles that hold them: at least one, which may hold none.
struct AttnSpan {
    int begin, end, tile0, tiles;
};
__device__ __forceinline__ AttnSpan attn_span(const AttnArgs& a, const AttnRow& w, int block) {
    AttnSpan s;
    // (packed rows fit 32 bits: tokens x query heads does)
    const uint32_t r0 = (uint32_t)block * a.block, r1 = min(r0 + a.block, (uint32_t)w.n * a.G) - 1;
    const int p0 = w.len - w.n + (int)(r0 / (uint32_t)a.G), p1 = w.len - w.n + (int)(r1 / (uint32_t)a.G);
    s.end = w.seq < 0 ? 0 : max(p1 + 1, 0);
    s.begin = a.window ? max(p0 - a.window + 1, 0) : 0;
    if (s.begin >= s.end) s.begin = s.end = 0;
    s.tile0 = s.begin / a.tile;
    s.tiles = max((s.end + a.tile - 1) / a.tile - s.tile0, 1);
    return s;
}
__device__ __forceinline__ int attn_blocks(const AttnArgs& a, int n) { return (int)(((int64_t)n * a.G + a.block - 1) / a.block); }

// The spans of the CTAs over a total cost.
struct AttnCut {
    int64_t total;
    int ctas;
    __device__ __forceinline__ AttnCut(const AttnArgs& a, int64_t t) : total(t), ctas((int)(t < a.ctas ? t : a.ctas)) {}
    __device__ __forceinline__ int64_t begin(int c) const { return total * c / ctas; }
    __device__ __forceinline__ int owner(int64_t x) const { return (int)(((x + 1) * ctas + total - 1) / total) - 1; }   // begin(owner) <= x
};

// The units of a call: read from the plan's arrays, or, where every row is one unit and the rows are few (direct), counted by
// every CTA for itself, which saves the plan's launch.
constexpr int kAttnDirectRows = 512;
struct AttnUnits {
    int units;
    const int64_t* start;
    __device__ __forceinline__ int64_t cost(const AttnArgs& a) const { return start[units] * a.Hkv; }
};
// All threads of a CTA; own: [kAttnDirectRows + 1] in shared memory.
__device__ __forceinline__ AttnUnits attn_units(const AttnArgs& a, int64_t* own) {
    AttnUnits s;
    cudaTriggerProgrammaticLaunchCompletion();       // the join may be launched
    if (threadIdx.x == 0) a.shared[blockIdx.x].rows = 0;
    if (!a.direct) {
        cudaGridDependencySynchronize();             // (the plan)
        s.units = *a.units;
        s.start = a.start;
        return s;
    }
    for (int r = threadIdx.x; r < a.rows; r += blockDim.x) own[r + 1] = attn_span(a, attn_row(a, r, blockIdx.x == 0), 0).tiles + a.extra;
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int64_t before = 0;
        for (int r0 = 0; r0 < a.rows; r0 += 32) {
            int64_t x = r0 + lane < a.rows ? own[r0 + lane + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t up = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += up;
            }
            x += before;
            if (r0 + lane < a.rows) own[r0 + lane + 1] = x;
            before = __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) own[0] = 0;
    }
    __syncthreads();
    s.units = a.rows;
    s.start = own;
    return s;
}

// The pieces of a CTA's span, one after the other: tiles [t0, t1) of an item's `tiles`.
struct AttnWalk {
    int u, head, t0, t1, tiles, row, block;
    int64_t item, end;                   // where the item's cost begins, and where the span ends
    AttnRow w;
    AttnSpan s;
    __device__ __forceinline__ AttnWalk(const AttnArgs& a, const AttnUnits& n, const AttnCut& cut, int cta) {
        const int64_t x = cut.begin(cta);
        end = cut.begin(cta + 1);
        int lo = 0, hi = n.units - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (n.start[mid] * a.Hkv <= x) lo = mid; else hi = mid - 1;
        }
        u = lo;
        unit(a, n);
        const int cost = tiles + a.extra;
        item = n.start[u] * a.Hkv;
        head = (int)((x - item) / cost);
        item += (int64_t)head * cost;
        t0 = max((int)(x - item) - a.extra, 0);
        if (!cut_off(a)) next(a, n);
    }
    __device__ __forceinline__ void unit(const AttnArgs& a, const AttnUnits& n) {
        row = a.direct ? u : a.unit_row[u];
        block = a.direct ? 0 : a.unit_row[a.units_most + u];
        w = attn_row(a, row, false);
        s = attn_span(a, w, block);
        tiles = (int)(n.start[u + 1] - n.start[u]) - a.extra;
    }
    // Whether the span reaches a tile of the item.
    __device__ __forceinline__ bool cut_off(const AttnArgs& a) {
        const int64_t left = end - item - a.extra;
        t1 = (int)(left < tiles ? left : tiles);
        return t1 > t0;
    }
    __device__ __forceinline__ bool more() const { return item < end; }
    __device__ __forceinline__ void next(const AttnArgs& a, const AttnUnits& n) {
        item += tiles + a.extra;
        if (item >= end) return;
        t0 = 0;
        if (++head == a.Hkv) {
            head = 0;
            ++u;
            unit(a, n);
        }
        if (!cut_off(a)) item = end;         // (what is left pays for the next CTA's beginning)
    }
    __device__ __forceinline__ bool whole() const { return t1 - t0 == tiles; }
    // Tells the join of an item that this CTA begins and does not finish (by thread 0).
    __device__ __forceinline__ void tell_join(const AttnArgs& a, const AttnCut& cut, int cta) const {
        if (t0 == 0 && t1 < tiles)
            a.shared[cta] = {w.first, head * a.G, (int)first_row(a), rows(a), cut.owner(item + a.extra + tiles - 1)};
    }
    // where its sums go: a CTA shares at most the item it starts inside of and the one it does not finish
    __device__ __forceinline__ int slot(int cta) const { return 2 * cta + (t0 == 0); }
    __device__ __forceinline__ uint32_t first_row(const AttnArgs& a) const { return (uint32_t)block * a.block; }
    __device__ __forceinline__ int rows(const AttnArgs& a) const { return (int)min((uint32_t)w.n * a.G - first_row(a), (uint32_t)a.block); }
    // The token and the query head of packed row i of the block.
    struct Place {
        int token, head;
    };
    __device__ __forceinline__ Place place(const AttnArgs& a, int i) const {
        const uint32_t r = first_row(a) + i, t = r / (uint32_t)a.G;
        return {w.first + (int)t, head * a.G + (int)(r - t * a.G)};
    }
    __device__ __forceinline__ int position(const AttnArgs& a, int i) const { return w.len - w.n + (int)((first_row(a) + i) / (uint32_t)a.G); }
};

__device__ __forceinline__ size_t attn_part_floats(const AttnArgs& a) { return (size_t)a.block * (a.D + 2); }

// Address of a page's keys (values: + Hkv page_tokens D elements) for key head h; nullptr where the table names none.
__device__ __forceinline__ const char* attn_page(const AttnArgs& a, int seq, int key, int head, int es) {
    const int page = a.table[(size_t)seq * a.max_pages + key / a.pt];
    if (page < 0 || page >= a.pages) {
        record_error(a.status, KDA_ERR_INVALID_ARG);
        return nullptr;
    }
    const size_t head_bytes = (size_t)a.pt * a.D * es;
    return static_cast<const char*>(a.pool) + ((size_t)page * 2 * a.Hkv + head) * head_bytes + (size_t)(key % a.pt) * a.D * es;
}

// The kernels.  mma: bf16, D a multiple of 8, 16-byte aligned pool; blocks of 16 packed rows.
constexpr int kAttnMmaRows = 16, kAttnMmaKeys = 64;
// Launches a kernel; early: while the one before it in the stream still runs (it begins with a wait for that one's end).
template <typename... P, typename... A>
cudaError_t attn_launch(void (*kernel)(P...), dim3 grid, int threads, size_t shared, bool early, cudaStream_t st, const A&... args) {
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = shared;
    c.stream = st;
    c.attrs = &at;
    c.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
}

cudaError_t launch_attn_mma(const AttnArgs& a, cudaStream_t st);
// tc: bf16, D a multiple of 8 up to 128, 16-byte aligned pool; two tiles of 128 packed rows against tiles of 128 keys.
constexpr int kAttnTcRows = 256, kAttnTcKeys = 128;
cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t st);
cudaError_t launch_attn_simt(const AttnArgs& a, cudaStream_t st);

}  // namespace kda
