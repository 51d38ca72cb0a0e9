// kda_pages.cu -- the pages of a cache: copying, forking, extending, freeing and compacting.
//
// refs is the only record of what is free (refs <= 0), so there is no free list to keep in step with it,
// and "the i-th free page by index" is one answer whatever the GPU's order of work.  It costs a pass over
// refs per allocating call: 4 bytes per page against the 2 x page_bytes x layers that a copied page moves.
// The passes are
//   count    free (or live) pages of each tile of kTile pages; the requests' needs and their ranks (one
//            more CTA); separate output arrays filled from the inputs;
//   assign   ranks of the pages, tile by tile, from the counts before it: the page of each rank;
//   apply    rows, references and the pages' data.
// A rank needs the counts of every tile before it, and a grid-wide wait inside one kernel would cost about what
// a launch does.  Up to kDirectTiles tiles the first two passes are one launch: each tile's CTA counts all
// tiles before its own, which it reads from L2.  Copies are bound by memory: 24 forks of 8 layers of 1 MB take
// 66 us for their 403 MB (6.1 TB/s), moving some 3000 pages of 16 KB in 4 layers 68 us for 407 MB.
#include <limits.h>
#include <string.h>

#include "kda.h"
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {

namespace {

constexpr int kThreads = 1024, kPer = 4, kTile = kThreads * kPer;
constexpr int kCopyThreads = 256, kCopyUnroll = 4;
// A page is copied in parts, each by a team of threads, 64 bytes a thread: a warp for pages up to 8 KB, so that
// many small pages are in flight at once, else a CTA (16384 pages compacted: pages of 4 KB 12.1 us by warps,
// 16.1 by CTAs, of 8 KB 17.0 and 19.6; four layers of 16 KB 88.2 and 87.5).
constexpr int64_t kPartBytes = 16 * kCopyUnroll;

enum Mode { kFork, kExtend, kCompact };

struct PageArgs {
    int layers, P, S, M, pt, n, tiles, mode, direct, team;
    int64_t page_bytes, layer_stride;
    uint8_t* pool;
    const int32_t *table, *lengths, *refs, *ra, *rb;   // ra, rb: the requests (parents, children | seqs, new lengths)
    int32_t *table_o, *lengths_o, *refs_o, *ok, *map;
    // workspace
    int32_t* head;      // [0] pages wanted, [1] free pages (kCompact: [0] pages to move, [1] live pages)
    int32_t* counts;    // [tiles]
    int32_t* need;      // [n] pages wanted by request i, -1: refused
    int32_t* rank;      // [n] pages wanted before it
    int32_t* list;      // [P] page of rank r (kCompact: holes)
    int32_t* movers;    // [P] kCompact: the k-th highest live page at or above L
    int32_t* to;        // [P] kCompact: p where it stays, -1 free, -2 - k the k-th mover
};

__device__ __forceinline__ bool page_ok(const PageArgs& a, int p) { return (unsigned)p < (unsigned)a.P; }
__device__ __forceinline__ int pages_of(const PageArgs& a, int len) { return len <= 0 ? 0 : (len - 1) / a.pt + 1; }

// Exclusive prefix sum of x over the CTA; total in every thread.
template <typename T>
__device__ __forceinline__ T block_scan(T x, T* total) {
    __shared__ T part[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    __syncthreads();   // part is free again
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        T w = part[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        part[lane] = w;
    }
    __syncthreads();
    *total = part[31];
    return inc - x + (warp ? part[warp - 1] : 0);
}

__device__ void request_needs(const PageArgs& a) {
    long long before = 0;
    for (int i0 = 0; i0 < a.n; i0 += kThreads) {
        const int i = i0 + threadIdx.x;
        int need = -1;
        if (i < a.n) {
            const int s = a.ra[i];
            if ((unsigned)s < (unsigned)a.S) {
                const int len = a.lengths[s];
                if (a.mode == kFork) {
                    const int ch = a.rb[i];
                    if ((unsigned)ch < (unsigned)a.S && ch != s && a.lengths[ch] <= 0 && pages_of(a, len) <= a.M) {
                        const bool part = len > 0 && len % a.pt != 0;
                        if (!part) need = 0;
                        else if (page_ok(a, a.table[(size_t)s * a.M + len / a.pt])) need = 1;
                    }
                } else {
                    const int nl = a.rb[i];
                    if (nl >= 0 && nl >= len && pages_of(a, nl) <= a.M) need = pages_of(a, nl) - pages_of(a, len);
                }
            }
        }
        long long total;
        const long long ex = before + block_scan<long long>(need > 0 ? need : 0, &total);
        before += total;
        if (i < a.n) {
            a.need[i] = need;
            a.rank[i] = (int)(ex < INT_MAX ? ex : INT_MAX);
        }
    }
    if (threadIdx.x == 0) a.head[0] = (int)(before < INT_MAX ? before : INT_MAX);
}

__device__ __forceinline__ void copy_ints(int32_t* dst, const int32_t* src, size_t n) {
    if (!dst || dst == src) return;
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (size_t)gridDim.x * blockDim.x)
        dst[i] = src[i];
}

// Output arrays of their own filled from the inputs, and the requests' CTA (true there: nothing is left to do).
__device__ __forceinline__ bool requests(const PageArgs& a) {
    if (a.mode == kCompact) return false;      // it has no requests, and writes its outputs in full by itself
    copy_ints(a.table_o, a.table, (size_t)a.S * a.M);
    copy_ints(a.lengths_o, a.lengths, a.S);
    copy_ints(a.refs_o, a.refs, a.P);
    if ((int)blockIdx.x < a.tiles) return false;
    request_needs(a);
    return true;
}

__global__ void __launch_bounds__(kThreads) pages_count_kernel(PageArgs a) {
    if (requests(a)) return;
    const bool live = a.mode == kCompact;
    int cnt = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const long long p = (long long)blockIdx.x * kTile + threadIdx.x * kPer + e;
        if (p < a.P) cnt += (a.refs[p] > 0) == live;
    }
    int total;
    block_scan<int>(cnt, &total);
    if (threadIdx.x == 0) a.counts[blockIdx.x] = total;
}

// Free (live) pages of the tiles before the CTA's, and (all) of all tiles.
__device__ int pages_before(const PageArgs& a, int tile, bool live, int* all) {
    const int upto = all ? a.tiles : tile;
    int before = 0, sum = 0;
    if (a.direct) {
        const int64_t own = (int64_t)tile * kTile, end = (int64_t)upto * kTile < a.P ? (int64_t)upto * kTile : a.P;
        for (int64_t p0 = 0; p0 < end; p0 += kTile) {
            int r[kPer];
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const int64_t p = p0 + e * kThreads + threadIdx.x;
                r[e] = p < end ? a.refs[p] : 0;
            }
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const int64_t p = p0 + e * kThreads + threadIdx.x;
                const int hit = p < end && (r[e] > 0) == live;
                sum += hit;
                before += hit && p < own;
            }
        }
    } else {
        for (int i = threadIdx.x; i < upto; i += kThreads) {
            const int c = a.counts[i];
            sum += c;
            before += i < tile ? c : 0;
        }
    }
    long long total;
    block_scan<long long>((long long)sum << 32 | before, &total);
    if (all) *all = (int)(total >> 32);
    return (int)total;
}

__global__ void __launch_bounds__(kThreads) pages_assign_kernel(PageArgs a) {
    if (a.direct && requests(a)) return;
    const bool live = a.mode == kCompact;
    int all = 0;
    const int base = pages_before(a, blockIdx.x, live, live ? &all : nullptr);
    const int want = live ? 0 : a.direct ? a.P : a.head[0];
    bool hit[kPer];
    int cnt = 0;
    const long long p0 = (long long)blockIdx.x * kTile + threadIdx.x * kPer;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        hit[e] = p0 + e < a.P && (a.refs[p0 + e] > 0) == live;
        cnt += hit[e];
    }
    int total;
    int r = base + block_scan<int>(cnt, &total);
    if (!live) {
        if ((int)blockIdx.x == a.tiles - 1 && threadIdx.x == 0) a.head[1] = base + total;
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            if (hit[e]) {
                if (r < want) a.list[r] = (int)(p0 + e);
                ++r;
            }
        return;
    }
    const int L = all;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.head[1] = L;
        if (L == a.P) a.head[0] = 0;
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const long long p = p0 + e;
        if (p >= a.P) break;
        if (p == L) a.head[0] = L - r;      // holes below L = live pages not below it
        int to = -1;
        if (hit[e]) {
            if (p < L) to = (int)p;
            else {
                const int k = L - 1 - r;
                a.movers[k] = (int)p;
                to = -2 - k;
            }
            ++r;
        } else if (p < L) {
            a.list[p - r] = (int)p;
        }
        a.to[p] = to;
    }
}

// A team's place in the grid.
struct Team {
    int size, rank;          // threads, this thread's number
    int64_t first, step;     // the first work item, and from one to the next
};
__device__ __forceinline__ Team team_of(int size) {
    const int per = kCopyThreads / size;
    return {size, (int)threadIdx.x % size, (int64_t)blockIdx.x * per + threadIdx.x / size, (int64_t)gridDim.x * per};
}
__host__ __device__ __forceinline__ int64_t parts_of(int64_t page_bytes, int team) {
    return (page_bytes + kPartBytes * team - 1) / (kPartBytes * team);
}

// Part k of a page.
template <typename V>
__device__ __forceinline__ void copy_part(const Team& t, uint8_t* dst, const uint8_t* src, int64_t k, int64_t page_bytes) {
    constexpr int U = kCopyUnroll * 16 / sizeof(V) > 16 ? 16 : kCopyUnroll * 16 / sizeof(V);
    const int64_t at = k * kPartBytes * t.size, step = t.size * (int64_t)sizeof(V);
    const int64_t stop = at + kPartBytes * t.size < page_bytes ? at + kPartBytes * t.size : page_bytes;
    for (int64_t o = at + t.rank * sizeof(V); o < stop; o += U * step) {
        V v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (o + u * step < stop) v[u] = __ldcs(reinterpret_cast<const V*>(src + o + u * step));
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (o + u * step < stop) __stcs(reinterpret_cast<V*>(dst + o + u * step), v[u]);
    }
}

template <typename V>
__global__ void __launch_bounds__(kCopyThreads) pages_fork_kernel(PageArgs a) {
    const Team t = team_of(a.team);
    const int64_t parts = parts_of(a.page_bytes, t.size), per = parts * a.layers, items = per * a.n;
    for (int64_t w = t.first; w < items; w += t.step) {
        const int i = (int)(w / per);
        const int64_t rest = w - i * per;
        const int need = a.need[i], rank = a.rank[i];
        const bool ok = need == 0 || (need > 0 && rank < a.head[1]);
        if (rest == 0 && t.rank == 0) a.ok[i] = ok;
        if (!ok) continue;
        const int s = a.ra[i], ch = a.rb[i], len = a.lengths[s];
        const int full = len > 0 ? len / a.pt : 0;
        const int fresh = need > 0 ? a.list[rank] : -1;
        const int32_t* row = a.table + (size_t)s * a.M;
        if (rest == 0) {
            for (int j = t.rank; j < a.M; j += t.size) {
                const int p = row[j];
                a.table_o[(size_t)ch * a.M + j] = j < full ? p : (j == full && need > 0 ? fresh : -1);
                if (j < full && page_ok(a, p)) atomicAdd(&a.refs_o[p], 1);
            }
            if (t.rank == 0) {
                a.lengths_o[ch] = len;
                if (need > 0) a.refs_o[fresh] = 1;
            }
        }
        if (need > 0) {
            const int l = (int)(rest / parts);
            uint8_t* base = a.pool + l * a.layer_stride;
            copy_part<V>(t, base + fresh * a.page_bytes, base + row[full] * a.page_bytes, rest - l * parts, a.page_bytes);
        }
    }
}

__global__ void __launch_bounds__(kCopyThreads) pages_extend_kernel(PageArgs a) {
    for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
        const int need = a.need[i], rank = a.rank[i];
        const bool ok = need >= 0 && (long long)rank + need <= a.head[1];
        const bool done = ok || need == 0;
        if (threadIdx.x == 0) a.ok[i] = done;
        if (!done) continue;
        // (the length may be another's already where a row is named twice: what the request was checked with stays
        // inside the row)
        const int s = a.ra[i], had = pages_of(a, a.rb[i]) - need;
        for (int j = threadIdx.x; j < need; j += kCopyThreads) {
            const int p = a.list[rank + j];
            a.table_o[(size_t)s * a.M + had + j] = p;
            a.refs_o[p] = 1;
        }
        if (threadIdx.x == 0) a.lengths_o[s] = a.rb[i];
    }
}

__global__ void __launch_bounds__(kCopyThreads) pages_fill_kernel(PageArgs a) {
    copy_ints(a.table_o, a.table, (size_t)a.S * a.M);
    copy_ints(a.lengths_o, a.lengths, a.S);
    copy_ints(a.refs_o, a.refs, a.P);
}

__global__ void __launch_bounds__(128) pages_free_kernel(PageArgs a) {
    const int s = a.ra[blockIdx.x];
    if ((unsigned)s >= (unsigned)a.S) return;
    for (int j = threadIdx.x; j < a.M; j += 128) {
        const int p = a.table[(size_t)s * a.M + j];
        if (page_ok(a, p)) atomicSub(&a.refs_o[p], 1);
        a.table_o[(size_t)s * a.M + j] = -1;
    }
    if (threadIdx.x == 0) a.lengths_o[s] = 0;
}

template <typename V>
__global__ void __launch_bounds__(kCopyThreads) pages_compact_kernel(PageArgs a) {
    const int moves = a.head[0], L = a.head[1];
    const int64_t step = (int64_t)gridDim.x * kCopyThreads, t0 = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x;
    for (int64_t p = t0; p < a.P; p += step) {
        const int to = a.to[p];
        if (to >= 0) a.refs_o[p] = a.refs[p];
        else if (to == -1) {
            if (p >= L) a.refs_o[p] = 0;     // a hole below L is written by the page that moves there
        } else {
            a.refs_o[a.list[-2 - to]] = a.refs[p];
            a.refs_o[p] = 0;
        }
        if (a.map) a.map[p] = to < -1 ? a.list[-2 - to] : to;
    }
    for (int64_t i = t0; i < (int64_t)a.S * a.M; i += step) {
        int p = a.table[i];
        if (page_ok(a, p)) {
            const int to = a.to[p];
            p = to < -1 ? a.list[-2 - to] : to;
        }
        a.table_o[i] = p;
    }
    const Team t = team_of(a.team);
    const int64_t parts = parts_of(a.page_bytes, t.size), per = parts * a.layers, items = per * moves;
    for (int64_t w = t.first; w < items; w += t.step) {
        const int k = (int)(w / per);
        const int64_t rest = w - k * per;
        const int l = (int)(rest / parts);
        uint8_t* base = a.pool + l * a.layer_stride;
        copy_part<V>(t, base + a.list[k] * a.page_bytes, base + a.movers[k] * a.page_bytes, rest - l * parts, a.page_bytes);
    }
}

struct CopyArgs {
    int layers, n, src_pages, dst_pages, team;
    int64_t page_bytes, src_stride, dst_stride;
    uint8_t* dst_pool;
    const uint8_t* src_pool;
    const int32_t *src, *dst;
};

template <typename V>
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(CopyArgs a) {
    const Team t = team_of(a.team);
    const int64_t parts = parts_of(a.page_bytes, t.size), per = parts * a.layers, items = per * a.n;
    for (int64_t w = t.first; w < items; w += t.step) {
        const int i = (int)(w / per);
        const int64_t rest = w - i * per;
        const int s = a.src[i], d = a.dst[i];
        if ((unsigned)s >= (unsigned)a.src_pages || (unsigned)d >= (unsigned)a.dst_pages) continue;
        const int l = (int)(rest / parts);
        copy_part<V>(t, a.dst_pool + l * a.dst_stride + d * a.page_bytes, a.src_pool + l * a.src_stride + s * a.page_bytes,
                     rest - l * parts, a.page_bytes);
    }
}

// The widest access that every page of the pool starts and ends on: 16, 4 or 1 bytes.
int access_bytes(const void* base, int64_t page_bytes, int64_t stride) {
    const uint64_t m = reinterpret_cast<uintptr_t>(base) | (uint64_t)page_bytes | (uint64_t)stride;
    return m % 16 == 0 ? 16 : m % 4 == 0 ? 4 : 1;
}

int copy_grid(int64_t items) {
    const int64_t most = 8 * 152;   // eight CTAs of 256 threads fill an SM
    return (int)(items < 1 ? 1 : items < most ? items : most);
}

int team_size(int64_t page_bytes) { return page_bytes <= 8192 ? 32 : kCopyThreads; }
// CTAs for the copies of n pages of every layer.
int pages_grid(int64_t page_bytes, int team, int layers, int64_t n) {
    const int per = kCopyThreads / team;
    return copy_grid((parts_of(page_bytes, team) * layers * n + per - 1) / per);
}

int tiles_of(int pages) { return (int)(((int64_t)pages + kTile - 1) / kTile); }

kda_status pages_check(const kda_pages_dims* d, int n, bool data) {
    if (!d || n < 0) return KDA_ERR_INVALID_ARG;
    if (d->num_pages < 1 || d->num_seqs < 1 || d->max_pages < 1 || d->page_tokens < 1) return KDA_ERR_INVALID_ARG;
    if (data && (d->layers < 1 || d->page_bytes < 1)) return KDA_ERR_INVALID_ARG;
    if (d->num_pages > (1 << 30) || n > (1 << 30) || (int64_t)d->num_seqs * d->max_pages > (1LL << 30)) return KDA_ERR_UNSUPPORTED;
    if (data) {
        if (d->page_bytes > (1LL << 40) / d->num_pages) return KDA_ERR_UNSUPPORTED;
        if (d->layers > 1 && d->layer_stride < d->page_bytes * d->num_pages) return KDA_ERR_INVALID_ARG;
    }
    return KDA_OK;
}

size_t pages_ws(const kda_pages_dims* d, int n) {
    return sizeof(int32_t) * (64 + (size_t)tiles_of(d->num_pages) + 2 * (size_t)n + 3 * (size_t)d->num_pages);
}

PageArgs page_args(const kda_pages_dims* d, int n, void* ws, int mode) {
    PageArgs a;
    memset(&a, 0, sizeof(a));
    a.layers = d->layers; a.P = d->num_pages; a.S = d->num_seqs; a.M = d->max_pages; a.pt = d->page_tokens;
    a.n = n; a.tiles = tiles_of(d->num_pages); a.mode = mode;
    a.page_bytes = d->page_bytes; a.layer_stride = d->layers > 1 ? d->layer_stride : 0;
    a.team = team_size(d->page_bytes);
    if (ws) {
        int32_t* w = static_cast<int32_t*>(ws);
        a.head = w; w += 64;
        a.counts = w; w += a.tiles;
        a.need = w; w += n;
        a.rank = w; w += n;
        a.list = w; w += a.P;
        a.movers = w; w += a.P;
        a.to = w;
    }
    return a;
}

bool ws_ok(const kda_pages_dims* d, int n, void* ws, size_t bytes) {
    return ws && bytes >= pages_ws(d, n) && reinterpret_cast<uintptr_t>(ws) % 256 == 0;
}

// Tiles up to which one launch is quicker: a fork in 4096, 16384 and 65536 pages takes 7.6, 8.7 and 13.8 us, in two
// launches 9.8, 10.0 and 10.2; a compaction 8.3, 10.4 and 17.9, 10.0, 15.1 and 32.0 (the latter with CTAs for teams).
constexpr int kDirectTiles = 4;

cudaError_t run_plan(PageArgs a, cudaStream_t stream) {
    a.direct = a.tiles <= kDirectTiles;
    const int requests = a.mode != kCompact;
    if (!a.direct) {
        timing_pre(stream, K_PAGES_COUNT);
        pages_count_kernel<<<a.tiles + requests, kThreads, 0, stream>>>(a);
        timing_post(stream);
        if (cudaError_t e = cudaGetLastError()) return e;
    }
    timing_pre(stream, K_PAGES_ASSIGN);
    pages_assign_kernel<<<a.tiles + (a.direct ? requests : 0), kThreads, 0, stream>>>(a);
    timing_post(stream);
    return cudaGetLastError();
}

cudaError_t run_fill(const PageArgs& a, cudaStream_t stream) {
    if (a.table_o == a.table && a.lengths_o == a.lengths && a.refs_o == a.refs) return cudaSuccess;
    const int64_t ints = (int64_t)a.S * a.M > a.P ? (int64_t)a.S * a.M : a.P;
    timing_pre(stream, K_PAGES_COUNT);
    pages_fill_kernel<<<copy_grid((ints + kCopyThreads - 1) / kCopyThreads), kCopyThreads, 0, stream>>>(a);
    timing_post(stream);
    return cudaGetLastError();
}

#define KDA_PAGES_LAUNCH(KERNEL, grid, a, bytes, st)                                  \
    do {                                                                              \
        if ((bytes) == 16) KERNEL<uint4><<<grid, kCopyThreads, 0, st>>>(a);           \
        else if ((bytes) == 4) KERNEL<unsigned><<<grid, kCopyThreads, 0, st>>>(a);    \
        else KERNEL<unsigned char><<<grid, kCopyThreads, 0, st>>>(a);                 \
    } while (0)

}  // namespace

}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_pages_workspace_size(const kda_pages_dims* dims, int n) {
    if (pages_check(dims, n, false) != KDA_OK) return 0;
    return (pages_ws(dims, n) + 255) / 256 * 256;
}

kda_status kda_pages_copy(int layers, int64_t page_bytes, void* dst_pool, int64_t dst_layer_stride, int dst_pages,
                          const void* src_pool, int64_t src_layer_stride, int src_pages, const int32_t* src,
                          const int32_t* dst, int n, cudaStream_t stream) {
    if (layers < 1 || page_bytes < 1 || dst_pages < 1 || src_pages < 1 || n < 0) return KDA_ERR_INVALID_ARG;
    if (!dst_pool || !src_pool || (n && (!src || !dst))) return KDA_ERR_INVALID_ARG;
    const int most = dst_pages > src_pages ? dst_pages : src_pages;
    if (most > (1 << 30) || n > (1 << 30) || page_bytes > (1LL << 40) / most) return KDA_ERR_UNSUPPORTED;
    if (layers > 1 && (dst_layer_stride < page_bytes * dst_pages || src_layer_stride < page_bytes * src_pages))
        return KDA_ERR_INVALID_ARG;
    if (n == 0) return KDA_OK;
    CopyArgs a;
    memset(&a, 0, sizeof(a));
    a.layers = layers; a.n = n; a.src_pages = src_pages; a.dst_pages = dst_pages; a.page_bytes = page_bytes;
    a.src_stride = layers > 1 ? src_layer_stride : 0;
    a.dst_stride = layers > 1 ? dst_layer_stride : 0;
    a.dst_pool = static_cast<uint8_t*>(dst_pool); a.src_pool = static_cast<const uint8_t*>(src_pool);
    a.src = src; a.dst = dst;
    const int w1 = access_bytes(dst_pool, page_bytes, a.dst_stride), w2 = access_bytes(src_pool, page_bytes, a.src_stride);
    a.team = team_size(page_bytes);
    const int grid = pages_grid(page_bytes, a.team, layers, n);
    timing_pre(stream, K_PAGES_COPY);
    KDA_PAGES_LAUNCH(pages_copy_kernel, grid, a, (w1 < w2 ? w1 : w2), stream);
    timing_post(stream);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_pages_fork(const kda_pages_dims* dims, void* pool, const int32_t* table, const int32_t* lengths,
                          const int32_t* refs, const int32_t* parents, const int32_t* children, int n,
                          int32_t* table_out, int32_t* lengths_out, int32_t* refs_out, int32_t* ok, void* workspace,
                          size_t workspace_bytes, cudaStream_t stream) {
    kda_status st = pages_check(dims, n, true);
    if (st != KDA_OK) return st;
    if (!pool || !table || !lengths || !refs || !table_out || !lengths_out || !refs_out) return KDA_ERR_INVALID_ARG;
    if (n && (!parents || !children || !ok)) return KDA_ERR_INVALID_ARG;
    if (!ws_ok(dims, n, workspace, workspace_bytes)) return KDA_ERR_WORKSPACE;
    PageArgs a = page_args(dims, n, workspace, kFork);
    a.pool = static_cast<uint8_t*>(pool);
    a.table = table; a.lengths = lengths; a.refs = refs; a.ra = parents; a.rb = children;
    a.table_o = table_out; a.lengths_o = lengths_out; a.refs_o = refs_out; a.ok = ok;
    if (n == 0) return run_fill(a, stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    if (run_plan(a, stream) != cudaSuccess) return KDA_ERR_CUDA;
    const int grid = pages_grid(a.page_bytes, a.team, a.layers, n);
    timing_pre(stream, K_PAGES_APPLY);
    KDA_PAGES_LAUNCH(pages_fork_kernel, grid, a, access_bytes(pool, a.page_bytes, a.layer_stride), stream);
    timing_post(stream);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_pages_extend(const kda_pages_dims* dims, const int32_t* table, const int32_t* lengths,
                            const int32_t* refs, const int32_t* seqs, const int32_t* new_lengths, int n,
                            int32_t* table_out, int32_t* lengths_out, int32_t* refs_out, int32_t* ok, void* workspace,
                            size_t workspace_bytes, cudaStream_t stream) {
    kda_status st = pages_check(dims, n, false);
    if (st != KDA_OK) return st;
    if (!table || !lengths || !refs || !table_out || !lengths_out || !refs_out) return KDA_ERR_INVALID_ARG;
    if (n && (!seqs || !new_lengths || !ok)) return KDA_ERR_INVALID_ARG;
    if (!ws_ok(dims, n, workspace, workspace_bytes)) return KDA_ERR_WORKSPACE;
    PageArgs a = page_args(dims, n, workspace, kExtend);
    a.table = table; a.lengths = lengths; a.refs = refs; a.ra = seqs; a.rb = new_lengths;
    a.table_o = table_out; a.lengths_o = lengths_out; a.refs_o = refs_out; a.ok = ok;
    if (n == 0) return run_fill(a, stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    if (run_plan(a, stream) != cudaSuccess) return KDA_ERR_CUDA;
    timing_pre(stream, K_PAGES_APPLY);
    pages_extend_kernel<<<copy_grid(n), kCopyThreads, 0, stream>>>(a);
    timing_post(stream);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_pages_free(const kda_pages_dims* dims, const int32_t* table, const int32_t* lengths,
                          const int32_t* refs, const int32_t* seqs, int n, int32_t* table_out, int32_t* lengths_out,
                          int32_t* refs_out, cudaStream_t stream) {
    kda_status st = pages_check(dims, n, false);
    if (st != KDA_OK) return st;
    if (!table || !lengths || !refs || !table_out || !lengths_out || !refs_out || (n && !seqs)) return KDA_ERR_INVALID_ARG;
    PageArgs a = page_args(dims, n, nullptr, kFork);
    a.table = table; a.lengths = lengths; a.refs = refs; a.ra = seqs;
    a.table_o = table_out; a.lengths_o = lengths_out; a.refs_o = refs_out;
    if (run_fill(a, stream) != cudaSuccess) return KDA_ERR_CUDA;
    if (n == 0) return KDA_OK;
    timing_pre(stream, K_PAGES_APPLY);
    pages_free_kernel<<<n, 128, 0, stream>>>(a);
    timing_post(stream);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_pages_compact(const kda_pages_dims* dims, void* pool, const int32_t* table, const int32_t* refs,
                             int32_t* table_out, int32_t* refs_out, int32_t* page_map, void* workspace,
                             size_t workspace_bytes, cudaStream_t stream) {
    kda_status st = pages_check(dims, 0, true);
    if (st != KDA_OK) return st;
    if (!pool || !table || !refs || !table_out || !refs_out) return KDA_ERR_INVALID_ARG;
    if (!ws_ok(dims, 0, workspace, workspace_bytes)) return KDA_ERR_WORKSPACE;
    PageArgs a = page_args(dims, 0, workspace, kCompact);
    a.pool = static_cast<uint8_t*>(pool);
    a.table = table; a.refs = refs; a.table_o = table_out; a.refs_o = refs_out; a.map = page_map;
    if (run_plan(a, stream) != cudaSuccess) return KDA_ERR_CUDA;
    // the number of moves is known on the device only: at most half the pages
    const int grid = pages_grid(a.page_bytes, a.team, a.layers, (a.P + 1) / 2);
    timing_pre(stream, K_PAGES_APPLY);
    KDA_PAGES_LAUNCH(pages_compact_kernel, grid, a, access_bytes(pool, a.page_bytes, a.layer_stride), stream);
    timing_post(stream);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
