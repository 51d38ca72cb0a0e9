// kda_gated.h -- a tile of the gated linear recurrence: what a thread has of it, and which rows begin and end there.
// (Host code compiles it as well: the tests follow a thread's reads of the rows' states through it.)
#pragma once

#ifdef __CUDACC__
#define KDA_BOTH __host__ __device__ __forceinline__
#else
#define KDA_BOTH inline
#endif

namespace kda {

// Eight warps do a tile's arithmetic, a ninth joins it to the chain of tiles.
constexpr int kGatedThreads = 256, kGatedWarps = kGatedThreads / 32;
constexpr int kGatedTok = 8, kGatedTile = kGatedWarps * kGatedTok;      // tokens of a thread and of a CTA

// What a thread has of a tile: its channels, and where its tokens lie.
struct GatedSpot {
    int tile, col, warp, lane, c, t0, tb, n;      // c: first channel; tb, n: first token and how many there are, 0 past the last channel
    bool in;
};
template <int VEC> KDA_BOTH GatedSpot gated_spot(int tokens, int C, int tile, int col, int thread) {
    GatedSpot s;
    s.tile = tile;
    s.col = col;
    s.warp = thread >> 5;
    s.lane = thread & 31;
    s.c = (col * 32 + s.lane) * VEC;
    s.in = s.c < C;
    s.t0 = tile * kGatedTile;
    s.tb = s.t0 + s.warp * kGatedTok;
    const int left = tokens - s.tb;
    s.n = !s.in || left < 0 ? 0 : left < kGatedTok ? left : kGatedTok;
    return s;
}

// Which rows begin at and end with a token of the tile, -1: none.  The lists are the CTA's, and a thread whose channels lie
// past the last has none of their tokens: it asks for no row's state, which may end where the last channel does.
struct GatedEdges {
    int first[kGatedTile], last[kGatedTile];
    KDA_BOTH int begins(const GatedSpot& s, int k) const { return k < s.n ? first[s.warp * kGatedTok + k] : -1; }
    KDA_BOTH int ends(const GatedSpot& s, int k) const { return k < s.n ? last[s.warp * kGatedTok + k] : -1; }
};

}  // namespace kda
