// pda_window.cuh -- the list of pda_decode_window: which tiles a step over a sliding window reads.  Integers only, so that the
// same code also compiles for the host, where the tiles are checked.
#pragma once

namespace pda {

// The tiles of a window: the first tokens' (none where the window reaches them), then the window's.  Only whole tokens that
// are seen are counted in a tile, and every tile counts a prefix of its 16 places: the tile in which the window begins is
// copied from the first token seen on (its places past the block's end come as zeros).  So a masked token is past a tile's
// count, as behind a context's end, and one before the window is not even read.
struct WindowTiles {
    int ctx, first, start;   // tokens; first tokens of their own; where the window begins
    int head, tiles;         // tiles of the first tokens, and of all
    __device__ __forceinline__ WindowTiles(int ctx_, int window, int num_first) : ctx(ctx_) {
        start = max(ctx - window, 0);
        first = min(num_first, ctx);
        if (start <= first) start = first = 0;
        head = (first + 15) >> 4;
        tiles = ctx > 0 ? head + ((ctx - 1) >> 4) - (start >> 4) + 1 : 0;
    }
    __device__ __forceinline__ int token(int t) const {   // a tile's first token
        return t < head ? 16 * t : t == head ? start : ((start >> 4) + t - head) * 16;
    }
    __device__ __forceinline__ int count(int t) const {   // and its tokens
        const int k = token(t);
        return t < head ? min(16, first - k) : min((k | 15) + 1, ctx) - k;
    }
};

}  // namespace pda
