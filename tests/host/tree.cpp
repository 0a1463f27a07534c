// The lists of the token operators, compiled for the host: the pieces of pda_decode_tree's passes, in the order in which every CTA
// takes them, and the tiles of pda_decode_window.
#include "warp.h"

#include "pda_split.cuh"
#include "pda_window.cuh"

extern "C" {

// out: rows of 12 ints {CTA, sequence, KV head, row tile, first token, rows, length, first step, steps, rotation, slot,
// pieces}.  Returns their number, or -1 where `cap` rows do not hold them; scalars: {error bits, places of a run, in all, a tile's
// own, refused}.
int tree_pieces_of(int NG, const int* starts, const int* lens, int tokens, int QG, int Hk, int MB, int BS, int P, int window,
                   int num_first, int ctas, int* out, int cap, int* scalars) {
    pda::TreeArgs a = {};
    a.group_starts = starts;
    a.prefix_lens = lens;
    int err = 0;
    a.err_word = &err;
    a.B = tokens, a.NG = NG, a.Hk = Hk, a.QG = QG, a.MP = MB, a.BS = BS, a.P = P, a.slots = P + 1;
    a.window = window, a.num_first = num_first;
    int n = 0;
    for (int cta = 0; cta < ctas && n >= 0; ++cta)
        host_warp::run([&] {
            const bool lead = threadIdx.x == 0;
            const auto split = pda::make_split(a, ctas, cta == 0);
            int at = (int)std::min((long long)cta * split.per, (long long)split.total);
            const int end = at + std::min(split.per, split.total - at);
            if (lead) scalars[1] = split.per, scalars[2] = split.total, scalars[3] = split.whole, scalars[4] = split.refused;
            for (;;) {
                const pda::Unit u = pda::find_unit(a, split, at, end);
                if (u.steps == 0) break;
                if (lead && n >= 0) {
                    if (n == cap) {
                        n = -1;
                    } else {
                        const int row[12] = {cta, u.g, u.h, u.rt, u.seq0, u.rows, u.len, u.step0, u.steps, u.rot, u.slot, u.pieces};
                        memcpy(out + 12 * n++, row, sizeof row);
                    }
                }
            }
        });
    scalars[0] = err;
    return n;
}

// {ctx, drafted, hole0, hole1, at, skip}
void tree_sight(int window, int num_first, int len, int drafted, int* out) {
    pda::TreeArgs a = {};
    a.window = window, a.num_first = num_first;
    const pda::Sight x = pda::sight_of(a, len, drafted);
    const int row[6] = {x.ctx, x.drafted, x.hole0, x.hole1, x.at, x.skip};
    memcpy(out, row, sizeof row);
}

// rows of {first token, tokens}; returns their number
int window_tiles(int ctx, int window, int num_first, int* out, int cap) {
    const pda::WindowTiles w(ctx, window, num_first);
    for (int t = 0; t < w.tiles && t < cap; ++t) out[2 * t] = w.token(t), out[2 * t + 1] = w.count(t);
    return w.tiles;
}

}  // extern "C"
