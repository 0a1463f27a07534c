// The split of decode_shared's prefix pass, compiled for the host: every CTA's pieces, in the order in which it takes them.
#include "warp.h"

#include "pda_split.cuh"

extern "C" {

// out: rows of 12 ints {CTA, group, KV head, row tile, first sequence, rows, length, first step, steps, rotation, slot, pieces}.
// Returns their number, or -1 where `cap` rows do not hold them; scalars: {error bits, places of a run, places in all, a tile's own}.
int split_pieces(int NG, const int* starts, const int* plens, int B, int QG, int Hk, int MP, int BS, int P, int ctas, int* out,
                 int cap, int* scalars) {
    pda::SharedArgs a = {};
    a.group_starts = starts;
    a.prefix_lens = plens;
    int err = 0;
    a.err_word = &err;
    a.B = B, a.NG = NG, a.Hk = Hk, a.QG = QG, a.MP = MP, a.BS = BS, a.P = P, a.slots = P + 1;
    int n = 0;
    for (int cta = 0; cta < ctas && n >= 0; ++cta)
        host_warp::run([&] {
            const bool lead = threadIdx.x == 0;
            const pda::Split split = pda::make_split(a, ctas, cta == 0);
            int at = (int)std::min((long long)cta * split.per, (long long)split.total);
            const int end = at + std::min(split.per, split.total - at);
            if (lead) scalars[1] = split.per, scalars[2] = split.total, scalars[3] = split.whole;
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

}  // extern "C"
