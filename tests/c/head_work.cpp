/* Follows how the LM-head loss's products are dealt out, on the host.
 *   argv: N H V pairs kept hidden weights (kept: rows that are not ignored; hidden, weights: which gradients)
 * Prints the plan, and for every piece of the vocabulary its size, then the tiles of every pair in their order:
 *   loss/score: pair m0 n0 stages;  grad: pair product m0 n0 k0 stages split */
#include <cstdio>
#include <cstdlib>

#include "head_work.cuh"

using namespace df2::head;

template <int MODE>
static void walk(const char *name, const Work &a, int pairs)
{
    for (int pair = 0; pair < pairs; ++pair)
        for (int i = 0;; ++i) {
            const Tile t = tile_of<MODE>(a, pair, pairs, i);
            if (!t.live)
                break;
            std::printf("%s %d %d %d %d %d %d %d\n", name, pair, t.product, t.m0, t.n0, t.k0, t.stages, t.split);
        }
}

int main(int argc, char **argv)
{
    if (argc != 8)
        return 2;
    auto arg = [&](int i) { return std::atoi(argv[i]); };
    const int N = arg(1), H = arg(2), V = arg(3), pairs = arg(4), kept = arg(5);
    Work a{};
    a.N = N;
    a.H = H;
    a.V = V;
    a.h_tiles = ceil_div(H, kTile);
    a.row_tiles = ceil_div(N, kTile);
    a.col_tiles = ceil_div(V, kTile);
    walk<kLoss>("loss", a, pairs);
    const GradPlan p = grad_plan(N, H, V);
    std::printf("plan %d %d %d %d\n", p.piece, p.splits, p.pitch, p.parts);
    a.parts = p.parts;
    a.hidden = arg(6);
    a.weights = arg(7);
    for (int v0 = 0; v0 < V; v0 += p.piece) {
        a.N = N;
        a.v0 = v0;
        a.col_tiles = ceil_div(std::min(p.piece, V - v0), kTile);
        a.width = a.col_tiles * kTile;
        a.splits = std::min(p.splits, a.width / kStageK);
        keep_rows(a, kept);
        share_out(a, pairs);
        std::printf("piece %d %d %d %d %d %d\n", v0, a.width, a.row_tiles, a.splits, a.hidden_tiles, a.weight_tiles);
        walk<kScore>("score", a, pairs);
        walk<kGrad>("grad", a, pairs);
    }
    return 0;
}
