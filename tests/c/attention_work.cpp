/* Follows the attention kernel's walk over its work on the host.
 *   argv: mode, causal, window, span, item_cost, heads, grid, then n and len of each sequence
 *   walk:  a line for every segment of every CTA
 *   begin: a line for every CTA: its share, and where its walk begins */
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "attention_work.cuh"

using namespace df2;

int main(int argc, char **argv)
{
    if (argc < 10 || (argc - 8) % 2 != 0)
        return 2;
    auto arg = [&](int i) { return std::atoi(argv[i]); };
    const WorkShape w{arg(2), arg(3), arg(4), arg(5), arg(6)};
    std::vector<Sequence> all;
    int start = 0;
    for (int i = 8; i < argc; i += 2) {
        all.push_back(Sequence{start, arg(i), arg(i + 1)});
        start += arg(i);
    }
    std::vector<long long> ahead{0};
    for (const Sequence &s : all)
        ahead.push_back(ahead.back() + units_of(w, s, 0, 1));
    const long long units = ahead.back() * w.heads;
    const int grid = static_cast<int>(min(static_cast<long long>(arg(7)), max(units, 1ll)));
    const Shares shares(units, grid);
    auto sequence = [&](int b) { return all[static_cast<size_t>(b)]; };
    for (int c = 0; c < grid && units > 0; ++c) {
        const long long u = shares.begin(c);
        int b = 0;
        while (b + 1 < static_cast<int>(all.size()) && ahead[b + 1] * w.heads <= u)
            ++b;
        Walk walk;
        walk.begin(w, sequence, u, shares.begin(c + 1), b, ahead[b], ahead[b + 1] - ahead[b]);
        if (std::strcmp(argv[1], "begin") == 0) {
            std::printf("%lld %lld %d %d %d %d\n", walk.u, walk.u_end, walk.b, walk.kvh, walk.qt, walk.off);
            continue;
        }
        for (Segment g;;) {
            walk.next(w, sequence, c, shares, g);
            if (g.tiles == 0)
                break;
            std::printf("%d %d %d %d %d %d %d %d %d %d %d\n", c, g.b, g.kvh, g.start, g.item.tok0, g.tile, g.tiles,
                        g.first, g.last, g.slot, g.first && !g.last ? g.end_cta : -1);
        }
    }
    return 0;
}
