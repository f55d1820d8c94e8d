// head_work.cuh -- how the LM-head loss's products are cut into tiles and dealt out to the pairs of CTAs.  Arithmetic
// alone, so that a test can compile it for the host and follow every pair's share.
#pragma once

#include <algorithm>
#include <cstdint>

#ifdef __CUDACC__
#define DF2_HEAD_WORK __host__ __device__ __forceinline__
#else
#define DF2_HEAD_WORK inline
#endif

namespace df2 {
namespace head {

constexpr int kRows = 128;                        // of the accumulator a CTA
constexpr int kTile = 256;                        // rows and columns of a pair's tile
constexpr int kBlock = 64;                        // columns of an operand's box: one 128-byte swizzle row
constexpr int kStageK = 2 * kBlock;               // elements of K a stage

enum Mode { kLoss = 0, kScore = 1, kGrad = 2 };
enum Product { kHiddenGrad = 1, kWeightGrad = 2 };  // of a tile; 0: h . W^T

// What a launch of the matrix kernel has to do.
struct Work {
    int N, H, V;
    int v0, width;        // the piece's columns: [v0, v0 + width), width a multiple of 256, past V too
    int row_tiles, col_tiles, h_tiles;
    int parts;            // of dz
    // gradient products: tiles of d_hidden first, see tile_of
    int hidden, weights, splits, first;
    int hidden_tiles, weight_tiles, early;  // see share_out
};

struct Tile {
    int product;
    int m0, n0;           // rows of A and of B
    int k0, stages;       // in stages
    int split;
    bool live;
};

DF2_HEAD_WORK int larger(int a, int b) { return a > b ? a : b; }

DF2_HEAD_WORK int ceil_div(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

// Of the rows n are there; with none left one tile of zeros makes d_W's.
DF2_HEAD_WORK void keep_rows(Work &a, int n)
{
    a.N = n;
    a.row_tiles = larger(1, (n + kTile - 1) / kTile);
}

// The gradient's tiles, and how many turns of d_W's tiles take as long as one of d_hidden's: stages, and half of one
// for a tile's ends.
DF2_HEAD_WORK void share_out(Work &a, int pairs)
{
    a.hidden_tiles = a.hidden ? a.row_tiles * a.h_tiles * a.splits : 0;
    a.weight_tiles = a.weights ? a.col_tiles * a.h_tiles : 0;
    a.early = a.hidden_tiles % pairs == 0 ? 0
                                          : larger(1, (2 * (a.width / kStageK / a.splits) + 1) /
                                                          (2 * larger(1, (a.N * a.parts + kStageK - 1) / kStageK) + 1));
}

// The pair's i-th tile.
template <int MODE>
DF2_HEAD_WORK Tile tile_of(const Work &a, int pair, int pairs, int i)
{
    Tile t{};
    if constexpr (MODE != kGrad) {
        // (counts of tiles fit 32 bits: 16384 rows of the loss at a time, 2^28 elements of dz)
        const uint32_t u = static_cast<uint32_t>(pair + i * pairs), rows = static_cast<uint32_t>(a.row_tiles);
        const uint32_t n = u / rows;
        t.live = n < static_cast<uint32_t>(a.col_tiles);
        t.m0 = static_cast<int>(u - n * rows) * kTile;
        t.n0 = static_cast<int>(n) * kTile;
        t.stages = (a.H + kStageK - 1) / kStageK;
    } else {
        // d_hidden's tiles are long and few: they are dealt out first.  Pairs that get one less than the others
        // work on d_W's tiles meanwhile, for `early` turns, so that all end together.
        const int rest = a.hidden_tiles % pairs;
        const int mine = a.hidden_tiles / pairs + (pair < rest ? 1 : 0);
        const int others = pairs - rest;  // that have one less
        if (i < mine) {
            const int j = pair + i * pairs;
            const int per = a.row_tiles * a.h_tiles, in = j % per;
            const int ks = a.width / kStageK;
            t.product = kHiddenGrad;
            t.live = true;
            t.split = j / per;
            t.m0 = in / a.h_tiles * kTile;
            t.n0 = in % a.h_tiles * kTile;
            t.k0 = ks * t.split / a.splits;
            t.stages = ks * (t.split + 1) / a.splits - t.k0;
        } else {
            i -= mine;
            int j = a.early * others + i * pairs + pair;
            if (pair >= rest)
                j = i < a.early ? i * others + (pair - rest) : j - a.early * pairs;
            t.product = kWeightGrad;
            t.live = j < a.weight_tiles;
            const int down = static_cast<int>(static_cast<uint32_t>(j) / static_cast<uint32_t>(a.h_tiles));
            t.m0 = down * kTile;
            t.n0 = (j - down * a.h_tiles) * kTile;
            t.stages = larger(1, (a.N * a.parts + kStageK - 1) / kStageK);
        }
    }
    return t;
}

// How the gradient of the LM head's loss is cut up, from its sizes alone.
struct GradPlan {
    int piece;    // columns of the vocabulary at a time, a multiple of 256
    int splits;   // parts of a piece whose d_hidden is summed apart
    int pitch;    // elements of a row of the packed hidden states, a multiple of 64
    int parts;    // bf16 numbers that dz is held in: 2 with few rows
};

inline GradPlan grad_plan(int N, int H, int V)
{
    GradPlan p;
    N = larger(N, 1);
    // Few rows leave half of a tile's rows, and of a stage's, empty: dz goes there a second time, as what its rounding to
    // bf16 left, and the products are those of float32's dz at nearly the same cost (64 x 5120 x 152064: 807 us, 778
    // without; d_hidden and d_W are off by 1.7e-3, as their own rounding leaves them, instead of 2.1e-3 to 2.6e-3)
    p.parts = N <= kRows ? 2 : 1;
    // dz of a piece takes at most half a gigabyte (and the pieces are of one size)
    const long long most = std::max(1ll, (1ll << 28) / (N * p.parts) / kTile) * kTile;
    const int pieces = ceil_div(V, most);
    p.piece = ceil_div(ceil_div(V, pieces), kTile) * kTile;
    // d_hidden has few tiles where there are few rows: parts of the piece, of two stages at least, are then summed apart,
    // so that its tiles keep 48 of 76 pairs while the others begin with d_W's (10 x 744 x 114074: 128 us, 132 with tiles
    // for two turns of all pairs; 254 x 2032 x 18994: 72, 82; 43 x 2792 x 225575: 755, 804).  One row of many tiles is
    // bound by HBM, which reads and then writes faster than both at once: nearly two turns (16 x 4096 x 151936: 617 us,
    // 641 with 48; 64 x 5120 x 152064: 807, 820).
    const int row_tiles = ceil_div(N, kTile), h_tiles = ceil_div(H, kTile);
    const long long tiles = static_cast<long long>(row_tiles) * h_tiles;
    const long long most_tiles = row_tiles == 1 && h_tiles >= 12 ? 128 : 48;
    const long long most_parts = std::min(static_cast<long long>(p.piece / kStageK / 2), most_tiles / tiles);
    p.splits = static_cast<int>(std::max(1ll, most_parts));
    p.pitch = ceil_div(H, kBlock) * kBlock;
    return p;
}

}  // namespace head
}  // namespace df2
