// attention_work.cuh -- how the attention kernel's work is cut up among the CTAs.  Arithmetic alone, so
// that a test can compile it for the host and follow every CTA's share.
//
// Counts of work are 64-bit: a causal prompt of 1.5 million tokens with 64 query heads on a cache head
// has 2^31 units, and the limits on sizes allow some 2^46.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define DF2_WORK __device__ __forceinline__
#else
#include <algorithm>
#define DF2_WORK inline
#endif

namespace df2 {

#ifndef __CUDACC__
using std::max;
using std::min;
#endif

constexpr int BN = 128;  // keys of a tile

struct WorkShape {
    int causal, window;
    int span;       // tokens of an item
    int item_cost;  // key tiles that an item costs besides its own
    int heads;      // of the cache
};

struct Sequence {
    int start, n, len;  // first packed token, new tokens, length with them
};

struct Item {
    int tok0, ntok;    // first token in its sequence, tokens
    int p0;            // position of the first
    int lo, hi;        // positions some row sees
    int tile0, tiles;  // key tiles (one, empty, if nothing is seen)

    DF2_WORK int units(const WorkShape &w) const { return tiles + w.item_cost; }
};

DF2_WORK Item item_at(const WorkShape &w, const Sequence &s, int qt)
{
    Item it;
    it.tok0 = qt * w.span;
    it.ntok = min(s.n - it.tok0, w.span);
    it.p0 = s.len - s.n + it.tok0;
    it.hi = w.causal ? min(s.len, it.p0 + it.ntok) : s.len;
    it.lo = w.window > 0 && it.p0 >= w.window ? it.p0 - w.window + 1 : 0;
    if (it.hi <= it.lo) {
        it.lo = it.hi = it.tile0 = 0;
        it.tiles = 1;
    } else {
        it.tile0 = it.lo / BN;
        it.tiles = (it.hi - 1) / BN - it.tile0 + 1;
    }
    return it;
}

DF2_WORK int items_of(const WorkShape &w, const Sequence &s)
{
    return static_cast<int>((static_cast<unsigned>(s.n) + w.span - 1) / w.span);
}

// Units of every step-th item of a sequence from `first` on, for one cache head.
DF2_WORK long long units_of(const WorkShape &w, const Sequence &s, int first, int step)
{
    const int nq = items_of(w, s);
    long long t = 0;
    for (int qt = first; qt < nq; qt += step)
        t += item_at(w, s, qt).units(w);
    return t;
}

// A run of key tiles of one item.
struct Segment {
    Item item;
    int b, kvh, start;   // start: the sequence's first packed token
    int tile, tiles;
    int first, last;     // has the item's first / last tile
    int slot;            // where a piece of an item goes
    int end_cta;         // of an item that begins here and ends elsewhere: the CTA with its last tile
    int spoilt;          // a value row that its tiles hold is not finite (8-bit caches; set on the way)
};

DF2_WORK long long quotient(long long a, long long b)
{
    return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

// `units` cut into `grid` shares, share c beginning at floor(c units / grid).
struct Shares {
    long long units, each;
    int grid, more;

    DF2_WORK Shares(long long n, int g) : units(n), each(quotient(n, g)), grid(g)
    {
        more = static_cast<int>(n - each * g);
    }
    DF2_WORK long long begin(int c) const
    {
        return c * each + static_cast<unsigned>(c * more) / static_cast<unsigned>(grid);
    }
    DF2_WORK int owner(long long u) const { return static_cast<int>(((u + 1) * grid - 1) / units); }
};

// The segments of a CTA's share [u, u_end) of the units, cache head by cache head, item by item.  An
// item has a unit for each key tile and, before them, some for its queries, its first score and its
// results: CTAs with short items would else finish last.
struct Walk {
    long long u, u_end;
    int pieces;
    int b, kvh, qt, off, nq;  // off: units of the item that are over
    Sequence s;

    // Sequence b0, whose units begin at heads * ahead and which has `units` of them for a cache head, is
    // the last one that begins at or before u0.
    template <class Sequences>
    DF2_WORK void begin(const WorkShape &w, const Sequences &sequence, long long u0, long long u1, int b0,
                        long long ahead, long long units)
    {
        u = u0;
        u_end = u1;
        pieces = 0;
        b = b0;
        s = sequence(b);
        nq = items_of(w, s);
        const long long per_head = max(units, 1ll), r = u - ahead * w.heads;
        kvh = static_cast<int>(quotient(r, per_head));
        long long left = r - kvh * per_head;
        for (qt = 0; qt + 1 < nq; ++qt) {
            const int t = item_at(w, s, qt).units(w);
            if (left < t)
                break;
            left -= t;
        }
        off = static_cast<int>(left);
    }

    template <class Sequences>
    DF2_WORK void next(const WorkShape &w, const Sequences &sequence, int cta, const Shares &shares, Segment &g)
    {
        g.tiles = 0;
        while (g.tiles == 0 && u < u_end) {
            while (kvh == w.heads) {  // the next sequence that has tokens
                ++b;
                s = sequence(b);
                nq = items_of(w, s);
                kvh = nq > 0 ? 0 : w.heads;
            }
            g.item = item_at(w, s, qt);
            g.b = b;
            g.kvh = kvh;
            g.start = s.start;
            const int n = static_cast<int>(min(static_cast<long long>(g.item.units(w) - off), u_end - u));
            const int from = max(off - w.item_cost, 0), to = off + n - w.item_cost;
            u += n;
            off += n;
            if (to > from) {
                g.tile = g.item.tile0 + from;
                g.tiles = to - from;
                g.first = from == 0;
                g.last = to == g.item.tiles;
                g.slot = 2 * cta + pieces++;
                if (g.first && !g.last)
                    g.end_cta = shares.owner(u - off + g.item.units(w) - 1);
            }
            if (off == g.item.units(w)) {
                off = 0;
                if (++qt == nq) {
                    qt = 0;
                    ++kvh;
                }
            }
        }
        pieces = min(pieces, 1);  // only a CTA's first and last segments can be pieces
    }
};

}  // namespace df2
