// paged.cuh -- device helpers of the paged cache: where a token's rows are.
#pragma once

#include <cstdint>

#include "internal.h"

namespace df2 {

// The sequence that packed token n belongs to: the largest b with token_start[b] <= n.  One
// warp, 32 probes a step (B <= 2048: three loads deep at most).
__device__ __forceinline__ int warp_sequence_of(const int32_t *token_start, int B, int n, int lane)
{
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const bool below = at < hi && __ldg(token_start + at) <= n;
        const int c = __popc(__ballot_sync(0xffffffffu, below));
        lo += c > 0 ? (c - 1) * step : 0;
        hi = min(lo + step, hi);
    }
    return lo;
}

// Token n's position in its sequence, and the index of its row (of head 0) in units of rows of
// the cache: ((page * heads + head) * page_size + slot).  row < 0: the token has no place.
struct TokenPlace {
    int pos;
    long long row;
};

__device__ __forceinline__ TokenPlace place_in(const PagedCache &c, const TokenBatch &t, int b, int n)
{
    const int pos = __ldg(t.kv_len + b) - __ldg(t.token_start + b + 1) + n;
    TokenPlace p{pos, -1};
    if (pos >= 0 && static_cast<long long>(pos) < static_cast<long long>(t.max_pages) * c.page_size) {
        const int page = __ldg(t.page_table + static_cast<long long>(b) * t.max_pages + pos / c.page_size);
        if (page >= 0 && page < c.pages)
            p.row = static_cast<long long>(page) * c.heads * c.page_size + pos % c.page_size;
    }
    return p;
}

// Token n's place; one warp.
__device__ __forceinline__ TokenPlace token_place(const PagedCache &c, const TokenBatch &t, int n, int lane)
{
    return place_in(c, t, warp_sequence_of(t.token_start, t.B, n, lane), n);
}

// The places of the tokens n0 .. n0 + count - 1 (count <= 32), a lane each; one warp.
__device__ __forceinline__ TokenPlace lane_token_place(const PagedCache &c, const TokenBatch &t, int n0, int count,
                                                       int lane)
{
    int b = warp_sequence_of(t.token_start, t.B, n0, lane);
    if (lane >= count)
        return TokenPlace{0, -1};
    while (b + 1 < t.B && __ldg(t.token_start + b + 1) <= n0 + lane)
        ++b;
    return place_in(c, t, b, n0 + lane);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two floats rounded to nearest even, `a` in the low half.
__device__ __forceinline__ uint32_t bf16_pack(float a, float b)
{
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    return d;
}

}  // namespace df2
