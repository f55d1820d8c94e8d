// cache.cu -- rotary positions, and the paged cache's quantising write and read-back.
//
// Rotation: pair i of a head turns by the angle position * f_i,
//   (a, b) -> (a c_i - b s_i, b c_i + a s_i),
// an orthogonal map, so its transpose (the gradient) is the same with -s_i.  Cosines and sines
// come from a table made once in double: in float32 the angle itself is off by position * 2^-24
// radians, 6e-3 at position 100,000.
// Quantisation of a row x (one token, one head): m = max |x|, scale = m / M, code = rn(x M / m).
// M / m and m / M are correctly rounded divisions, one each per row; a multiplication per element
// in place of a division changes a code only where x M / m is within 2 ulp of a rounding boundary.
//
// Both kernels only move data: 2 bytes in and 2 (bf16) or 1 (8-bit) out per element, a few
// operations each, so HBM bounds long calls and latency short ones.  A row is at most 256 bytes (512
// where it is only rotated): 16 (32) lanes hold one, 8 elements or 16 bytes a lane.  A warp works on
// rows of one token, so the sequence lookup, the page lookup and the cosines and sines in registers
// serve all of its rows, and every pair's partner is in the lane itself or one shuffle away.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace df2 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kTiny = 1e-30f;  // rows below this are held as zeros (M / m would overflow near 1e-36)

enum CacheType { kBf16 = 0, kE4m3 = 1, kInt8 = 2 };

struct RowsArgs {
    PagedCache cache;
    TokenBatch tokens;
    RopeTable rope;
    HeadRows q, q_out, k, v;
    const int32_t *positions;  // plain rotation: positions of the tokens (no cache)
    int N, dim;
    float sine_sign;
    int rows;            // rows of a token: q heads, then cache heads of k, then of v
    int units_per_token;
    int vec_table;  // cosines and sines in 16-byte loads
    int shuffle;    // half layout: partners are whole chunks of other lanes
};

// Row h of token n: of q, then of k, then of v.
template <bool CACHE>
__device__ __forceinline__ const uint16_t *source_row(const RowsArgs &a, int n, int h)
{
    const int qh = a.q.heads, kvh = CACHE ? a.cache.heads : 0;
    if (!CACHE || h < qh)
        return a.q.data + n * a.q.token_stride + h * a.q.head_stride;
    const HeadRows &s = h < qh + kvh ? a.k : a.v;
    return s.data + n * s.token_stride + (h - (h < qh + kvh ? qh : qh + kvh)) * s.head_stride;
}

// Cosines and signed sines of the 8 elements of chunk `c`.
__device__ __forceinline__ void load_turn(const RowsArgs &a, int pos, int c, float (&cs)[8], float (&sn)[8])
{
    const int rot = a.rope.rot, half = rot / 2;
    const float *t = a.rope.table + static_cast<long long>(min(max(pos, 0), a.rope.max_pos - 1)) * rot;
    const float sg = a.sine_sign;
    if (a.vec_table && 8 * c < rot) {  // rot a multiple of 8: the chunk turns whole
        if (a.rope.interleaved) {
            const float4 x = __ldg(reinterpret_cast<const float4 *>(t + 4 * c));
            const float4 y = __ldg(reinterpret_cast<const float4 *>(t + half + 4 * c));
            cs[0] = cs[1] = x.x, cs[2] = cs[3] = x.y, cs[4] = cs[5] = x.z, cs[6] = cs[7] = x.w;
            sn[1] = sg * y.x, sn[3] = sg * y.y, sn[5] = sg * y.z, sn[7] = sg * y.w;
            sn[0] = -sn[1], sn[2] = -sn[3], sn[4] = -sn[5], sn[6] = -sn[7];
            return;
        }
        if (a.shuffle) {
            const bool second = 8 * c >= half;
            const float *p = t + 8 * c - (second ? half : 0);
            const float s = second ? sg : -sg;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 x = __ldg(reinterpret_cast<const float4 *>(p) + i);
                const float4 y = __ldg(reinterpret_cast<const float4 *>(p + half) + i);
                cs[4 * i] = x.x, cs[4 * i + 1] = x.y, cs[4 * i + 2] = x.z, cs[4 * i + 3] = x.w;
                sn[4 * i] = s * y.x, sn[4 * i + 1] = s * y.y, sn[4 * i + 2] = s * y.z, sn[4 * i + 3] = s * y.w;
            }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int e = 8 * c + j;
        cs[j] = 1.f, sn[j] = 0.f;
        if (e < rot) {
            const int i = a.rope.interleaved ? e >> 1 : (e < half ? e : e - half);
            const bool second = a.rope.interleaved ? (e & 1) != 0 : e >= half;
            cs[j] = __ldg(t + i);
            sn[j] = second ? sg * __ldg(t + half + i) : -sg * __ldg(t + half + i);
        }
    }
}

// x (8 elements of chunk c of row h of token n) turned in place.  All lanes of the warp call it.
template <int LG, bool CACHE>
__device__ __forceinline__ void turn(const RowsArgs &a, int n, int h, const uint4 &raw, bool live, int c, int lane,
                                     const float (&cs)[8], const float (&sn)[8], float (&x)[8])
{
    const int rot = a.rope.rot, half = rot / 2;
    float p[8];
    if (a.rope.interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            p[j] = x[j ^ 1];
    } else if (a.shuffle) {
        const int h8 = half / 8;
        const int src = c < h8 ? c + h8 : c < 2 * h8 ? c - h8 : c;
        const int from = (lane & ~(LG - 1)) | src;
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t o = __shfl_sync(0xffffffffu, w[i], from);
            p[2 * i] = bf16_lo(o), p[2 * i + 1] = bf16_hi(o);
        }
    } else {  // pairs that start inside a chunk
        const uint16_t *row = source_row<CACHE>(a, n, live ? h : 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = 8 * c + j;
            p[j] = live && e < rot ? bf16_lo(row[e < half ? e + half : e - half]) : 0.f;
        }
    }
    // one by one: a packed product and a packed sum come out as one rounding (measured), and the codes
    // of an 8-bit cache are to be those of the formula's separate operations
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (8 * c + j < rot)
            x[j] = __fadd_rn(__fmul_rn(x[j], cs[j]), __fmul_rn(p[j], sn[j]));
}

__device__ __forceinline__ void widen(const uint4 &r, float (&x)[8])
{
    x[0] = bf16_lo(r.x), x[1] = bf16_hi(r.x), x[2] = bf16_lo(r.y), x[3] = bf16_hi(r.y);
    x[4] = bf16_lo(r.z), x[5] = bf16_hi(r.z), x[6] = bf16_lo(r.w), x[7] = bf16_hi(r.w);
}

__device__ __forceinline__ uint4 narrow(const float (&x)[8])
{
    return make_uint4(bf16_pack(x[0], x[1]), bf16_pack(x[2], x[3]), bf16_pack(x[4], x[5]), bf16_pack(x[6], x[7]));
}

__device__ __forceinline__ uint32_t e4m3x4(const float *x)
{
    uint16_t a, b;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(a) : "f"(x[1]), "f"(x[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(x[3]), "f"(x[2]));
    return static_cast<uint32_t>(a) | static_cast<uint32_t>(b) << 16;
}

__device__ __forceinline__ uint32_t int8x4(const float *x)
{
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w |= (static_cast<uint32_t>(min(max(__float2int_rn(x[i]), -127), 127)) & 0xFFu) << (8 * i);
    return w;
}

// One row (16-byte chunk c of it in `raw`), rotated and written where it belongs.  All lanes of the
// warp call it.
template <int LG, bool CACHE>
__device__ __forceinline__ void put_row(const RowsArgs &a, const uint4 &raw, int h, int n, int c,
                                        int lane, bool turns, const float (&cs)[8], const float (&sn)[8],
                                        const TokenPlace &place)
{
    const bool in_dim = 8 * c < a.dim, live = h < a.rows;
    const int qh = a.q.heads, kvh = CACHE ? a.cache.heads : 0;
    float x[8];
    widen(raw, x);
    // values are not rotated: a warp that has only those skips it
    const bool turned = turns && live && (!CACHE || h < qh + kvh);
    if (__any_sync(0xffffffffu, turned)) {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            y[j] = x[j];
        turn<LG, CACHE>(a, n, h, raw, live && in_dim, c, lane, cs, sn, y);
        if (turned) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = y[j];
        }
        __syncwarp();  // q_out may be q: partners are read before any lane writes
    }
    if (!CACHE || h < qh) {
        if (live && in_dim)
            *reinterpret_cast<uint4 *>(a.q_out.data + n * a.q_out.token_stride + h * a.q_out.head_stride + 8 * c) =
                narrow(x);
    }
    if constexpr (CACHE) {
        const bool is_v = h >= qh + kvh;
        const int hh = h - qh - (is_v ? kvh : 0);
        const bool put = live && h >= qh && place.row >= 0;
        const long long row = place.row + static_cast<long long>(hh) * a.cache.page_size;
        if (a.cache.type == kBf16) {
            if (put && in_dim)
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(is_v ? a.cache.v : a.cache.k) + row * a.dim + 8 * c) =
                    narrow(x);
            return;
        }
        if (!__any_sync(0xffffffffu, put))  // queries only
            return;
        // magnitudes compare as integers, with infinities and NaN above every finite value
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            m = max(m, __float_as_uint(x[j]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = LG / 2; o > 0; o >>= 1)
            m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float top = a.cache.type == kE4m3 ? 448.f : 127.f;
        const float mf = __uint_as_float(m);
        const bool finite = m < 0x7F800000u, held = finite && mf >= kTiny;
        const float inv = held ? __fdiv_rn(top, mf) : 0.f;
        const float scale = held ? __fdiv_rn(mf, top) : finite ? 0.f : __uint_as_float(0x7FC00000u);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = held ? __fmul_rn(x[j], inv) : 0.f;
        if (put && in_dim) {
            uint2 w;
            if (a.cache.type == kE4m3)
                w = make_uint2(e4m3x4(x), e4m3x4(x + 4));
            else
                w = make_uint2(int8x4(x), int8x4(x + 4));
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(is_v ? a.cache.v : a.cache.k) + row * a.dim + 8 * c) = w;
            if (c == 0)
                (is_v ? a.cache.v_scale : a.cache.k_scale)[row] = scale;
        }
    }
}

// LG lanes a row, R rows a lane at a time.  CACHE: append (q rotated to q_out, k and v into the
// cache), else plain rotation of q to q_out.
// One step (few tokens): a warp takes R * 32 / LG rows of a token.
template <int LG, int R, bool CACHE>
__global__ void __launch_bounds__(kThreads, 4) rows_kernel(const RowsArgs a)
{
    constexpr int kGroups = 32 / LG;
    const int lane = threadIdx.x & 31, c = lane & (LG - 1), grp = lane / LG;
    const int unit = blockIdx.x * kWarps + static_cast<int>(threadIdx.x >> 5);
    griddep_launch_dependents();
    griddep_wait();
    const int n = unit / a.units_per_token;
    if (n >= a.N)
        return;
    const int first = (unit - n * a.units_per_token) * R * kGroups + grp;
    uint4 raw[R];  // loaded before the lookups, which they do not wait for
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int h = first + i * kGroups;
        raw[i] = h < a.rows && 8 * c < a.dim ? *reinterpret_cast<const uint4 *>(source_row<CACHE>(a, n, h) + 8 * c)
                                             : make_uint4(0, 0, 0, 0);
    }
    TokenPlace place{0, -1};
    if constexpr (CACHE)
        place = token_place(a.cache, a.tokens, n, lane);
    else
        place.pos = __ldg(a.positions + n);
    float cs[8], sn[8];
    const bool turns = a.rope.table != nullptr;
    if (turns)
        load_turn(a, place.pos, c, cs, sn);
#pragma unroll
    for (int i = 0; i < R; ++i)
        put_row<LG, CACHE>(a, raw[i], first + i * kGroups, n, c, lane, turns, cs, sn, place);
}

// Many tokens: a warp takes all rows of `run` tokens in a row, the next R rows a lane on their way
// while R are worked on.  The tokens' places are looked up at once, a lane each, and the next
// token's cosines and sines are asked for when only values, which do not turn, are left of this one.
// At the 64 registers that four CTAs an SM leave, a thread spills 40 to 64 bytes.
template <int LG, int R, bool CACHE>
__global__ void __launch_bounds__(kThreads, 4) rows_run_kernel(const RowsArgs a, int run)
{
    constexpr int kGroups = 32 / LG, kStep = R * kGroups;
    const int lane = threadIdx.x & 31, c = lane & (LG - 1), grp = lane / LG;
    const int n0 = (blockIdx.x * kWarps + static_cast<int>(threadIdx.x >> 5)) * run;
    griddep_launch_dependents();
    griddep_wait();
    if (n0 >= a.N)
        return;
    const int count = min(run, a.N - n0);
    uint4 raw[R], next[R];
    auto load = [&](int n, int h0, uint4(&to)[R]) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int h = h0 + grp + i * kGroups;
            to[i] = h < a.rows && 8 * c < a.dim ? *reinterpret_cast<const uint4 *>(source_row<CACHE>(a, n, h) + 8 * c)
                                                : make_uint4(0, 0, 0, 0);
        }
    };
    load(n0, 0, raw);
    TokenPlace mine{0, -1};  // of token n0 + lane
    if constexpr (CACHE)
        mine = lane_token_place(a.cache, a.tokens, n0, count, lane);
    else
        mine.pos = lane < count ? __ldg(a.positions + n0 + lane) : 0;
    float cs[8], sn[8];
    const bool turns = a.rope.table != nullptr;
    const int turned = CACHE ? a.q.heads + a.cache.heads : a.rows;  // rows that turn
    if (turns)
        load_turn(a, __shfl_sync(0xffffffffu, mine.pos, 0), c, cs, sn);
    for (int t = 0; t < count; ++t) {
        const int n = n0 + t;
        const TokenPlace place{0, __shfl_sync(0xffffffffu, mine.row, t)};
        const int next_pos = __shfl_sync(0xffffffffu, mine.pos, min(t + 1, count - 1));
        for (int h0 = 0; h0 < a.rows; h0 += kStep) {
            const bool more = h0 + kStep < a.rows;
            load(more ? n : min(n + 1, n0 + count - 1), more ? h0 + kStep : 0, next);
#pragma unroll
            for (int i = 0; i < R; ++i)
                put_row<LG, CACHE>(a, raw[i], h0 + grp + i * kGroups, n, c, lane, turns, cs, sn, place);
            if (turns && h0 < turned && h0 + kStep >= turned)
                load_turn(a, next_pos, c, cs, sn);
#pragma unroll
            for (int i = 0; i < R; ++i)
                raw[i] = next[i];
        }
    }
}

struct ReadArgs {
    PagedCache cache;
    TokenBatch tokens;
    HeadRows k, v;
    int rows, units_per_token;
};

__device__ __forceinline__ void e4m3_widen(uint32_t w, float *x)
{
    uint32_t a, b;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"(static_cast<uint16_t>(w)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"(static_cast<uint16_t>(w >> 16)));
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}" : "=f"(x[0]), "=f"(x[1]) : "r"(a));
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}" : "=f"(x[2]), "=f"(x[3]) : "r"(b));
}

template <int R>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadArgs a)
{
    const int lane = threadIdx.x & 31, c = lane & 15, grp = lane >> 4;
    const int unit = blockIdx.x * kWarps + static_cast<int>(threadIdx.x >> 5);
    griddep_launch_dependents();
    griddep_wait();
    const int n = unit / a.units_per_token;
    if (n >= a.tokens.N)
        return;
    const int row0 = (unit - n * a.units_per_token) * (R * 2) + grp;
    const int kvh = a.cache.heads, dim = a.cache.dim;
    const bool in_dim = 8 * c < dim;
    const TokenPlace place = token_place(a.cache, a.tokens, n, lane);
    uint4 raw[R];
    float scale[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int h = row0 + 2 * i;
        raw[i] = make_uint4(0, 0, 0, 0);
        scale[i] = 0.f;
        const bool is_v = h >= kvh;
        if (h < a.rows && place.row >= 0 && in_dim && (is_v ? a.v.data : a.k.data)) {
            const long long row = place.row + static_cast<long long>(h - (is_v ? kvh : 0)) * a.cache.page_size;
            const void *base = is_v ? a.cache.v : a.cache.k;
            if (a.cache.type == kBf16) {
                raw[i] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + row * dim + 8 * c);
            } else {
                const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(base) + row * dim + 8 * c);
                raw[i].x = w.x, raw[i].y = w.y;
                scale[i] = (is_v ? a.cache.v_scale : a.cache.k_scale)[row];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int h = row0 + 2 * i;
        if (h >= a.rows || !in_dim)
            continue;
        const bool is_v = h >= kvh;
        const HeadRows &o = is_v ? a.v : a.k;
        if (!o.data)
            continue;
        if (a.cache.type != kBf16) {
            float x[8];
            if (a.cache.type == kE4m3) {
                e4m3_widen(raw[i].x, x);
                e4m3_widen(raw[i].y, x + 4);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[j] = static_cast<float>(static_cast<int8_t>((j < 4 ? raw[i].x : raw[i].y) >> (8 * (j & 3))));
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = __fmul_rn(x[j], scale[i]);
            raw[i] = narrow(x);
        }
        *reinterpret_cast<uint4 *>(o.data + n * o.token_stride + (h - (is_v ? kvh : 0)) * o.head_stride + 8 * c) = raw[i];
    }
}

// cos and sin of position * f_i in double, one thread a pair.
__global__ void rope_table_kernel(const RopeScaling s, int max_pos, int rot, float *table)
{
    const int half = rot / 2;
    const long long at = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    griddep_launch_dependents();
    griddep_wait();
    if (at >= static_cast<long long>(max_pos) * half)
        return;
    const int pos = static_cast<int>(at / half), i = static_cast<int>(at % half);
    const double two_pi = 6.283185307179586476925286766559;
    const double theta = s.kind == 2 ? s.theta * pow(s.factor, rot / (rot - 2.0)) : s.theta;
    double f = pow(theta, -2.0 * i / rot);
    if (s.kind == 1) {
        f /= s.factor;
    } else if (s.kind == 3) {
        // pair index at which a pair turns r times within original_len positions
        const double per = rot / (2.0 * log(s.theta));
        const double lo = fmax(floor(per * log(s.original_len / (s.high * two_pi))), 0.0);
        const double hi = fmin(ceil(per * log(s.original_len / (s.low * two_pi))), rot - 1.0);
        const double ramp = fmin(fmax((i - lo) / fmax(hi - lo, 1e-3), 0.0), 1.0);
        f = f * (1.0 - ramp) + f / s.factor * ramp;
    } else if (s.kind == 4) {
        const double turns = s.original_len * f / two_pi;
        const double keep = fmin(fmax((turns - s.low) / (s.high - s.low), 0.0), 1.0);
        f = f * keep + f / s.factor * (1.0 - keep);
    }
    double sn, cs;
    sincos(pos * f, &sn, &cs);
    float *t = table + static_cast<long long>(pos) * rot;
    t[i] = static_cast<float>(cs * s.multiplier);
    t[half + i] = static_cast<float>(sn * s.multiplier);
}

template <int LG, int R, bool CACHE>
cudaError_t launch_step(RowsArgs a, cudaStream_t stream)
{
    constexpr int kPerWarp = R * (32 / LG);
    a.units_per_token = (a.rows + kPerWarp - 1) / kPerWarp;
    const long long units = static_cast<long long>(a.N) * a.units_per_token;
    const unsigned grid = static_cast<unsigned>((units + kWarps - 1) / kWarps);
    return launch_dependent(rows_kernel<LG, R, CACHE>, dim3(grid), dim3(kThreads), 0, stream, a);
}

template <int LG, bool CACHE>
cudaError_t launch_rows(RowsArgs a, cudaStream_t stream)
{
    const int rot = a.rope.rot;
    a.vec_table = rot % 8 == 0 && reinterpret_cast<uintptr_t>(a.rope.table) % 16 == 0;
    a.shuffle = !a.rope.interleaved && (rot / 2) % 8 == 0;
    // A warp's life is a chain of loads (the sequence, its length, the page, the cosines) whatever it
    // carries, so it should carry much while enough warps are left: a row a lane while that fits 32
    // warps an SM, then four, then whole tokens with the next rows on their way, and several tokens
    // where they have few rows.  Measured on GB300, four rows a lane against whole tokens: 2048
    // tokens of 48 rows to int8 19.1 and 28.4 us, 8195 of 32 rows turned 29.8 and 28.8, 16384 of 48
    // to e4m3 107.6 and 88.9; one token a warp against twenty: 100,000 of 4 rows 74 and 54 us.
    const long long rows = static_cast<long long>(a.N) * a.rows, wave = 32LL * device_sm_count();
    if (rows <= wave * (32 / LG))
        return launch_step<LG, 1, CACHE>(a, stream);
    if (rows <= 16 * wave * (32 / LG))
        return launch_step<LG, 4, CACHE>(a, stream);
    const int run = a.rows >= 32 ? 1 : static_cast<int>(std::max<long long>(1, std::min<long long>(std::min(32, 96 / a.rows), (a.N + wave - 1) / wave)));
    const unsigned grid = static_cast<unsigned>((static_cast<long long>(a.N) + run * kWarps - 1) / (run * kWarps));
    return launch_dependent(rows_run_kernel<LG, 2, CACHE>, dim3(grid), dim3(kThreads), 0, stream, a, run);
}

}  // namespace

cudaError_t launch_rope_table(const RopeScaling &s, int max_pos, int rot, float *table, cudaStream_t stream)
{
    const long long n = static_cast<long long>(max_pos) * (rot / 2);
    return launch_dependent(rope_table_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, stream, s,
                            max_pos, rot, table);
}

cudaError_t launch_rope(const RopeTable &rope, int N, int dim, const HeadRows &x, const int32_t *positions,
                        float sine_sign, const HeadRows &y, cudaStream_t stream)
{
    RowsArgs a{};
    a.rope = rope;
    a.q = x;
    a.q_out = y;
    a.positions = positions;
    a.N = N;
    a.dim = dim;
    a.sine_sign = sine_sign;
    a.rows = x.heads;
    return dim > 128 ? launch_rows<32, false>(a, stream) : launch_rows<16, false>(a, stream);
}

cudaError_t launch_cache_append(const PagedCache &cache, const TokenBatch &tokens, const RopeTable &rope,
                                const HeadRows &q, const HeadRows &q_out, const HeadRows &k, const HeadRows &v,
                                cudaStream_t stream)
{
    RowsArgs a{};
    a.cache = cache;
    a.tokens = tokens;
    a.rope = rope;
    a.q = q;
    a.q_out = q_out;
    a.k = k;
    a.v = v;
    a.N = tokens.N;
    a.dim = cache.dim;
    a.sine_sign = 1.f;
    a.rows = q.heads + 2 * cache.heads;
    return launch_rows<16, true>(a, stream);  // a cache's dim is at most 128
}

cudaError_t launch_cache_read(const PagedCache &cache, const TokenBatch &tokens, const HeadRows &k_out,
                              const HeadRows &v_out, cudaStream_t stream)
{
    ReadArgs a{};
    a.cache = cache;
    a.tokens = tokens;
    a.k = k_out;
    a.v = v_out;
    a.rows = 2 * cache.heads;
    // rows a lane holds at once: more of them share a lookup, but the call must spread over the SMs
    // (65536 tokens of 2 * 8 rows 73.7 us at 4, 70.3 at 8; 5,000 of 2 * 3 rows 5.1 and 6.1 us)
    const long long rows = static_cast<long long>(tokens.N) * a.rows;
    const int per_lane = rows <= 16LL * device_sm_count() * kWarps ? 1 : rows <= 256LL * device_sm_count() * kWarps ? 4 : 8;
    a.units_per_token = (a.rows + 2 * per_lane - 1) / (2 * per_lane);
    const long long units = static_cast<long long>(tokens.N) * a.units_per_token;
    const dim3 grid(static_cast<unsigned>((units + kWarps - 1) / kWarps));
    const auto kernel = per_lane == 1 ? read_kernel<1> : per_lane == 4 ? read_kernel<4> : read_kernel<8>;
    return launch_dependent(kernel, grid, dim3(kThreads), 0, stream, a);
}

}  // namespace df2
