// norm.cu -- root-mean-square norm of hidden states with the residual's addition, and its gradient.
//
//   z = x + residual,  n = sqrt(mean(z^2) + eps),  y = gamma z / n
//   dz = (u - z mean(u z) / n^2) / n  with u = gamma dy,   dgamma = sum over rows of dy z / n
//
// HBM-bound: a row is read once, kept in registers between the reduction and the result, and written
// once.  Bytes a row of C: 8 C forward with a residual (6 C + C + 4 with 8-bit codes in place of y), 8 C
// backward with the residual stream's gradient.
//
// A row is a warp's up to 1024 channels and a CTA's beyond; a thread keeps up to four 16-byte chunks (eight channels)
// of each tensor, as many as leave the fewest threads without one.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "f32x2.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace df2 {
namespace {

constexpr int kMaxWarps = 32;     // of a CTA
constexpr int kSmem = 227 * 1024; // of an SM
constexpr float kTiny = 1e-30f;   // a row of codes whose largest magnitude is below this is held as zeros
// The sum of squares is taken as it is between these; outside, squares may have been lost or overflowed.
constexpr float kLeast = 1e-24f, kMost = 1e36f;
// In the gradient it stands next to the sum of u z, which has to hold for any u from 1e-32 to 1e32: a row whose root of
// the sum is below a thousandth or above a million is brought near one first.
constexpr float kGradLeast = 1e-6f, kGradMost = 1e12f;

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8])
{
    f[0] = lo(v.x), f[1] = hi(v.x), f[2] = lo(v.y), f[3] = hi(v.y);
    f[4] = lo(v.z), f[5] = hi(v.z), f[6] = lo(v.w), f[7] = hi(v.w);
}

// Eight bf16 as four pairs of float32.
__device__ __forceinline__ void unpack8x2(const uint4 &v, uint64_t (&p)[4])
{
    p[0] = f2(lo(v.x), hi(v.x));
    p[1] = f2(lo(v.y), hi(v.y));
    p[2] = f2(lo(v.z), hi(v.z));
    p[3] = f2(lo(v.w), hi(v.w));
}

__device__ __forceinline__ uint32_t pack2x(uint64_t v)
{
    const float2 f = f2_split(v);
    return pack2(f.x, f.y);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
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
        w |= (static_cast<uint32_t>(__float2int_rn(fminf(fmaxf(x[i], -127.f), 127.f))) & 0xFFu) << (8 * i);
    return w;
}

struct Sum {
    __device__ static float apply(float a, float b) { return a + b; }
};
// NaN wins over everything, so that a row that holds one is found out by its maximum.
struct Max {
    __device__ static float apply(float a, float b) { return a > b || a != a ? a : b; }
};

// The N values of each thread reduced over the threads of a row (WARP: a warp, otherwise the CTA), in one order;
// every thread gets them.  `slots` holds two turns of kMaxWarps values for each of MOST, the most that the kernel
// reduces at once; `turn` tells a call's from the one's before, whose values another warp may still be reading.
template <bool WARP, typename Op, int MOST, int N>
__device__ __forceinline__ void row_reduce(float (&v)[N], float *slots, int &turn)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int d = 16; d > 0; d /= 2)
            v[i] = Op::apply(v[i], __shfl_xor_sync(0xffffffffu, v[i], d));
    if constexpr (!WARP) {
        const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        float *mine = slots + turn * MOST * kMaxWarps;
        turn ^= 1;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < N; ++i)
                mine[i * kMaxWarps + warp] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float t = mine[i * kMaxWarps];
            for (int w = 1; w < warps; ++w)
                t = Op::apply(t, mine[i * kMaxWarps + w]);
            v[i] = t;
        }
    }
}

// The power of two that brings m (finite, positive) into [1, 2), kept within what float32 holds.
__device__ __forceinline__ float scale_to_one(float m)
{
    const int e = min(max(static_cast<int>(__float_as_uint(m) >> 23) - 127, -126), 126);
    return __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

// What a row of largest magnitude m is multiplied by before its squares are summed: m comes near one, but
// eps k^2 stays below four (beyond, the row is nothing next to eps).
__device__ __forceinline__ float row_scale(float m, float eps)
{
    if (!(m > 0.f && m <= 3.4028234e38f))
        return 1.f;
    const float k = scale_to_one(m);
    return eps > 0.f ? fminf(k, scale_to_one(sqrtf(eps))) : k;
}

struct NormArgs {
    int N, C;
    const uint4 *x, *residual, *gamma;
    float eps;
    uint4 *sum, *y;
    uint2 *codes;
    float *scale;
    int e4m3;  // codes' type, or int8
};

template <bool WARP, int THREADS, int kChunks>
__global__ void __launch_bounds__(THREADS) norm_kernel(const NormArgs a)
{
    constexpr int kRows = WARP ? THREADS / 32 : 1;
    __shared__ float s_slots[2 * kMaxWarps];
    int turn = 0;
    const int TPR = WARP ? 32 : blockDim.x;
    const int slot = WARP ? threadIdx.x / 32 : 0, lane = WARP ? threadIdx.x % 32 : threadIdx.x;
    const int chunks = a.C / 8;
    const long long row = static_cast<long long>(blockIdx.x) * kRows + slot;
    const bool live = row < a.N;
    const long long at = row * chunks;
    griddep_launch_dependents();
    griddep_wait();
    float z[kChunks][8];
    uint4 g[kChunks];
    {
        uint4 x[kChunks], r[kChunks];
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int c = lane + i * TPR;
            const bool in = live && c < chunks;
            x[i] = in ? __ldcs(a.x + at + c) : make_uint4(0, 0, 0, 0);
            r[i] = in && a.residual ? __ldcs(a.residual + at + c) : make_uint4(0, 0, 0, 0);
            g[i] = c < chunks ? a.gamma[c] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            float f[8];
            unpack8(x[i], z[i]);
            if (a.residual) {
                unpack8(r[i], f);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    z[i][j] += f[j];
            }
        }
    }
    float sums[1] = {0.f};
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sums[0] = fmaf(z[i][j], z[i][j], sums[0]);
    row_reduce<WARP, Sum, 1>(sums, s_slots, turn);
    const float C = static_cast<float>(a.C);
    float k = 1.f;  // of the row, before its squares are summed
    // the same for all threads of a row, which are a warp or the whole CTA: the reductions inside may have barriers
    if (!(sums[0] >= kLeast && sums[0] <= kMost)) {
        float m[1] = {0.f};
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                m[0] = Max::apply(m[0], fabsf(z[i][j]));
        row_reduce<WARP, Max, 1>(m, s_slots, turn);
        k = row_scale(m[0], a.eps);
        sums[0] = 0.f;
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float t = z[i][j] * k;
                sums[0] = fmaf(t, t, sums[0]);
            }
        row_reduce<WARP, Sum, 1>(sums, s_slots, turn);
    }
    const float under = sums[0] / C + a.eps * k * k;  // mean((z k)^2) + eps k^2
    const float inv = under == 0.f ? 0.f : 1.f / sqrtf(under);
    float m[1] = {0.f};
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int c = lane + i * TPR;
        const bool in = live && c < chunks;
        float f[8];
        if (a.sum && in)
            __stcs(a.sum + at + c, pack8(z[i]));
        unpack8(g[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            z[i][j] = z[i][j] * k * inv * f[j];
            m[0] = Max::apply(m[0], fabsf(z[i][j]));
        }
        if (a.y && in)
            __stcs(a.y + at + c, pack8(z[i]));
    }
    if (a.codes) {
        row_reduce<WARP, Max, 1>(m, s_slots, turn);
        const float top = a.e4m3 ? 448.f : 127.f;
        const bool finite = m[0] <= 3.4028234e38f;
        const float by = finite && m[0] >= kTiny ? top / m[0] : 0.f;
        if (live && lane == 0)
            a.scale[row] = !finite ? __uint_as_float(0x7fc00000u) : m[0] >= kTiny ? m[0] / top : 0.f;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int c = lane + i * TPR;
            if (!live || c >= chunks)
                continue;
            float q[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                q[j] = finite ? z[i][j] * by : 0.f;
            a.codes[at + c] = a.e4m3 ? make_uint2(e4m3x4(q), e4m3x4(q + 4)) : make_uint2(int8x4(q), int8x4(q + 4));
        }
    }
}

struct NormGradArgs {
    int N, C;
    const uint4 *z, *gamma, *dy, *d_sum;
    float eps;
    uint4 *dx;
    float *partial;  // [gridDim.x, C] of dgamma, 8-byte aligned, or null
};

// Persistent over rows, so that a thread sums its channels' dgamma in registers.  Each thread copies its own chunks
// of the next DEPTH - 1 rows into shared memory (cp.async: no registers, and nothing to wait for but its own copies):
// the loads of one row would leave HBM idle while the row is reduced (8195 x 5120: 70.4 us without, 56.3 now, 5.97
// TB/s; 40 instructions an element bound it then, hence pairs of float32).  160 threads with four chunks instead of
// 320 with two: 95 us.

// CTAs of the gradient that an SM holds at once, as far as registers go: a thread of four chunks takes up to 128, of
// two or one 64 (80 where a row is a warp's).
__host__ __device__ constexpr int grad_resident(bool warp, int threads, int chunks)
{
    return warp ? (chunks == 4 ? 512 : 768) / threads : 1024 / threads;
}

template <bool WARP, int THREADS, int CHUNKS, int DEPTH>
__global__ void __launch_bounds__(THREADS, grad_resident(WARP, THREADS, CHUNKS)) norm_grad_kernel(const NormGradArgs a)
{
    constexpr int kRows = WARP ? THREADS / 32 : 1;
    __shared__ float s_slots[4 * kMaxWarps];
    int turn = 0;
    extern __shared__ uint4 s_rows[];  // [DEPTH][z, dy, d_sum if any][CHUNKS][threads]; later the rows' sums of dgamma
    const int TPR = WARP ? 32 : blockDim.x;
    const int slot = WARP ? threadIdx.x / 32 : 0, lane = WARP ? threadIdx.x % 32 : threadIdx.x;
    const int chunks = a.C / 8;
    const float inv_C = 1.f / static_cast<float>(a.C);
    griddep_launch_dependents();
    griddep_wait();
    uint64_t dg[CHUNKS][4] = {};  // pairs of float32
    uint64_t gamma[CHUNKS][4];
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i)
        unpack8x2(lane + i * TPR < chunks ? a.gamma[lane + i * TPR] : make_uint4(0, 0, 0, 0), gamma[i]);
    const long long step = static_cast<long long>(gridDim.x) * kRows;
    // this thread's chunk i of tensor `which` in the place of a row that starts at `at`
    const uint32_t chunk_step = blockDim.x * 16, tensor_step = CHUNKS * chunk_step;
    const uint32_t row_step = (a.d_sum ? 3 : 2) * tensor_step, begin = smem_u32(s_rows) + threadIdx.x * 16;
    const uint32_t end = begin + DEPTH * row_step;
    auto place = [&](uint32_t at, int which, int i) { return at + which * tensor_step + i * chunk_step; };
    auto fetch = [&](long long row, uint32_t to) {
        if (row < a.N) {
#pragma unroll
            for (int i = 0; i < CHUNKS; ++i) {
                const int c = lane + i * TPR;
                if (c >= chunks)
                    continue;
                const long long at = row * chunks + c;
                cp_async16(place(to, 0, i), a.z + at);
                cp_async16(place(to, 1, i), a.dy + at);
                if (a.d_sum)
                    cp_async16(place(to, 2, i), a.d_sum + at);
            }
        }
        cp_async_commit();
    };
    const long long first = static_cast<long long>(blockIdx.x) * kRows;
    for (int d = 0; d < DEPTH - 1; ++d)
        fetch(first + slot + d * step, begin + d * row_step);
    uint32_t here = begin;
    for (long long base = first; base < a.N; base += step, here = here + row_step == end ? begin : here + row_step) {
        const long long row = base + slot;
        const bool live = row < a.N;
        const long long at = row * chunks;
        fetch(row + (DEPTH - 1) * step, (here == begin ? end : here) - row_step);
        cp_async_wait<DEPTH - 1>();
        auto held = [&](int which, int i) {  // read again where it is needed again: registers are short
            uint4 v = make_uint4(0, 0, 0, 0);
            if (live && lane + i * TPR < chunks)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                             : "r"(place(here, which, i))
                             : "memory");
            return v;
        };
        float v[2];  // sum z^2, sum u z, of the row as it is held
        auto add_up = [&]() {
            uint64_t zz = 0, uz = 0;
#pragma unroll
            for (int i = 0; i < CHUNKS; ++i) {
                uint64_t z[4], dy[4];
                unpack8x2(held(0, i), z);
                unpack8x2(held(1, i), dy);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    zz = fma2(z[j], z[j], zz);
                    uz = fma2(mul2(dy[j], gamma[i][j]), z[j], uz);
                }
            }
            const float2 x = f2_split(zz), y = f2_split(uz);
            v[0] = x.x + x.y;
            v[1] = y.x + y.y;
            row_reduce<WARP, Sum, 2>(v, s_slots, turn);
        };
        add_up();
        float k = 1.f;
        if (!(v[0] >= kGradLeast && v[0] <= kGradMost)) {  // all threads of a row alike
            float m[1] = {0.f};
#pragma unroll
            for (int i = 0; i < CHUNKS; ++i) {
                float z[8];
                unpack8(held(0, i), z);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    m[0] = Max::apply(m[0], fabsf(z[j]));
            }
            row_reduce<WARP, Max, 2>(m, s_slots, turn);
            k = row_scale(m[0], a.eps);
            if (k != 1.f) {
                // the row is held as z k from here on: exact, but for elements that are nothing next to its largest
#pragma unroll
                for (int i = 0; i < CHUNKS; ++i) {
                    float z[8];
                    unpack8(held(0, i), z);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        z[j] *= k;
                    const uint4 w = pack8(z);
                    if (live && lane + i * TPR < chunks)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(place(here, 0, i)), "r"(w.x),
                                     "r"(w.y), "r"(w.z), "r"(w.w)
                                     : "memory");
                }
                add_up();
            }
        }
        const float under = v[0] * inv_C + a.eps * k * k;
        const float inv = under == 0.f ? 0.f : rsqrtf(under);  // 1 / (n k)
        const float back = v[1] * inv_C * inv;                 // mean(u z / n)
        const uint64_t inv2 = f2(inv, inv), back2 = f2(-back, -back);
        // (1 / n of a row below float32's normal range is more than float32 holds: 1 / (n k) and k come one after the
        // other.  The loop twice, because every instruction of it counts: 0 to 0.7% slower than one that could not do
        // this, 2 to 7% up to 512 channels; k where each element is finished costs 12% at 16384 x 4096.)
        auto finish = [&](auto scaled) {
            const uint64_t k2 = f2(k, k);
#pragma unroll
            for (int i = 0; i < CHUNKS; ++i) {
                const int c = lane + i * TPR;
                uint64_t z[4], dy[4], s[4];
                unpack8x2(held(0, i), z);
                unpack8x2(held(1, i), dy);
                unpack8x2(a.d_sum ? held(2, i) : make_uint4(0, 0, 0, 0), s);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint64_t t = mul2(z[j], inv2);  // z / n
                    dg[i][j] = fma2(dy[j], t, dg[i][j]);
                    const uint64_t u = fma2(t, back2, mul2(dy[j], gamma[i][j]));
                    s[j] = scaled.value ? fma2(mul2(u, inv2), k2, s[j]) : fma2(u, inv2, s[j]);
                }
                if (live && c < chunks)
                    __stcs(a.dx + at + c, make_uint4(pack2x(s[0]), pack2x(s[1]), pack2x(s[2]), pack2x(s[3])));
            }
        };
        if (__builtin_expect(k == 1.f, 1))
            finish(std::false_type{});
        else
            finish(std::true_type{});
    }
    if (!a.partial)
        return;
    float *out = a.partial + static_cast<long long>(blockIdx.x) * a.C;
    if constexpr (kRows == 1) {
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
            const int c = lane + i * TPR;
            if (c < chunks) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<float2 *>(out + 8 * c + 2 * j) = f2_split(dg[i][j]);
            }
        }
    } else {
        float *s_gamma = reinterpret_cast<float *>(s_rows);  // [kRows, C]
        cp_async_wait<0>();
        __syncthreads();
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
            const int c = lane + i * TPR;
            if (c < chunks)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<float2 *>(s_gamma + slot * a.C + 8 * c + 2 * j) = f2_split(dg[i][j]);
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.C; c += THREADS) {
            float t = s_gamma[c];
#pragma unroll
            for (int r = 1; r < kRows; ++r)
                t += s_gamma[r * a.C + c];
            out[c] = t;
        }
    }
}

// dgamma = the CTAs' sums added up: 32 channels a CTA, 32 threads each, so that many loads are in flight.
__global__ void __launch_bounds__(1024) gamma_kernel(const float *partial, int parts, int C, float *dgamma)
{
    __shared__ float s_part[32][33];
    griddep_launch_dependents();
    griddep_wait();
    const int c = blockIdx.x * 32 + threadIdx.x % 32, w = threadIdx.x / 32;
    float t = 0.f;
    if (c < C)
#pragma unroll 8
        for (int p = w; p < parts; p += 32)
            t += partial[static_cast<long long>(p) * C + c];
    s_part[w][threadIdx.x % 32] = t;
    __syncthreads();
    t = s_part[threadIdx.x % 32][w];  // a warp adds a channel's up
#pragma unroll
    for (int d = 16; d > 0; d /= 2)
        t += __shfl_xor_sync(0xffffffffu, t, d);
    if (threadIdx.x % 32 == 0 && blockIdx.x * 32 + w < C)
        dgamma[blockIdx.x * 32 + w] = t;
}

// Threads that a row of more than 1024 channels takes: no more than its chunks need.
int threads_for(int C, int chunks) { return (C / 8 + 32 * chunks - 1) / (32 * chunks) * 32; }

template <bool WARP, int THREADS, int CHUNKS>
cudaError_t norm(const NormArgs &a, cudaStream_t stream)
{
    const long long rows = WARP ? THREADS / 32 : 1;
    return launch_dependent(norm_kernel<WARP, THREADS, CHUNKS>, dim3(static_cast<unsigned>((a.N + rows - 1) / rows)),
                            dim3(WARP ? THREADS : threads_for(a.C, CHUNKS)), 0, stream, a);
}

template <bool WARP, int THREADS, int CHUNKS, int DEPTH>
cudaError_t norm_grad(NormGradArgs a, float *dgamma, cudaStream_t stream)
{
    auto kernel = norm_grad_kernel<WARP, THREADS, CHUNKS, DEPTH>;
    const int rows = WARP ? THREADS / 32 : 1, threads = WARP ? THREADS : threads_for(a.C, CHUNKS);
    // (the rows' C floats of dgamma fit where DEPTH of their bf16 did)
    const int smem = DEPTH * (a.d_sum ? 3 : 2) * CHUNKS * threads * 16;
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), smem);
    if (e != cudaSuccess)
        return e;
    const int resident = std::max(1, std::min({grad_resident(WARP, threads, CHUNKS), kSmem / (smem + 1280), 16}));
    const int parts = std::min({(a.N - 1) / rows + 1, norm_parts(a.C), device_sm_count() * resident});
    // one CTA's sums are the result, and go there at once if it may be written in pairs (the caller's need not be
    // aligned to more than a float)
    const bool whole = parts == 1 && reinterpret_cast<uintptr_t>(dgamma) % 8 == 0;
    if (a.partial && whole)
        a.partial = dgamma;
    e = launch_dependent(kernel, dim3(static_cast<unsigned>(parts)), dim3(threads), smem, stream, a);
    if (e != cudaSuccess || !a.partial || whole)
        return e;
    return launch_dependent(gamma_kernel, dim3(static_cast<unsigned>((a.C + 31) / 32)), dim3(1024), 0, stream,
                            static_cast<const float *>(a.partial), parts, a.C, dgamma);
}

// Whether a row of a CTA leaves fewer threads without a chunk with two chunks a thread than with four.
bool two_fit_better(int C)
{
    const int n = C / 8;
    return (n + 63) / 64 * 64 < (n + 127) / 128 * 128;
}

}  // namespace

cudaError_t launch_residual_norm(int N, int C, const void *x, const void *residual, const void *gamma, float eps,
                                 void *sum, void *y, void *codes, bool e4m3, float *scale, cudaStream_t stream)
{
    NormArgs a{};
    a.N = N;
    a.C = C;
    a.x = static_cast<const uint4 *>(x);
    a.residual = static_cast<const uint4 *>(residual);
    a.gamma = static_cast<const uint4 *>(gamma);
    a.eps = eps;
    a.sum = static_cast<uint4 *>(sum);
    a.y = static_cast<uint4 *>(y);
    a.codes = static_cast<uint2 *>(codes);
    a.scale = scale;
    a.e4m3 = e4m3;
    // 57617 x 400 to bf16 and codes: 27.9 us with two chunks a thread, 41.2 with four; 5385 x 1120 to codes: 10.8, 11.6
    if (C <= 256)
        return norm<true, 128, 1>(a, stream);
    if (C <= 512)
        return norm<true, 128, 2>(a, stream);
    if (C <= 1024)
        return norm<true, 128, 4>(a, stream);
    return two_fit_better(C) ? norm<false, 1024, 2>(a, stream) : norm<false, 512, 4>(a, stream);
}

cudaError_t launch_residual_norm_grad(int N, int C, const void *z, const void *gamma, const void *dy,
                                      const void *d_sum, float eps, void *dx, float *dgamma, float *partial,
                                      cudaStream_t stream)
{
    NormGradArgs a{};
    a.N = N;
    a.C = C;
    a.z = static_cast<const uint4 *>(z);
    a.gamma = static_cast<const uint4 *>(gamma);
    a.dy = static_cast<const uint4 *>(dy);
    a.d_sum = static_cast<const uint4 *>(d_sum);
    a.eps = eps;
    a.dx = static_cast<uint4 *>(dx);
    a.partial = dgamma ? partial : nullptr;
    // 16659 x 312: 13.9 us with two chunks a thread, 20.0 with four
    if (C <= 256)
        return norm_grad<true, 128, 1, 4>(a, dgamma, stream);
    if (C <= 512)
        return norm_grad<true, 128, 2, 4>(a, dgamma, stream);
    if (C <= 1024)
        return norm_grad<true, 128, 4, 3>(a, dgamma, stream);
    // places for as many rows of a CTA's as let two CTAs share an SM (16384 x 4096: 87 us with four, 99 with three;
    // 8195 x 5120: 56.3 us with three, 59.0 with two, 74.1 with four, which leave room for one CTA)
    const int threads = threads_for(C, 2);
    if (threads <= 256)
        return norm_grad<false, 256, 2, 4>(a, dgamma, stream);
    if (threads <= 384)
        return norm_grad<false, 512, 2, 3>(a, dgamma, stream);
    if (C <= 512 * 8 * 2)
        return norm_grad<false, 512, 2, 2>(a, dgamma, stream);
    return norm_grad<false, 1024, 2, 2>(a, dgamma, stream);
}

}  // namespace df2
