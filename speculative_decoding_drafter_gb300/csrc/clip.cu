// clip.cu -- the norm of many gradients together, and the gradients scaled so that it has a bound.
//
//   norm = sqrt(sum x^2) or max |x| over every element of every tensor;  out = x min(1, max_norm / norm)
//
// HBM-bound: every element is read for the norm, and read and written again for the scaling, which cannot start
// before the norm is known.  All tensors are one line of units of 16 KB, cut into equal shares, a CTA each, whatever
// the tensors' sizes; the scaling walks each share from its end, where L2 may still hold what the norm read last.
// Two reads and a write of 1.8 GB of bf16: 832 us, 6.5 TB/s; the norm alone of 0.5 GB in 777 tensors 79 us, 6.3 TB/s;
// of 12 MB in 7 tensors 10.2 us: two launches, each with a chain of arguments -> tensors -> sums.
//
// The tensors' addresses and lengths travel in the kernels' arguments (up to 1000 a launch), so a call uploads
// nothing and leaves no host memory behind that a captured graph would read again.
//
// No atomics: each CTA leaves its sum in double, and whoever needs the norm adds the sums up in one order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "dflash2.h"
#include "internal.h"
#include "ptx.cuh"

namespace df2 {
namespace {

constexpr int kThreads = 256;
constexpr int kVectors = 4;                                // of 16 bytes, a thread and turn
constexpr int kUnit = kThreads * kVectors * 16;            // bytes
constexpr int kCtasPerSm = 4;
constexpr int kMaxCtas = 2048;                             // shares of a launch
constexpr int kFew = 64, kMany = 1000;                     // tensors a launch
constexpr double kLeast = 1e-24, kMost = 1e37;             // squares beyond may have been lost or overflowed

// Side by side, so that a CTA finds what it needs of a tensor in one line of the arguments.
struct Entry {
    const void *data;
    void *out;
    long long count_type;  // count * 4 + type
    int unit, pad;         // the units before the tensor
};

template <int M>
struct Batch {
    Entry tensor[M + 1];  // [n].unit is the number of units
    int n;
};
static_assert(sizeof(Batch<kMany>) <= 32700, "kernel arguments");

// What a share has of one tensor.  Offsets count bytes from `base`, the tensor's address rounded down to 16; the
// tensor is [lo, hi) of them.
struct Span {
    const uint8_t *base;
    long long lo, hi;
    long long first, last;  // the share's full vectors (16 bytes of the tensor each)
    bool head, tail;        // the vector before `first`, the one from `last` on: the tensor's, but not whole
    int type;
};

template <int M>
__device__ __forceinline__ Span span_of(const Batch<M> &b, int t, int u0, int u1)
{
    Span r;
    const Entry &e = b.tensor[t];
    const uintptr_t p = reinterpret_cast<uintptr_t>(e.data);
    r.type = static_cast<int>(e.count_type & 3);
    r.base = reinterpret_cast<const uint8_t *>(p & ~uintptr_t(15));
    r.lo = static_cast<long long>(p & 15);
    r.hi = r.lo + (e.count_type >> 2) * (r.type == DF2_F32 ? 4 : 2);
    const long long from = static_cast<long long>(max(u0, e.unit) - e.unit) * (kUnit / 16);
    const long long to = static_cast<long long>(min(u1, b.tensor[t + 1].unit) - e.unit) * (kUnit / 16);
    r.head = from == 0 && r.lo > 0;
    r.first = r.head ? 1 : from;
    r.last = min(to, r.hi / 16);
    r.tail = r.last >= r.first && r.last < to && r.hi % 16 != 0;
    if (r.last < r.first) {  // the tensor lies within its first vector, whose other end is cut off too
        r.last = r.first;
        r.tail = false;
    }
    return r;
}

// Byte offset of the element that this thread takes of the two vectors that are not whole, or -1.
__device__ __forceinline__ long long edge_element(const Span &s, int size)
{
    const int j = static_cast<int>(threadIdx.x % 32) * size;
    if (threadIdx.x >= 64 || j >= 16)
        return -1;
    if (threadIdx.x < 32)
        return s.head && j >= s.lo && j < s.hi ? j : -1;
    return s.tail && s.last * 16 + j < s.hi ? s.last * 16 + j : -1;
}

__device__ __forceinline__ void widen(uint32_t w, int type, float &a, float &b)
{
    if (type == DF2_BF16) {
        a = __uint_as_float(w << 16);
        b = __uint_as_float(w & 0xFFFF0000u);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        a = f.x;
        b = f.y;
    }
}

__device__ __forceinline__ uint32_t narrow(float a, float b, int type)
{
    if (type == DF2_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A thread's sum of squares and largest magnitudes (16-bit types: two a word, as bits).
struct Part {
    float sum[2] = {0.f, 0.f};
    uint32_t max32 = 0, max_bf16 = 0, max_f16 = 0;
};

// The same in float32's bits, whose order is that of the values, infinity and NaN above them.
__device__ __forceinline__ uint32_t max_bits(const Part &p)
{
    uint32_t m = max(p.max32, max(p.max_bf16 << 16, p.max_bf16 & 0xFFFF0000u));
    float a, b;
    widen(p.max_f16, DF2_F16, a, b);
    return max(m, max(__float_as_uint(a), __float_as_uint(b)) & 0x7FFFFFFFu);
}

template <bool SCALED, int WHICH = 0>
__device__ __forceinline__ void add_word(Part &p, uint32_t w, int type, float k)
{
    if (type == DF2_F32) {
        float a = __uint_as_float(w);
        if (SCALED)
            a *= k;
        p.sum[WHICH] = fmaf(a, a, p.sum[WHICH]);
        p.max32 = max(p.max32, w & 0x7FFFFFFFu);
    } else {
        float a, b;
        widen(w, type, a, b);
        if (SCALED)
            a *= k, b *= k;
        p.sum[0] = fmaf(a, a, p.sum[0]);
        p.sum[1] = fmaf(b, b, p.sum[1]);
        uint32_t &m = type == DF2_BF16 ? p.max_bf16 : p.max_f16;
        m = __vmaxu2(m, w & 0x7FFF7FFFu);
    }
}

// The first tensor whose units reach past u (tensors without elements have none).
template <int M>
__device__ __forceinline__ int tensor_of(const Batch<M> &b, int u)
{
    int lo = 0, hi = b.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (b.tensor[mid + 1].unit > u)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

template <int M>
__device__ __forceinline__ void share_of(const Batch<M> &b, int &u0, int &u1)
{
    const long long units = b.tensor[b.n].unit;
    u0 = static_cast<int>(units * blockIdx.x / gridDim.x);
    u1 = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x);
}

// ONCE: nobody reads the tensors after, so they need not push others' lines out of L2 (norm of 400 MB beside a cache
// of written lines: 74 us, 85 otherwise; where they are scaled after, 50 MB take 38 us instead of 31).
template <int TYPE, bool SCALED, bool ONCE>
__device__ __forceinline__ void add_span(Part &p, const Span &s, float k)
{
    const uint4 *x = reinterpret_cast<const uint4 *>(s.base);
    long long v = s.first + threadIdx.x;
    auto add = [&](const uint4 &w) {
        add_word<SCALED, 0>(p, w.x, TYPE, k), add_word<SCALED, 1>(p, w.y, TYPE, k);
        add_word<SCALED, 0>(p, w.z, TYPE, k), add_word<SCALED, 1>(p, w.w, TYPE, k);
    };
    for (; v + (kVectors - 1) * kThreads < s.last; v += kVectors * kThreads) {
        uint4 w[kVectors];
#pragma unroll
        for (int i = 0; i < kVectors; ++i)
            w[i] = ONCE ? __ldcs(x + v + i * kThreads) : x[v + i * kThreads];
        // the turn's squares are summed by themselves: a long sum then rounds once a turn
        const float before[2] = {p.sum[0], p.sum[1]};
        p.sum[0] = p.sum[1] = 0.f;
#pragma unroll
        for (int i = 0; i < kVectors; ++i)
            add(w[i]);
        p.sum[0] += before[0];
        p.sum[1] += before[1];
    }
    for (; v < s.last; v += kThreads)
        add(ONCE ? __ldcs(x + v) : x[v]);
    const long long e = edge_element(s, TYPE == DF2_F32 ? 4 : 2);
    if (e >= 0)
        add_word<SCALED>(p, TYPE == DF2_F32 ? *reinterpret_cast<const uint32_t *>(s.base + e)
                                            : *reinterpret_cast<const uint16_t *>(s.base + e),
                         TYPE, k);
}

template <int M, bool SCALED, bool ONCE>
__device__ __forceinline__ Part add_share(const Batch<M> &b, float k)
{
    int u0, u1;
    share_of(b, u0, u1);
    Part p;
    if (u0 >= u1)
        return p;
    for (int t = tensor_of(b, u0); t < b.n && b.tensor[t].unit < u1; ++t) {
        if (b.tensor[t].unit == b.tensor[t + 1].unit)
            continue;
        const Span s = span_of(b, t, u0, u1);
        if (s.type == DF2_F32)
            add_span<DF2_F32, SCALED, ONCE>(p, s, k);
        else if (s.type == DF2_BF16)
            add_span<DF2_BF16, SCALED, ONCE>(p, s, k);
        else
            add_span<DF2_F16, SCALED, ONCE>(p, s, k);
    }
    return p;
}

// Over the CTA's threads, for thread 0.  The SM has two units for double: only one thread adds in it.
__device__ __forceinline__ double cta_sum(float v)
{
    __shared__ float s[kThreads / 32];
#pragma unroll
    for (int d = 16; d > 0; d /= 2)
        v += __shfl_xor_sync(0xffffffffu, v, d);
    __syncthreads();
    if (threadIdx.x % 32 == 0)
        s[threadIdx.x / 32] = v;
    __syncthreads();
    double t = 0;
    if (threadIdx.x == 0)
        for (int i = 0; i < kThreads / 32; ++i)
            t += s[i];
    return t;
}

__device__ __forceinline__ uint32_t cta_max(uint32_t v)
{
    __shared__ uint32_t s[kThreads / 32];
    v = __reduce_max_sync(0xffffffffu, v);
    __syncthreads();
    if (threadIdx.x % 32 == 0)
        s[threadIdx.x / 32] = v;
    __syncthreads();
    v = s[0];
    for (int i = 1; i < kThreads / 32; ++i)
        v = max(v, s[i]);
    return v;
}

// partial[CTA] = the share's sum of squares, or its largest magnitude.
template <int M, bool ONCE>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) sum_kernel(const __grid_constant__ Batch<M> b, int kind,
                                                                   double *partial)
{
    griddep_launch_dependents();
    griddep_wait();
    Part p = add_share<M, false, ONCE>(b, 1.f);
    const uint32_t bits = cta_max(max_bits(p));
    if (kind == DF2_NORM_MAX) {
        if (threadIdx.x == 0)
            partial[blockIdx.x] = __uint_as_float(bits);
        return;
    }
    __shared__ int s_again;
    double value = cta_sum(p.sum[0] + p.sum[1]);
    if (threadIdx.x == 0)
        // a largest magnitude is there, finite, and its square may have been lost or overflowed
        s_again = bits != 0 && bits < 0x7F800000u && !(value >= kLeast && value <= kMost);
    __syncthreads();
    if (s_again) {
        const int e = min(max(static_cast<int>(bits >> 23) - 127, -126), 126);
        p = add_share<M, true, ONCE>(b, __uint_as_float(static_cast<uint32_t>(127 - e) << 23));
        value = cta_sum(p.sum[0] + p.sum[1]);
        value *= __hiloint2double((1023 + 2 * e) << 20, 0);  // 2^(2e)
    }
    if (threadIdx.x == 0)
        partial[blockIdx.x] = value;
}

// The norm out of the shares' sums, the same in every CTA: one warp adds them up (see cta_sum).
__device__ __forceinline__ float norm_of(const double *partial, int parts, int kind)
{
    __shared__ float s_norm;
    if (threadIdx.x < 32) {
        float norm;
        if (kind == DF2_NORM_MAX) {
            uint32_t m = 0;
            for (int i = threadIdx.x; i < parts; i += 32)
                m = max(m, __float_as_uint(static_cast<float>(partial[i])));
            norm = __uint_as_float(__reduce_max_sync(0xffffffffu, m));
        } else {
            double v = 0;
#pragma unroll 8
            for (int i = threadIdx.x; i < parts; i += 32)
                v += partial[i];
#pragma unroll
            for (int d = 16; d > 0; d /= 2)
                v += __shfl_xor_sync(0xffffffffu, v, d);
            // sqrt(m 2^2e) = sqrt(m) 2^e with m in [1, 4), for which float32 will do
            const int e = (__double2hiint(v) >> 20) - 1023;
            if (v == 0 || e == 1024) {
                norm = static_cast<float>(v);  // nothing, or not finite
            } else {
                const int half = e >> 1;
                const double m = __hiloint2double(__double2hiint(v) - (half << 21), __double2loint(v));
                norm = ldexpf(sqrtf(static_cast<float>(m)), half);
            }
        }
        if (threadIdx.x == 0)
            s_norm = norm;
    }
    __syncthreads();
    return s_norm;
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const double *partial, int parts, int kind, float *norm)
{
    griddep_launch_dependents();
    griddep_wait();
    const float v = norm_of(partial, parts, kind);
    if (threadIdx.x == 0)
        *norm = v;
}

// What the elements are multiplied by, one after the other.
struct Factor {
    float f, by;
};

// max_norm / total.  A quotient down to 2^-277 is less than float32 holds, or holds in full, and its product with an
// element may be any number: it goes in two factors, of which the second is a power of two.
__device__ __forceinline__ Factor factor_of(float max_norm, float total)
{
    int e_max, e_total;
    const float m = frexpf(max_norm, &e_max), t = frexpf(total, &e_total);
    const int e = e_max - e_total;
    if (max_norm == 0.f || e >= -120)
        return Factor{max_norm / total, 1.f};
    return Factor{ldexpf(m / t, -120), ldexpf(1.f, e + 120)};
}

__device__ __forceinline__ uint32_t scale_word(uint32_t w, int type, Factor k)
{
    if (k.f == 1.f)
        return w;  // a NaN's bits too
    if (type == DF2_F32)
        return __float_as_uint(__uint_as_float(w) * k.f * k.by);
    float a, b;
    widen(w, type, a, b);
    return narrow(a * k.f * k.by, b * k.f * k.by, type);
}

// From the span's end to its start.
template <int TYPE>
__device__ __forceinline__ void scale_span(const Span &s, uint8_t *out, Factor f)
{
    constexpr int kSize = TYPE == DF2_F32 ? 4 : 2;
    const uint4 *x = reinterpret_cast<const uint4 *>(s.base);
    uint8_t *y = out - s.lo;  // offsets as the input's
    const bool aligned = (reinterpret_cast<uintptr_t>(y) & 15) == 0;
    auto scaled = [&](const uint4 &w) {
        return make_uint4(scale_word(w.x, TYPE, f), scale_word(w.y, TYPE, f), scale_word(w.z, TYPE, f),
                          scale_word(w.w, TYPE, f));
    };
    long long v = s.last - 1 - threadIdx.x;
    if (aligned) {
        for (; v - (kVectors - 1) * kThreads >= s.first; v -= kVectors * kThreads) {
            uint4 w[kVectors];
#pragma unroll
            for (int i = 0; i < kVectors; ++i)
                w[i] = __ldcs(x + v - i * kThreads);
#pragma unroll
            for (int i = 0; i < kVectors; ++i)
                __stcs(reinterpret_cast<uint4 *>(y) + v - i * kThreads, scaled(w[i]));
        }
        for (; v >= s.first; v -= kThreads)
            __stcs(reinterpret_cast<uint4 *>(y) + v, scaled(__ldcs(x + v)));
    } else {
        for (; v >= s.first; v -= kThreads) {
            const uint4 q = scaled(__ldcs(x + v));
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (kSize == 4) {
                    *reinterpret_cast<uint32_t *>(y + 16 * v + 4 * i) = w[i];
                } else {
                    *reinterpret_cast<uint16_t *>(y + 16 * v + 4 * i) = static_cast<uint16_t>(w[i]);
                    *reinterpret_cast<uint16_t *>(y + 16 * v + 4 * i + 2) = static_cast<uint16_t>(w[i] >> 16);
                }
            }
        }
    }
    const long long e = edge_element(s, kSize);
    if (e >= 0) {
        if constexpr (kSize == 4)
            *reinterpret_cast<uint32_t *>(y + e) =
                scale_word(*reinterpret_cast<const uint32_t *>(s.base + e), TYPE, f);
        else
            *reinterpret_cast<uint16_t *>(y + e) = static_cast<uint16_t>(
                scale_word(*reinterpret_cast<const uint16_t *>(s.base + e), TYPE, f));
    }
}

template <int M>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) scale_kernel(const __grid_constant__ Batch<M> b, int kind,
                                                                     float max_norm, const double *partial, int parts,
                                                                     float *norm)
{
    griddep_launch_dependents();
    griddep_wait();
    const float total = norm_of(partial, parts, kind);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0)
        *norm = total;
    // a norm that is not finite leaves the gradients as they are
    const bool over = total > max_norm && total <= 3.4028234e38f;
    const Factor f = over ? factor_of(max_norm, total) : Factor{1.f, 1.f};
    int u0, u1;
    share_of(b, u0, u1);
    if (u0 >= u1)
        return;
    for (int t = tensor_of(b, u1 - 1); t >= 0 && b.tensor[t + 1].unit > u0; --t) {
        uint8_t *out = static_cast<uint8_t *>(b.tensor[t].out);
        if ((!over && out == b.tensor[t].data) || b.tensor[t].unit == b.tensor[t + 1].unit)
            continue;
        const Span s = span_of(b, t, u0, u1);
        if (s.type == DF2_F32)
            scale_span<DF2_F32>(s, out, f);
        else if (s.type == DF2_BF16)
            scale_span<DF2_BF16>(s, out, f);
        else
            scale_span<DF2_F16>(s, out, f);
    }
}

long long units_of(const df2_tensor &t)
{
    const long long size = t.type == DF2_F32 ? 4 : 2;
    const long long lead = static_cast<long long>(reinterpret_cast<uintptr_t>(t.data) & 15);
    return t.count ? (lead + t.count * size + kUnit - 1) / kUnit : 0;
}

// What one launch walks: the tensors from `at` on, up to M.
template <int M>
int fill(Batch<M> &b, const df2_tensor *tensors, int at, int n)
{
    b.n = std::min(M, n - at);
    long long units = 0;
    for (int i = 0; i < b.n; ++i) {
        const df2_tensor &t = tensors[at + i];
        b.tensor[i] = Entry{t.data, t.out, t.count * 4 + t.type, static_cast<int>(units), 0};
        units += units_of(t);
    }
    b.tensor[b.n].unit = static_cast<int>(units);
    return static_cast<int>(units);
}

int ctas_for(int units) { return std::max(1, std::min({units, kMaxCtas, device_sm_count() * kCtasPerSm})); }

template <int M>
cudaError_t clip(const df2_tensor *tensors, int n, int kind, float max_norm, bool write, float *norm, double *partial,
                 cudaStream_t stream)
{
    Batch<M> b;
    int parts = 0;
    cudaError_t e = cudaSuccess;
    for (int at = 0; at < n; at += M) {
        const int grid = ctas_for(fill(b, tensors, at, n));
        e = launch_dependent(write ? sum_kernel<M, false> : sum_kernel<M, true>, dim3(grid), dim3(kThreads), 0, stream,
                             b, kind, partial + parts);
        if (e != cudaSuccess)
            return e;
        parts += grid;
    }
    if (!write || n == 0)
        return launch_dependent(norm_kernel, dim3(1), dim3(kThreads), 0, stream,
                                static_cast<const double *>(partial), parts, kind, norm);
    // the tensors read last come first
    for (int at = (n - 1) / M * M; at >= 0; at -= M) {
        const int grid = ctas_for(fill(b, tensors, at, n));
        e = launch_dependent(scale_kernel<M>, dim3(grid), dim3(kThreads), 0, stream, b, kind, max_norm,
                             static_cast<const double *>(partial), parts,
                             at == 0 ? norm : static_cast<float *>(nullptr));
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

}  // namespace

size_t grad_clip_scratch(int n)
{
    // a launch of up to kMany tensors leaves up to kMaxCtas sums
    return sizeof(double) * kMaxCtas * static_cast<size_t>(std::max(1, (n + kMany - 1) / kMany));
}

cudaError_t launch_grad_clip(const df2_tensor *tensors, int n, int kind, float max_norm, bool write, float *norm,
                             void *scratch, cudaStream_t stream)
{
    double *partial = static_cast<double *>(scratch);
    // few tensors' arguments are a fifteenth of the 32 KB that many take, which every launch copies
    if (n <= kFew)
        return clip<kFew>(tensors, n, kind, max_norm, write, norm, partial, stream);
    return clip<kMany>(tensors, n, kind, max_norm, write, norm, partial, stream);
}

}  // namespace df2
