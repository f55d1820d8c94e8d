// attention.cu -- attention of a block of new tokens over the paged cache.
//
// The plain kernel: one warp a row (token, query head), 32 keys at a time, each lane the score of
// one key, with the running maximum m and sum l of the softmax:
//   m' = max(m, s_j), l' = l 2^(m - m') + sum 2^(s_j - m'), o' = o 2^(m - m') + sum 2^(s_j - m') v_j
// (scores in units of log 2), then each lane four dimensions of o over the 32 values.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace df2 {
namespace {

constexpr int kWarps = 8;

struct AttnArgs {
    PagedCache cache;
    TokenBatch tokens;
    HeadRows q, out;
    float *lse;
    float scale_log2;
    int causal, window, group;
};

// Element d of cached row `row`, without its scale.
__device__ __forceinline__ float code_at(const PagedCache &c, const void *base, long long row, int d)
{
    const long long at = row * c.dim + d;
    if (c.type == 0)
        return bf16_lo(static_cast<const uint16_t *>(base)[at]);
    if (c.type == 2)
        return static_cast<const int8_t *>(base)[at];
    uint32_t w;
    float f;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(w) : "h"(static_cast<uint16_t>(static_cast<const uint8_t *>(base)[at])));
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.f32.f16 %0, l;}" : "=f"(f) : "r"(w));
    return f;
}

__global__ void __launch_bounds__(kWarps * 32) attention_kernel(const AttnArgs a)
{
    __shared__ float qs[kWarps][128];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int heads = a.q.heads, dim = a.cache.dim, ps = a.cache.page_size;
    const long long r = static_cast<long long>(blockIdx.x) * kWarps + warp;
    griddep_launch_dependents();
    griddep_wait();
    if (r >= static_cast<long long>(a.tokens.N) * heads)
        return;
    const int n = static_cast<int>(r / heads), h = static_cast<int>(r % heads), kvh = h / a.group;
    const int b = warp_sequence_of(a.tokens.token_start, a.tokens.B, n, lane);
    const int kv_len = a.tokens.kv_len[b];
    const int pos = kv_len - a.tokens.token_start[b + 1] + n;
    const int held = static_cast<int>(min(static_cast<long long>(kv_len), static_cast<long long>(a.tokens.max_pages) * ps));
    const int hi = a.causal ? min(held, pos + 1) : held;
    const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
    for (int d = lane; d < dim; d += 32)
        qs[warp][d] = bf16_lo(a.q.data[n * a.q.token_stride + h * a.q.head_stride + d]) * a.scale_log2;
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = lo; j0 < hi; j0 += 32) {
        const int j = j0 + lane;
        long long row = -1;
        float s = -INFINITY, vs = 0.f;
        if (j < hi) {
            const int page = a.tokens.page_table[static_cast<long long>(b) * a.tokens.max_pages + j / ps];
            if (page >= 0 && page < a.cache.pages)
                row = (static_cast<long long>(page) * a.cache.heads + kvh) * ps + j % ps;
            s = 0.f;
            if (row >= 0) {
                for (int d = 0; d < dim; ++d)
                    s = fmaf(qs[warp][d], code_at(a.cache, a.cache.k, row, d), s);
                vs = 1.f;
                if (a.cache.type != 0) {
                    s *= a.cache.k_scale[row];
                    vs = a.cache.v_scale[row];
                }
            }
        }
        float top = s;
        for (int x = 16; x > 0; x >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        const float m2 = fmaxf(m, top);
        const float keep = m2 == -INFINITY ? 0.f : exp2f(m - m2);
        const float p = m2 == -INFINITY ? 0.f : exp2f(s - m2);
        float sum = p;
        for (int x = 16; x > 0; x >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, x);
        l = l * keep + sum;
        m = m2;
        for (int i = 0; i < 4; ++i)
            o[i] *= keep;
        for (int k = 0; k < 32 && j0 + k < hi; ++k) {
            const long long rk = __shfl_sync(0xffffffffu, row, k);
            const float pk = __shfl_sync(0xffffffffu, p * vs, k);
            if (rk >= 0)
                for (int i = 0; i < 4; ++i)
                    if (lane + 32 * i < dim)
                        o[i] = fmaf(pk, code_at(a.cache, a.cache.v, rk, lane + 32 * i), o[i]);
        }
    }
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
    for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < dim)
            a.out.data[n * a.out.token_stride + h * a.out.head_stride + lane + 32 * i] =
                static_cast<uint16_t>(bf16_pack(o[i] * inv, 0.f));
    if (a.lse && lane == 0)
        a.lse[static_cast<long long>(n) * heads + h] = (m + log2f(l)) * 0.69314718055994530942f;
}

}  // namespace

size_t paged_attention_scratch(const PagedCache &, const TokenBatch &, int) { return 0; }

cudaError_t launch_paged_attention(const PagedCache &cache, const TokenBatch &tokens, const AttentionOptions &opt,
                                   const HeadRows &q, const HeadRows &out, float *lse, uint32_t *, void *,
                                   cudaStream_t stream)
{
    AttnArgs a{};
    a.cache = cache;
    a.tokens = tokens;
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.scale_log2 = opt.scale * 1.44269504088896340736f;
    a.causal = opt.causal;
    a.window = opt.window;
    a.group = q.heads / cache.heads;
    const long long rows = static_cast<long long>(tokens.N) * q.heads;
    return launch_dependent(attention_kernel, dim3(static_cast<unsigned>((rows + kWarps - 1) / kWarps)),
                            dim3(kWarps * 32), 0, stream, a);
}

}  // namespace df2
