// head_loss.cu -- cross entropy of the LM head and its gradient on tcgen05 tensor cores, without the logits.
//
//   z = h . W^T,  lse = log sum exp z,  loss = lse - z[label]
//   dz = (exp(z - lse) - [label]) grad,  d_hidden = dz . W,  d_W = dz^T . h
//
// One matrix kernel serves all four products.  A pair of CTAs (a cluster on two SMs) works on tiles of 256 x 256
// (tcgen05.mma.cta_group::2, M = 256, N = 256, K = 16 an instruction): each CTA loads its 128 rows of A and its
// 128 of B's 256 and holds 128 rows of the float32 accumulator in TMEM, two buffers of 256 columns, so that the
// epilogue of a tile runs under the products of the next.
//   warp 0      TMA producer: a stage is 128 elements of K of both operands, one box of 64 x 128 x 2 each
//               (32 KB); three stages.
//   warp 1      allocates TMEM; in the even CTA it issues the products.  (Warps 2 and 3 fill up the warpgroup.)
//   warps 4-11  epilogue, a thread half a row of the accumulator.
// Tiles are dealt out to the pairs in turn, so that pairs at work at the same time share operands in L2.
//
// All operands are boxes of three matrices, h [N, H], W [V, H] and dz [N, piece], each box 64 columns x 128 rows x
// 2 blocks of columns, 128-byte swizzled.  What differs is which axis is summed over: as h . W^T sums over the columns
// of both, the boxes are K-major; d_hidden sums over W's rows and d_W over dz's and h's, and the same boxes are
// MN-major operands there (the descriptors say which).
//
//   loss      epilogue of h . W^T: a tile leaves each row's sum of exponentials over 128 columns with an exponent
//             (8 bytes), and the label's logit where it has it; rows_kernel joins them.  8 / 512 of what float32
//             logits would write.
//   gradient  in pieces of the vocabulary: h . W^T again, epilogue dz in bf16 (through shared memory and TMA stores);
//             then one launch for d_W's tiles and d_hidden's, which need the same dz.  d_hidden sums over the
//             vocabulary: its tiles run over a whole piece (or a part of it, where there are few) and add their float32
//             results to those of the pieces before; hidden_grad_kernel rounds them at the end.  Ignored rows are
//             left out before (pack_kernel): their number is known on the device alone, so the kernels count their
//             tiles themselves.
// Every element is added to by one tile a launch, in the pieces' order: no result depends on which tile is first.
//
// What bounds it (one GB300): the products, from about 256 rows on.  Loss of 1024 x 5376 x 262144: 1495 us in short
// runs, 1.93 PFLOP/s (cuBLAS's bare bf16 product measured 1.89 to 1.95); 1674-1744 back to back, at the power cap.
// Gradient of 2048 x 4096 x 151936 with 1792 rows kept (seven tiles): 3540 us, 1.89 PFLOP/s of the rows kept, and 3985
// back to back, 1.68; 1794 rows, an eighth tile: 3870 and 4365.  The feed of operands is next: MMAs wait a quarter of
// their time for boxes in single launches.  Rows of W that do not start on 128-byte lines (H no multiple of 64) are
// read with a fifth sector in four: 1003 x 1032 x 50021 79 us, 1003 x 1088 72.  Few rows: HBM; loss of 16 x 4096 x
// 151936 201-207 us (6.0-6.2 TB/s), gradient of 64 x 5120 x 152064 807-835 us, of which W read twice and d_W written
// take 690.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "dflash2.h"
#include "f32x2.cuh"
#include "head_work.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "tensor_map.h"

namespace df2 {
namespace {

using namespace head;

constexpr int kBox = kRows * 128;                 // bytes of one block of columns of a box
constexpr int kStage = 4 * kBox;                  // A's two blocks, B's two blocks
constexpr int kStages = 3;
constexpr long long kSpread = 128 << 10, kSpreadFrom = 64 << 20;  // bytes of few rows' copies, and of W that make them
constexpr int kGroup = 6;                         // stages of a logit that one accumulator sums at most
constexpr int kBufs = 2;                          // accumulators
constexpr int kEpilogue = 8;                      // warps of the epilogue: 32 rows and half of the columns each
constexpr int kCols = kTile / 2;                  // of a warp
constexpr int kWarpBox = 32 * 128;                // bytes of a warp's staging buffer: 128 of each of its 32 rows
constexpr int kThreads = 128 + 32 * kEpilogue;
constexpr int kBars = 256;
constexpr int kStaging = kEpilogue * kWarpBox;
constexpr int kSmem = 1024 + kStages * kStage + kStaging + kBars;
static_assert(kSmem <= 227 * 1024, "shared memory of an SM");
constexpr uint32_t kTmemCols = 512;
// Registers of the logits' launches: the epilogue holds up to 128 sums a thread and takes what the first four warps
// need not.
constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8, kControlRegs = 72, kSumRegs = 216;
static_assert(kControlRegs + 2 * kSumRegs <= 3 * kLaunchRegs, "setmaxnreg.inc would wait forever");
constexpr float kLog2e = 1.4426950408889634f;

struct Args : Work {
    int blocks_w;         // whole blocks of 64 columns that W's boxes may be cut from two at a time
    int copies, copy_blocks;  // of the rows side by side, and a copy's blocks of 64 columns (logits; see hidden_copies)
    const int *count;     // rows that are not ignored, packed (null: all N)
    const uint4 *raw;     // the rows as they came, and where the scores' launch puts them for the products (or null)
    uint4 *packed;
    uint16_t *dz;         // [parts, N, pitch of dz] and
    float *sums;          // [splits, parts, N, H], where the epilogue writes few rows itself
    int dz_pitch;
    const int32_t *labels;
    const float *lse, *grad;
    float2 *part;         // [2 col_tiles, N] exponent and sum of exponentials (Running)
    float *label_logit;   // [N]
    int d_w_f32;
    uint32_t *status;
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// The element `at` of 32 (any where it is none of them).
__device__ __forceinline__ float pick(const uint32_t (&r)[32], int at)
{
    uint32_t z = 0;
    if (at >= 0 && at < 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            z = j == at ? r[j] : z;
    }
    return __uint_as_float(z);
}

template <int N>
__device__ __forceinline__ void reg_dec()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int N>
__device__ __forceinline__ void reg_inc()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// What the epilogue needs of a row.
struct RowData {
    int label;  // -1: none
    float lse, grad;
};

template <int MODE>
__device__ __forceinline__ RowData row_data(const Args &a, int m)
{
    RowData r{-1, 0.f, 0.f};
    if (MODE != kGrad && m < a.N) {
        r.label = a.labels[m];
        if (r.label >= a.V)
            r.label = -1;
        if (MODE == kScore) {
            r.lse = a.lse[m];
            r.grad = a.grad[m];
        }
    }
    return r;
}

// A running sum of exponentials: sum 2^exponent, the exponent a whole number (so that only the sum is ever rounded),
// not below the largest logit's.
struct Running {
    float exponent = -INFINITY, sum = 0.f;

    __device__ __forceinline__ void add(const uint32_t (&r)[32])
    {
        float b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            b[j] = fmaxf(fmaxf(__uint_as_float(r[j]), __uint_as_float(r[j + 8])),
                         fmaxf(__uint_as_float(r[j + 16]), __uint_as_float(r[j + 24])));
        const float high = ceilf(kLog2e * fmaxf(fmaxf(fmaxf(b[0], b[1]), fmaxf(b[2], b[3])),
                                                fmaxf(fmaxf(b[4], b[5]), fmaxf(b[6], b[7]))));
        if (high > exponent) {
            sum *= ex2(exponent - high);  // (0 for the first)
            exponent = high;
        }
        const float less = exponent == -INFINITY ? 0.f : -exponent;
        const uint64_t by = f2(kLog2e, kLog2e), from = f2(less, less);
        uint64_t e[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float2 x = f2_split(fma2(f2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), by, from));
            e[j % 2] = add2(e[j % 2], f2(ex2(x.x), ex2(x.y)));
        }
        const float2 s = f2_split(add2(e[0], e[1]));
        sum += s.x + s.y;
    }
};

// Calls f(columns, block) for each block of 32 columns of a thread's row, the next block on its way from TMEM
// meanwhile; release() once all have been read.
template <typename Release, typename F>
__device__ __forceinline__ void for_blocks(uint32_t acc, Release release, F f)
{
    uint32_t r0[32], r1[32];
    tmem_ld_32x32b_x32(acc, r0);
    tmem_wait_ld(r0);
#pragma unroll 1
    for (int cb = 0; cb < kCols / 32; cb += 2) {
        tmem_ld_32x32b_x32(acc + cb * 32 + 32, r1);
        f(r0, cb);
        tmem_wait_ld(r1);
        if (cb + 2 < kCols / 32)
            tmem_ld_32x32b_x32(acc + cb * 32 + 64, r0);
        else
            release();
        f(r1, cb + 1);
        if (cb + 2 < kCols / 32)
            tmem_wait_ld(r0);
    }
}

// As for_blocks, with one copy of f in the code and a copy of the registers instead.  The loss alone takes it, whose
// f is long and stands behind the sums of its groups as well: 16 x 4096 x 151936 205 us with it, 210 with for_blocks,
// 1024 x 5376 x 262144 1497 and 1507; a head so narrow that the epilogue bounds it loses by it, 1003 x 256 x 50021
// 31.9 and 29.9.
template <typename Release, typename F>
__device__ __forceinline__ void for_blocks_once(uint32_t acc, Release release, F f)
{
    uint32_t r[32], next[32];
    tmem_ld_32x32b_x32(acc, r);
    tmem_wait_ld(r);
#pragma unroll 1
    for (int cb = 0; cb < kCols / 32; ++cb) {
        const bool more = cb + 1 < kCols / 32;
        if (more)
            tmem_ld_32x32b_x32(acc + cb * 32 + 32, next);
        else
            release();
        f(r, cb);
        if (more) {
            tmem_wait_ld(next);
#pragma unroll
            for (int j = 0; j < 32; ++j)
                r[j] = next[j];
        }
    }
}

// Waits without looking at the abort flag; used only to drain in-flight work after an abort.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity)
{
    const unsigned long long t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > kWaitTimeoutNs / 10)
            return;
}

// Two blocks of 64 columns from block `block` on, 128 rows from `row` on: one box where both are among the `blocks`
// whole ones, otherwise (the tail of a matrix whose columns are no multiple of 64, or past its end) one by one.
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, const CUtensorMap *tail, int blocks,
                                         uint32_t bar, int row, int block)
{
    if (block + 1 < blocks) {
        tma_load_3d_pair(dst, map, bar, 0, row, block);
    } else {
        tma_load_2d_pair(dst, tail, bar, block * kBlock, row);
        tma_load_2d_pair(dst + kBox, tail, bar, (block + 1) * kBlock, row);
    }
}

// A lane's 128 bytes into its warp's staging buffer of 32 rows, swizzled as TMA reads them.
__device__ __forceinline__ void stage_row(uint32_t buf, int lane, const uint32_t (&w)[32])
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + lane * 128 + ((j ^ (lane & 7)) * 16)),
                     "r"(w[4 * j]), "r"(w[4 * j + 1]), "r"(w[4 * j + 2]), "r"(w[4 * j + 3])
                     : "memory");
}

// Logits of many products: the stages are cut into even groups, whose sums the epilogue adds up rounded to nearest.
// An accumulator cuts off what does not fit (256 times for 4096 products: lse is then off by 1.8e-6 of it).  Groups
// of at most 6 stages leave 5.7e-7 in the worst of a dozen sizes, of 14 1.4e-6, of 4 3.9e-7; 1024 x 5376 x 262144
// takes 1484 us with 6, 1486 to 1500 with 14, 1495 with 4; 1003 x 1024 x 50021 66.2, 65.9, 66.5. The gradient's
// logits are the same sums, bit by bit: what a label's logit is off by is then in its row's lse too, and 1 - p of a
// row that is nearly fitted keeps its value (1 - p from 2e-6 to 1e-3, H = 4096: the worst row's d_hidden is off by 5
// to 15%, which is lse's own rounding; by 21 to 47 times its size if the gradient's logits had one accumulator.  64 x
// 5120 x 152064 takes 0.4% more with groups).
__device__ __forceinline__ int group_of(int stages)
{
    const int groups = (stages + kGroup - 1) / kGroup;
    return (stages + groups - 1) / groups;
}

struct Maps {
    CUtensorMap h, w, w_tail;         // operands
    CUtensorMap z, z_part[2];         // dz, all of its parts' rows and each part's
    CUtensorMap z_out, dh, dw;        // results
};

// A lane's 128 bytes to where they go, 32 at a time up to `count` of them.
__device__ __forceinline__ void store_row(void *to, int count, const uint32_t (&w)[32])
{
    uint8_t *p = static_cast<uint8_t *>(to);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < count)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + 32 * j), "r"(w[8 * j]),
                         "r"(w[8 * j + 1]), "r"(w[8 * j + 2]), "r"(w[8 * j + 3]), "r"(w[8 * j + 4]), "r"(w[8 * j + 5]),
                         "r"(w[8 * j + 6]), "r"(w[8 * j + 7])
                         : "memory");
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ Maps maps, const Args args)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t stage0 = smem_u32(smem), staging = stage0 + kStages * kStage;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kStages * kStage + kStaging);
    const uint32_t bar0 = smem_u32(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };
    auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * kStages + b); };
    auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * kStages + kBufs + b); };
    const uint32_t drain_bar = bar0 + 8u * (2 * kStages + 2 * kBufs);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * kStages + 2 * kBufs + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;

    griddep_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < kBufs; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), 2 * kEpilogue);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&maps.h);
        prefetch_tmap(&maps.w);
        if (MODE == kGrad)
            prefetch_tmap(&maps.z);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the issuer's barriers are initialised before either CTA signals them
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();
    Args a = args;
    if (MODE != kLoss && a.count)
        keep_rows(a, *a.count);  // ignored rows are not there
    if (MODE == kGrad)
        share_out(a, pairs);

    if (warp < 4) {
        // One place for the whole warpgroup: setmaxnreg wants all its warps at the same instruction, and the
        // epilogue's wait for what it gives back has no limit.
        if constexpr (MODE != kGrad)
            reg_dec<kControlRegs>();
        if (warp == 0 && lane == 0) {
            // ---------------- TMA producer: both CTAs' loads complete on the even CTA's barriers
            int stage = 0;
            uint32_t phase = 0;
            long long issued = 0;
            bool ok = true;
            const int copy = MODE == kGrad ? 0 : pair % a.copies * a.copy_blocks;
            for (int i = 0; ok; ++i) {
                const Tile t = tile_of<MODE>(a, pair, pairs, i);
                if (!t.live)
                    break;
                const int half = static_cast<int>(rank) * kRows;
                for (int s = 0; s < t.stages; ++s) {
                    if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = stage0 + stage * kStage;
                    const uint32_t bar = mapa_shared(full_bar(stage), 0u);
                    if (rank == 0)
                        mbar_arrive_expect_tx(full_bar(stage), 2 * kStage);
                    const int k = t.k0 + s;
                    if (MODE != kGrad) {
                        tma_load_3d_pair(dst, &maps.h, bar, 0, t.m0 + half, copy + 2 * k);
                        load_box(dst + 2 * kBox, &maps.w, &maps.w_tail, a.blocks_w, bar, a.v0 + t.n0 + half, 2 * k);
                    } else if (t.product == kHiddenGrad) {
                        // (dz in two parts: one CTA's rows are the first's, the other's the second's)
                        if (a.parts == 2)
                            tma_load_3d_pair(dst, &maps.z_part[rank], bar, 0, 0, 2 * k);
                        else
                            tma_load_3d_pair(dst, &maps.z, bar, 0, t.m0 + half, 2 * k);
                        load_box(dst + 2 * kBox, &maps.w, &maps.w_tail, a.blocks_w, bar, a.v0 + k * kStageK,
                                 (t.n0 + half) / kBlock);
                    } else {
                        tma_load_3d_pair(dst, &maps.z, bar, 0, k * kStageK, (t.m0 + half) / kBlock);
                        tma_load_3d_pair(dst + 2 * kBox, &maps.h, bar, 0, k * kStageK, (t.n0 + half) / kBlock);
                    }
                    ++issued;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {
                // let the copies already issued land before the CTA leaves (the odd CTA cannot wait on the even
                // one's barriers: it gives them a fixed 100 us)
                if (rank != 0) {
                    const unsigned long long t0 = globaltimer_ns();
                    while (globaltimer_ns() - t0 < 100000ull) {
                    }
                } else {
                    for (long long n = issued > kStages ? issued - kStages : 0; n < issued; ++n)
                        drain_wait(full_bar(static_cast<int>(n % kStages)), static_cast<uint32_t>((n / kStages) & 1));
                }
            }
        }
        if (warp == 1 && lane == 0 && rank == 0) {
            // ---------------- products
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            int use = 0;  // accumulators filled so far
            for (int i = 0; ok; ++i) {
                const Tile t = tile_of<MODE>(a, pair, pairs, i);
                if (!t.live)
                    break;
                const bool a_mn = MODE == kGrad && t.product == kWeightGrad;
                const uint32_t idesc = idesc_bf16_f32(kTile, kTile) | (a_mn ? 1u << 15 : 0u) |
                                       (MODE == kGrad ? 1u << 16 : 0u);
                const int group = group_of(t.stages);
                for (int s = 0; s < t.stages && ok; ++use) {
                    const int buf = use % kBufs;
                    if (!mbar_wait(tempty_bar(buf), (static_cast<uint32_t>(use / kBufs) & 1u) ^ 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem + static_cast<uint32_t>(buf * kTile);
                    const int first = s, last = MODE != kGrad ? min(t.stages, s + group) : t.stages;
                    for (; s < last; ++s) {
                        if (!mbar_wait(full_bar(stage), phase, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t at = stage0 + stage * kStage, bt = at + 2 * kBox;
#pragma unroll
                        for (int k = 0; k < kStageK / 16; ++k) {
                            // 16 elements of K: 32 bytes on in a row, or 16 rows on
                            const uint32_t major = (k / 4) * kBox + (k % 4) * 32, minor = k * 16 * 128;
                            const uint64_t ad = a_mn ? sw128_mnmajor_desc(at + minor, kBox)
                                                     : sw128_kmajor_desc(at + major);
                            const uint64_t bd = MODE == kGrad ? sw128_mnmajor_desc(bt + minor, kBox)
                                                              : sw128_kmajor_desc(bt + major);
                            umma_bf16_pair(d, ad, bd, idesc, s != first || k != 0 ? 1u : 0u);
                        }
                        umma_commit_pair_both(empty_bar(stage));
                        if (++stage == kStages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (ok)
                        umma_commit_pair_both(tfull_bar(buf));
                }
            }
            if (!ok) {
                umma_commit_pair(drain_bar);  // every product issued so far ends before TMEM is released
                drain_wait(drain_bar, 0);
            }
        }
    } else {
        if constexpr (MODE != kGrad)
            reg_inc<kSumRegs>();
        // ---------------- epilogue: a thread is half a row; a warp stores what it has by itself
        const int q = warp & 3;  // the quarter of TMEM's lanes that this warp may read
        const int first_col = (warp - 4) / 4 * kCols;
        const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
        const uint32_t mine = staging + (warp - 4) * kWarpBox;
        // 128 bytes of each row go to the buffer, once the store before has read it, and from there to
        // `map` at (x, y) if `in`; z < 0: a matrix
        auto store = [&](const uint32_t(&w)[32], const CUtensorMap *map, bool in, int x, int y, int z, bool add) {
            if (lane == 0)
                bulk_wait_read<0>();
            __syncwarp();
            stage_row(mine, lane, w);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                if (in) {
                    if (z < 0)
                        tma_store_2d(map, mine, x, y);
                    else if (add)
                        tma_add_3d(map, mine, x, y, z);
                    else
                        tma_store_3d(map, mine, x, y, z);
                }
                bulk_commit();
            }
        };
        if (MODE == kScore && a.raw) {
            // under the first tile's products: ignored rows become zeros, for what they hold must not reach d_W (0 .
            // NaN)
            const int chunks = a.H / 8, total = a.N * chunks;
            for (int i = blockIdx.x * 32 * kEpilogue + threadIdx.x - 128; i < total; i += gridDim.x * 32 * kEpilogue) {
                const int label = a.labels[i / chunks];
                const uint4 v = label >= 0 && label < a.V ? a.raw[i] : make_uint4(0, 0, 0, 0);
                for (int part = 0; part < a.parts; ++part)
                    a.packed[part * total + i] = v;
            }
        }
        Tile t = tile_of<MODE>(a, pair, pairs, 0);
        RowData next = row_data<MODE>(a, t.m0 + static_cast<int>(rank) * kRows + q * 32 + lane);
        int use = 0;  // accumulators emptied so far
        for (int i = 0; t.live; ++i) {
            const int m_first = t.m0 + static_cast<int>(rank) * kRows + q * 32;
            const int m = m_first + lane;  // row of the product
            const int label = next.label;
            const float lse = next.lse, g = next.grad;
            // the next accumulator: false if it does not come
            uint32_t acc = 0;
            auto await = [&]() {
                const int buf = use % kBufs;
                acc = tmem + lanes + static_cast<uint32_t>(buf * kTile + first_col);
                const bool ready = mbar_wait(tfull_bar(buf), static_cast<uint32_t>(use / kBufs) & 1u, abort_flag);
                tc_fence_after();
                return __all_sync(0xffffffffu, ready) != 0;
            };
            // it has been read; whoever waits looks at nothing else of this warp's
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster_relaxed(mapa_shared(tempty_bar(use % kBufs), 0u));
                ++use;
            };
            if (!await())
                break;
            const Tile after = tile_of<MODE>(a, pair, pairs, i + 1);
            if (MODE != kGrad)  // on its way while this tile is worked on
                next = row_data<MODE>(a, after.live ? after.m0 + static_cast<int>(rank) * kRows + q * 32 + lane : a.N);
            // a warp whose rows all lie past the last has nothing to do but to let the accumulators go
            const bool two = MODE == kGrad && t.product == kHiddenGrad && a.parts == 2;
            const int row_first = two ? q * 32 : m_first;
            if (row_first >= (MODE != kGrad ? args.N : t.product == kHiddenGrad ? a.N : a.V - a.v0)) {
                release();
                bool there = true;
                if (MODE != kGrad)
                    for (int s = group_of(t.stages); s < t.stages && (there = await()); s += group_of(t.stages))
                        release();
                if (!there)
                    break;
                t = after;
                continue;
            }
            // The logits of a tile of several groups (this one's accumulator is the first's): their sums, block by
            // block, to f. False if an accumulator does not come.
            auto for_groups = [&](auto f) {
                uint32_t sum[kCols / 32][32] = {};
                const int group = group_of(t.stages);
                for (int s = 0; s < t.stages; s += group) {
                    if (s && !await())
                        return false;
#pragma unroll
                    for (int cb = 0; cb < kCols / 32; ++cb) {
                        uint32_t r[32];
                        tmem_ld_32x32b_x32(acc + cb * 32, r);
                        tmem_wait_ld(r);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            sum[cb][j] = __float_as_uint(__uint_as_float(sum[cb][j]) + __uint_as_float(r[j]));
                    }
                    release();
                }
#pragma unroll
                for (int cb = 0; cb < kCols / 32; ++cb)
                    f(sum[cb], cb);
                return true;
            };
            const int n_first = t.n0 + first_col;
            const int col0 = a.v0 + n_first;  // MODE != kGrad: the first token
            if constexpr (MODE == kLoss) {
                Running run;
                auto take = [&](uint32_t(&r)[32], int cb) {
                    const int c = col0 + cb * 32;
                    if (c + 32 > a.V) {  // columns past the vocabulary count as -inf
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            r[j] = c + j < a.V ? r[j] : 0xFF800000u;
                    }
                    const int at = label - c;
                    if (label >= 0 && at >= 0 && at < 32) {
                        uint32_t z = 0;
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            z = j == at ? r[j] : z;
                        a.label_logit[m] = __uint_as_float(z);
                    }
                    run.add(r);
                };
                if (group_of(t.stages) == t.stages)
                    for_blocks_once(acc, release, take);
                else if (!for_groups(take))
                    break;
                if (m < a.N)
                    a.part[static_cast<long long>(n_first / kCols) * a.N + m] = make_float2(run.exponent, run.sum);
            } else if (MODE == kGrad && (t.product == kHiddenGrad || a.d_w_f32)) {
                // float32: 32 columns are 128 bytes
                const bool hidden = t.product == kHiddenGrad;
                const CUtensorMap *map = hidden ? &maps.dh : &maps.dw;
                const int y = hidden ? row_first : a.v0 + m_first;
                const int z = !hidden ? -1 : two ? 2 * t.split + static_cast<int>(rank) : t.split;
                for_blocks(acc, release, [&](uint32_t(&r)[32], int cb) {
                    const int x = n_first + cb * 32;
                    if (two && a.first) {
                        if (y + lane < a.N)
                            store_row(a.sums + (static_cast<long long>(z) * a.N + y + lane) * a.H + x, (a.H - x) / 8,
                                      r);
                    } else {
                        store(r, map, x < a.H, x, y, z, !a.first);
                    }
                });
            } else {
                // bf16: 64 columns are 128 bytes
                const CUtensorMap *map = MODE == kScore ? &maps.z_out : &maps.dw;
                const int y = MODE == kScore ? m_first : a.v0 + m_first;
                // p = 2^(z log2e - lse log2e), the latter as a whole number and the rest: near p = 1 no more is lost
                // than lse's own rounding
                const float whole = rintf(lse * kLog2e), rest = fmaf(lse, kLog2e, -whole);
                const uint64_t by = f2(kLog2e, kLog2e), less = f2(-whole, -whole), lesser = f2(-rest, -rest);
                const uint64_t g2 = f2(g, g);
                uint32_t w[32], rest_w[32];
                auto take = [&](uint32_t(&r)[32], int cb) {
                    const int half = cb % 2;
                    if constexpr (MODE == kScore) {
                        const int c = col0 + cb * 32, at = label - c;
                        const float z_label = pick(r, at);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float2 e = f2_split(add2(
                                fma2(f2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), by, less), lesser));
                            const float2 d = f2_split(mul2(f2(ex2(e.x), ex2(e.y)), g2));
                            r[2 * j] = __float_as_uint(d.x);
                            r[2 * j + 1] = __float_as_uint(d.y);
                        }
                        if (at >= 0 && at < 32) {
                            const uint32_t d = __float_as_uint((ex2(fmaf(z_label, kLog2e, -whole) - rest) - 1.f) * g);
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                r[j] = j == at ? d : r[j];
                        }
                        // a row past the last is nothing whatever it holds, and so is a column past the vocabulary
                        if (label < 0 || c + 32 > a.V) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                r[j] = label >= 0 && c + j < a.V ? r[j] : 0u;
                        }
                    }
                    // (`half` is known where the calls are unrolled)
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        w[half ? 16 + j : j] = pack2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
                    if constexpr (MODE == kScore)
                        if (a.parts == 2) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const uint32_t v = w[half ? 16 + j : j];
                                rest_w[half ? 16 + j : j] =
                                    pack2(__uint_as_float(r[2 * j]) - __uint_as_float(v << 16),
                                          __uint_as_float(r[2 * j + 1]) - __uint_as_float(v & 0xFFFF0000u));
                            }
                        }
                    if (half) {
                        const int x = n_first + (cb - 1) * 32;
                        if (MODE == kScore && a.parts == 2) {
                            // few rows: each lane's by itself, without waiting for a staging buffer to be read (8 x
                            // 256 x 4096: 16.9 us, 17.5 through staging)
                            if (m < a.N) {
                                uint16_t *to = a.dz + static_cast<long long>(m) * a.dz_pitch + x;
                                store_row(to, 4, w);
                                store_row(to + static_cast<long long>(a.N) * a.dz_pitch, 4, rest_w);
                            }
                        } else {
                            store(w, map, MODE == kScore || x < a.H, x, y, -1, false);
                        }
                    }
                };
                if (MODE == kGrad || group_of(t.stages) == t.stages)
                    for_blocks(acc, release, take);
                else if (!for_groups(take))
                    break;
            }
            t = after;
        }
        if (lane == 0)
            bulk_wait_all();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while the other may still signal or read it
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
    if (threadIdx.x == 0 && *abort_flag)
        atomicOr(a.status, kStatusTimeoutGemm);
}

// Joins the tiles' sums of each row: eight rows a CTA, 128 threads each, so that few rows' tiles are read in
// a few turns.
__global__ void __launch_bounds__(1024) rows_kernel(const float2 *part, int tiles, int N, int V, const int32_t *labels,
                                                    const float *label_logit, float *loss, float *lse)
{
    __shared__ float2 s_part[8][33];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    auto join = [](float2 x, float2 y) {
        const float top = fmaxf(x.x, y.x);
        const float from = top == -INFINITY ? 0.f : top;
        return make_float2(top, x.y * ex2(x.x - from) + y.y * ex2(y.x - from));
    };
    auto join_lane = [&](float2 x, int d) {
        return join(x, make_float2(__shfl_xor_sync(0xffffffffu, x.x, d), __shfl_xor_sync(0xffffffffu, x.y, d)));
    };
    const int row = blockIdx.x * 8 + lane % 8;
    float2 t = make_float2(-INFINITY, 0.f);
    if (row < N) {
        int c = warp * 4 + lane / 8;
        for (; c + 3 * 128 < tiles; c += 4 * 128) {
            float2 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = part[static_cast<long long>(c + i * 128) * N + row];
            t = join(join(t, join(x[0], x[1])), join(x[2], x[3]));
        }
        for (; c < tiles; c += 128)
            t = join(t, part[static_cast<long long>(c) * N + row]);
    }
    t = join_lane(join_lane(t, 8), 16);
    if (lane < 8)
        s_part[lane][warp] = t;
    __syncthreads();
    if (warp < 8 && blockIdx.x * 8 + warp < N) {
        t = s_part[warp][lane];
#pragma unroll
        for (int d = 16; d > 0; d /= 2)
            t = join_lane(t, d);
        if (lane == 0) {
            const int r = blockIdx.x * 8 + warp;
            // sum 2^exponent: the exponent times ln 2 in two parts, so that it is as good as exact
            const float l = fmaf(t.x, 0.693147182464599609375f, fmaf(t.x, -1.9046542121259336e-9f, logf(t.y)));
            const int label = labels[r];
            lse[r] = l;
            loss[r] = label >= 0 && label < V ? l - label_logit[r] : 0.f;
        }
    }
}

// Rows of H elements, a multiple of 8, as rows of `pitch`, a multiple of 64: boxes of rows that start on a 128-byte
// line each are read from L2 without a fifth sector in four.  With labels, ignored rows become zeros (what they hold
// must not reach a product: 0 . NaN); the whole is written `times` times, `step` chunks apart, rows `row_step`.
__global__ void __launch_bounds__(256) pad_kernel(const uint4 *hidden, const int32_t *labels, int N, int V, int whole,
                                                  int chunks, int times, long long step, int row_step, uint4 *padded)
{
    griddep_launch_dependents();
    griddep_wait();
    const long long total = static_cast<long long>(N) * chunks;
#pragma unroll 4
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const int row = static_cast<int>(i / chunks), c = static_cast<int>(i - static_cast<long long>(row) * chunks);
        const int label = labels ? labels[row] : 0;
        const uint4 v = c < whole && label >= 0 && label < V ? hidden[static_cast<long long>(row) * whole + c]
                                                             : make_uint4(0, 0, 0, 0);
        for (int t = 0; t < times; ++t)
            padded[t * step + static_cast<long long>(row) * row_step + c] = v;
    }
}

// What the gradient keeps of its rows: those that are not ignored, one after another in their order.
struct Packed {
    uint4 *hidden;      // rows of `pitch` elements, a multiple of 64
    int32_t *label;
    float *lse, *grad;
    int32_t *place;     // of each row among them, or -1
    int *count;
};

// Packs the rows (what an ignored one holds must not reach a product, 0 . NaN, and takes no work).  A CTA has `per`
// consecutive rows and counts those before them itself.  Rows behind the last are zeros up to a whole stage.
__global__ void __launch_bounds__(256) pack_kernel(const uint4 *hidden, const int32_t *labels, const float *lse,
                                                   const float *grad, int N, int H, int V, int pitch, int per, Packed p)
{
    __shared__ int s_before[8], s_row[32];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int r0 = blockIdx.x * per, r1 = min(N, r0 + per);
    const int chunks = pitch / 8, whole = H / 8;
    auto seen = [&](int label) { return label >= 0 && label < V; };
    int before = 0;
#pragma unroll 4
    for (int r = threadIdx.x; r < r0; r += 256)
        before += seen(labels[r]);
    before = __reduce_add_sync(0xffffffffu, before);
    if (lane == 0)
        s_before[warp] = before;
    __syncthreads();
    before = 0;
    for (int w = 0; w < 8; ++w)
        before += s_before[w];
    for (int base = r0; base < r1; base += 32) {
        const int row = base + lane;
        const int label = row < r1 ? labels[row] : -1;
        const uint32_t mask = __ballot_sync(0xffffffffu, row < r1 && seen(label));
        const int to = before + __popc(mask & ((1u << lane) - 1u));
        if (warp == 0 && row < r1) {
            const bool keep = mask >> lane & 1u;
            p.place[row] = keep ? to : -1;
            if (keep) {
                p.label[to] = label;
                p.lse[to] = lse[row];
                p.grad[to] = grad[row];
            }
        }
        __syncthreads();  // the rows before have been read from s_row
        if (warp == 0 && (mask >> lane & 1u))
            s_row[to - before] = row;
        __syncthreads();
        const int total = __popc(mask) * chunks;
        uint4 *dst = p.hidden + static_cast<long long>(before) * chunks;
#pragma unroll 4
        for (int i = threadIdx.x; i < total; i += 256) {
            const int c = i % chunks;
            dst[i] = c < whole ? hidden[static_cast<long long>(s_row[i / chunks]) * whole + c] : make_uint4(0, 0, 0, 0);
        }
        before += __popc(mask);
    }
    if (r1 == N) {
        if (threadIdx.x == 0)
            *p.count = before;
        const int padded = min(N, (max(before, 1) + kStageK - 1) / kStageK * kStageK);
        const long long end = static_cast<long long>(padded) * chunks;
        for (long long c = static_cast<long long>(before) * chunks + threadIdx.x; c < end; c += 256)
            p.hidden[c] = make_uint4(0, 0, 0, 0);
    }
}

// d_hidden = the sums of the splits and of dz's parts, rounded; zeros for ignored rows.  place: where a row's sums
// are (null: in its own place).  GROUP threads share eight elements, where many sums are read for few of them.
template <int GROUP>
__global__ void __launch_bounds__(256) hidden_grad_kernel(const float4 *sums, int count, int N, int chunks,
                                                          const int32_t *place, const int32_t *labels, int V,
                                                          uint4 *d_hidden)
{
    griddep_launch_dependents();
    griddep_wait();
    const long long total = static_cast<long long>(N) * chunks;
    const int g = threadIdx.x % GROUP;
    for (long long i = (blockIdx.x * 256ll + threadIdx.x) / GROUP; i < total; i += gridDim.x * 256ll / GROUP) {
        const int row = static_cast<int>(i / chunks), c = static_cast<int>(i % chunks);
        const int label = labels[row];
        const int from = place ? place[row] : label >= 0 && label < V ? row : -1;
        float x[8] = {};
        if (from >= 0) {
            const float4 *at = sums + (static_cast<long long>(from) * chunks + c) * 2;
#pragma unroll 4
            for (int s = g; s < count; s += GROUP) {
                const float4 u = __ldcs(at + s * total * 2), v = __ldcs(at + s * total * 2 + 1);
                x[0] += u.x, x[1] += u.y, x[2] += u.z, x[3] += u.w;
                x[4] += v.x, x[5] += v.y, x[6] += v.z, x[7] += v.w;
            }
        }
#pragma unroll
        for (int d = GROUP / 2; d > 0; d /= 2)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] += __shfl_xor_sync(
                    GROUP == 1 ? 0xffffffffu : ((1u << GROUP) - 1u) << (threadIdx.x % 32 / GROUP * GROUP), x[j], d);
        if (g == 0)
            d_hidden[i] = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
    }
}

// ---------------------------------------------------------------------------------------------- host

// A row-major matrix's boxes of 64 columns x 128 rows, 128-byte swizzled: two blocks of columns at once (three
// dimensions: columns of a block, rows, whole blocks), or one (`tail`).
cudaError_t load_map(CUtensorMap *map, const void *p, long long rows, int cols, int pitch, bool tail)
{
    auto encode = tensor_map_encoder();
    if (!encode)
        return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(tail ? cols : kBlock), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(cols / kBlock)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(pitch) * 2, kBlock * 2};
    const cuuint32_t box[3] = {kBlock, kRows, 2};
    const cuuint32_t step[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, tail ? 2 : 3, const_cast<void *>(p), dims, strides,
                              box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Both maps of a matrix, and how many blocks load_box may take from the first (with columns that are a multiple of 64
// that is any: past the end it reads zeros).
cudaError_t load_maps(CUtensorMap *map, CUtensorMap *tail, int *blocks, const void *p, long long rows, int cols)
{
    *blocks = cols % kBlock == 0 ? 1 << 30 : cols / kBlock;
    const cudaError_t e = load_map(tail, p, rows, cols, cols, true);
    if (e != cudaSuccess)
        return e;
    if (cols >= kBlock)
        return load_map(map, p, rows, cols, cols, false);
    *map = *tail;  // never used
    return cudaSuccess;
}

// Boxes of 128 bytes x 32 rows that a warp of the epilogue stores; splits > 0: a stack of that many matrices.
cudaError_t store_map(CUtensorMap *map, void *p, bool f32, long long rows, int cols, int splits)
{
    auto encode = tensor_map_encoder();
    if (!encode)
        return cudaErrorNotSupported;
    const int size = f32 ? 4 : 2;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(splits)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * size, static_cast<cuuint64_t>(cols) * size * rows};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / size), 32, 1};
    const cuuint32_t step[3] = {1, 1, 1};
    const CUresult r = encode(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                              splits ? 3 : 2, p, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Pairs resident at once on the current device (clusters of two need two SMs of one GPC); cached per device,
// safe to call from several host threads.
int resident_pairs()
{
    static std::mutex mu;
    static int cache[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        (void)cudaGetLastError();
        return std::max(1, device_sm_count() / 2);
    }
    std::lock_guard<std::mutex> lock(mu);
    if (cache[dev] == 0) {
        (void)ensure_dynamic_smem(reinterpret_cast<const void *>(product_kernel<kLoss>), kSmem);
        cudaLaunchConfig_t c = {};
        c.gridDim = dim3(static_cast<unsigned>(2 * device_sm_count()));
        c.blockDim = dim3(kThreads);
        c.dynamicSmemBytes = kSmem;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 2;
        at[0].val.clusterDim.y = 1;
        at[0].val.clusterDim.z = 1;
        c.attrs = at;
        c.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, reinterpret_cast<const void *>(product_kernel<kLoss>), &c) !=
                cudaSuccess ||
            n < 1) {
            (void)cudaGetLastError();
            n = std::max(1, device_sm_count() / 2);
        }
        cache[dev] = n;
    }
    return cache[dev];
}

template <int MODE>
cudaError_t launch(const Maps &m, const Args &a, int pairs, cudaStream_t stream)
{
    auto kern = product_kernel<MODE>;
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kern), kSmem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if ((e = cudaLaunchKernelEx(&cfg, kern, m, a)) != cudaSuccess)
        return e;
    return cudaGetLastError();
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

// Rows that the loss takes at a time: what their tiles leave takes at most 256 MB (or 256 rows).
static int loss_rows(int N, int V)
{
    const long long rows = (1ll << 28) / (2 * sizeof(float2) * ceil_div(V, kTile)) / kTile * kTile;
    return static_cast<int>(std::min<long long>(N, std::max(1ll * kTile, std::min(16384ll, rows))));
}

// Copies of few rows that the logits' launch reads, each pair of CTAs one of them: all pairs read all rows while W
// streams by, and that is slow where the rows lie in less than 128 KB, by how their address falls (they are then few
// slices of L2's work): loss of 1 x 4096 x 151936 207 us, 293 to 390 without copies; 8 rows 207, 240 to 332; 1 x 4560
// x 223738 341, 549; with 64 KB 288, 236 and 403.  16 rows, 128 KB, take 206 wherever they lie.  The launch that
// makes the copies costs more than it gives for a small W (41 MB: 18.4 to 20 us, 17.8 to 19.4 without; 131 MB: 34 to
// 36, 40 to 47).
static int hidden_copies(int N, int H, int V)
{
    const long long bytes = static_cast<long long>(N) * ceil_div(H, kStageK) * kStageK * 2;
    if (N < 1 || N > kRows || bytes >= kSpread || static_cast<long long>(V) * H * 2 < kSpreadFrom)
        return 1;
    return static_cast<int>(std::min(64ll, (kSpread + bytes - 1) / bytes));
}

// Columns of the logits' rows, as the launch that pads them leaves them: 0 if it need not.
static int copied_pitch(int N, int H, int V)
{
    return hidden_copies(N, H, V) > 1 ? ceil_div(H, kStageK) * kStageK : H % kBlock ? ceil_div(H, kBlock) * kBlock : 0;
}

size_t lm_head_loss_scratch(int N, int H, int V)
{
    const size_t rows = static_cast<size_t>(loss_rows(N, V));
    return round256(rows * hidden_copies(N, H, V) * copied_pitch(N, H, V) * 2) +
           round256(rows * 2 * ceil_div(V, kTile) * sizeof(float2)) +
           round256(rows * sizeof(float));
}

// The gradient's scratch, each part 256-byte aligned.
struct GradScratch {
    Packed packed;
    uint4 *copies;  // for the logits
    void *dz;
    float *sums;
    size_t bytes;
};

static GradScratch carve(int N, int H, int V, void *base)
{
    const GradPlan p = grad_plan(N, H, V);
    const size_t n = static_cast<size_t>(N);
    uint8_t *at = static_cast<uint8_t *>(base);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        uint8_t *q = at ? at + off : nullptr;
        off += round256(bytes);
        return static_cast<void *>(q);
    };
    GradScratch g{};
    g.packed.hidden = static_cast<uint4 *>(take(n * p.parts * p.pitch * 2));
    const int copies = hidden_copies(N, H, V);
    g.copies = copies > 1 ? static_cast<uint4 *>(take(n * copies * copied_pitch(N, H, V) * 2)) : nullptr;
    g.packed.label = static_cast<int32_t *>(take(n * 4));
    g.packed.lse = static_cast<float *>(take(n * 4));
    g.packed.grad = static_cast<float *>(take(n * 4));
    g.packed.place = static_cast<int32_t *>(take(n * 4));
    g.packed.count = static_cast<int *>(take(4));
    g.dz = take(n * p.parts * p.piece * 2);
    g.sums = static_cast<float *>(take(n * p.parts * H * p.splits * sizeof(float)));
    g.bytes = off;
    return g;
}

size_t lm_head_loss_grad_scratch(int N, int H, int V) { return carve(N, H, V, nullptr).bytes; }

cudaError_t launch_lm_head_loss(int N, int H, int V, const void *hidden, const void *W, const int32_t *labels,
                                float *loss, float *lse, uint32_t *status, void *scratch, cudaStream_t stream)
{
    Maps m{};
    Args a{};
    a.H = H;
    a.V = V;
    a.col_tiles = ceil_div(V, kTile);
    a.width = a.col_tiles * kTile;
    a.status = status;
    const int pitch = copied_pitch(N, H, V), rows = loss_rows(N, V);
    a.copies = hidden_copies(N, H, V);  // (more than one: all rows are taken at once)
    a.copy_blocks = pitch / kBlock;
    uint8_t *at = static_cast<uint8_t *>(scratch);
    uint4 *const padded = pitch ? reinterpret_cast<uint4 *>(at) : nullptr;
    at += round256(static_cast<size_t>(rows) * a.copies * pitch * 2);
    a.part = reinterpret_cast<float2 *>(at);
    at += round256(static_cast<size_t>(rows) * 2 * a.col_tiles * sizeof(float2));
    a.label_logit = reinterpret_cast<float *>(at);
    cudaError_t e = load_maps(&m.w, &m.w_tail, &a.blocks_w, W, V, H);
    if (e != cudaSuccess)
        return e;
    for (int r0 = 0; r0 < N; r0 += rows) {
        a.N = std::min(rows, N - r0);
        a.row_tiles = ceil_div(a.N, kTile);
        a.labels = labels + r0;
        const uint16_t *h = static_cast<const uint16_t *>(hidden) + static_cast<long long>(r0) * H;
        if (padded) {
            const long long chunks = static_cast<long long>(a.N) * (pitch / 8);
            e = launch_dependent(pad_kernel, dim3(static_cast<unsigned>(std::min(1216ll, (chunks + 255) / 256))),
                                 dim3(256), 0, stream, reinterpret_cast<const uint4 *>(h),
                                 static_cast<const int32_t *>(nullptr), a.N, V, H / 8, pitch / 8, a.copies,
                                 static_cast<long long>(pitch / 8), a.copies * (pitch / 8), padded);
            if (e != cudaSuccess)
                return e;
            h = reinterpret_cast<const uint16_t *>(padded);
        }
        const int cols = padded ? a.copies * pitch : H;
        if ((e = load_map(&m.h, h, a.N, cols, cols, false)) != cudaSuccess)
            return e;
        const int pairs = static_cast<int>(
            std::min<long long>(resident_pairs(), static_cast<long long>(a.row_tiles) * a.col_tiles));
        if ((e = launch<kLoss>(m, a, pairs, stream)) != cudaSuccess)
            return e;
        if ((e = launch_dependent(rows_kernel, dim3(static_cast<unsigned>(ceil_div(a.N, 8))), dim3(1024), 0, stream,
                                  static_cast<const float2 *>(a.part), 2 * a.col_tiles, a.N, V, a.labels,
                                  static_cast<const float *>(a.label_logit), loss + r0, lse + r0)) != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

cudaError_t launch_lm_head_loss_grad(int N, int H, int V, const void *hidden, const void *W, const int32_t *labels,
                                     const float *lse, const float *grad, void *d_hidden, void *d_W, bool d_W_f32,
                                     uint32_t *status, void *scratch, cudaStream_t stream)
{
    const GradPlan p = grad_plan(N, H, V);
    const GradScratch g = carve(N, H, V, scratch);
    // One tile of rows takes the same work with its ignored rows as without: it needs no packing, only zeros in their
    // place, which the scores' launch writes where its boxes can be the caller's rows (a launch less: 3.7 of 20.8 us
    // at 8 x 256 x 4096).
    const bool in_place = N <= kTile && H % kBlock == 0, few = in_place || p.parts == 2;
    cudaError_t e = cudaSuccess;
    if (!few) {
        const int per = ceil_div(N, 1024);
        e = launch_dependent(pack_kernel, dim3(static_cast<unsigned>(ceil_div(N, per))), dim3(256), 0, stream,
                             static_cast<const uint4 *>(hidden), labels, lse, grad, N, H, V, p.pitch, per, g.packed);
    } else if (!in_place) {
        const long long chunks = static_cast<long long>(N) * (p.pitch / 8);
        e = launch_dependent(pad_kernel, dim3(static_cast<unsigned>((chunks + 255) / 256)), dim3(256), 0, stream,
                             static_cast<const uint4 *>(hidden), labels, N, V, H / 8, p.pitch / 8, p.parts, chunks,
                             p.pitch / 8, g.packed.hidden);
    }
    const int copies = hidden_copies(N, H, V), copied = copied_pitch(N, H, V);
    if (e == cudaSuccess && copies > 1) {  // (few rows)
        const int chunks = copied / 8;
        e = launch_dependent(pad_kernel,
                             dim3(static_cast<unsigned>(ceil_div(static_cast<long long>(N) * chunks, 256))), dim3(256),
                             0, stream, static_cast<const uint4 *>(hidden), labels, N, V, H / 8, chunks, copies,
                             static_cast<long long>(chunks), copies * chunks, g.copies);
    }
    if (e != cudaSuccess)
        return e;
    Maps m{};
    Args a{};
    a.N = N;
    a.H = H;
    a.V = V;
    a.h_tiles = ceil_div(H, kTile);
    a.count = few ? nullptr : g.packed.count;
    a.labels = few ? labels : g.packed.label;
    a.lse = few ? lse : g.packed.lse;
    a.grad = few ? grad : g.packed.grad;
    a.row_tiles = 1;
    a.parts = p.parts;
    a.dz = static_cast<uint16_t *>(g.dz);
    a.sums = g.sums;
    a.dz_pitch = p.piece;
    a.hidden = d_hidden != nullptr;
    a.weights = d_W != nullptr;
    a.d_w_f32 = d_W_f32;
    a.status = status;
    const int rows = N * p.parts;  // that d_W's products sum over
    if ((e = load_map(&m.h, g.packed.hidden, rows, p.pitch, p.pitch, false)) != cudaSuccess ||
        (e = load_maps(&m.w, &m.w_tail, &a.blocks_w, W, V, H)) != cudaSuccess ||
        (e = load_map(&m.z, g.dz, rows, p.piece, p.piece, false)) != cudaSuccess ||
        (e = store_map(&m.z_out, g.dz, false, N, p.piece, 0)) != cudaSuccess ||
        (e = store_map(&m.dh, g.sums, true, N, H, p.splits * p.parts)) != cudaSuccess ||
        (e = d_W ? store_map(&m.dw, d_W, d_W_f32, V, H, 0) : cudaSuccess) != cudaSuccess)
        return e;
    for (int part = 0; part < p.parts; ++part) {
        void *dz = static_cast<uint16_t *>(g.dz) + static_cast<size_t>(part) * N * p.piece;
        if ((e = load_map(&m.z_part[part], dz, N, p.piece, p.piece, false)) != cudaSuccess)
            return e;
    }
    Maps score = m;  // (the rows once)
    a.copies = copies;
    a.copy_blocks = copied / kBlock;
    if (few && (e = copies > 1 ? load_map(&score.h, g.copies, N, copies * copied, copies * copied, false)
                    : in_place ? load_map(&score.h, hidden, N, H, H, false)
                             : load_map(&score.h, g.packed.hidden, N, p.pitch, p.pitch, false)) != cudaSuccess)
        return e;
    const long long resident = resident_pairs(), row_tiles = ceil_div(N, kTile);
    for (int v0 = 0; v0 < V; v0 += p.piece) {
        a.v0 = v0;
        a.col_tiles = ceil_div(std::min(p.piece, V - v0), kTile);
        a.width = a.col_tiles * kTile;
        a.first = v0 == 0;
        a.raw = in_place && a.first ? static_cast<const uint4 *>(hidden) : nullptr;
        a.packed = g.packed.hidden;
        if ((e = launch<kScore>(score, a, static_cast<int>(std::min(resident, row_tiles * a.col_tiles)), stream)) !=
            cudaSuccess)
            return e;
        // parts beyond a short last piece's stages would be empty (their sums are those of the pieces before)
        a.splits = std::min(p.splits, a.width / kStageK);
        const long long tiles = (d_hidden ? row_tiles * a.h_tiles * a.splits : 0) +
                                (d_W ? static_cast<long long>(a.col_tiles) * a.h_tiles : 0);
        if ((e = launch<kGrad>(m, a, static_cast<int>(std::min(resident, tiles)), stream)) != cudaSuccess)
            return e;
    }
    if (!d_hidden)
        return cudaSuccess;
    const long long chunks = static_cast<long long>(N) * (H / 8);
    const int sums = p.splits * p.parts;
    const bool share = sums >= 8;
    const long long threads = chunks * (share ? 8 : 1);
    return launch_dependent(
        share ? hidden_grad_kernel<8> : hidden_grad_kernel<1>,
        dim3(static_cast<unsigned>(std::min<long long>(device_sm_count() * 8ll, (threads + 255) / 256))), dim3(256), 0,
        stream, reinterpret_cast<const float4 *>(g.sums), sums, N, H / 8,
        static_cast<const int32_t *>(few ? nullptr : g.packed.place), labels, V, static_cast<uint4 *>(d_hidden));
}

}  // namespace df2
