// attention.cu -- attention of a block of new tokens over the paged cache, on tcgen05 tensor cores.
//
// For query row r (a token and a query head) over the keys j it sees:
//   x_j = scale log2(e) q_r . k_j,   m = max x_j,   l = sum 2^(x_j - m),   o = sum 2^(x_j - m) v_j / l
// in one pass over tiles of 128 keys with a running m: when a tile raises it, l and o are scaled by
// 2^(m_old - m_new).  As long as it rises by no more than 8 (a factor 256, harmless in float32 and
// in the 16-bit probabilities) the old m is kept, so o is seldom touched.
//
// A work item is a sequence, a cache head and a run of its new tokens: the query heads that share
// the cache head are rows of the same tile (token major), 128 rows a tile, one or two tiles (two when
// a sequence may have more rows than one holds: they share every K and V tile read).  Each CTA (one
// per SM) takes an equal share of all (item, key tile) pairs in order, so lengths may differ at will
// and few items still fill the GPU; an item that crosses a border is finished by the combine kernel
// from partial (o, m, l), pieces in order, so results do not depend on timing.
//
// Roles of a CTA:
//   warp 0     walks the work and hands segments to the others; loads K tiles by TMA, a box per run of
//              rows of a page (gcd(page_size, 128) of them), pages looked up 32 at a time
//   warp 3     loads V tiles;   warp 2   (8-bit cache) fetches and prepares the tiles' scales
//   warp 1     one elected lane issues the MMAs
//   a warpgroup per row tile: softmax, a thread per row, S read from and P written back to TMEM
//   two warpgroups (8-bit cache): widen codes to f16 in shared memory, one K's and one V's
//   S = Q K^T   K from shared memory as it lies, Q from TMEM (one row tile) or shared memory (two)
//   O += P V    P from TMEM over S, V as it lies (its rows are the K dimension: MN-major B)
// One row tile: two S take turns, so the next S is ready when a softmax ends.  Two row tiles: one S
// each (TMEM is full), and the products of one run under the softmax of the other.
//
// Few rows (a draft block of one cache head is often 8 to 64 of them) leave most of a 128-row tile
// empty, and a thread that walks 128 scores is then the longest step of a tile.  With an 8-bit cache
// the tile holds such rows FOLD = 2 or 4 times over: every copy takes 128 / FOLD of a tile's keys (its
// P is zero elsewhere), with its own m and l, and the copies are added up at the end of the item.
// 8-bit caches: codes are exact in f16, so K's scale multiplies the score, and V's goes into the
// exponent: x'_j = x_j + log2(vs_j), P'_j = 2^(x'_j - m'), o = sum P'_j code_j, l = sum P'_j / vs_j,
// which keeps P' in f16's range whatever the values' size (2^7 P' is what is rounded, see kAbove).
// Value rows of zeros, and those that are not finite, get a scale that leaves m' to the others; the
// latter mark their run of tiles, whose rows of o end as NaN.  Queries go to f16 by a power of two per
// row that brings the row's largest magnitude to 2^14..2^15 (smaller parts lose bits only below
// 2^-24 of it).  With a bf16 cache everything stays bf16; P is rounded once, to bf16 or f16, as the
// MMA's operand; scores, sums and o are float32.
//
// What bounds it, and measured on one GB300 (copy 6768 GB/s, cuBLAS bf16 1957 TFLOP/s burst):
//   32 sequences x 16 tokens, up to 8192 keys, 32 / 8 heads of 128, bf16: HBM; 131 us, 5.9 TB/s
//     (the kernel alone 126 us and 1.01 times the algorithmic bytes; the rest is the combine kernel)
//   32 x 8 tokens, up to 16384 keys, e4m3: shared memory, which the codes cross three times (TMA in,
//     widening, MMA: some 1,540 of the 2,190 cycles of a tile); 171 to 177 us, 4.5 to 4.6 TB/s
//   one sequence, 2048 tokens over 18432 keys, bf16: the chain of a tile's softmax and products;
//     373 us cold, 1.57 PFLOP/s, 382 to 406 back to back under the power cap; over e4m3 661 to 672,
//     every CTA widening each key tile again for its own 256 rows
//   one token over 777 keys: a chain of latencies (lengths, pages, tile, softmax, combine); 9.8 to 10.3 us
// The code of all roles has to fit the instruction cache: with the walk in every role and loops
// unrolled (11,200 instructions) warps waited for instructions and the e4m3 case took 330 us.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <numeric>

#include "attention_work.cuh"
#include "f32x2.cuh"
#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "tensor_map.h"

namespace df2 {
namespace {

constexpr int BM = 128;  // rows of a tile
constexpr int HALF_BYTES = 128 * 128;  // 128 rows of 64 16-bit elements
constexpr int SMEM_LIMIT = 227 * 1024;
constexpr int MAX_RING = 12;
constexpr int MAX_WIDE = 4;
constexpr int SEGMENTS = 4;  // segments that the walking warp may be ahead
constexpr int MAX_SCALES = 4;
constexpr float kLeastScale = -108.f;  // log2 of the least scale a cache holds, 1e-30 / 448
constexpr float LAZY = 8.f;   // how far the running maximum may lag, in powers of two
// An 8-bit cache's P' are f16 with the maximum at 2^7, so at most 2^15 while it lags: what is up to
// 2^-32 of the maximum is not lost (at 1 it was 2^-25: 3% of a result over a million such keys).
constexpr float kAbove = 7.f, kBelow = 0x1p-7f;

struct SplitRecord {  // an item whose pieces the combine kernel joins
    int32_t valid, first_slot, c0, c1, kvh, tok0, ntok, pad;
};

struct Args {
    PagedCache cache;
    TokenBatch tokens;
    HeadRows q, out;
    float *lse;
    float scale_log2;
    uint32_t q_and, q_xor;  // scale 0 clears q, a negative one flips its sign
    WorkShape work;
    int group;             // query heads of a cache head
    int q_wide, out_wide;  // rows begin on 32-byte borders
    int tpm;               // tokens of a row tile
    uint32_t page_magic, page_shift;  // token / page_size = umulhi(token, magic) >> shift
    int box;   // rows of a TMA box: gcd(page_size, 128)
    int ring;  // stages of the TMA ring
    SplitRecord *records;
    float2 *part_ml;  // [2 * grid][rows]: (maximum, logarithm of the sum), in powers of two
    float *part_o;    // [2 * grid][rows][dim]
    uint32_t *status;
};

// token / page_size for 0 <= token < 2^31.
__device__ __forceinline__ int page_of_token(const Args &a, int token)
{
    return static_cast<int>(__umulhi(static_cast<uint32_t>(token), a.page_magic) >> a.page_shift);
}

constexpr int NEAR = 32;              // sequences whose numbers a CTA keeps in shared memory
constexpr uint32_t MANY = 0xFFFFFFFFu;  // units of a sequence that are counted anew where they are wanted

__device__ __forceinline__ Sequence load_sequence(const Args &a, int b)
{
    Sequence s;
    s.start = min(max(__ldg(a.tokens.token_start + b), 0), a.tokens.N);
    s.n = min(max(__ldg(a.tokens.token_start + b + 1), s.start), a.tokens.N) - s.start;
    s.len = min(max(__ldg(a.tokens.kv_len + b), 0), a.tokens.max_pages * a.cache.page_size);
    return s;
}

// Where one kind of operand is in a ring that both share: operand 2 j is tile j's K, 2 j + 1 its V,
// operand i is in slot i mod size, for the (i / size)-th time.
struct RingSlot {
    int slot, round;
    __device__ __forceinline__ void step(int size)
    {
        slot += 2;
        if (slot >= size) {
            slot -= size;
            ++round;
        }
    }
    // The n-th time (from 0) that this kind takes the slot over from its last user; -1: it was free.
    // In a ring of odd size a slot holds the two kinds in turn.
    __device__ __forceinline__ int turn(int size, int kv) const
    {
        return (size & 1) == 0 ? round - 1 : (round >> 1) - ((slot & 1) == kv ? 1 : 0);
    }
};

// Position in a ring of `size` slots, two items (a K and a V) at a time.
struct RingAt {
    int slot;
    uint32_t phase;
    __device__ __forceinline__ void step(int size)
    {
        slot += 2;
        if (slot >= size) {
            slot -= size;
            phase ^= 1u;
        }
    }
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log2(2^a + 2^b)
__device__ __forceinline__ float log_sum(float a, float b)
{
    const float top = fmaxf(a, b);
    return top + __log2f(ex2(a - top) + ex2(b - top));
}

__device__ __forceinline__ uint32_t f16_pack(float a, float b)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    return d;
}

// Four codes of an 8-bit cache as f16 (exact).
template <int TYPE>
__device__ __forceinline__ uint2 widen4(uint32_t w)
{
    uint2 r;
    if constexpr (TYPE == 1) {
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r.x) : "h"(static_cast<uint16_t>(w)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r.y) : "h"(static_cast<uint16_t>(w >> 16)));
    } else {
        // 0x6400 | u is the f16 number 1024 + u; u = code + 128
        w ^= 0x80808080u;
        const uint32_t lo = __byte_perm(w, 0x64646464u, 0x4140), hi = __byte_perm(w, 0x64646464u, 0x4342);
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r.x) : "r"(lo), "r"(0x64806480u));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r.y) : "r"(hi), "r"(0x64806480u));
    }
    return r;
}

template <int QT, int TYPE>
struct Shape {
    // widened tiles: two K and two V; with two row tiles there is room for three in rotation
    static constexpr int kWideRing = QT == 1 ? 4 : 3;
    // tiles whose scales are held, ready (see soft_done) and as they lie
    static constexpr int kScales = QT == 1 ? 2 : 4, kRaws = QT == 1 ? 4 : 2;
    static constexpr int kThreads = 128 * (1 + QT + (TYPE ? 2 : 0));
    // registers of a thread after the roles part: control, softmax, widening (their sum times 128
    // is at most what the launch holds: 65536 / threads, a multiple of 8, times the threads)
    static constexpr int kSoftRegs = TYPE == 0 ? 200 : QT == 2 ? 128 : 184;
    static constexpr int kWideRegs = QT == 2 ? 64 : 112;
    static constexpr int kControlRegs = TYPE == 0 ? 104 : QT == 2 ? 96 : 104;
    static constexpr bool kSplitRegs = kThreads > 256;
    static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;
    static_assert(!kSplitRegs || kControlRegs + QT * kSoftRegs + (TYPE ? 2 * kWideRegs : 0) <=
                                     kThreads / 128 * kLaunchRegs, "setmaxnreg.inc would wait forever");
};

// Shared memory: Q tiles (two row tiles; one tile's queries are in TMEM) | TMA ring | widened ring
// (8-bit) | scales, and as they lie (8-bit) | place to add copies up, their (m, l) | barriers | segments | sequences | their units.
struct Layout {
    int q, ring, ring_stage, wide, scales, raw, fold, bars, segs, near, counts, bytes;
};

constexpr int BAR_COUNT = 4 * MAX_RING + 3 * MAX_WIDE + 2 + 2 + 2 + 2 + MAX_SCALES + 1 + 1 + 2 + 2 * SEGMENTS;  // tmem slot and abort flag follow

template <int DP, int QT, int TYPE, int FOLD>
__host__ __device__ constexpr Layout layout_of(int ring, int dim, int B)
{
    Layout l{};
    const int tile = DP / 64 * HALF_BYTES;
    l.q = 0;
    l.ring = QT == 2 ? QT * tile : 0;
    l.ring_stage = TYPE ? 128 * dim : tile;
    l.wide = l.ring + ring * l.ring_stage;
    l.scales = l.wide + (TYPE ? Shape<QT, TYPE>::kWideRing * tile : 0);
    l.raw = l.scales + (TYPE ? Shape<QT, TYPE>::kScales * 3 * BN * 4 : 0);
    l.fold = l.raw + (TYPE ? Shape<QT, TYPE>::kRaws * 2 * BN * 4 : 0);
    l.bars = l.fold + (FOLD > 1 ? BM * 16 * 4 + BM * 8 : 0);
    l.segs = l.bars + BAR_COUNT * 8 + 8;
    l.near = l.segs + SEGMENTS * static_cast<int>(sizeof(Segment));
    l.counts = l.near + NEAR * static_cast<int>(sizeof(Sequence));
    l.bytes = l.counts + B * 4;
    return l;
}

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity)
{
    const unsigned long long t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > kWaitTimeoutNs / 10)
            return;
}

// 16 bytes of shared memory.  volatile keeps a batch of them together and ahead of the wait that
// follows: behind the widening warps' stores each takes some 250 cycles, so they must all be in flight.
__device__ __forceinline__ float4 lds4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

// 32 bytes a lane: rows are a lane each, so an access touches as many lines as it has lanes and costs
// as many cycles; half as many accesses are half the time.
__device__ __forceinline__ void ldg8(const void *p, uint32_t *v)
{
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(__cvta_generic_to_global(p)));
}

__device__ __forceinline__ void stg8(void *p, const uint32_t *v)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(__cvta_generic_to_global(p)), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

__device__ __forceinline__ uint64_t load2(const uint32_t *v) { return f2(__uint_as_float(v[0]), __uint_as_float(v[1])); }

__device__ __forceinline__ void store2(uint32_t *v, uint64_t x)
{
    const float2 f = f2_split(x);
    v[0] = __float_as_uint(f.x);
    v[1] = __float_as_uint(f.y);
}

// A converged warp's wait for the phase of parity `parity`; false when another role gave up, or
// after kWaitCycles, when it gives up itself.  (As short as it can be: it is inlined everywhere.)
constexpr long long kWaitCycles = 2000000000;  // about a second
// For warps that have no part in an item while the others work through all of its tiles: up to 2^23 of
// them, a microsecond and more each.  Should one of the others give up, these see its flag.
constexpr long long kIdleCycles = 64 * kWaitCycles;

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                          long long limit = kWaitCycles)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
        return true;
    const long long t0 = clock64();
    while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
        if (__any_sync(0xffffffffu, *abort_flag != 0 || clock64() - t0 > limit)) {
            *abort_flag = 1;
            return false;
        }
    }
    return true;
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

template <int DP, int QT, int TYPE, int FOLD>
__global__ void __launch_bounds__(Shape<QT, TYPE>::kThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const __grid_constant__ Args a)
{
    constexpr int kThreads = Shape<QT, TYPE>::kThreads;
    constexpr int kHalves = DP / 64;
    constexpr int kTile = kHalves * HALF_BYTES;
    constexpr bool kQuant = TYPE != 0;
    constexpr int kWide = Shape<QT, TYPE>::kWideRing;
    constexpr int kScales = Shape<QT, TYPE>::kScales, kRaws = Shape<QT, TYPE>::kRaws;
    constexpr int kRows = BM / FOLD;  // distinct rows of a tile
    constexpr int kCols = BN / FOLD;  // keys of a tile that a thread takes
    constexpr int kQCol = 384;        // TMEM: two S at 0 and 128, O at 256 (and 384), one tile's Q at 384
    extern __shared__ uint8_t smem_raw[];
    // an offset into the array, not a rounded address: the compiler must see shared memory, or every
    // access becomes a generic one (the scales' reads were the longest step of a tile)
    uint8_t *smem = smem_raw + (1024u - (smem_u32(smem_raw) & 1023u)) % 1024u;
    const Layout lay = layout_of<DP, QT, TYPE, FOLD>(a.ring, a.cache.dim, a.tokens.B);
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + lay.bars;
    // A barrier's phases are told apart by parity, so whoever waits on one must wait for every phase
    // of it.  The slots of a ring of odd size hold a K and a V in turn, which different warps load and
    // widen: each has barriers of its own (next_kv: what the slot becomes free for).  Where a phase is
    // skipped, the one before must be known to be over: pv_done has a barrier for each S, not each row
    // tile, because with one row tile an S that is ready says that the products two tiles back are in,
    // not those of the last tile, and after a late V a wait on one barrier let go two phases early.
    auto ring_full = [&](int s, int kv) { return bar0 + 8u * (s + (kQuant ? kv * MAX_RING : 0)); };
    auto ring_empty = [&](int s, int next_kv) { return bar0 + 8u * (MAX_RING * (2 + next_kv) + s); };
    auto wide_full = [&](int s) { return bar0 + 8u * (4 * MAX_RING + s); };
    auto wide_empty = [&](int s, int next_kv) { return bar0 + 8u * (4 * MAX_RING + MAX_WIDE * (1 + next_kv) + s); };
    constexpr int kRest = 4 * MAX_RING + 3 * MAX_WIDE;
    auto s_full = [&](int x) { return bar0 + 8u * (kRest + x); };
    auto p_full = [&](int x) { return bar0 + 8u * (kRest + 2 + x); };
    auto pv_done = [&](int s) { return bar0 + 8u * (kRest + 4 + s); };
    auto q_full = [&](int s) { return bar0 + 8u * (kRest + 6 + s); };
    auto scale_full = [&](int s) { return bar0 + 8u * (kRest + 8 + s); };
    constexpr int kMore = kRest + 8 + MAX_SCALES;
    const uint32_t drain_bar = bar0 + 8u * kMore;
    const uint32_t meet_bar = bar0 + 8u * (kMore + 1);
    auto soft_done = [&](int x) { return bar0 + 8u * (kMore + 2 + x); };
    auto seg_full = [&](int i) { return bar0 + 8u * (kMore + 4 + i); };
    auto seg_empty = [&](int i) { return bar0 + 8u * (kMore + 4 + SEGMENTS + i); };
    static_assert(kMore + 4 + 2 * SEGMENTS == BAR_COUNT, "barriers");
    // what the MMAs read: the TMA ring itself, or the widened one
    const int op_size = kQuant ? kWide : a.ring;
    const uint32_t op_base = sbase + (kQuant ? lay.wide : lay.ring);
    auto op_full = [&](int s) { return kQuant ? wide_full(s) : ring_full(s, 0); };
    auto op_empty = [&](int s, int kv) { return kQuant ? wide_empty(s, kWide & 1 ? 1 - kv : kv) : ring_empty(s, a.ring & 1 ? 1 - kv : kv); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + lay.bars + BAR_COUNT * 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    uint32_t *counts = reinterpret_cast<uint32_t *>(smem + lay.counts);
    Sequence *near = reinterpret_cast<Sequence *>(smem + lay.near);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        griddep_launch_dependents();
        for (int s = 0; s < a.ring; ++s) {
            mbar_init(ring_full(s, 0), 1);
            if (kQuant)
                mbar_init(ring_full(s, 1), 1);
            mbar_init(ring_empty(s, 0), kQuant ? 4 : 1);
            mbar_init(ring_empty(s, 1), kQuant ? 4 : 1);
        }
        for (int s = 0; s < kWide; ++s) {
            mbar_init(wide_full(s), 4);
            mbar_init(wide_empty(s, 0), 1);
            mbar_init(wide_empty(s, 1), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(s_full(s), 1);
            mbar_init(p_full(s), 4);
            mbar_init(pv_done(s), 1);
            mbar_init(q_full(s), 4);
            mbar_init(soft_done(s), 4);
        }
        for (int s = 0; s < kScales; ++s) {
            mbar_init(scale_full(s), 1);
        }
        for (int s = 0; s < SEGMENTS; ++s) {
            mbar_init(seg_full(s), 1);
            mbar_init(seg_empty(s), 2 + 4 * QT + (kQuant ? 1 + 8 : 0));  // warps that read it
        }
        mbar_init(drain_bar, 1);
        mbar_init(meet_bar, 4);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&map_k);
        prefetch_tmap(&map_v);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();

    // Units of each sequence (for one cache head), as many as 32 bits hold.  Up to 32 sequences warp 0
    // does it alone and the others need not wait.
    const int B = a.tokens.B;
    auto sequence = [&](int b) { return b < NEAR ? near[b] : load_sequence(a, b); };
    auto count = [&](int b, long long n) { counts[b] = static_cast<uint32_t>(min(n, static_cast<long long>(MANY))); };
    if (B > NEAR) {
        for (int b = threadIdx.x; b < B; b += kThreads) {
            const Sequence s = load_sequence(a, b);
            if (b < NEAR)
                near[b] = s;
            count(b, units_of(a.work, s, 0, 1));
        }
        __syncthreads();
    } else if (warp == 0) {
        Sequence s{0, 0, 0};
        if (lane < B)
            near[lane] = s = load_sequence(a, lane);
        if (__all_sync(0xffffffffu, items_of(a.work, s) <= 4)) {
            if (lane < B)
                count(lane, units_of(a.work, s, 0, 1));
        } else {
            __syncwarp();
            for (int b = 0; b < B; ++b) {
                long long t = units_of(a.work, near[b], lane, 32);
                for (int o = 16; o > 0; o >>= 1)
                    t += __shfl_xor_sync(0xffffffffu, t, o);
                if (lane == 0)
                    count(b, t);
            }
        }
        __syncwarp();
    }
    const int cta = blockIdx.x;
    Segment *segs = reinterpret_cast<Segment *>(smem + lay.segs);
    // the CTA's n-th segment (tiles == 0: there is none), and done with it
    auto seg_wait = [&](int n, long long limit = kWaitCycles) {
        return warp_wait(seg_full(n % SEGMENTS), (n / SEGMENTS) & 1, abort_flag, limit);
    };
    auto seg_done = [&](int n) {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(seg_empty(n % SEGMENTS));
    };

    if (warp < 4) {
        // One place for the whole warpgroup: setmaxnreg wants all its warps at the same instruction, and
        // the softmax warps' wait for what it gives back has no limit.
        if constexpr (Shape<QT, TYPE>::kSplitRegs)
            reg_dec<Shape<QT, TYPE>::kControlRegs>();
        if (warp == 0 || warp == 3) {
            // ---------------------------------------------------------------- TMA producers: K, V
            // Warp 0 also walks.  One lane issues with warp-uniform operands, box after box: lanes that
            // issue their own boxes are taken one by one anyhow, at several times the cost.
            const int kv = warp == 0 ? 0 : 1;
            const CUtensorMap *map = kv ? &map_v : &map_k;
            Shares shares(1, 1);
            Walk walk;
            walk.u = walk.u_end = 0;
            if (kv == 0) {
                auto units_in = [&](int b) -> long long {
                    if (b >= B)
                        return 0;
                    const uint32_t n = counts[b];
                    return n < MANY ? n : units_of(a.work, sequence(b), 0, 1);
                };
                auto running = [&](long long t) {  // this lane's and those of the lanes before it
                    for (int o = 1; o < 32; o <<= 1) {
                        const long long x = __shfl_up_sync(0xffffffffu, t, o);
                        t += lane >= o ? x : 0;
                    }
                    return t;
                };
                // Sequences 32 at a time; a lane keeps what is ahead of runs `lane` and `lane + 32`.
                long long sum = 0, mine = 0, upto = 0, ahead_lo = 0, ahead_hi = 0;
                const int runs = (B + 31) / 32;
                for (int i = 0; i < runs; ++i) {
                    mine = units_in(32 * i + lane);
                    upto = running(mine);
                    if (lane == (i & 31)) {
                        if (i < 32)
                            ahead_lo = sum;
                        else
                            ahead_hi = sum;
                    }
                    sum += __shfl_sync(0xffffffffu, upto, 31);
                }
                const long long units = sum * a.work.heads;
                const int grid = static_cast<int>(min(static_cast<long long>(gridDim.x), max(units, 1ll)));
                shares = Shares(units, grid);
                if (cta < grid && units > 0) {
                    // the last run, and in it the last sequence, that begins at or before the share
                    const long long u = shares.begin(cta);
                    int run = 0;
                    if (runs > 1) {
                        run = __popc(__ballot_sync(0xffffffffu, lane < runs && ahead_lo * a.work.heads <= u)) +
                              __popc(__ballot_sync(0xffffffffu, lane + 32 < runs && ahead_hi * a.work.heads <= u)) - 1;
                        mine = units_in(32 * run + lane);
                        upto = running(mine);
                    }
                    const long long ahead = __shfl_sync(0xffffffffu, run < 32 ? ahead_lo : ahead_hi, run & 31) + upto - mine;
                    const uint32_t before = __ballot_sync(0xffffffffu, 32 * run + lane < B && ahead * a.work.heads <= u);
                    const int at = 31 - __clz(before);
                    walk.begin(a.work, sequence, u, shares.begin(cta + 1), 32 * run + at,
                               __shfl_sync(0xffffffffu, ahead, at), __shfl_sync(0xffffffffu, mine, at));
                }
            }
            const int boxes = BN / a.box, per_batch = 32 / boxes;  // boxes of a tile, tiles of a batch of 32
            const int ps = a.cache.page_size, dim = a.cache.dim;
            const uint32_t box_bytes = kQuant ? a.box * dim : a.box * 128 * kHalves;
            RingSlot rs{kv, 0};
            int tcnt = 0;  // tiles begun
            bool ok = true;
            for (int n = 0; ok; ++n) {
                const Segment &g = segs[n % SEGMENTS];
                if (kv == 0) {
                    if (n >= SEGMENTS)
                        ok = warp_wait(seg_empty(n % SEGMENTS), (n / SEGMENTS - 1) & 1, abort_flag);
                    if (!ok)
                        break;
                    Segment next;
                    walk.next(a.work, sequence, cta, shares, next);
                    if (lane == 0) {
                        if constexpr (kQuant)
                        next.spoilt = 0;
                    segs[n % SEGMENTS] = next;
                        mbar_arrive(seg_full(n % SEGMENTS));
                    }
                    __syncwarp();
                } else {
                    ok = seg_wait(n);
                }
                const int tiles = g.tiles, kvh = g.kvh;
                if (!ok || tiles == 0)
                    break;
                const int32_t *pt = a.tokens.page_table + static_cast<long long>(g.b) * a.tokens.max_pages;
                const int tok0 = g.tile * BN, lo = g.item.lo, hi = g.item.hi;
                // 32 boxes' pages at a time, a lane each, the next 32 on their way: a load waits hundreds of
                // cycles, too long to be met at every tile
                auto pages_at = [&](int j) {
                    const int tok = tok0 + j * BN + lane * a.box;
                    const bool need = tok < hi && tok + a.box > lo;
                    return need ? min(max(__ldg(pt + page_of_token(a, tok)), 0), a.cache.pages - 1) : -1;
                };
                int batch = pages_at(0), next_batch = pages_at(per_batch), at = 0;
                uint32_t needed = __ballot_sync(0xffffffffu, batch >= 0);
                for (int j = 0; j < tiles; ++j) {
                    if (at == 32) {
                        at = 0;
                        batch = next_batch;
                        needed = __ballot_sync(0xffffffffu, batch >= 0);
                        next_batch = pages_at(j + per_batch);
                    }
                    const int tok = tok0 + j * BN;
                    const int here = __popc(needed >> at & ((1u << boxes) - 1u));
                    const int turn = rs.turn(a.ring, kv);
                    if (turn >= 0)
                        ok = warp_wait(ring_empty(rs.slot, kv), turn & 1, abort_flag);
                    if (!ok)
                        break;
                    const uint32_t full = ring_full(rs.slot, kv);
                    if (elect_one())
                        mbar_arrive_expect_tx(full, here * box_bytes);
                    __syncwarp();
                    uint32_t dst = sbase + lay.ring + rs.slot * lay.ring_stage;
                    int in_page = tok - page_of_token(a, tok) * ps;
#pragma unroll 1
                    for (int i = 0; i < boxes; i += 4) {
                        int page[4], x[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            page[k] = __shfl_sync(0xffffffffu, batch, (at + i + k) & 31);
                            page[k] = i + k < boxes ? page[k] : -1;
                            x[k] = in_page;
                            in_page += a.box;
                            in_page = in_page == ps ? 0 : in_page;
                        }
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if (page[k] >= 0) {
                                    const uint32_t to = dst + k * a.box * (kQuant ? dim : 128);
                                    if constexpr (kQuant) {
                                        tma_load_4d(to, map, full, 0, x[k], kvh, page[k]);
                                    } else {
#pragma unroll
                                        for (int h = 0; h < kHalves; ++h)
                                            tma_load_4d(to + h * HALF_BYTES, map, full, h * 64, x[k], kvh, page[k]);
                                    }
                                }
                            }
                        }
                        __syncwarp();
                        dst += 4 * a.box * (kQuant ? dim : 128);
                    }
                    at += boxes;
                    rs.step(a.ring);
                    ++tcnt;
                }
                if (ok && kv == 1)
                    seg_done(n);
            }
            if (!ok) {  // let the copies already issued land before the CTA leaves
                for (int n = max(tcnt - a.ring, 0); n < tcnt; ++n) {
                    const int i = 2 * n + kv, round = i / a.ring;
                    drain_wait(ring_full(i % a.ring, kv), (kQuant && (a.ring & 1) ? round >> 1 : round) & 1);
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issuer
            // The warp walks and waits together and one elected lane issues: operands are then
            // warp-uniform for the compiler, which costs far less per MMA than a lone lane's.
            const uint32_t fmt = kQuant ? 0u : (1u << 7 | 1u << 10);  // f16 or bf16 operands
            const uint32_t shape = (1u << 4) | static_cast<uint32_t>(BM >> 4) << 24;
            const uint32_t idesc_qk = fmt | shape | static_cast<uint32_t>(BN >> 3) << 17;
            const uint32_t idesc_pv = fmt | shape | static_cast<uint32_t>(DP >> 3) << 17 | 1u << 16;  // V is MN-major
            const uint64_t k_desc = sw128_kmajor_desc(0), v_desc = sw128_mnmajor_desc(0, HALF_BYTES);
            const uint32_t k_lo = static_cast<uint32_t>(k_desc), k_hi = static_cast<uint32_t>(k_desc >> 32);
            const uint32_t v_lo = static_cast<uint32_t>(v_desc), v_hi = static_cast<uint32_t>(v_desc >> 32);
            RingAt kr{0, 0}, vr{1, 0};
            int cnt[2] = {0, 0};  // tiles done, per row tile (QT = 2) or in all (QT = 1, cnt[0])
            uint32_t q_phase[2] = {0, 0};
            bool ok = true;
            auto qk = [&](int s, int sbuf, int slot) {
                const uint32_t q = k_lo + ((sbase + lay.q + s * kTile) >> 4);
                const uint32_t k = k_lo + ((op_base + __shfl_sync(0xffffffffu, slot, 0) * kTile) >> 4);
                const uint32_t d = tmem + __shfl_sync(0xffffffffu, sbuf, 0) * BN;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < DP / 16; ++kk) {
                        const uint32_t o = ((kk / 4) * HALF_BYTES + (kk % 4) * 32) >> 4;
                        if constexpr (QT == 1)
                            umma_f16_tmem_a(d, tmem + kQCol + kk * 8, desc_at(k + o, k_hi), idesc_qk, kk > 0);
                        else
                            umma_bf16(d, desc_at(q + o, k_hi), desc_at(k + o, k_hi), idesc_qk, kk > 0);
                    }
                    umma_commit(s_full(sbuf));
                }
                __syncwarp();
            };
            auto pv = [&](int s, int sbuf, int slot, bool first) {
                const uint32_t v = v_lo + ((op_base + __shfl_sync(0xffffffffu, slot, 0) * kTile) >> 4);
                const uint32_t p = tmem + __shfl_sync(0xffffffffu, sbuf, 0) * BN;
                const uint32_t d = tmem + 256 + s * 128;
                const uint32_t acc = __shfl_sync(0xffffffffu, first ? 0u : 1u, 0);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < BN / 16; ++kk)
                        umma_f16_tmem_a(d, p + kk * 8, desc_at(v + kk * (2048 >> 4), v_hi), idesc_pv, kk > 0 ? 1u : acc);
                    umma_commit(pv_done(sbuf));
                }
                __syncwarp();
            };
            auto commit = [&](uint32_t bar) {
                if (elect_one())
                    umma_commit(bar);
                __syncwarp();
            };
#define DF2_WAIT(bar, parity)                                               \
    if (!warp_wait(bar, parity, abort_flag)) {                              \
        ok = false;                                                         \
        break;                                                              \
    }
            for (int n = 0; ok; ++n) {
                DF2_WAIT(seg_full(n % SEGMENTS), (n / SEGMENTS) & 1);
                const Segment &g = segs[n % SEGMENTS];
                const int tiles = g.tiles;
                if (tiles == 0)
                    break;
                // one call site each for the two products, again for the instruction cache
                if constexpr (QT == 2) {
                    // PV of a row tile, then its next S: while one tile's softmax runs, the other's
                    // products do
                    const int mt = g.item.ntok > a.tpm ? 2 : 1;
#pragma unroll 1
                    for (int j = -1; j < tiles && ok; ++j) {
                        const bool more = j + 1 < tiles;
                        if (j >= 0) {
                            DF2_WAIT(op_full(vr.slot), vr.phase);
                        }
                        if (more) {
                            DF2_WAIT(op_full(kr.slot), kr.phase);
                        }
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            if (s == mt)
                                break;
                            if (j >= 0) {
                                DF2_WAIT(p_full(s), cnt[s] & 1);
                                ++cnt[s];
                            } else {
                                DF2_WAIT(q_full(s), q_phase[s]);
                                q_phase[s] ^= 1u;
                            }
                            tc_fence_after();
                            if (j >= 0) {
                                pv(s, s, vr.slot, j == 0);
                                if (s == mt - 1)
                                    commit(op_empty(vr.slot, 1));
                            }
                            if (more)
                                qk(s, s, kr.slot);
                        }
                        if (!ok)
                            break;
                        if (j >= 0)
                            vr.step(op_size);
                        if (more) {
                            commit(op_empty(kr.slot, 0));
                            kr.step(op_size);
                        }
                    }
                } else {
                    // the next S, then PV: the softmax always has an S waiting
                    DF2_WAIT(q_full(0), q_phase[0]);
                    q_phase[0] ^= 1u;
#pragma unroll 1
                    for (int j = 0; j <= tiles; ++j) {
                        if (j < tiles) {
                            DF2_WAIT(op_full(kr.slot), kr.phase);
                            tc_fence_after();  // the queries in TMEM too
                            qk(0, (cnt[0] + (j > 0 ? 1 : 0)) & 1, kr.slot);
                            commit(op_empty(kr.slot, 0));
                            kr.step(op_size);
                        }
                        if (j > 0) {
                            const int sbuf = cnt[0] & 1;
                            DF2_WAIT(op_full(vr.slot), vr.phase);
                            DF2_WAIT(p_full(sbuf), (cnt[0] >> 1) & 1);
                            ++cnt[0];
                            tc_fence_after();
                            pv(0, sbuf, vr.slot, j == 1);
                            commit(op_empty(vr.slot, 1));
                            vr.step(op_size);
                        }
                    }
                }
                seg_done(n);
            }
#undef DF2_WAIT
            // every MMA issued must finish before TMEM is released (in a healthy run all have)
            commit(drain_bar);
            drain_wait(drain_bar, 0);
        } else if (kQuant && warp == 2) {
            // ------------------------------------------------------------ scales of the keys and values
            // A tile's scales become (ks, log2 vs, 1 / vs).  A lane copies four keys' of them, up to kRaws
            // tiles ahead and into the segments that are known by then, and prepares the same four.
            // (Bulk copies by the producers, one for each box, doubled what these issue: 32 x 8 tokens over
            // up to 16384 keys in e4m3 took 215 instead of 181 us with pages of 16, 304 instead of 230 with 24.)
            int tcnt = 0, asked = 0;  // tiles prepared, tiles whose copies are on their way
            int an = 0, aj = 0, at_end = 0, a_tiles = 0, a_tok = 0, a_lo = 0, a_hi = 0, page = -1;  // the next to ask for
            const int32_t *a_pt = nullptr;
            int a_kvh = 0;
            bool ok = true;
            auto page_at = [&](int tok) {  // -1: no key of the four is seen
                return tok < a_hi && tok + 4 > a_lo ? min(max(__ldg(a_pt + page_of_token(a, tok)), 0), a.cache.pages - 1) : -1;
            };
            auto ask = [&]() {  // false: nothing more is known
                if (aj == a_tiles) {
                    if (at_end || !__all_sync(0xffffffffu, mbar_test_wait(seg_full(an % SEGMENTS), (an / SEGMENTS) & 1)))
                        return false;
                    const Segment &x = segs[an % SEGMENTS];
                    a_tiles = x.tiles;
                    if (a_tiles == 0) {
                        at_end = 1;
                        aj = 0;
                        return false;
                    }
                    aj = 0;
                    a_lo = x.item.lo, a_hi = x.item.hi, a_kvh = x.kvh;
                    a_pt = a.tokens.page_table + static_cast<long long>(x.b) * a.tokens.max_pages;
                    a_tok = x.tile * BN + 4 * lane;
                    page = page_at(a_tok);
                    ++an;
                }
                if (page >= 0) {
                    const int ps = a.cache.page_size;
                    const long long from = (static_cast<long long>(page) * a.cache.heads + a_kvh) * ps + a_tok - page_of_token(a, a_tok) * ps;
                    const uint32_t to = sbase + lay.raw + (asked % kRaws * 2 * BN + 4 * lane) * 4;
                    cp_async16(to, a.cache.k_scale + from);
                    cp_async16(to + BN * 4, a.cache.v_scale + from);
                }
                cp_async_commit();
                a_tok += BN;
                page = ++aj < a_tiles ? page_at(a_tok) : -1;
                ++asked;
                return true;
            };
            for (int n = 0; ok; ++n) {
                ok = seg_wait(n);
                if (!ok || segs[n % SEGMENTS].tiles == 0)
                    break;
                const Segment &g = segs[n % SEGMENTS];
                const int tiles = g.tiles, lo = g.item.lo - g.tile * BN, hi = g.item.hi - g.tile * BN;
                float top_lv = -INFINITY;  // this lane's largest log2 of a value scale in the segment
                bool spoilt = false;
                for (int j = 0; j < tiles; ++j) {
#pragma unroll 1
                    while (asked - tcnt < kRaws && ask())
                        ;
                    // the first softmax warpgroup is done with the tile two back, so a second one (which
                    // the order of the MMAs keeps less than two tiles behind) with the one four back:
                    // the tile whose place this is
                    if (tcnt >= 2)
                        ok = warp_wait(soft_done(tcnt & 1), ((tcnt >> 1) - 1) & 1, abort_flag);
                    if (!ok)
                        break;
                    const int ahead = asked - tcnt;
                    if (ahead >= 4)
                        cp_async_wait<3>();
                    else if (ahead == 3)
                        cp_async_wait<2>();
                    else if (ahead == 2)
                        cp_async_wait<1>();
                    else
                        cp_async_wait<0>();
                    const float4 k4 = lds4(sbase + lay.raw + (tcnt % kRaws * 2 * BN + 4 * lane) * 4);
                    const float4 v4 = lds4(sbase + lay.raw + (tcnt % kRaws * 2 * BN + BN + 4 * lane) * 4);
                    float ks[4] = {k4.x, k4.y, k4.z, k4.w}, vs[4] = {v4.x, v4.y, v4.z, v4.w}, lv[4], rv[4];
                    bool zero = false;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int k = j * BN + 4 * lane + i;
                        const bool held = k >= lo && k < hi;
                        ks[i] = held ? ks[i] : 0.f;
                        vs[i] = held ? vs[i] : 1.f;
                        if (!(vs[i] >= 0.f && vs[i] < INFINITY))
                            vs[i] = 0.f, spoilt = true;
                        lv[i] = __log2f(vs[i]);
                        rv[i] = __fdividef(kBelow, vs[i]);
                        if (held && vs[i] > 0.f)
                            top_lv = fmaxf(top_lv, lv[i]);
                        zero = zero || vs[i] == 0.f;
                    }
                    if (__any_sync(0xffffffffu, zero)) {
                        // A row of zeros adds to l alone (so does one that is not finite, whose rows of out
                        // are made NaN at the end); any scale serves its codes.  One 2^60 below
                        // the largest seen keeps it from setting m' (P' of the others would fall out
                        // of f16) and its own P' far above float32's least.
                        float ref = top_lv;
                        for (int o = 16; o > 0; o >>= 1)
                            ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
                        ref = fmaxf(floorf(ref) - 60.f, kLeastScale);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (vs[i] == 0.f)
                                lv[i] = ref, rv[i] = kBelow * exp2f(-ref);
                    }
                    float4 *sm = reinterpret_cast<float4 *>(smem + lay.scales + tcnt % kScales * 3 * BN * 4) + lane;
                    sm[0] = make_float4(ks[0], ks[1], ks[2], ks[3]);
                    sm[BN / 4] = make_float4(lv[0], lv[1], lv[2], lv[3]);
                    sm[BN / 2] = make_float4(rv[0], rv[1], rv[2], rv[3]);
                    if (spoilt)
                        segs[n % SEGMENTS].spoilt = 1;
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(scale_full(tcnt % kScales));
                    ++tcnt;
                }
                seg_done(n);
            }
            cp_async_wait<0>();
        }
    } else if (warp < 4 + 4 * QT) {
        // -------------------------------------------------------------------- softmax, a thread per row
        if constexpr (Shape<QT, TYPE>::kSplitRegs)
            reg_inc<Shape<QT, TYPE>::kSoftRegs>();
        const int s = QT == 2 ? (warp - 4) >> 2 : 0;
        const int row = threadIdx.x - 128 - 128 * s;  // of the tile
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp & 3) << 21);
        const int trow = row % kRows;
        const int col0 = row / kRows * kCols;  // this copy's keys
        const int rt = trow / a.group;  // token of the row within its tile
        const int gi = trow - rt * a.group;
        const bool in_tile = trow < a.tpm * a.group;
        const int dim = a.cache.dim;
        RingAt vr{1, 0};
        int cnt = 0;   // tiles this warpgroup has done
        int tcnt = 0;  // tiles of the CTA
        bool ok = true;
        float qscale = 1.f, next_qscale = 1.f;  // 8-bit: row's scale * log2(e) * 2^-shift
        if (s == 0 && row == 0)
            a.records[cta].valid = 0;

        // Q row of a segment's item: into shared memory (swizzled, K-major), or with one row tile
        // into TMEM, where it costs the MMAs no shared-memory reads
        auto active = [&](const Segment &x) { return s * a.tpm < x.item.ntok; };
        auto row_live = [&](const Segment &x) { return in_tile && s * a.tpm + rt < x.item.ntok; };
        auto load_q = [&](const Segment &x) {
            const bool in = row_live(x);
            uint32_t v[DP / 2];
            const uint16_t *src = a.q.data +
                                  static_cast<long long>(x.start + x.item.tok0 + s * a.tpm + rt) * a.q.token_stride +
                                  static_cast<long long>(x.kvh * a.group + gi) * a.q.head_stride;
#pragma unroll
            for (int i = 0; i < DP / 2; ++i)
                v[i] = 0;
            if (in && a.q_wide) {
#pragma unroll
                for (int i = 0; i < DP / 16; ++i)
                    if (16 * i < dim)
                        ldg8(src + 16 * i, v + 8 * i);
            } else if (in) {
#pragma unroll
                for (int i = 0; i < DP / 8; ++i)
                    if (8 * i < dim) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(src + 8 * i);
                        v[4 * i] = w.x, v[4 * i + 1] = w.y, v[4 * i + 2] = w.z, v[4 * i + 3] = w.w;
                    }
            }
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < DP / 2; ++i) {
                v[i] = (v[i] & a.q_and) ^ a.q_xor;
                if constexpr (kQuant)
                    top = __vmaxu2(top, v[i] & 0x7F807F80u);  // exponents
            }
            if constexpr (kQuant) {
                const int e = static_cast<int>(max(top & 0xFFFFu, top >> 16) >> 7);  // biased
                const int shift = e == 0 ? 0 : min(14 - (e - 127), 126);
                const float up = __uint_as_float(static_cast<uint32_t>(shift + 127) << 23);
                next_qscale = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
#pragma unroll
                for (int i = 0; i < DP / 2; ++i)
                    v[i] = f16_pack(bf16_lo(v[i]) * up, bf16_hi(v[i]) * up);
            }
            if constexpr (QT == 1) {
#pragma unroll
                for (int i = 0; i < DP / 2; i += 32)
                    tmem_st_32x32b_x32(lane_base + kQCol + i, reinterpret_cast<const uint32_t(&)[32]>(v[i]));
                tmem_wait_st();
                tc_fence_before();
            } else {
                uint8_t *dst = smem + lay.q + s * kTile + row * 128;
#pragma unroll
                for (int i = 0; i < DP / 8; ++i)
                    *reinterpret_cast<uint4 *>(dst + (i / 8) * HALF_BYTES + (((i & 7) ^ (row & 7)) << 4)) =
                        make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                fence_proxy_async();
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(q_full(s));
        };

        // the four warps of the (one) softmax warpgroup meet; false on a timeout
        uint32_t meet_phase = 0;
        auto group_sync = [&]() {
            __syncwarp();
            if (lane == 0)
                mbar_arrive(meet_bar);
            const bool met = warp_wait(meet_bar, meet_phase, abort_flag);
            meet_phase ^= 1u;
            return met;
        };

        // waits for the products of tile cnt - 1
        auto products_in = [&]() {
            const int t = cnt - 1;
            return QT == 2 ? warp_wait(pv_done(s), t & 1, abort_flag) : warp_wait(pv_done(t & 1), (t >> 1) & 1, abort_flag);
        };

        // Segment n after segment n; before the first there is only its queries to load.
        bool more = true;
        for (int n = -1; more; ++n) {
            const Segment &g = segs[n & (SEGMENTS - 1)];
            const bool started = n >= 0;
            qscale = next_qscale;
            const bool act = started && active(g);
            const bool live = started && row_live(g);
            const bool warp_live = __any_sync(0xffffffffu, live);
            // keys the row sees, relative to the segment's tiles
            int hi = 0x7FFFFFFF, lo = 0;  // rows of no token: whatever comes out goes nowhere
            if (live) {
                const int pos = g.item.p0 + s * a.tpm + rt;
                hi = a.work.causal ? min(g.item.hi, pos + 1) : g.item.hi;
                lo = a.work.window > 0 && pos >= a.work.window ? pos - a.work.window + 1 : 0;
            }
            // With an 8-bit cache a row of zeros, or of values next to the least, adds up to 2^116 to l, which
            // holds a few thousand of them.  What would not fit goes to log_more, a logarithm that no move touches.
            float m = -INFINITY, l = 0.f, log_more = -INFINITY;
            const float sl2 = kQuant ? 1.f : a.scale_log2;
            if (act) {
                for (int j = 0, stop; ok && j < g.tiles;) {
                    stop = kQuant ? min(g.tiles, j + 16) : g.tiles;  // a tile adds at most 2^123 to l
                    for (; j < stop; ++j) {
                        const int t0 = (g.tile + j) * BN;
                        const int sbuf = QT == 2 ? s : cnt & 1;
                        const uint32_t s_phase = QT == 2 ? cnt & 1 : (cnt >> 1) & 1;
                        ok = warp_wait(s_full(sbuf), s_phase, abort_flag);
                        if (!ok)
                            break;
                        if constexpr (kQuant) {
                            ok = warp_wait(scale_full(tcnt % kScales), (tcnt / kScales) & 1, abort_flag);
                            if (!ok)
                                break;
                        }
                        tc_fence_after();
                        const uint32_t s_addr = lane_base + sbuf * BN;
                        const uint32_t scales = sbase + lay.scales + ((tcnt % kScales) * 3 * BN + col0) * 4;
                        if (warp_live) {
                            // An 8-bit cache's scores of 128 keys do not fit the registers beside everything
                            // else: scaled, they go back to TMEM until the maximum is known.
                            constexpr bool kKeep = !kQuant || kCols <= 64;
                            uint32_t v[kKeep ? kCols / 32 : 1][32];
                            const int rlo = lo - t0 - col0, rhi = hi - t0 - col0;
                            const bool edge = __any_sync(0xffffffffu, rlo > 0 || rhi < kCols);
                            // keys c0 .. c0 + 31 that the row sees, a bit each; the others' scores go
                            auto mask = [&](uint32_t(&x)[32], int c0) {
                                const int below = min(max(rlo - c0, 0), 32), up_to = min(max(rhi - c0, 0), 32);
                                const uint32_t seen = static_cast<uint32_t>((1ull << up_to) - 1) &
                                                      ~static_cast<uint32_t>((1ull << below) - 1);
#pragma unroll
                                for (int c = 0; c < 32; ++c)
                                    if (!(seen & (1u << c)))
                                        x[c] = 0xFF800000u;
                            };
                            // x_j of 32 keys from c0 (of this copy's), their S taken out of TMEM into x
                            auto scores = [&](uint32_t(&x)[32], int c0) {
                                tmem_ld_32x32b_x32(s_addr + col0 + c0, x);
                                if constexpr (kQuant) {
                                    float4 ks[8], lv[8];
#pragma unroll
                                    for (int i = 0; i < 8; ++i)
                                        ks[i] = lds4(scales + (c0 + 4 * i) * 4);
#pragma unroll
                                    for (int i = 0; i < 8; ++i)
                                        lv[i] = lds4(scales + (BN + c0 + 4 * i) * 4);
                                    tmem_wait_ld(x);
                                    const uint64_t qs2 = f2(qscale, qscale);
#pragma unroll
                                    for (int i = 0; i < 8; ++i) {
                                        store2(x + 4 * i, fma2(mul2(load2(x + 4 * i), f2(ks[i].x, ks[i].y)), qs2,
                                                               f2(lv[i].x, lv[i].y)));
                                        store2(x + 4 * i + 2, fma2(mul2(load2(x + 4 * i + 2), f2(ks[i].z, ks[i].w)), qs2,
                                                                   f2(lv[i].z, lv[i].w)));
                                    }
                                } else {
                                    tmem_wait_ld(x);
                                }
                                if (edge)
                                    mask(x, c0);
                            };
                            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                            auto raise = [&](const uint32_t(&x)[32]) {
#pragma unroll
                                for (int c = 0; c < 32; c += 8)
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        top[i] = fmaxf(top[i], fmaxf(__uint_as_float(x[c + 2 * i]), __uint_as_float(x[c + 2 * i + 1])));
                            };
                            if constexpr (kQuant) {
#pragma unroll(kKeep ? 4 : 1)
                                for (int i = 0; i < kCols / 32; ++i) {
                                    scores(v[kKeep ? i : 0], 32 * i);
                                    raise(v[kKeep ? i : 0]);
                                    if constexpr (!kKeep)
                                        tmem_st_32x32b_x32(s_addr + col0 + 32 * i, v[0]);
                                }
                            } else {
#pragma unroll
                                for (int i = 0; i < kCols / 32; ++i)
                                    tmem_ld_32x32b_x32(s_addr + col0 + 32 * i, v[i]);
#pragma unroll
                                for (int i = 0; i < kCols / 32; ++i)
                                    tmem_wait_ld(v[i]);
                                if (edge) {
#pragma unroll
                                    for (int i = 0; i < kCols / 32; ++i)
                                        mask(v[i], 32 * i);
                                }
#pragma unroll
                                for (int i = 0; i < kCols / 32; ++i)
                                    raise(v[i]);
                            }
                            if constexpr (!kKeep)
                                tmem_wait_st();
                            const float tile_top = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                            const float rise = tile_top > m ? (tile_top - m) * sl2 : 0.f;  // inf from -inf
                            const bool move = live && rise > LAZY;
                            if (j > 0 && __any_sync(0xffffffffu, move)) {
                                // the products so far must be in before they are scaled
                                ok = products_in();
                                if (!ok)
                                    break;
                                tc_fence_after();
                                const float keep = move ? ex2(-rise) : 1.f;
                                l = kQuant && move ? l * ex2(-0.5f * rise) * ex2(-0.5f * rise) : l * keep;
#pragma unroll 1
                                for (int c = 0; c < DP; c += 16) {
                                    uint32_t o[16];
                                    tmem_ld_32x32b_x16(lane_base + 256 + s * 128 + c, o);
                                    tmem_wait_ld(o);
#pragma unroll
                                    for (int k = 0; k < 16; ++k)
                                        o[k] = __float_as_uint(__uint_as_float(o[k]) * keep);
                                    tmem_st_32x32b_x16(lane_base + 256 + s * 128 + c, o);
                                }
                            }
                            if (move)
                                m = tile_top;
                            const float base = m == -INFINITY ? 0.f : (kQuant ? kAbove : 0.f) - m * sl2;
                            const uint64_t base2 = f2(base, base), sl22 = f2(sl2, sl2);
                            uint64_t sum2[2] = {0, 0};
                            if constexpr (FOLD > 1) {  // the other copies' keys
                                uint32_t z[16];
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    z[k] = 0;
#pragma unroll
                                for (int c = 0; c < BN / 2; c += 16)
                                    if (2 * c < col0 || 2 * c >= col0 + kCols)
                                        tmem_st_32x32b_x16(s_addr + c, z);
                            }
#pragma unroll(kKeep ? 4 : 1)
                            for (int c0 = 0; c0 < kCols; c0 += 32) {
                                uint32_t p[16];
                                float4 rv[8];
                                if constexpr (kQuant) {
#pragma unroll
                                    for (int i = 0; i < 8; ++i)
                                        rv[i] = lds4(scales + (2 * BN + c0 + 4 * i) * 4);
                                }
                                if constexpr (!kKeep) {  // P goes where x has been read already
                                    tmem_ld_32x32b_x32(s_addr + col0 + c0, v[0]);
                                    tmem_wait_ld(v[0]);
                                }
                                const uint32_t(&vc)[32] = v[kKeep ? c0 / 32 : 0];
#pragma unroll
                                for (int c = 0; c < 32; c += 4) {
                                    uint64_t x0 = load2(vc + c), x1 = load2(vc + c + 2);
                                    if constexpr (kQuant) {
                                        x0 = add2(x0, base2), x1 = add2(x1, base2);
                                    } else {
                                        x0 = fma2(x0, sl22, base2), x1 = fma2(x1, sl22, base2);
                                    }
                                    const float2 y0 = f2_split(x0), y1 = f2_split(x1);
                                    const float p0 = ex2(y0.x), p1 = ex2(y0.y), p2 = ex2(y1.x), p3 = ex2(y1.y);
                                    if constexpr (kQuant) {
                                        sum2[0] = fma2(f2(p0, p1), f2(rv[c / 4].x, rv[c / 4].y), sum2[0]);
                                        sum2[1] = fma2(f2(p2, p3), f2(rv[c / 4].z, rv[c / 4].w), sum2[1]);
                                        p[c / 2] = f16_pack(p0, p1), p[c / 2 + 1] = f16_pack(p2, p3);
                                    } else {
                                        sum2[0] = add2(sum2[0], f2(p0, p1));
                                        sum2[1] = add2(sum2[1], f2(p2, p3));
                                        p[c / 2] = bf16_pack(p0, p1), p[c / 2 + 1] = bf16_pack(p2, p3);
                                    }
                                }
                                tmem_st_32x32b_x16(s_addr + (col0 + c0) / 2, p);
                            }
                            const float2 sums = f2_split(add2(sum2[0], sum2[1]));
                            l += sums.x + sums.y;
                            tmem_wait_st();
                        }
                        if constexpr (!kQuant) {
                            // rows of V that no row of the item sees may hold anything: 0 * NaN must not happen
                            if (s == 0 && (t0 < g.item.lo || t0 + BN > g.item.hi)) {
                                ok = warp_wait(ring_full(vr.slot, 0), vr.phase, abort_flag);
                                if (!ok)
                                    break;
                                if (t0 + row < g.item.lo || t0 + row >= g.item.hi) {
                                    uint8_t *vrow = smem + lay.ring + vr.slot * lay.ring_stage + row * 128;
#pragma unroll
                                    for (int h = 0; h < kHalves; ++h)
#pragma unroll
                                        for (int i = 0; i < 8; ++i)
                                            *reinterpret_cast<uint4 *>(vrow + h * HALF_BYTES + 16 * i) =
                                                make_uint4(0, 0, 0, 0);
                                }
                                fence_proxy_async();
                            }
                            vr.step(a.ring);
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(p_full(sbuf));
                            if (kQuant && s == 0)
                                mbar_arrive(soft_done(tcnt & 1));
                        }
                        ++cnt;
                        ++tcnt;
                    }
                    if (kQuant && l > 0x1p80f) {
                        log_more = log_sum(log_more, m + __log2f(l));
                        l = 0.f;
                    }
                }
            } else if (started) {
                tcnt += g.tiles;
            }
            if (!ok)
                break;
            // the next item's queries go in while the last product of this one runs
            const Segment &next = segs[(n + 1) & (SEGMENTS - 1)];
            ok = seg_wait(n + 1, QT == 2 && !act ? kIdleCycles : kWaitCycles);
            if (!ok)
                break;
            more = next.tiles != 0;
            if (more && active(next))
                load_q(next);
            if (!act) {
                if (started)
                    seg_done(n);
                continue;
            }
            const int tok = g.start + g.item.tok0 + s * a.tpm + rt;
            const int head = g.kvh * a.group + gi;
            const bool whole = g.first && g.last;
            const long long part = static_cast<long long>(g.slot) * (QT * BM) + s * BM + trow;
            uint16_t *dst = a.out.data + static_cast<long long>(tok) * a.out.token_stride +
                            static_cast<long long>(head) * a.out.head_stride;
            ok = products_in();
            if (!ok)
                break;
            tc_fence_after();
            float weight = 1.f;
            float log_l = log2f(l);
            if constexpr (kQuant) {
                if (log_more > -INFINITY)
                    log_l = log_sum(log_l, log_more - m);
                m -= kAbove, log_l += kAbove;  // o is in units of 2^(m - 7)
            }
            if constexpr (FOLD > 1) {
                // the copies' common maximum; each copy's weight; the sum of their sums
                float2 *ml = reinterpret_cast<float2 *>(smem + lay.fold + BM * 16 * 4);
                ml[row] = make_float2(m, log_l);
                ok = group_sync();
                if (!ok)
                    break;
                float top = -INFINITY, far = -INFINITY;
#pragma unroll
                for (int f = 0; f < FOLD; ++f) {
                    const float2 x = ml[f * kRows + trow];
                    top = fmaxf(top, x.x);
                    far = fmaxf(far, x.x + x.y);
                }
                const float b = top == -INFINITY ? 0.f : top;
                weight = exp2f(m - b);
                far = far == -INFINITY ? 0.f : far - b;
                float sum = 0.f;
#pragma unroll
                for (int f = 0; f < FOLD; ++f) {
                    const float2 x = ml[f * kRows + trow];
                    sum += exp2f(x.x - b + x.y - far);  // in one power, as in the combine kernel
                }
                log_l = far + log2f(sum);
                m = top;
            } else {
                m *= sl2;
            }
            float inv = 1.f;
            if (whole) {
                if constexpr (kQuant)
                    inv = log_l == -INFINITY ? 0.f : exp2f(-log_l);
                else
                    inv = l > 0.f ? __fdividef(1.f, l) : l == 0.f ? 0.f : l;
            }
            // a value row that is not finite is in out and not in the sum
            const bool spoilt = kQuant && g.spoilt != 0 && log_l > -INFINITY;
            if (spoilt)
                inv = NAN;
            if (warp_live || FOLD > 1) {
                constexpr int kChunk = FOLD > 1 ? 16 : 32;     // columns at a time
                constexpr int kPer = kChunk / FOLD;            // ... of which this thread writes
                const int k0 = FOLD > 1 ? row / kRows * kPer : 0;
#pragma unroll 1
                for (int c = 0; c < DP; c += kChunk) {
                    uint32_t o[kChunk];
                    const uint32_t src = lane_base + 256 + s * 128 + c;
                    if constexpr (FOLD > 1) {
                        // through shared memory: rows of 16 words, word k of row r at k ^ (r / 2 mod 16)
                        tmem_ld_32x32b_x16(src, o);
                        tmem_wait_ld(o);
                        float *x = reinterpret_cast<float *>(smem + lay.fold);
                        const int flip = (lane >> 1) & 15;
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            x[row * 16 + (k ^ flip)] = weight == 0.f ? 0.f : __uint_as_float(o[k]) * weight;
                        ok = ok && group_sync();
#pragma unroll
                        for (int k = 0; k < kPer; ++k) {
                            float sum = 0.f;
#pragma unroll
                            for (int f = 0; f < FOLD; ++f)
                                sum += x[(f * kRows + trow) * 16 + ((k0 + k) ^ flip)];
                            o[k] = __float_as_uint(sum);
                        }
                        ok = ok && group_sync();
                    } else {
                        tmem_ld_32x32b_x32(src, o);
                        tmem_wait_ld(o);
                    }
                    if (live && whole) {
                        uint32_t w[kPer / 2];
#pragma unroll
                        for (int k = 0; k < kPer / 2; ++k)
                            w[k] = bf16_pack(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
                        uint16_t *to = dst + c + k0;
                        if constexpr (kPer >= 16) {
                            if (a.out_wide) {
#pragma unroll
                                for (int k = 0; k < kPer / 2; k += 8)
                                    if (c + 2 * k < dim)
                                        stg8(to + 2 * k, w + k);
                            } else {
#pragma unroll
                                for (int k = 0; k < kPer / 2; k += 4)
                                    if (c + 2 * k < dim)
                                        *reinterpret_cast<uint4 *>(to + 2 * k) = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
                            }
                        } else if (c + k0 < dim) {
#pragma unroll
                            for (int k = 0; k < kPer / 2; k += 2)
                                *reinterpret_cast<uint2 *>(to + 2 * k) = make_uint2(w[k], w[k + 1]);
                        }
                    } else if (live) {
                        if (spoilt) {
#pragma unroll
                            for (int k = 0; k < kPer; ++k)
                                o[k] = 0x7FC00000u;
                        }
                        float *to = a.part_o + part * dim + c + k0;
                        if constexpr (kPer >= 8) {
#pragma unroll
                            for (int k = 0; k < kPer; k += 8)
                                if (c + k0 + k < dim)
                                    stg8(to + k, o + k);
                        } else if (c + k0 < dim) {
                            *reinterpret_cast<uint4 *>(to) = make_uint4(o[0], o[1], o[2], o[3]);
                        }
                    }
                }
            }
            if (live && col0 == 0) {
                if (!whole)
                    a.part_ml[part] = make_float2(m, log_l);
                else if (a.lse)
                    a.lse[static_cast<long long>(tok) * a.q.heads + head] = (m + log_l) * 0.69314718055994530942f;
            }
            if (s == 0 && row == 0 && g.first && !g.last) {
                SplitRecord rec;
                rec.valid = 1;
                rec.pad = 0;
                rec.first_slot = g.slot;
                rec.c0 = cta;
                rec.c1 = g.end_cta;
                rec.kvh = g.kvh;
                rec.tok0 = g.start + g.item.tok0;
                rec.ntok = g.item.ntok;
                a.records[cta] = rec;
            }
            tc_fence_before();
            seg_done(n);
        }
    } else {
        // -------------------------------------------------------------------- 8-bit codes to f16
        if constexpr (kQuant) {
            reg_dec<Shape<QT, TYPE>::kWideRegs>();
            const int kv = warp >= 8 + 4 * QT ? 1 : 0;
            const int t = threadIdx.x & 127;
            const int dim = a.cache.dim;
            constexpr int kChunks = DP / 16;
            RingSlot rs{kv, 0}, ws{kv, 0};  // in the TMA ring, in the widened one
            bool ok = true;
            for (int n = 0; ok; ++n) {
                ok = seg_wait(n);
                if (!ok || segs[n % SEGMENTS].tiles == 0)
                    break;
                const Segment &g = segs[n % SEGMENTS];
                const int tiles = g.tiles, first = g.tile * BN, item_lo = g.item.lo, item_hi = g.item.hi;
                for (int j = 0; j < tiles && ok; ++j) {
                    const int t0 = first + j * BN;
                    const int turn = ws.turn(kWide, kv);
                    if (turn >= 0)
                        ok = warp_wait(wide_empty(ws.slot, kv), turn & 1, abort_flag);
                    if (!ok)
                        break;
                    const uint32_t r_phase = rs.round >> (a.ring & 1) & 1;
                    ok = warp_wait(ring_full(rs.slot, kv), r_phase, abort_flag);
                    if (!ok)
                        break;
                    const uint8_t *src = smem + lay.ring + rs.slot * lay.ring_stage;
                    uint8_t *dst = smem + lay.wide + ws.slot * kTile;
                    // sixteen codes at a time; a code of zero is the number zero in both types
                    const int c = t % kChunks, odd = c >> 2, c0 = 2 * (c & 3);
                    const bool edge = t0 < item_lo || t0 + BN > item_hi || c * 16 >= dim;
#pragma unroll 1
                    for (int r0 = t / kChunks; r0 < BN; r0 += 4 * (128 / kChunks)) {
                        uint4 v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = r0 + i * (128 / kChunks);
                            v[i] = *reinterpret_cast<const uint4 *>(src + r * dim + c * 16);
                        }
                        if (edge) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int r = r0 + i * (128 / kChunks);
                                if (t0 + r < item_lo || t0 + r >= item_hi || c * 16 >= dim)
                                    v[i] = make_uint4(0, 0, 0, 0);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = r0 + i * (128 / kChunks);
                            // lanes of the two halves write opposite chunks of a pair, so eight lanes
                            // cover all banks
                            const uint2 w0 = widen4<TYPE>(odd ? v[i].z : v[i].x), w1 = widen4<TYPE>(odd ? v[i].w : v[i].y),
                                        w2 = widen4<TYPE>(odd ? v[i].x : v[i].z), w3 = widen4<TYPE>(odd ? v[i].y : v[i].w);
                            uint8_t *d = dst + odd * HALF_BYTES + r * 128;
                            *reinterpret_cast<uint4 *>(d + (((c0 + odd) ^ (r & 7)) << 4)) =
                                make_uint4(w0.x, w0.y, w1.x, w1.y);
                            *reinterpret_cast<uint4 *>(d + (((c0 + 1 - odd) ^ (r & 7)) << 4)) =
                                make_uint4(w2.x, w2.y, w3.x, w3.y);
                        }
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(ring_empty(rs.slot, a.ring & 1 ? 1 - kv : kv));
                        mbar_arrive(wide_full(ws.slot));
                    }
                    rs.step(a.ring);
                    ws.step(kWide);
                }
                seg_done(n);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && *abort_flag)
        atomicOr(a.status, kStatusTimeoutAttention);
}

// Joins the pieces of the items that several CTAs worked on, in CTA order: a warp a row, a lane
// four dimensions.  It is a chain of loads (the record, then the pieces' maxima and sums), so the
// first pieces of o are asked for before their weights are known.
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ Args a, int rows)
{
    constexpr int kEarly = 8;
    griddep_launch_dependents();
    griddep_wait();
    const SplitRecord rec = a.records[blockIdx.x];
    const int row = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int tile = row / BM, r = row % BM, rt = r / a.group, gi = r - rt * a.group;
    const int t = tile * a.tpm + rt, dim = a.cache.dim;
    if (!rec.valid || rt >= a.tpm || t >= rec.ntok)
        return;
    const int n = rec.c1 - rec.c0 + 1;
    auto at = [&](int i) { return static_cast<long long>(i == 0 ? rec.first_slot : 2 * (rec.c0 + i)) * rows + row; };
    auto piece = [&](int i) {
        return i < n && 4 * lane < dim ? *reinterpret_cast<const float4 *>(a.part_o + at(i) * dim + 4 * lane)
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    float4 early[kEarly];
#pragma unroll
    for (int i = 0; i < kEarly; ++i)
        early[i] = piece(i);
    float2 ml = lane < n ? a.part_ml[at(lane)] : make_float2(-INFINITY, -INFINITY);
    float top = ml.x, far = ml.x + ml.y;
    for (int i = lane + 32; i < n; i += 32) {
        const float2 x = a.part_ml[at(i)];
        top = fmaxf(top, x.x);
        far = fmaxf(far, x.x + x.y);
    }
    for (int o = 16; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float base = top == -INFINITY ? 0.f : top;
    // with an 8-bit cache the maximum carries a value's scale and a sum may be far from it
    if (a.cache.type != 0) {
        for (int o = 16; o > 0; o >>= 1)
            far = fmaxf(far, __shfl_xor_sync(0xffffffffu, far, o));
        far = far == -INFINITY ? 0.f : far - base;
    } else {
        far = 0.f;
    }
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float w, const float4 &o) {
        acc.x = fmaf(w, o.x, acc.x), acc.y = fmaf(w, o.y, acc.y);
        acc.z = fmaf(w, o.z, acc.z), acc.w = fmaf(w, o.w, acc.w);
    };
    for (int i0 = 0; i0 < n; i0 += 32) {
        if (i0 > 0)
            ml = i0 + lane < n ? a.part_ml[at(i0 + lane)] : make_float2(-INFINITY, -INFINITY);
        const float wgt = exp2f(ml.x - base);
        l += exp2f(ml.x - base + ml.y - far);  // in one power: the weight alone may fall below what float32 holds
        int i = 0;
        if (i0 == 0) {
#pragma unroll
            for (; i < kEarly; ++i)
                add(__shfl_sync(0xffffffffu, wgt, i), early[i]);
        }
        const int m = min(32, n - i0);
#pragma unroll 4
        for (; i < m; ++i)
            add(__shfl_sync(0xffffffffu, wgt, i), piece(i0 + i));
    }
    for (int o = 16; o > 0; o >>= 1)
        l += __shfl_xor_sync(0xffffffffu, l, o);
    const float inv = l > 0.f ? exp2f(-far) / l : l == 0.f ? 0.f : l;
    const long long token = rec.tok0 + t;
    const int head = rec.kvh * a.group + gi;
    if (4 * lane < dim)
        *reinterpret_cast<uint2 *>(a.out.data + token * a.out.token_stride + head * a.out.head_stride + 4 * lane) =
            make_uint2(bf16_pack(acc.x * inv, acc.y * inv), bf16_pack(acc.z * inv, acc.w * inv));
    if (a.lse && lane == 0)
        a.lse[token * a.q.heads + head] = (top + (far + log2f(l))) * 0.69314718055994530942f;
}

// Row tiles an item has: two when some sequence may have more rows than one holds.
int row_tiles(const TokenBatch &t, int group) { return t.max_new > BM / group ? 2 : 1; }

// Copies of the rows in a tile: with an 8-bit cache as many as fit.  A bf16 tile takes twice as long
// to arrive, which hides the softmax of one copy, and adding copies up costs at the item's end.
int row_copies(const PagedCache &c, const TokenBatch &t, int group)
{
    if (c.type == 0)
        return 1;
    const long long rows = static_cast<long long>(t.max_new) * group;
    return rows <= BM / 4 ? 4 : rows <= BM / 2 ? 2 : 1;
}

struct Scratch {
    size_t records, ml, o, bytes;
};

Scratch scratch_of(int sms, int tiles, int dim)
{
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    Scratch s{};
    const size_t rows = static_cast<size_t>(2) * sms * tiles * BM;
    s.records = 0;
    s.ml = up(static_cast<size_t>(sms) * sizeof(SplitRecord));
    s.o = s.ml + up(rows * sizeof(float2));
    s.bytes = s.o + up(rows * dim * sizeof(float));
    return s;
}

// A cache tensor [pages, heads, page_size, dim]: boxes of `box` rows of one page, 64 bf16 elements
// wide with the 128-byte swizzle, or whole rows of 8-bit codes as they lie.
cudaError_t encode_cache(CUtensorMap *map, const PagedCache &c, const void *base, int box)
{
    auto encode = tensor_map_encoder();
    if (!encode)
        return cudaErrorNotSupported;
    const bool wide = c.type == 0;
    const cuuint64_t es = wide ? 2 : 1;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.dim), static_cast<cuuint64_t>(c.page_size),
                                static_cast<cuuint64_t>(c.heads), static_cast<cuuint64_t>(c.pages)};
    const cuuint64_t strides[3] = {dims[0] * es, dims[0] * dims[1] * es, dims[0] * dims[1] * dims[2] * es};
    const cuuint32_t boxes[4] = {static_cast<cuuint32_t>(wide ? 64 : c.dim), static_cast<cuuint32_t>(box), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUresult r = encode(map, wide ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4,
                              const_cast<void *>(base), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              wide ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int DP, int QT, int TYPE, int FOLD>
cudaError_t launch(Args a, int sms, cudaStream_t stream)
{
    a.ring = MAX_RING;
    while (a.ring > 3 && layout_of<DP, QT, TYPE, FOLD>(a.ring, a.cache.dim, a.tokens.B).bytes + 1024 > SMEM_LIMIT)
        --a.ring;
    const int smem = layout_of<DP, QT, TYPE, FOLD>(a.ring, a.cache.dim, a.tokens.B).bytes + 1024;
    if (smem > SMEM_LIMIT)
        return cudaErrorInvalidConfiguration;
    CUtensorMap mk, mv;
    cudaError_t e;
    if ((e = encode_cache(&mk, a.cache, a.cache.k, a.box)) != cudaSuccess ||
        (e = encode_cache(&mv, a.cache, a.cache.v, a.box)) != cudaSuccess)
        return e;
    auto kern = attention_kernel<DP, QT, TYPE, FOLD>;
    if ((e = ensure_dynamic_smem(reinterpret_cast<const void *>(kern), smem)) != cudaSuccess)
        return e;
    return launch_dependent(kern, dim3(static_cast<unsigned>(sms)), dim3(Shape<QT, TYPE>::kThreads),
                            static_cast<size_t>(smem), stream, mk, mv, a);
}

template <int DP, int QT, int FOLD>
cudaError_t launch_type(const Args &a, int sms, cudaStream_t stream)
{
    switch (a.cache.type) {
    case 0: return launch<DP, QT, 0, FOLD>(a, sms, stream);
    case 1: return launch<DP, QT, 1, FOLD>(a, sms, stream);
    default: return launch<DP, QT, 2, FOLD>(a, sms, stream);
    }
}

template <int DP>
cudaError_t launch_rows(const Args &a, int tiles, int fold, int sms, cudaStream_t stream)
{
    if (tiles == 2)
        return launch_type<DP, 2, 1>(a, sms, stream);
    if (fold == 4)
        return a.cache.type == 1 ? launch<DP, 1, 1, 4>(a, sms, stream) : launch<DP, 1, 2, 4>(a, sms, stream);
    if (fold == 2)
        return a.cache.type == 1 ? launch<DP, 1, 1, 2>(a, sms, stream) : launch<DP, 1, 2, 2>(a, sms, stream);
    return launch_type<DP, 1, 1>(a, sms, stream);
}

}  // namespace

size_t paged_attention_scratch(const PagedCache &cache, const TokenBatch &tokens, int q_heads)
{
    return scratch_of(device_sm_count(), row_tiles(tokens, q_heads / cache.heads), cache.dim).bytes;
}

cudaError_t launch_paged_attention(const PagedCache &cache, const TokenBatch &tokens, const AttentionOptions &opt,
                                   const HeadRows &q, const HeadRows &out, float *lse, uint32_t *status,
                                   void *scratch, cudaStream_t stream)
{
    const int sms = device_sm_count();
    Args a{};
    a.cache = cache;
    a.tokens = tokens;
    a.q = q;
    a.out = out;
    a.lse = lse;
    const float scale = opt.scale == 0.f ? 1.f : std::fabs(opt.scale);
    a.scale_log2 = scale * 1.44269504088896340736f;
    a.q_and = opt.scale == 0.f ? 0u : 0xFFFFFFFFu;
    a.q_xor = opt.scale < 0.f ? 0x80008000u : 0u;
    a.work.causal = opt.causal;
    auto wide = [](const HeadRows &r) {
        return reinterpret_cast<uintptr_t>(r.data) % 32 == 0 && r.token_stride % 16 == 0 && r.head_stride % 16 == 0;
    };
    a.q_wide = wide(q);
    a.out_wide = wide(out);
    a.work.window = opt.window >= tokens.max_pages * cache.page_size ? 0 : opt.window;
    a.group = q.heads / cache.heads;
    const int tiles = row_tiles(tokens, a.group);
    const int fold = row_copies(cache, tokens, a.group);
    a.tpm = BM / fold / a.group;
    // no item has more rows than the combine kernel looks at, even where a sequence has more than max_new
    a.work.span = tiles == 2 ? 2 * a.tpm : std::min(a.tpm, tokens.max_new);
    a.work.heads = cache.heads;
    // Measured on GB300: 2048 tokens over their own 2048 keys (two row tiles) 100.7, 84.4, 76.5, 73.2,
    // 70.5 and 71.4 us at 0, 1, 2, 3, 4 and 6; 7 blocks of 16 over 1000 keys (one) 20.3, 17.4 and
    // 19.4 us at 0, 1 and 3.
    a.work.item_cost = tiles == 2 ? 4 : 1;
    a.box = std::gcd(cache.page_size, BN);
    // ceil(2^(31 + b) / page_size) with b = ceil(log2(page_size)) gives the exact quotient below 2^31
    int bits = 3;
    while ((1 << bits) < cache.page_size)
        ++bits;
    a.page_magic = static_cast<uint32_t>(((1ull << (31 + bits)) + cache.page_size - 1) / cache.page_size);
    a.page_shift = static_cast<uint32_t>(bits - 1);
    a.status = status;
    const Scratch s = scratch_of(sms, tiles, cache.dim);
    uint8_t *p = static_cast<uint8_t *>(scratch);
    a.records = reinterpret_cast<SplitRecord *>(p + s.records);
    a.part_ml = reinterpret_cast<float2 *>(p + s.ml);
    a.part_o = reinterpret_cast<float *>(p + s.o);
    cudaError_t e;
    e = cache.dim <= 64 ? launch_rows<64>(a, tiles, fold, sms, stream) : launch_rows<128>(a, tiles, fold, sms, stream);
    if (e != cudaSuccess)
        return e;
    // the rows that an item can have, eight to a CTA
    const int most = tiles == 2 ? 2 * BM : a.work.span * a.group;
    const unsigned y = static_cast<unsigned>((most + 7) / 8);
    return launch_dependent(combine_kernel, dim3(static_cast<unsigned>(sms), y), dim3(256), 0, stream, a, tiles * BM);
}

}  // namespace df2
