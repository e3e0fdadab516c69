// qs_fp8mm.cu -- e4m3 x e4m3 product with fp32 scales per 128 of the inner dimension, for one
// matrix and for rows sorted by expert (sm_103a).
//
//   out[m, n] = sum_b sa[m, b] * sw[e, n/128, b] * (sum over k in block b of a[m, k] * w[e, n, k])
//
// The inner sums run on the tensor cores (tcgen05.mma kind::f8f6f4, fp32 accumulators in tensor
// memory), one block of 128 at a time; since every block has its own scales, an accumulator holds one
// block only and the sum over blocks is kept in registers.  Four roles work at their own pace:
//   warp 0     TMA: a stage is a block (narrow tiles: two or four) of the tile's rows of a and of its weight rows
//   warps 1-2  MMA, taking turns: four instructions a block and accumulator, overwriting
//   warp 3     brings the scales of eight blocks at a time to shared memory
//   warps 4-11 read an accumulator (a thread a row, half of its columns), add it, scaled, to their registers,
//              and after the last block send the tile out through shared memory
// A thread owns a row of the tile, so a block's scale is one number a thread (two where its columns are of two
// weight blocks) and a step costs one multiply-add an element.
// Tiles are 128 rows by BN weight rows, or, where there is work for all SMs in them, 256 x 256 of two CTAs, or, for few
// rows, 64 or 128 weight rows by 16 or 32 rows with the operands' parts changed about.  A CTA takes tiles blockIdx.x,
// + gridDim.x, ... and its stages run on from one tile to the next.
// Bound: weights from HBM where there are few rows a weight (2048 tokens to 8 of 256 experts, 2048 x 1024 each:
// 93 us, 96 % of the copy rate), latency where a matrix is small (one row by 4096 x 2048: 4.0 us with the weights in L2, 4.9 with them in HBM, for
// 1.25 us of weights), and for long prompts the tensor cores and the sums between them: 8192 x 8192 x 4096 takes 180 us
// in a burst of 20 ms, 3.05 PFLOP/s (without the reads of accumulators 165, without the copies 169, without both 145), and
// 204 to 214 us for longer, at the card's power cap.  With 64 rows at most the
// stage's row part is only as high as the rows there are (the matrix instruction reads on into whatever follows:
// rows of the result that no thread stores), so that nearly all of shared memory holds weights in flight.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "qs_fp8tiles.h"
#include "qs_internal.h"
#include "qs_rows.cuh"
#include "qs_tc.cuh"

namespace qs {

namespace {

constexpr int kMaxStages = 32;
constexpr int kFirstSum = 4;  // first of the warps that sum
constexpr int kRowBox = 16;  // rows of the small TMA box of a are a multiple of this

struct MmParams {
    // a as [block of K][row][128 columns] and w as [expert][block][row][128 columns], boxes of a group's blocks;
    // where K is no multiple of 128, one block deep over whole rows, boxes of one block (columns past K read as 0)
    CUtensorMap tfew;   // a, boxes of box_rows rows
    CUtensorMap ta128;  // a, boxes of 128 rows
    CUtensorMap tw;     // w, boxes of BN rows
    CUtensorMap tout;   // out, boxes of 32 rows x 64 bytes
    const float* sa;
    const float* sw;
    const int32_t* offsets;
    void* out;
    uint32_t* status;
    int64_t sa_stride, out_stride;
    int M, N, E, KB, NB;  // KB: blocks of K, NB: 128-row blocks of N
    int out_dtype, out_vec, out_tma;
    int a_bytes, stages;  // bytes of a block's row part
    int box_rows, blocked;
    int out_at;           // where the summing warps' staging rows begin in shared memory, a multiple of 1024
};

// Scales on their way to the summing warps: kScaleRing groups of kScaleGroup blocks.  Rows are 132 apart
// so that the eight blocks of a row, read together, are stored to different banks.
constexpr int kScaleGroup = 8, kScaleRing = 2;
struct alignas(16) MmScales {
    float a[kScaleGroup][kTileRows + 4];
    float w[2][kScaleGroup];  // of the tile's first and second 128 columns
};

struct MmCtl {
    MmScales scales[kScaleRing];
    uint64_t scfull[kScaleRing], scempty[kScaleRing];
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t accfull[4], accempty[4];
    uint64_t drain;
    uint32_t tmem;
    int abort;
};

__device__ __noinline__ void mm_timeout(uint32_t* status, uint32_t code) {
    if (atomicCAS(status, 0u, (uint32_t)QS_ERR_TIMEOUT) == 0u) {
        status[1] = code;
        status[2] = blockIdx.x;
        __threadfence();
    }
}

// Whether a phase is complete, without waiting.
__device__ __forceinline__ bool mbar_done(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Bounded wait of the calling thread; false once the CTA gives up.
__device__ __forceinline__ bool mm_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* status,
                                        uint32_t code) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        if (mbar_try_wait_sleep(bar, parity, 20000)) return true;
        if (*abort) return false;
        if (global_timer_ns() - t0 > kWaitNs) {
            *abort = 1;
            mm_timeout(status, code);
            return false;
        }
    }
}

// Boxes of a (columns, row, block) and of w (columns, row, block, expert).
__device__ __forceinline__ void tma_a(void* dst, const CUtensorMap* m, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_u32(dst)),
        "l"(m), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_w(void* dst, const CUtensorMap* m, int x, int y, int z, int e, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            smem_u32(dst)),
        "l"(m), "r"(x), "r"(y), "r"(z), "r"(e), "r"(smem_u32(bar))
        : "memory");
}

// One lane of a converged warp, the same one each time.  Code under it is known to run in a single
// thread, so descriptors stay in uniform registers: issuing a block takes a fraction of what it takes
// under `lane == 0`.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// ---- two CTAs that share a tile (a cluster of 2; the even one leads)

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// shared::cluster address of the leader's copy of a shared variable
__device__ __forceinline__ uint32_t leader_addr(const void* p) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
    return a;
}
// TMA into this CTA's shared memory, counted on the leader's barrier
__device__ __forceinline__ void tma_a_pair(void* dst, const CUtensorMap* m, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_u32(dst)),
        "l"(m), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_w_pair(void* dst, const CUtensorMap* m, int x, int y, int z, int e, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            smem_u32(dst)),
        "l"(m), "r"(x), "r"(y), "r"(z), "r"(e), "r"(bar)
        : "memory");
}
// D[tmem of both] = A[smem of both] * B[smem of both]^T: 256 rows, 128 and half of B's rows in each CTA
__device__ __forceinline__ void mma_f8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t id, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(id), "r"(accumulate)
        : "memory");
}
// arrive on the barrier of both CTAs when the MMAs issued so far are done
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
// Arrive on a barrier of this CTA, or (PAIR) of either.  What it orders is tensor memory, by the tcgen05
// fences: no release at cluster scope, which costs a step of the sum more than the step.
template <bool PAIR>
__device__ __forceinline__ void arrive_at(uint32_t bar) {
    if (PAIR) asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
    else asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// D[tmem] = A[smem] * B[smem]^T (accumulate: added), e4m3, 32 of K
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t id, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(id), "r"(accumulate)
        : "memory");
}

template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[N]);
template <>
__device__ __forceinline__ void tmem_load<32>(uint32_t addr, uint32_t (&r)[32]) { tc::ld32(addr, r); }
template <>
__device__ __forceinline__ void tmem_load<16>(uint32_t addr, uint32_t (&r)[16]) { tc::ld16(addr, r); }
template <>
__device__ __forceinline__ void tmem_load<8>(uint32_t addr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr)
                 : "memory");
}

struct Tile {
    int e, row0, rows, n0;  // expert, first row of a, rows that are the tile's, first weight row
};

// The call's groups of rows, in shared memory (every role looks up every tile): for each expert its first row
// (entries of `offsets` clipped to the rows there are; one group without them) and the row tiles of the experts
// before it among its 32, and for each 32 experts their row tiles.
struct Groups {
    int first[1025], before[1056], total[33];
};

// Row tiles of 32 experts that count, at most.  Groups that do not overlap have fewer in all.  Offsets that are not
// ascending may name a row 512 times; sums of these stay inside 32 bits all the same (one that wrapped numbered tiles outside
// the rows), and a tile's number leads to rows of the tile's expert.
constexpr int kSpanTiles = 1 << 25;
static_assert(kMmMaxRows / kTileRows + kMmMaxExperts <= kSpanTiles, "all tiles of ascending groups count");
static_assert(kFewAverage * kMmMaxExperts <= kSpanTiles, "and those of few rows");
static_assert((int64_t)kMmMaxExperts / 32 * kSpanTiles + 32ll * (kMmMaxRows / kTileRows) <= INT32_MAX, "an expert's first tile");

// A warp's view: lane c has the row tiles before the experts 32 c ..; `all` of them.
struct Lookup {
    int base, all;
};
__device__ __forceinline__ Lookup lookup_of(const Groups& g, int E) {
    const int lane = threadIdx.x & 31, c = lane < (E + 31) / 32 ? g.total[lane] : 0;
    int s = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += v;
    }
    return {s - c, __shfl_sync(0xffffffffu, s, 31)};
}

// Tiles of the call, by number: experts ascending, inside one the weight tiles, inside one the row
// tiles, so that CTAs side by side share a weight tile.  A warp looks for the expert together: the last of the
// 32 spans, and of its 32 experts, that begins at or before the tile (it has tiles: the next begins later).
template <int ROWS>
__device__ __forceinline__ Tile tile_at(const MmParams& p, const Groups& g, const Lookup& look, int nt, int BN, int64_t tile) {
    Tile t;
    const int lane = threadIdx.x & 31, spans = (p.E + 31) / 32;
    const int span = 31 - __clz(__ballot_sync(0xffffffffu, lane < spans && (int64_t)look.base * nt <= tile));
    const int from = __shfl_sync(0xffffffffu, look.base, span), e = span * 32 + lane;
    const int mine = from + (e < p.E ? g.before[e] : 0);
    const int at = 31 - __clz(__ballot_sync(0xffffffffu, e < p.E && (int64_t)mine * nt <= tile));
    t.e = span * 32 + at;
    const int first = g.first[t.e], last = g.first[t.e + 1], mt = (last - first + ROWS - 1) / ROWS;
    const int local = (int)(tile - (int64_t)__shfl_sync(0xffffffffu, mine, at) * nt);
    const int n = mt == 1 ? local : local / mt, m = local - n * mt;
    t.row0 = first + m * ROWS;
    t.rows = min(ROWS, last - t.row0);
    t.n0 = n * BN;
    return t;
}

constexpr int kStage = 2048;  // bytes of a summing warp's staging rows: 32 of 64 bytes

// FEW (0, 16 or 32): the accumulator's rows are BN weight rows and its columns FEW rows of a.  A block's instructions cost
// about the same whoever the 128 rows are: by 4096 x 16384 a group of four blocks took 0.52 us with 32 weight rows across
// and one row of a among the 128 down, 0.42 us with 64 weight rows down.
template <int BN, int FEW = 0>
struct MmShape {
    static_assert(FEW == 0 || BN == 64 || BN == 128, "an accumulator's rows");
    // The widest tile is two accumulators of 128 columns, filled and read one after the other: with one of
    // 256 the time from a read back to the next fill stood open, 700 cycles a block.
    static constexpr int kHalves = BN == 256 ? 2 : 1;
    static constexpr int kAccCols = FEW ? FEW : BN / kHalves;
    static constexpr int kAcc = 4;                                       // accumulators in tensor memory
    // Blocks of K that pass through the roles as one: a stage, an accumulator (side by side, each block with its
    // own columns) and one round of barriers.  Waits, issue and release take 300 to 400 cycles whatever the
    // width, which is all a narrow tile's time: one row by 4096 x 2048 took 6.0 us with one block at a time, 4.8 so (then in tiles of 32).
    static constexpr int kGroup = FEW ? (BN == 64 ? 4 : 2) : BN >= 128 ? 1 : BN == 64 ? 2 : 4;
    static constexpr int kAccStep = kAccCols * kGroup;                   // columns of an accumulator
    static constexpr int kTmemCols = kAccStep * kAcc;                    // 256 or 512
    static constexpr int kSumWarps = 8;
    static constexpr int kThreads = 32 * (kFirstSum + kSumWarps);
    static constexpr int kCols = (FEW ? FEW : BN) * 4 / kSumWarps;  // columns of a summing thread, in runs of 64 at most:
    static constexpr int kRun = kCols < 64 ? kCols : 64;        // what lies together in a pair's accumulator and in w
    static constexpr int kRuns = kCols / kRun;
    static constexpr int kLoad = BN == 256 ? 16 : kRun < 32 ? kRun : 32;  // columns of one tensor-memory load
    static constexpr int kSumBytes = FEW ? 0 : kSumWarps * kStage;  // staging rows of the summing warps
};

// Registers a thread of the widest tile: the launch's 168 x 384 are dealt out as 56 for warps 0-3 and
// 224 for the others, (56 + 2 x 224) x 128 <= 168 x 384.
constexpr int kLaunchRegs = 168, kFewRegs = 56, kSumRegs = 224;
static_assert((kFewRegs + 2 * kSumRegs) * 128 <= kLaunchRegs * MmShape<256>::kThreads, "more registers than launched");

// a + b * s in both halves
__device__ __forceinline__ float2 fma2(uint32_t b0, uint32_t b1, float s, float2 a) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tmov.b64 z, {%5, %6};\n\t"
        "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "r"(b0), "r"(b1), "f"(s), "f"(a.x), "f"(a.y));
    return d;
}

// acc += scale * the thread's columns of an accumulator, which is free once its last columns are in
// registers.  With two buffers the next columns are read while these are added.
template <int BN, bool PAIR>
__device__ __forceinline__ void add_block(float2 (&acc)[MmShape<BN>::kRuns][MmShape<BN>::kRun / 2], uint32_t src,
                                          const float (&scale)[MmShape<BN>::kRuns], uint32_t empty, int lane) {
    using S = MmShape<BN>;
    constexpr int kSteps = S::kCols / S::kLoad;
    uint32_t d[2][S::kLoad];
    tc::fence_after();
    tmem_load<S::kLoad>(src, d[0]);
#pragma unroll
    for (int j = 0; j < kSteps; j++) {
        tc::wait_ld();
        if (j + 1 == kSteps) {
            tc::fence_before();
            __syncwarp();
            if (lane == 0) arrive_at<PAIR>(empty);
        } else {
            tmem_load<S::kLoad>(src + (j + 1) * S::kLoad, d[(j + 1) % 2]);
        }
        constexpr int kPer = S::kRun / S::kLoad;  // loads of a run
#pragma unroll
        for (int i = 0; i < S::kLoad / 2; i++) {
            float2& v = acc[j / kPer][j % kPer * (S::kLoad / 2) + i];
            v = fma2(d[j % 2][2 * i], d[j % 2][2 * i + 1], scale[j / kPer], v);
        }
    }
}

// The same for the blocks of a narrow tile's accumulator (n of them are there), all read at once.
template <int BN, bool PAIR>
__device__ __forceinline__ void add_group(float2 (&acc)[MmShape<BN>::kRun / 2], uint32_t src,
                                          const float (&scale)[MmShape<BN>::kGroup], int n, uint32_t empty, int lane) {
    using S = MmShape<BN>;
    static_assert(S::kRuns == 1 && S::kLoad == S::kCols, "one load a block");
    uint32_t d[S::kGroup][S::kLoad];
    tc::fence_after();
#pragma unroll
    for (int g = 0; g < S::kGroup; g++) tmem_load<S::kLoad>(src + g * S::kAccCols, d[g]);
    tc::wait_ld();
    tc::fence_before();
    __syncwarp();
    if (lane == 0) arrive_at<PAIR>(empty);
#pragma unroll
    for (int g = 0; g < S::kGroup; g++) {
        if (g < n) {
#pragma unroll
            for (int i = 0; i < S::kLoad / 2; i++) acc[i] = fma2(d[g][2 * i], d[g][2 * i + 1], scale[g], acc[i]);
        }
    }
}

// The same for a tile of few rows: a thread's columns are rows of a, each with its own scale (of block g at
// scale + g * step).
template <int BN, int FEW>
__device__ __forceinline__ void add_few(float2 (&acc)[MmShape<BN, FEW>::kRun / 2], uint32_t src, const float* scale, int step,
                                        int n, uint32_t empty, int lane) {
    using S = MmShape<BN, FEW>;
    uint32_t d[S::kGroup][S::kLoad];
    tc::fence_after();
#pragma unroll
    for (int g = 0; g < S::kGroup; g++) tmem_load<S::kLoad>(src + g * S::kAccCols, d[g]);
    tc::wait_ld();
    tc::fence_before();
    __syncwarp();
    if (lane == 0) arrive_at<false>(empty);
#pragma unroll
    for (int g = 0; g < S::kGroup; g++) {
        if (g < n) {
#pragma unroll
            for (int i = 0; i < S::kLoad; i += 4) {
                const float4 f = *reinterpret_cast<const float4*>(scale + g * step + i);
                acc[i / 2].x = fmaf(__uint_as_float(d[g][i]), f.x, acc[i / 2].x);
                acc[i / 2].y = fmaf(__uint_as_float(d[g][i + 1]), f.y, acc[i / 2].y);
                acc[i / 2 + 1].x = fmaf(__uint_as_float(d[g][i + 2]), f.z, acc[i / 2 + 1].x);
                acc[i / 2 + 1].y = fmaf(__uint_as_float(d[g][i + 3]), f.w, acc[i / 2 + 1].y);
            }
        }
    }
}

// Where byte b of row r lies in the staging rows: as the 64-byte swizzle of a tensor map has it, which
// spreads a column of 16-byte parts over all banks.
__device__ __forceinline__ int stage_at(int r, int b) { return r * 64 + ((((b >> 4) ^ (r >> 1)) & 3) << 4) + (b & 15); }

// A warp's 32 rows of the tile (a thread a row, COLS columns) to memory.  Pieces of up to 64 bytes a row
// go through the warp's staging rows (pieces of 128 took a stage's room, and time): whole pieces are then copied out by TMA while the warp goes on, or, where rows of the tile are
// not the call's or the output is not aligned for that, stored by neighbouring lanes.  (Stored from the
// registers as they lie, 32 rows at a time, a tile's end took 9000 cycles.)
template <int COLS, bool F32>
__device__ __forceinline__ void store_rows(const MmParams& p, const float2 (&acc)[COLS / 2], uint8_t* stage, int row0,
                                           int rows, int col0, int lane) {
    constexpr int kSize = F32 ? 4 : 2;
    constexpr int kPiece = COLS * kSize < 64 ? COLS * kSize : 64;  // bytes of a row stored at a time
    constexpr int kPieceCols = kPiece / kSize;
    constexpr int kLanes = kPiece / 16;                              // lanes a row
    constexpr int kStep = 32 / kLanes;                               // rows an instruction
    const bool tma = kPiece == 64 && p.out_tma && (rows >= 32 || !p.offsets);
#pragma unroll
    for (int c = 0; c < COLS; c += kPieceCols) {
        const int n = min(kPieceCols, p.N - col0 - c);  // columns of this piece that are there
        if (n <= 0) break;
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the piece before has left
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kLanes; i++) {
            uint4 w;
            if (F32) {
                const float2 a = acc[c / 2 + 2 * i], b = acc[c / 2 + 2 * i + 1];
                w = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
            } else {
                const float2* a = &acc[c / 2 + 4 * i];
                w = make_uint4(pack_bf16(a[0].x, a[0].y), pack_bf16(a[1].x, a[1].y), pack_bf16(a[2].x, a[2].y),
                               pack_bf16(a[3].x, a[3].y));
            }
            *reinterpret_cast<uint4*>(stage + stage_at(lane, 16 * i)) = w;
        }
        if (tma) fence_proxy_async_smem();
        __syncwarp();
        if (tma) {
            if (lane == 0) {
                asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(&p.tout),
                             "r"(col0 + c), "r"(row0), "r"(smem_u32(stage))
                             : "memory");
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
        } else if (p.out_vec) {  // rows 16-byte aligned, N a multiple of 8: a lane's 16 bytes are there or not as one
            const int l = lane % kLanes;
            uint8_t* o = static_cast<uint8_t*>(p.out) + (row0 * p.out_stride + col0 + c) * kSize + 16 * l;
#pragma unroll
            for (int r = lane / kLanes; r < 32; r += kStep)
                if (r < rows && l * (16 / kSize) < n)
                    *reinterpret_cast<uint4*>(o + r * p.out_stride * kSize) =
                        *reinterpret_cast<const uint4*>(stage + stage_at(r, 16 * l));
        } else {
            const int last = min(32, rows);
            for (int r = 0; r < last; r++)
                for (int j = lane; j < n; j += 32) {
                    const int64_t at = (row0 + r) * p.out_stride + col0 + c + j;
                    const uint8_t* v = stage + stage_at(r, kSize * j);
                    if (F32) static_cast<float*>(p.out)[at] = *reinterpret_cast<const float*>(v);
                    else static_cast<uint16_t*>(p.out)[at] = *reinterpret_cast<const uint16_t*>(v);
                }
        }
        __syncwarp();
    }
}

// A weight row's part of a tile of few rows: the first `left` of a thread's rows of column `col`.
template <int ROWS, typename T>
__device__ __forceinline__ void store_few(const MmParams& p, const float2 (&acc)[ROWS / 2], int row0, int left, int col) {
    T* out = static_cast<T*>(p.out) + (int64_t)row0 * p.out_stride + col;
#pragma unroll
    for (int i = 0; i < ROWS; i++, out += p.out_stride) {
        const float v = i % 2 ? acc[i / 2].y : acc[i / 2].x;
        if (i >= left) break;
        if constexpr (sizeof(T) == 4) *out = v;
        else *out = __float2bfloat16_rn(v);
    }
}

// PAIR: two CTAs take a tile of 256 rows together, each 128 rows and half of the weight rows; the
// leader issues the matrix instructions for both.
template <int BN, bool PAIR, int FEW = 0>
__global__ void __launch_bounds__(MmShape<BN, FEW>::kThreads, 1) fp8_mm_kernel(const __grid_constant__ MmParams p) {
    using S = MmShape<BN, FEW>;
    constexpr int kCtas = PAIR ? 2 : 1, kRows = FEW ? FEW : kTileRows * kCtas;
    constexpr int G = S::kGroup;
    constexpr int kWBytes = BN / kCtas * 128;  // a CTA's weight part of a block; a stage has G blocks
    extern __shared__ uint8_t mm_smem[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(mm_smem) + 1023) & ~(uintptr_t)1023);
    __shared__ MmCtl ctl;
    __shared__ Groups groups_of;
    // known to be the same in a warp, so that what follows from it may live in uniform registers
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = PAIR ? (int)cluster_rank() : 0;
    const unsigned first_tile = blockIdx.x / kCtas, tile_step = gridDim.x / kCtas;
    volatile int* abort = &ctl.abort;
    const int stages = p.stages;
    // weight parts first: the row part of the last stage is followed by the tail that keeps the matrix
    // instruction's 128 rows inside shared memory
    uint8_t* wst = sm;
    uint8_t* ast = sm + (size_t)stages * G * kWBytes;

    if (warp == 0) {  // the barriers of a stage a lane: in one thread they took a third of a microsecond
        static_assert(kMaxStages <= 32, "a lane a stage");
        if (lane < stages) {
            mbar_init(&ctl.full[lane], 1);
            mbar_init(&ctl.empty[lane], S::kHalves);
        }
        if (lane < S::kAcc) {
            mbar_init(&ctl.accfull[lane], 1);
            mbar_init(&ctl.accempty[lane], S::kSumWarps / S::kHalves * kCtas);
        }
        if (lane < kScaleRing) {
            mbar_init(&ctl.scfull[lane], 1);
            mbar_init(&ctl.scempty[lane], S::kSumWarps);
        }
        if (lane == 0) {
            mbar_init(&ctl.drain, 2);
            ctl.abort = 0;
        }
        fence_barrier_init();
        if (elect_one()) {
            prefetch_map(&p.tw);
            prefetch_map(&p.tfew);
            prefetch_map(&p.ta128);
        }
        __syncwarp();
    }
    if (warp == 1) {
        if (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl.tmem)),
                         "r"(S::kTmemCols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            tc::tmem_alloc(&ctl.tmem, S::kTmemCols);
            tc::tmem_relinquish();
        }
    }
    pdl_wait();
    pdl_launch_next();
    if (p.offsets) {
        for (int c = warp; c * 32 <= p.E; c += S::kThreads / 32) {  // 32 experts a warp
            const int e = c * 32 + lane;
            const int r0 = min(max(p.offsets[min(e, p.E)], 0), p.M), r1 = min(max(p.offsets[min(e + 1, p.E)], 0), p.M);
            const int mt = r1 > r0 ? (r1 - r0 + kRows - 1) / kRows : 0;
            int s = mt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += v;
            }
            if (e <= p.E) {
                groups_of.first[e] = r0;
                groups_of.before[e] = s - mt;
            }
            if (lane == 31) groups_of.total[c] = min(s, kSpanTiles);
        }
    } else if (threadIdx.x == 0) {
        groups_of.first[0] = groups_of.before[0] = 0;
        groups_of.first[1] = p.M;
        groups_of.total[0] = (p.M + kRows - 1) / kRows;
    }
    tc::fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();  // both CTAs' barriers are there
    tc::fence_after();
    const uint32_t tbase = ctl.tmem;
    const int nt = (p.N + BN - 1) / BN;
    const Lookup look = lookup_of(groups_of, p.E);
    const int64_t n_tiles = (int64_t)look.all * nt;

    if (warp < kFirstSum) {
        if (BN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
        if (warp == 0) {
            // ------------------------------------------------------ TMA
            int s = 0;            // stage to fill
            uint32_t phase = 1;   // parity of the phase of `empty` that frees it: the first round passes at once
            int64_t filled = 0;
            bool ok = true;
            for (int64_t u = first_tile; u < n_tiles && ok; u += tile_step) {
                const Tile t = tile_at<kRows>(p, groups_of, look, nt, BN, u);
                // rows by boxes of box_rows, or (0) by one of 128; boxes of several blocks lie as the blocks do
                // only if one holds all rows
                const int boxes = PAIR ? 0
                                : FEW || p.M <= kFewRows ? 1
                                : G == 1 && t.rows <= kFewRows ? (t.rows + p.box_rows - 1) / p.box_rows : 0;
                const int abytes = (boxes ? boxes * p.box_rows : kTileRows) * 128;
                for (int kb0 = 0; kb0 < p.KB; kb0 += G) {
                    ok = __all_sync(0xffffffffu, mm_wait(&ctl.empty[s], phase, abort, p.status, 1));
                    if (!ok) break;
                    const int n = p.blocked ? G : min(G, p.KB - kb0);  // blocks copied (past the last: zeros)
                    uint8_t *as = ast + s * G * p.a_bytes, *ws = wst + s * G * kWBytes;
                    if (elect_one()) {
                        if (rank == 0) mbar_arrive_expect_tx(&ctl.full[s], (uint32_t)(kCtas * n * (abytes + kWBytes)));
                        if (PAIR) {  // the leader's barrier counts both CTAs' bytes
                            const uint32_t bar = leader_addr(&ctl.full[s]);
                            const int x = p.blocked ? 0 : kb0 * 128, z = p.blocked ? kb0 : 0;
                            tma_w_pair(ws, &p.tw, x, t.n0 + rank * (BN / 2), z, t.e, bar);
                            tma_a_pair(as, &p.ta128, x, t.row0 + rank * kTileRows, z, bar);
                        } else {
                            // a copy takes the issuing thread 90 to 170 cycles: one for a group's blocks where there
                            // can be
                            for (int g = 0; g < (p.blocked ? 1 : n); g++) {
                                const int x = p.blocked ? 0 : (kb0 + g) * 128, z = p.blocked ? kb0 : 0;
                                tma_w(ws + g * kWBytes, &p.tw, x, t.n0, z, t.e, &ctl.full[s]);
                                if (boxes) {
                                    for (int b = 0; b < boxes; b++)
                                        tma_a(as + g * p.a_bytes + b * p.box_rows * 128, &p.tfew, x, t.row0 + b * p.box_rows, z,
                                              &ctl.full[s]);
                                } else {
                                    tma_a(as + g * p.a_bytes, &p.ta128, x, t.row0, z, &ctl.full[s]);
                                }
                            }
                        }
                    }
                    __syncwarp();
                    filled++;
                    if (++s == stages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
            // the matrix instructions' arrivals on `empty` land while the CTA is there: those of the last fills
            for (int64_t i = max((int64_t)0, filled - stages); i < filled && ok; i++)
                ok = __all_sync(0xffffffffu, mm_wait(&ctl.empty[i % stages], (uint32_t)(i / stages) & 1, abort, p.status, 5));
            // copies in flight end before the CTAs do
            if (rank == 0 && (!ok || *abort))
                for (int64_t i = max((int64_t)0, filled - stages); i < filled; i++)
                    (void)mbar_wait(&ctl.full[i % stages], (uint32_t)(i / stages) & 1, 1000000ull);
        } else if (warp < 3 && rank == 0) {
            // ------------------------------------------------------ MMA
            // Issuing a group's instructions and looking at its barriers takes one warp 400 cycles and more, as long as
            // the tensor cores take for it: two warps take turns.  Warp w has half w of every block of the widest
            // tile, else every second group; its accumulators are w and w + 2, and, the number of stages being
            // even, its stages every second one: it sees each phase of the barriers that it waits on.
            constexpr uint32_t id = tc::idesc(0 /* e4m3 */, FEW ? BN : kRows, S::kAccCols);
            constexpr int kTurn = 2 / S::kHalves;  // groups of blocks from one of the warp's to the next
            const int w = warp - 1, h = S::kHalves == 2 ? w : 0;
            const int per = (p.KB + G - 1) / G;    // groups of a tile
            int64_t groups = 0;                    // of this CTA
            if (first_tile < n_tiles) groups = ((n_tiles - 1 - first_tile) / tile_step + 1) * per;
            int at = S::kHalves == 2 ? 0 : w % per;  // the group's number in its tile
            int s = S::kHalves == 2 ? 0 : w % stages, a = w;
            uint32_t phase = S::kHalves == 2 ? 0 : (w / stages) & 1, aphase = 1;
            bool ok = true;
            for (int64_t c = S::kHalves == 2 ? 0 : w; c < groups && ok; c += kTurn) {
                // both are looked at together: most often they are complete, and two waits cost twice one
                const bool e = mbar_done(&ctl.accempty[a], aphase), f = mbar_done(&ctl.full[s], phase);
                if (!__all_sync(0xffffffffu, e && f)) {
                    ok = mm_wait(&ctl.accempty[a], aphase, abort, p.status, 3) &&
                         mm_wait(&ctl.full[s], phase, abort, p.status, 2);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                }
                tc::fence_after();
                if (elect_one()) {
                    const uint64_t ad = tc::sdesc_sw128(smem_u32(ast + s * G * p.a_bytes));
                    const uint64_t wd = tc::sdesc_sw128(smem_u32(wst + s * G * kWBytes + h * (kWBytes / S::kHalves)));
                    const int n = min(G, p.KB - at * G);
#pragma unroll
                    for (int g = 0; g < G; g++) {
                        if (g < n) {
                            const uint64_t ag = ad + (uint64_t)(g * (p.a_bytes >> 4)), wg = wd + (uint64_t)(g * (kWBytes >> 4));
#pragma unroll
                            for (int k = 0; k < 4; k++) {  // 32 of K: 32 bytes, 2 units of the descriptors
                                if (PAIR) mma_f8_pair(tbase + a * S::kAccStep, ag + 2 * k, wg + 2 * k, id, k > 0);
                                else mma_f8(tbase + a * S::kAccStep + g * S::kAccCols, (FEW ? wg : ag) + 2 * k, (FEW ? ag : wg) + 2 * k, id, k > 0);
                            }
                        }
                    }
                    if (PAIR) {
                        commit_pair(&ctl.accfull[a]);
                        commit_pair(&ctl.empty[s]);
                    } else {
                        tc::commit(&ctl.accfull[a]);
                        tc::commit(&ctl.empty[s]);
                    }
                }
                __syncwarp();
                at += kTurn;
                while (at >= per) at -= per;
                s += kTurn;
                while (s >= stages) {
                    s -= stages;
                    phase ^= 1;
                }
                a += 2;
                if (a >= S::kAcc) {
                    a = w;
                    aphase ^= 1;
                }
            }
            if (elect_one()) {
                if (PAIR) commit_pair(&ctl.drain);
                else tc::commit(&ctl.drain);
            }
            __syncwarp();
            (void)mbar_wait(&ctl.drain, 0);
        } else if (PAIR && warp == 1) {
            // the leader's last arrivals; a leader that gave up sends them too
            (void)mbar_wait(&ctl.drain, 0, 4 * kWaitNs);
        } else if (warp == 3) {
            // ------------------------------------------------------ scales
            // A lane takes block lane % 8 of every fourth row: 32 bytes of a row are read together, whatever the
            // rows' alignment, and the loads are far ahead of their use.  Read by the summing threads, each
            // along its own row, they took 500 to 1800 cycles out of every four blocks.
            const int b = lane & 7, r0 = lane >> 3;
            int slot = 0;
            uint32_t phase = 1;
            bool ok = true;
            for (int64_t u = first_tile; u < n_tiles && ok; u += tile_step) {
                const Tile t = tile_at<kRows>(p, groups_of, look, nt, BN, u);
                const int rows = min(kTileRows, t.rows - rank * kTileRows);
                const float* sa = p.sa + (int64_t)(t.row0 + rank * kTileRows) * p.sa_stride;
                for (int kb0 = 0; kb0 < p.KB; kb0 += kScaleGroup) {
                    const int kb = kb0 + b;
                    const bool on = kb < p.KB;
                    MmScales& sc = ctl.scales[slot];
                    float w = 0.0f;
                    if ((FEW || lane < 16) && on) {
                        const int nb = min(t.n0 / kScaleCols + (BN == 256 ? lane >> 3 : 0), p.NB - 1);
                        w = p.sw[((int64_t)t.e * p.NB + nb) * p.KB + kb];
                    }
                    constexpr int kReads = FEW ? FEW / 4 : 16;  // rows of a lane at a time
                    for (int r1 = 0; r1 < (FEW ? FEW : kTileRows); r1 += 4 * kReads) {
                        float v[kReads];
#pragma unroll
                        for (int i = 0; i < kReads; i++) {
                            const int r = r1 + r0 + 4 * i;
                            v[i] = on && r < rows ? sa[(int64_t)r * p.sa_stride + kb] : 0.0f;
                        }
                        if (r1 == 0) {
                            ok = __all_sync(0xffffffffu, mm_wait(&ctl.scempty[slot], phase, abort, p.status, 6));
                            if (!ok) break;
                        }
#pragma unroll
                        for (int i = 0; i < kReads; i++) sc.a[b][r1 + r0 + 4 * i] = FEW ? v[i] * w : v[i];
                    }
                    if (!ok) break;
                    if (lane < 16) sc.w[lane >> 3][b] = w;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl.scfull[slot]);
                    if (++slot == kScaleRing) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- sum over blocks, store
        if (BN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
        const int quad = warp & 3, part = (warp - kFirstSum) >> 2;  // the warp's rows and columns of the accumulators
        constexpr int kParts = S::kAccCols / S::kCols;               // column parts of an accumulator
        const int h = part / kParts, sub = part % kParts;
        // First column of the tile that a run of the warp's columns is.  An accumulator of a pair has half of
        // its columns from each CTA's weight rows, and those are 128 apart.
        auto col_at = [&](int q) {
            return PAIR ? h * (S::kAccCols / 2) + q * (BN / 2) : h * S::kAccCols + sub * S::kCols + q * S::kRun;
        };
        const int r = quad * 32 + lane;
        const uint32_t accempty = PAIR ? leader_addr(&ctl.accempty[0]) : smem_u32(&ctl.accempty[0]);
        int a = h;
        uint32_t aphase = 0;
        bool ok = true;
        uint8_t* stage = sm + p.out_at + (warp - kFirstSum) * kStage;
        int slot = 0;
        uint32_t scphase = 0;
        for (int64_t u = first_tile; u < n_tiles && ok; u += tile_step) {
            float2 acc[S::kRuns][S::kRun / 2];
#pragma unroll
            for (int i = 0; i < S::kCols / 2; i++) acc[i / (S::kRun / 2)][i % (S::kRun / 2)] = make_float2(0.0f, 0.0f);
            for (int kb0 = 0; kb0 < p.KB && ok; kb0 += kScaleGroup) {
                ok = __all_sync(0xffffffffu, mm_wait(&ctl.scfull[slot], scphase, abort, p.status, 7));
                if (!ok) break;
                const MmScales& sc = ctl.scales[slot];
                const int n = min(kScaleGroup, p.KB - kb0);
                for (int i = 0; i < n; i += G) {
                    // scales of the blocks (past the last: numbers that are not used), read before the accumulator is awaited
                    float scale[S::kRuns], more[G];
                    if constexpr (FEW == 0) {
#pragma unroll
                        for (int q = 0; q < S::kRuns; q++) scale[q] = sc.a[i][r] * sc.w[col_at(q) / kScaleCols][i];
#pragma unroll
                        for (int g = 0; g < G; g++) more[g] = g == 0 ? scale[0] : sc.a[i + g][r] * sc.w[0][i + g];
                    }
                    ok = __all_sync(0xffffffffu, mm_wait(&ctl.accfull[a], aphase, abort, p.status, 4));
                    if (!ok) break;
                    const uint32_t src = tc::taddr(tbase, quad * 32, a * S::kAccStep + sub * S::kCols), empty = accempty + a * 8;
                    if constexpr (FEW != 0) add_few<BN, FEW>(acc[0], src, &sc.a[i][sub * S::kCols], kTileRows + 4, n - i, empty, lane);
                    else if constexpr (G > 1) add_group<BN, PAIR>(acc[0], src, more, n - i, empty, lane);
                    else add_block<BN, PAIR>(acc, src, scale, empty, lane);
                    if ((a += S::kHalves) >= S::kAcc) {
                        a = h;
                        aphase ^= 1;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.scempty[slot]);
                if (++slot == kScaleRing) {
                    slot = 0;
                    scphase ^= 1;
                }
            }
            if (!ok) break;
            const Tile now = tile_at<kRows>(p, groups_of, look, nt, BN, u);
            if constexpr (FEW != 0) {  // a thread a weight row: a warp's lanes store neighbouring columns
                // 64 rows of an accumulator lie in the first 16 lanes of each 32
                const int col = now.n0 + (BN == 64 ? quad * 16 + lane : r), m0 = sub * S::kCols, left = now.rows - m0;
                if (left > 0 && col < p.N && (BN == 128 || lane < 16)) {
                    if (p.out_dtype == QS_F32) store_few<S::kCols, float>(p, acc[0], now.row0 + m0, left, col);
                    else store_few<S::kCols, __nv_bfloat16>(p, acc[0], now.row0 + m0, left, col);
                }
                continue;
            }
            const int row0 = now.row0 + rank * kTileRows + quad * 32, rows = now.rows - rank * kTileRows - quad * 32;
            if (rows <= 0) continue;
#pragma unroll
            for (int q = 0; q < S::kRuns; q++) {
                if (p.out_dtype == QS_F32) store_rows<S::kRun, true>(p, acc[q], stage, row0, rows, now.n0 + col_at(q), lane);
                else store_rows<S::kRun, false>(p, acc[q], stage, row0, rows, now.n0 + col_at(q), lane);
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // copies out end before the CTA does
        __syncwarp();
    }
    tc::fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();  // neither CTA's shared memory or accumulators are in use any more
    tc::fence_after();
    if (warp == 1) {
        if (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(S::kTmemCols) : "memory");
        else
            tc::tmem_dealloc(tbase, S::kTmemCols);
    }
}

// ================================================================== host side

using EncodeFn = PFN_cuTensorMapEncodeTiled_v12000;

EncodeFn get_encode() {
    static std::once_flag once;
    static EncodeFn fn = nullptr;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(f);
    });
    return fn;
}

bool encode_out(CUtensorMap* m, void* base, int dtype, const uint64_t* dims, uint64_t stride) {
    EncodeFn fn = get_encode();
    if (!fn) return false;
    const cuuint32_t box[2] = {(cuuint32_t)(64 / type_size(dtype)), 32}, es[2] = {1, 1};
    const cuuint64_t d[2] = {dims[0], dims[1]}, st[1] = {stride};
    return fn(m, dtype == QS_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, d, st, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// rows x K codes (E of them, one after the other, if it is w) as the kernel's boxes take them.
bool encode8(CUtensorMap* m, bool w, const void* base, int K, int64_t rows, int64_t stride, int E, int64_t expert_stride,
             bool blocked, uint32_t box_rows, uint32_t box_blocks) {
    EncodeFn fn = get_encode();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)(blocked ? 128 : K), (cuuint64_t)rows, (cuuint64_t)(blocked ? K / 128 : 1),
                                (cuuint64_t)E};
    const cuuint64_t strides[3] = {(cuuint64_t)stride, (cuuint64_t)(blocked ? 128 : stride), (cuuint64_t)expert_stride};
    const cuuint32_t box[4] = {128, box_rows, blocked ? box_blocks : 1, 1}, es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, w ? 4 : 3, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct MmFacts {
    int n_sm = 0;
    int smem = 0;  // dynamic shared memory a CTA may have beside the static part
    bool wide = false;  // whether the tiles of 256 weight rows may run
};

cudaError_t mm_facts(MmFacts** out) {
    static std::mutex mu;
    static MmFacts facts[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    MmFacts& f = facts[dev];
    if (f.n_sm == 0) {
        int optin = 0, n_sm = 0;
        if ((e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        if ((e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess) return e;
        f.smem = optin - (int)(sizeof(MmCtl) + sizeof(Groups) + 64);
        const void* fns[9] = {(const void*)fp8_mm_kernel<16, false>,  (const void*)fp8_mm_kernel<32, false>,
                              (const void*)fp8_mm_kernel<64, false>,  (const void*)fp8_mm_kernel<128, false>,
                              (const void*)fp8_mm_kernel<256, false>, (const void*)fp8_mm_kernel<256, true>,
                              (const void*)fp8_mm_kernel<64, false, kFewTile>, (const void*)fp8_mm_kernel<64, false, 2 * kFewTile>,
                              (const void*)fp8_mm_kernel<128, false, kFewTile>};
        for (const void* fn : fns)
            if ((e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, f.smem)) != cudaSuccess) return e;
        // The register split would wait forever on a launch with fewer registers: where a compiler gives those kernels
        // another number, the other tiles do their work.
        f.wide = true;
        for (const void* fn : {fns[4], fns[5]}) {
            cudaFuncAttributes wide;
            if ((e = cudaFuncGetAttributes(&wide, fn)) != cudaSuccess) return e;
            f.wide &= wide.numRegs == kLaunchRegs;
        }
        f.n_sm = n_sm;
    }
    *out = &f;
    return cudaSuccess;
}

template <int BN, bool PAIR, int FEW = 0>
cudaError_t mm_run(const Fp8MmArgs& g, MmParams& p, const MmFacts& f, int64_t tiles, cudaStream_t st) {
    constexpr int kCtas = PAIR ? 2 : 1;
    using S = MmShape<BN, FEW>;
    constexpr int G = S::kGroup;
    const bool few = g.n_rows <= kFewRows;
    p.blocked = g.n_inner % 128 == 0;
    p.box_rows = FEW ? FEW : few ? (g.n_rows + kRowBox - 1) / kRowBox * kRowBox : kRowBox;
    p.a_bytes = FEW || few ? p.box_rows * 128 : kTileRows * 128;
    if (!encode8(&p.tw, true, g.w, g.n_inner, g.n_cols, g.w_stride, g.n_experts, g.w_expert_stride, p.blocked, BN / kCtas, G) ||
        !encode8(&p.tfew, false, g.a, g.n_inner, g.n_rows, g.a_stride, 1, 0, p.blocked, p.box_rows, G) ||
        !encode8(&p.ta128, false, g.a, g.n_inner, g.n_rows, g.a_stride, 1, 0, p.blocked, kTileRows, G))
        return cudaErrorInvalidValue;
    const int stage = G * (p.a_bytes + BN / kCtas * 128);
    const int tail = FEW ? 0 : kTileRows * 128 - p.a_bytes;  // the last stage's matrix instruction reads 128 rows
    p.stages = std::min(kMaxStages, (f.smem - 1024 - tail - S::kSumBytes) / stage);
    // Where the issuing warps take groups in turn, a stage is always the same warp's: it has to see every
    // phase of the stage's barrier, or it takes the fill before last for the one it waits for.
    if (S::kHalves == 1) p.stages &= ~1;
    if (p.stages < 2) return cudaErrorInvalidConfiguration;
    p.out_at = p.stages * stage + tail;
    const size_t smem = 1024 + (size_t)p.out_at + S::kSumBytes;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(tiles, f.n_sm / kCtas) * kCtas);
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 2;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = PAIR ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, fp8_mm_kernel<BN, PAIR, FEW>, p);
}

}  // namespace

size_t fp8_matmul_workspace(int, int, int, int) { return kHeaderBytes; }

cudaError_t launch_fp8_matmul(const Fp8MmArgs& g, void* workspace, cudaStream_t st) {
    if (g.n_rows == 0) return cudaSuccess;
    MmFacts* f;
    cudaError_t e = mm_facts(&f);
    if (e != cudaSuccess) return e;
    MmParams p = {};
    p.sa = g.a_scale;
    p.sw = g.w_scale;
    p.offsets = g.offsets;
    p.out = g.out;
    p.status = static_cast<uint32_t*>(workspace);
    p.sa_stride = g.a_scale_stride;
    p.out_stride = g.out_stride;
    p.M = g.n_rows;
    p.N = g.n_cols;
    p.E = g.offsets ? g.n_experts : 1;
    p.KB = scale_blocks(g.n_inner);
    p.NB = scale_blocks(g.n_cols);
    p.out_dtype = g.out_dtype;
    p.out_vec = g.n_cols % 8 == 0 && ((uintptr_t)g.out & 15u) == 0 && (g.out_stride * type_size(g.out_dtype)) % 16 == 0;
    // copied out by TMA: rows on 16-byte boundaries, at a stride that a tensor map holds, and whole 16 bytes long
    // (a copy is cut at the last column's 16 bytes, not at the column)
    const int64_t out_bytes = g.out_stride * type_size(g.out_dtype), row_bytes = g.n_cols * (int64_t)type_size(g.out_dtype);
    p.out_tma = ((uintptr_t)g.out & 15u) == 0 && out_bytes % 16 == 0 && row_bytes % 16 == 0 && out_bytes >= row_bytes &&
                out_bytes < (1ll << 40);
    const uint64_t dout[2] = {(uint64_t)g.n_cols, (uint64_t)g.n_rows};
    if (p.out_tma && !encode_out(&p.tout, g.out, g.out_dtype, dout, (uint64_t)out_bytes)) return cudaErrorInvalidValue;
    const MmTiles t = pick_tiles(g.n_rows, g.n_cols, g.n_experts, g.offsets != nullptr, f->n_sm, f->wide);
    if (t.pair) return mm_run<256, true>(g, p, *f, t.count, st);
    if (t.few == kFewTile)
        return t.cols == 64 ? mm_run<64, false, kFewTile>(g, p, *f, t.count, st) : mm_run<128, false, kFewTile>(g, p, *f, t.count, st);
    if (t.few) return mm_run<64, false, 2 * kFewTile>(g, p, *f, t.count, st);
    switch (t.cols) {
        case 256: return mm_run<256, false>(g, p, *f, t.count, st);
        case 128: return mm_run<128, false>(g, p, *f, t.count, st);
        case 64: return mm_run<64, false>(g, p, *f, t.count, st);
        case 32: return mm_run<32, false>(g, p, *f, t.count, st);
        default: return mm_run<16, false>(g, p, *f, t.count, st);
    }
}

}  // namespace qs
