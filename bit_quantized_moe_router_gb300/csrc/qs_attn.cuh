// qs_attn.cuh -- attention of the newest tokens of each sequence over the paged key-value cache (sm_103a).
//
// Per token at position p and head h (key-value head h / group), over the positions i that it sees:
//   s_i = scale q . k_i,  out = sum_i 2^(s_i' - m) v_i / sum_i 2^(s_i' - m),  s' = s log2(e),  m the running maximum
// in one pass over keys and values.  Bound: HBM, each key and value once; at 8 rows (heads of a group, drafted tokens) to
// a key the products are 8 to 16 operations a byte.
//
// Work.  An item is a sequence, a key-value head and a tile of RT rows (a row: a new token and one of the group's
// heads).  Its positions are cut into tiles of TP.  All items' tiles in one line are dealt to the teams of warps in equal
// runs, wherever an item begins or ends: lengths are known on the device alone and may be uneven, and an even share of the
// line keeps every SM busy to the end.  Entering an item counts as kEnter places of the line (many short sequences 70 -> 34
// us), and an item of few places is not split over CTAs (many short windows 65 -> 48 us).  An item inside one team's run is written from its registers.  What a CTA's teams
// have of the same item is added up in shared memory when their runs end; what several CTAs have of one is joined by the
// last of them to finish (a counter an item, no waits), above kFan of them in two steps, always in the order of the
// positions, so the result does not depend on who was last.  (One CTA that read all 76 parts of a long sequence took 100 us.)
//
// A team of R x C warps has a ring of ST tiles in shared memory filled by 16-byte asynchronous copies, which run ahead over
// the ends of items: pages of any size and order, one lookup a position a tile ahead of its copies; positions that are not
// there are filled with zeros, never read.  The warps of a team share the tile; R of them have 8 NT rows each, C of them a
// share of the output's columns (where a tile is so large that one a warp would not fit).  With R = C = 1 no barrier wider
// than a warp is met before the run's end.  About 64 KB an SM are on their way: with 128 KB the SMs' shares of the memory
// became uneven and the last ones late (64 sequences of bf16 218 -> 179 us).
//
// Products.  mma.sync m16n8k16 in the cache's own 16-bit values: bf16, or e4m3 widened to fp16 (exact) in registers.
// tcgen05 takes 64 or 128 rows where there are mostly 8, its results have to be fetched for the softmax, and widened
// codes would go back to shared memory first; at 8 rows mma.sync's 1024 multiply-adds a cycle and SM are 2.5 times what HBM
// can feed.  At 64 rows (eight heads, eight drafted tokens) they are not, and the kernel reads 2 TB/s there.
// S^T = K Q^T: 16 positions down, rows across, so that 8 rows leave nothing empty (queries down: twice the products).  bf16 keys
// and values come by ldmatrix, values transposed; e4m3's are widened from 16- and 8-byte loads, values interleaved by
// position first.  A lane's weights are transposed by movmatrix into the second operand of O^T = V^T P^T.
//
// Roundings.  Scores, maxima, sums and O are fp32.  e4m3 scales stay out of the 16-bit operands: the key's multiplies
// the score, the value's the weight, and the running maximum is of s' + log2(value scale), so that fp16 weights stay below
// 2^(kLift + kSlack) whatever the scales are.  A weight goes into the product as PP 16-bit parts, each of what the ones before
// leave out: two of bf16 or one of fp16 for bf16 output (off by 2^-16, 2^-11 of the weight), three or two with fp32
// rows or codes (2^-24, 2^-22).  fp32 queries are QP such parts; for an fp16 product a row is scaled by a power of two.  Keys and
// values of bf16 may be infinite, so that its parts have one sign and none is zero alone (kOver).
//
// A position that a row does not see never touches it, NaN and infinity included: scores are replaced, and positions that
// some of an item's rows see and others do not (the drafted tokens' own, the first ones of a window) are added for those rows
// alone in fp32, their values then cleared before the product.
//
// Code that runs once an SM and call costs 3 to 6 cycles an instruction beyond 32 KB, so there is one copy of each part.
//
// Measured on one GB300, in a replayed graph, cold (HBM): 64 sequences of up to 8192 positions, 32 heads on 8 of 128
// columns, bf16 169 to 183 us (by the lengths drawn, 1.0 to 1.2 GB: 6.2 to 6.7 TB/s; fp32 rows 174, to codes 181), e4m3 to codes 111
// to 123 us (5.0 TB/s; 4-byte scales of one head are 32-byte sectors); one token over 131072 positions of 2 e4m3 heads of 256 39 us (3.4 TB/s:
// 20 us of it enter, add up and join); 1000 positions of 2 bf16 heads of 256 15 us; 16 sequences of up to eight drafted tokens
// over 16384 positions 101 us (e4m3 107; heads of 256 195, fp32 rows 313); 200 windows of 301 positions 47 us.
#pragma once

#include <algorithm>

#include "qs_cache.cuh"

namespace qs {

namespace attn {

constexpr float kSlack = 8.0f;    // a row's maximum may lag behind by this much (log2) before the sums are scaled
constexpr float kLift = 7.0f;     // fp16 weights are 2^(score - maximum + kLift), at most 2^15: small ones keep 7 more bits
// Over e4m3 the running maximum is of a score and the logarithm of the value's scale, kLeastScale at least (values that are all zero
// have 2^-109).  A weight may so be 2^(kLift + kSlack - kLeastScale) = 2^111, and a row has 2^30 of them at most: their sum is held in
// units of 2^kDown, below 2^127.  The other way a scale of 2^119, the largest that fp32 rows are written with, leaves a maximum's weight 2^-112,
// in these units fp32's smallest normal number.
constexpr float kLeastScale = -96.0f, kDown = 14.0f, kUnit = 0x1p-14f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kSmemMax = 227 * 1024;
constexpr int kFan = 12;          // parts of an item that one CTA joins at a time
constexpr int kMostTeams = 16;
constexpr int kAhead = 64 * 1024;  // bytes of copies on their way
constexpr int kStatic = 8 * 1024;  // shared memory for tables

// A kernel's sizes: cache type, columns (head_dim rounded up), 8 rows times NT a warp, teams of R warps with rows of their
// own times C with columns of their own, W warps a CTA, TP positions a tile, and whether queries and weights go into the
// products with all their parts.
template <bool E4_, int DP_, int NT_, int R_, int C_, int W_, int TP_, bool WIDE_>
struct Plan {
    static constexpr bool E4 = E4_, WIDE = WIDE_;
    static constexpr int DP = DP_, NT = NT_, R = R_, C = C_, kWarps = W_;
    static constexpr int kRowBytes = DP * (E4 ? 1 : 2), kChunks = kRowBytes / 16;
    static constexpr int kTeam = R * C, kTeams = kWarps / kTeam, kRows = 8 * NT, RT = R * kRows, kCols = DP / C;
    static constexpr int TP = TP_;
    static constexpr int kStage = 2 * TP * kRowBytes + (E4 ? 2 * TP * 4 : 0);  // keys, values, their scales
    static constexpr float kUp = E4 ? kLift : 0.0f;
    static constexpr int QP = WIDE ? (E4 ? 2 : 3) : 1, PP = WIDE ? (E4 ? 2 : 3) : (E4 ? 1 : 2);
    static constexpr int kSteps = DP / 16;            // of the first product
    // The queries' fragments: in registers where they fit beside the sums and about 80 others, else in shared memory.
    static constexpr int kQEach = 2 * NT * QP;         // registers of a step
    static constexpr int kRegs = 65536 / (32 * kWarps) < 255 ? 65536 / (32 * kWarps) : 255;  // of a thread
    static constexpr bool kQInRegs = kQEach * kSteps <= kRegs - 80 - kCols * NT / 4;
    static constexpr int kQBytes = kQInRegs ? 0 : kWarps * QP * NT * kSteps * 32 * 8;
    static constexpr int kPieces = kCols / 16;         // of the output: 16 columns of a warp's rows
    static constexpr int kRow = DP + 4, kPart = RT * (kRow + 2);  // floats of an item's part: rows of sums, maxima and sums of weights
    static constexpr int kRed = kTeams * kPart * 4;  // the teams' parts, over all of it
    static constexpr int kFit = (kSmemMax - kStatic - kQBytes) / (kTeams * kStage);
    static constexpr int kGoal = 1 + (kAhead + kTeams * kStage / 2) / (kTeams * kStage);
    static constexpr int ST = kGoal < 2 ? (kFit < 2 ? kFit : 2) : kGoal > kFit ? kFit : kGoal;
    static constexpr int kRing = kTeams * ST * kStage;
    static constexpr int kSmem = kQBytes + kRing > kRed ? kQBytes + kRing : kRed;
    // Places in the line.  A tile's: one, or where warps share it kTileBase and one more for each warp with rows (a tile takes
    // nearly as long for 8 rows as for 64).  Entering an item, two tiles' where queries are scaled and cut into parts (16 rows of
    // e4m3: 46.7 us, 49.0 with one, 48.9 with four), one's where they are taken as they lie (many short sequences: 33.5 us, 34.5
    // with two, 37.2 with four), four's where warps share them (drafted tokens: 102.4 us, 104.7 with two); the least share of a
    // team (one token over 1000 positions: 15.2 us with two places, 17.1 with four); the largest item that is not split over CTAs.
    static constexpr int kTileBase = 12, kEnter = R > 1 ? 4 * (kTileBase + R) : E4 || WIDE ? 2 : 1;
    static constexpr int kLeast = R == 1 ? 2 : kEnter + kTileBase, kUnsplit = 8 * (R == 1 ? 1 : kTileBase + R) * kTeams;
    static_assert(ST >= 2 && kSmem + kStatic <= kSmemMax, "shared memory");
    static_assert(kWarps % kTeam == 0 && 32 * kTeam % kChunks == 0 && TP * kChunks % (32 * kTeam) == 0, "copies");
    static_assert(kTeams <= (RT <= 16 ? kMostTeams : 3) && kTeams <= 16 && kCols % 64 == 0 && (kTeam == 1 || kTeams <= 15), "teams");
    static_assert(!WIDE || DP < kScaleCols || kCols >= kScaleCols, "a scale's columns are one warp's");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Warps that wait for one another: `warps` of them at barrier `id` (1 .. 15).
__device__ __forceinline__ void sync_warps(int id, int warps) {
    if (warps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(32 * warps) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool E4>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if (E4)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four 8 x 8 matrices of 16-bit values from shared memory, a row's address from each lane; as they lie or transposed.
template <bool TRANS>
__device__ __forceinline__ void load_matrices(uint32_t (&a)[4], uint32_t at) {
    if (TRANS) asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]) : "r"(at) : "memory");
    else asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]) : "r"(at) : "memory");
}
// An 8 x 8 matrix of 16-bit values, two of a row in a lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Two e4m3 codes as fp16.
__device__ __forceinline__ uint32_t widen(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)two));
    return r;
}

// Of bf16 keys and values one may be infinite, and its products with the parts of a query or a weight have to agree.  So all parts but the
// last are cut toward zero, and what they leave is taken from kOver of the value: of one sign, and never zero beside a value that is
// not (queries from 2^-80 on, weights from 2^-80 of the largest).  Two parts hold 16 bits, three 24.  kBack takes kOver back out where
// there are three, from the scores' factor and from the rows': with two it is far below what they leave out.
constexpr float kOver = 1.0f + 0x1p-23f, kBack = 1.0f - 0x1p-23f;

// The N 16-bit parts of two weights, each what the ones before leave out.
template <bool E4, int N>
__device__ __forceinline__ void weight_parts(uint32_t (&parts)[N], float lo, float hi) {
#pragma unroll
    for (int pl = 0; pl < N; pl++) {
        if (E4) {
            const __half2 h = __floats2half2_rn(lo, hi);
            const float2 f = __half22float2(h);
            lo -= f.x;
            hi -= f.y;
            parts[pl] = *reinterpret_cast<const uint32_t*>(&h);
        } else if (pl == N - 1) {
            parts[pl] = pack_bf16(lo, hi);
        } else {
            parts[pl] = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
            lo = fmaf(lo, kOver, -bf16_lo(parts[pl]));
            hi = fmaf(hi, kOver, -bf16_hi(parts[pl]));
        }
    }
}

// The next part of two queries, and what it leaves out.  Of an infinite query every part is infinite: where a row has one (`finite` is false)
// parts are not taken from one another, and what its other columns come to then does not count.  The last is rounded.
template <bool E4>
__device__ __forceinline__ uint32_t query_part(float& lo, float& hi, bool finite, bool last) {
    if (E4) {
        const __half2 h = __floats2half2_rn(lo, hi);
        const float2 f = __half22float2(h);
        if (finite) lo -= f.x;
        if (finite) hi -= f.y;
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    if (last) return pack_bf16(lo, hi);
    const uint32_t w = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
    if (finite) lo = fmaf(lo, kOver, -bf16_lo(w));
    if (finite) hi = fmaf(hi, kOver, -bf16_hi(w));
    return w;
}

// What a sequence has to do.  Positions are 32-bit numbers near enough to the table's (0 .. positions): a start far outside
// it is brought so near that its tokens see the same.
struct Seq {
    int first_token, tokens;  // the new tokens that are attended (max_new at most)
    int lo_base, hi_base;     // token j sees lo_base + j .. hi_base + j - 1, clipped to the table
    int lo;                   // the first position that any of them sees
    int tiles, row_tiles;     // of an item; row tiles of a head
    int weight;               // places in the line that a tile takes
};
// a / b, b > 0, a >= 0, in 32 bits where both fit.
__device__ __forceinline__ int64_t div_of(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}
__device__ __forceinline__ int near_pos(int64_t p, int n) { return (int)(p < -1024 ? -1024 : p > n ? n : p); }
__device__ __forceinline__ int clip_pos(int p, int n) { return min(max(p, 0), n); }

template <class P>
__device__ __forceinline__ Seq seq_of(const AttnArgs& p, int s) {
    constexpr int TP = P::TP, RT = P::RT;
    Seq q;
    q.first_token = s;
    q.tokens = 1;
    if (p.seqs.offsets) {
        // both clipped before they are subtracted: the difference stays in 32 bits and the rows inside the call's
        q.first_token = min(max(p.seqs.offsets[s], 0), p.n_tokens);
        q.tokens = min(max(min(max(p.seqs.offsets[s + 1], 0), p.n_tokens) - q.first_token, 0), p.max_new);
    }
    const int64_t start = p.seqs.starts ? p.seqs.starts[s] : 0;
    const int n = p.seqs.positions;
    q.lo_base = p.window ? near_pos(start - p.window + 1, n) : -1024;
    q.hi_base = near_pos(start + 1, n);
    q.lo = clip_pos(q.lo_base, n);
    q.tiles = max(1, (clip_pos(q.hi_base + q.tokens - 1, n) + TP - 1) / TP - q.lo / TP);  // one where nothing is seen: its rows are still written
    q.row_tiles = (q.tokens * p.group + RT - 1) / RT;
    // where warps share a tile, its time grows with those that have rows
    q.weight = P::R == 1 ? 1 : P::kTileBase + (min(q.tokens * p.group, RT) + P::kRows - 1) / P::kRows;
    return q;
}

// The token of an item's row.
__device__ __forceinline__ int token_of(const AttnArgs& p, int row) { return fast_div(row, p.group_div); }

// What an item's rows are and see, and what of it a team's run has: `count` tiles from the one at position pos0, a stretch.
struct Item {
    int first_token, rows, kv, row0;
    int lo_base, hi_base, tiles, marks;
    int count, pos0, at, weight;  // at: where the item begins in the line, from the run's start
};
enum { kOpens = 1, kEnds = 2 };  // the stretch has the item's first tile, its last
// What a team has of an item that is not whole in its run: where the item begins in the line (-1: nothing), and which.
struct Piece {
    int64_t at;
    int first_token, rows, kv, row0, tiles, weight;
};

// An output row: where it goes.
struct Row {
    int64_t token;
    int head;
    bool real;
};
template <class X>
__device__ __forceinline__ Row row_of(const AttnArgs& p, const X& x, int row) {
    const int at = token_of(p, row);
    return {x.first_token + at, x.kv * p.group + row - at * p.group, row < x.rows};
}
// From a row's sum of weights, which is held in units of 2^kDown over e4m3.
template <bool E4>
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.0f ? -INFINITY : (m + (log2f(l) + (E4 ? kDown : 0.0f))) * kLn2; }
template <bool E4, bool WIDE>
__device__ __forceinline__ float inverse_of(float l) { return l == 0.0f ? 0.0f : (E4 ? kUnit : WIDE ? kBack : 1.0f) / l; }

// Four columns of a row from col, of a warp that has 128 of it side by side: v is the sum of weighted values, l the sum of
// weights, m the maximum that they are relative to.
template <bool E4, bool WIDE>
__device__ __forceinline__ void finish(const AttnArgs& p, const Row& r, int col, float (&v)[4], float m, float l) {
    const float inv = inverse_of<E4, WIDE>(l);
#pragma unroll
    for (int q = 0; q < 4; q++) v[q] = l == 0.0f ? 0.0f : v[q] * inv;
    const int d = p.cache.head_dim;
    if (WIDE && p.codes) {
        const BlockCode code(lanes_max(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))), 16), 1.0f, kMinAmax);
        if (r.real) {
            const int i = r.head * d + col;
            *reinterpret_cast<uint32_t*>(p.codes + r.token * p.codes_stride + i) = code.pair(v[0], v[1]) | (code.pair(v[2], v[3]) << 16);
            if (i % kScaleCols == 0) p.codes_scale[r.token * p.codes_scale_stride + i / kScaleCols] = code.scale;
        }
    }
    if (!r.real || col >= d) return;
    if (p.out.data) {
        uint8_t* to = p.out.data + r.token * p.out.token_stride + r.head * p.out.head_stride;
        if (WIDE && p.out.dtype == QS_F32) *reinterpret_cast<float4*>(to + 4 * col) = make_float4(v[0], v[1], v[2], v[3]);
        else *reinterpret_cast<uint2*>(to + 2 * col) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    }
    if (p.lse && col == 0) p.lse[r.token * p.n_heads + r.head] = lse_of<E4>(m, l);
}

// A warp's output, acc[j][nt][2 h + e]: of piece j the column col_of_value(j, h) from the warp's first, of rows nt * 8 + 2 t + e.
// bf16: piece j is columns 16 j ..; e4m3: four pieces are 64 columns, of which a lane has eight neighbours.
template <bool E4>
__device__ __forceinline__ int col_of_value(int j, int h) {
    const int g = (threadIdx.x & 31) >> 2;
    return E4 ? 64 * (j / 4) + 8 * g + 2 * (j % 4) + h : 16 * j + 8 * h + g;
}

// An item's rows from the registers of the warps that have all their positions: columns col0 .. of rows w0 ...
template <class P, class X>
__device__ __forceinline__ void finish_rows(const AttnArgs& p, const X& x, int w0, int col0, const float (&top)[P::NT][2], const float (&sum)[P::NT][2],
                                            const float (&acc)[P::kPieces][P::NT][4]) {
    constexpr int NT = P::NT, kJ = P::kPieces;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, d = p.cache.head_dim;
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const float l = sum[nt][e], by = inverse_of<P::E4, P::WIDE>(l);
            const Row r = row_of(p, x, w0 + nt * 8 + 2 * t + e);
            if (p.lse && g == 0 && col0 == 0 && r.real) p.lse[r.token * p.n_heads + r.head] = lse_of<P::E4>(top[nt][e], l);
            float v[kJ][2];
#pragma unroll
            for (int j = 0; j < kJ; j++)
#pragma unroll
                for (int h = 0; h < 2; h++) v[j][h] = by == 0.0f ? 0.0f : acc[j][nt][2 * h + e] * by;
            if constexpr (P::WIDE && kJ >= 8) {  // a scale's 128 columns are in the eight lanes of the same t
                if (p.codes) {
#pragma unroll
                    for (int b = 0; b < kJ; b += 8) {
                        float a = 0.0f;
#pragma unroll
                        for (int j = b; j < b + 8; j++) a = fmaxf(a, fmaxf(fabsf(v[j][0]), fabsf(v[j][1])));
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
                        const BlockCode code(a, 1.0f, kMinAmax);
                        if (!r.real) continue;
                        const int i = r.head * d + col0 + 16 * b;
                        if (g == 0) p.codes_scale[r.token * p.codes_scale_stride + i / kScaleCols] = code.scale;
                        uint8_t* to = p.codes + r.token * p.codes_stride + r.head * d + col0;
#pragma unroll
                        for (int j = b; j < b + 8; j++) {
                            if (P::E4) *reinterpret_cast<uint16_t*>(to + col_of_value<P::E4>(j, 0)) = (uint16_t)code.pair(v[j][0], v[j][1]);
                            else
#pragma unroll
                                for (int h = 0; h < 2; h++) to[col_of_value<P::E4>(j, h)] = code.one(v[j][h]);
                        }
                    }
                }
            }
            if (!r.real || !p.out.data) continue;
            uint8_t* to = p.out.data + r.token * p.out.token_stride + r.head * p.out.head_stride;
            const bool f32 = P::WIDE && p.out.dtype == QS_F32;
            if (P::E4) {  // eight neighbours
#pragma unroll
                for (int j = 0; j < kJ; j += 4) {
                    const int col = col0 + col_of_value<true>(j, 0);
                    const float y[8] = {v[j][0], v[j][1], v[j + 1][0], v[j + 1][1], v[j + 2][0], v[j + 2][1], v[j + 3][0], v[j + 3][1]};
                    if (col < d) store8_row<true>(to, f32 ? QS_F32 : QS_BF16, col, d, y);
                }
            } else {  // the lanes of eight neighbouring columns store one each
#pragma unroll
                for (int j = 0; j < kJ; j++)
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const int col = col0 + col_of_value<false>(j, h);
                        if (col >= d) continue;
                        if (f32) reinterpret_cast<float*>(to)[col] = v[j][h];
                        else reinterpret_cast<__nv_bfloat16*>(to)[col] = __float2bfloat16_rn(v[j][h]);
                    }
            }
        }
}

// Where a row's 16-byte pieces lie in shared memory: piece c of row r at c ^ swap(r), so that the eight that are read at
// once have banks of their own.  bf16: a matrix's eight rows; e4m3 keys: two rows' four; e4m3 values: four rows' two.
template <bool E4, int NC>
__device__ __forceinline__ int key_swap(int row) { return E4 ? (NC >= 8 ? (row & 1) * 4 : 0) : row & 7; }
template <bool E4, int NC>
__device__ __forceinline__ int value_swap(int row) { return E4 ? ((row >> 1) & 3) * 2 & (NC - 1) : row & 7; }

// What a part with maximum ml.x counts beside the maximum m; one of no positions (-infinity, 0) nothing.
__device__ __forceinline__ float part_factor(float2 ml, float m) { return ml.x == -INFINITY ? (ml.y == 0.0f ? 0.0f : 1.0f) : ex2(ml.x - m); }

template <class P>
__global__ void __launch_bounds__(32 * P::kWarps, 1) attn_kernel(const AttnArgs p) {
    constexpr bool E4 = P::E4;
    constexpr int DP = P::DP, NT = P::NT, RT = P::RT, TP = P::TP, ST = P::ST, NC = P::kChunks, kJ = P::kPieces;
    constexpr int kWarps = P::kWarps, kThreads = 32 * kWarps;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t scan[kWarps], before_of[kThreads];
    __shared__ unsigned there_of[kWarps][ST];           // a tile's positions that are there
    __shared__ __align__(16) Item item_of[kWarps][ST];  // of the tiles that are a stretch's first
    __shared__ __align__(16) Piece piece_of[2 * P::kTeams];  // of each team: the stretch that begins inside an item and ends with it; the run's last
    __shared__ bool last_of[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int team = warp / P::kTeam, team_tid = tid % (32 * P::kTeam), row_warp = (warp % P::kTeam / P::C + team) % P::R , col_warp = warp % P::C;
    // (rows dealt to the SM's quarters in turn: an item's last warps may have none)
    const int n_pos = p.seqs.positions;
    uint8_t* const q_shared = smem + warp * (P::kQBytes / kWarps) + lane * 8;
    uint8_t* const ring = smem + P::kQBytes + team * ST * P::kStage;
    float* const red = reinterpret_cast<float*>(smem);  // a part a team, over all of it
    pdl_wait();
    pdl_launch_next();

    // ---- the CTA's run of the line [run0, run1), the team's share of it, and the sequence that this begins in.  An item
    // takes kEnter places before its tiles', about what entering and leaving it costs.
    const int per = (p.seqs.n_seqs + kThreads - 1) / kThreads;
    const int s0 = min(tid * per, p.seqs.n_seqs), s1 = min(s0 + per, p.seqs.n_seqs);
    auto places_of = [&](int s) {
        const Seq q = seq_of<P>(p, s);
        return (int64_t)(q.tiles * q.weight + P::kEnter) * (q.row_tiles * p.cache.n_kv);
    };
    int64_t mine = 0;
    for (int s = s0; s < s1; s++) mine += places_of(s);
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    before_of[tid] = upto - mine;  // within the warp
    if (lane == 31) scan[warp] = upto;
    if (tid < 2 * P::kTeams) piece_of[tid].at = -1;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; w++) total += scan[w];
    // as many CTAs as have kLeast places for each team
    const int64_t workers = min((int64_t)gridDim.x, div_of(total - 1, P::kTeams * P::kLeast) + 1);
    const int c = blockIdx.x;
    if (total == 0 || c >= workers) return;
    // equal runs, the first of them a place longer
    const int64_t each = div_of(total, workers), longer = total - each * workers;
    auto begin_of_cta = [&](int x) { return x * each + min((int64_t)x, longer); };
    // where a place lies: its sequence, and where that begins
    auto find = [&](int64_t place, int64_t& base) {
        base = 0;
        if (p.seqs.n_seqs <= 1) return 0;
        int of_warp = 0;
        int64_t sums = 0;
#pragma unroll
        for (int w = 0; w < kWarps; w++) {
            if (sums <= place) {
                of_warp = w;
                base = sums;
            }
            sums += scan[w];
        }
        // of that warp's threads the last whose sequences begin at or before it
        const int64_t mine_before = before_of[of_warp * 32 + lane];
        const unsigned at_or_before = __ballot_sync(0xffffffffu, base + mine_before <= place && (of_warp * 32 + lane) * per < p.seqs.n_seqs);
        const int of_lane = 31 - __clz(at_or_before);
        base += __shfl_sync(0xffffffffu, mine_before, of_lane);
        int s = (of_warp * 32 + of_lane) * per;
        for (int n = 1; n < per && s + 1 < p.seqs.n_seqs; n++, s++) {
            const int64_t x = places_of(s);
            if (place < base + x) break;
            base += x;
        }
        return s;
    };
    // Runs begin where they fall, but for items of few places, which one CTA has: what sharing such a one over two saves is
    // less than what joining it costs.
    auto whole_items = [&](int64_t place) {
        if (place <= 0 || place >= total) return place;
        int64_t base;
        const Seq q = seq_of<P>(p, find(place, base));
        const int span = q.tiles * q.weight + P::kEnter;
        if (span > P::kUnsplit) return place;
        const int in = (int)((place - base) - div_of(place - base, span) * span);
        return place - in + (2 * in < span ? 0 : span);
    };
    const int64_t run0 = whole_items(begin_of_cta(c)), run1 = whole_items(begin_of_cta(c + 1));
    const unsigned length = (unsigned)(run1 - run0);
    auto begin_of = [&](unsigned x) { return length / P::kTeams * x + length % P::kTeams * x / P::kTeams; };
    const int64_t from = run0 + begin_of(team);
    const int run = (int)(begin_of(team + 1) - begin_of(team));
    int64_t base;
    const int seq0 = find(min(from, total - 1), base);

    // ---- the next tile to copy, kept by all warps of a team alike
    struct {
        int seq, item, items, left, count, pos, lo, hi;
        const uint8_t *k, *v;
        const int32_t* table;
        const float *k_scale, *v_scale;
    } next = {};
    Item entered = {};
    bool first = false, entered_one = false;
    int ahead = -1;          // a lane's position's place, in units; -1: not there
    int64_t ahead_scale = 0;
    next.seq = seq0;
    next.left = run;
    // a thread copies the 16 bytes `chunk` of the rows chunk_row, chunk_row + kStep, ...; a row's bits above chunk_row's are
    // the pass's, and swap() is of bits
    constexpr int kStep = 32 * P::kTeam / NC, kPasses = TP / kStep;
    const int chunk = team_tid % NC, chunk_row = team_tid / NC;
    const bool chunk_in = chunk * 16 < p.cache.head_dim * (E4 ? 1 : 2), all_in = p.cache.head_dim == DP;
    const uint32_t key_to = smem_u32(ring) + chunk_row * P::kRowBytes, key_piece = (chunk ^ key_swap<E4, NC>(chunk_row)) * 16, value_piece = (chunk ^ value_swap<E4, NC>(chunk_row)) * 16;
    constexpr unsigned kAll = TP == 32 ? 0xffffffffu : (1u << (TP & 31)) - 1u;

    // ---- the rows of the item under way
    struct {
        int first_token, rows, kv, row0, lo_base, hi_base, tiles, marks, at, weight;
    } item = {};
    int remain = 0, pos0 = 0, w0 = 0, all_lo = 0, all_hi = 0, tile_lo = 0, tile_hi = 0;
    bool active = false;
    uint32_t qf[P::kQInRegs ? P::kSteps : 1][P::kQInRegs ? P::kQEach : 1];
    float row_scale[NT][2];
    float acc[kJ][NT][4];
    float top[NT][2], sum[NT][2];  // of rows 2 t, 2 t + 1: what weights are relative to (the maximum less kUp), and the sum of this lane's
    auto lo_of = [&](int base, int row) { return clip_pos(base + token_of(p, row), n_pos); };  // of lo_base or hi_base, and a row

    // queries as fragments in the order in which the keys' pieces lie
    auto begin = [&](const Item& x) {
        item = {x.first_token, x.rows, x.kv, x.row0, x.lo_base, x.hi_base, x.tiles, x.marks, x.at, x.weight};
        remain = x.count;
        pos0 = x.pos0;
        w0 = x.row0 + row_warp * P::kRows;
        active = w0 < x.rows;
        const int last = min(x.row0 + RT, x.rows) - 1;
        tile_lo = lo_of(x.lo_base, x.row0);
        tile_hi = lo_of(x.hi_base, last);
        all_lo = lo_of(x.lo_base, last);
        all_hi = lo_of(x.hi_base, x.row0);
        constexpr int kE = P::kQInRegs ? P::kQEach : 1, kS = P::kQInRegs ? P::kSteps : 1;
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            const Row r = row_of(p, x, w0 + nt * 8 + g);
            const uint8_t* q = p.q.data + r.token * p.q.token_stride + r.head * p.q.head_stride;
            const int n_cols = r.real ? p.cache.head_dim : 0;
            // a step's columns: two neighbours for the lower half of the step, two for the upper
            auto cols_of = [&](int step, int half) { return E4 ? 64 * (step / 4) + 16 * t + 4 * (step % 4) + 2 * half : 16 * step + 8 * half + 2 * t; };
            auto store = [&](int step, int pl, uint32_t lo, uint32_t hi) {
                if (P::kQInRegs) {
                    qf[step % kS][(2 * (pl * NT + nt)) % kE] = lo;
                    qf[step % kS][(2 * (pl * NT + nt) + 1) % kE] = hi;
                } else {
                    *reinterpret_cast<uint2*>(q_shared + ((pl * NT + nt) * P::kSteps + step) * 256) = make_uint2(lo, hi);
                }
            };
            float factor = 1.0f;
            if constexpr (!E4 && !P::WIDE) {  // bf16 as it lies
                uint32_t raw[P::kSteps][2];
#pragma unroll
                for (int step = 0; step < P::kSteps; step++)
#pragma unroll
                    for (int half = 0; half < 2; half++) {
                        raw[step][half] = 0u;
                        if (cols_of(step, half) < n_cols) raw[step][half] = *reinterpret_cast<const uint32_t*>(q + 2 * cols_of(step, half));
                    }
#pragma unroll
                for (int step = 0; step < P::kSteps; step++) store(step, 0, raw[step][0], raw[step][1]);
            } else {
                float2 v[P::kSteps][2];
                if (E4) {  // two steps' columns of a lane are neighbours
#pragma unroll
                    for (int step = 0; step < P::kSteps; step += 2) {
                        float y[8];
                        load8_row<true>(q, P::WIDE ? p.q.dtype : QS_BF16, cols_of(step, 0), n_cols, y);
                        v[step][0] = make_float2(y[0], y[1]);
                        v[step][1] = make_float2(y[2], y[3]);
                        v[step + 1][0] = make_float2(y[4], y[5]);
                        v[step + 1][1] = make_float2(y[6], y[7]);
                    }
                }
#pragma unroll
                for (int step = 0; step < (E4 ? 0 : P::kSteps); step++)
#pragma unroll
                    for (int half = 0; half < 2; half++) {
                        const int col = cols_of(step, half);
                        v[step][half] = make_float2(0.0f, 0.0f);
                        if (col >= n_cols) continue;
                        if (P::WIDE && p.q.dtype == QS_F32) {
                            v[step][half] = *reinterpret_cast<const float2*>(q + 4 * col);
                        } else {
                            const uint32_t w = *reinterpret_cast<const uint32_t*>(q + 2 * col);
                            v[step][half] = make_float2(bf16_lo(w), bf16_hi(w));
                        }
                    }
                float a = 0.0f;
#pragma unroll
                for (int step = 0; step < P::kSteps; step++)
#pragma unroll
                    for (int half = 0; half < 2; half++) a = fmaxf(a, fmaxf(fabsf(v[step][half].x), fabsf(v[step][half].y)));
                const bool finite = a < INFINITY;  // of this lane's columns
                if (E4) {  // a power of two that brings the row's largest into fp16's upper range (down from any that fp32 has)
                    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
                    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
                    const int e = min(max(14 - ((int)(__float_as_uint(a) >> 23) - 127), -113), 100);
                    factor = __uint_as_float((uint32_t)(127 + e) << 23);
                }
#pragma unroll
                for (int step = 0; step < P::kSteps; step++) {
                    float2 y = v[step][0], z = v[step][1];
                    y.x *= factor;
                    y.y *= factor;
                    z.x *= factor;
                    z.y *= factor;
#pragma unroll
                    for (int pl = 0; pl < P::QP; pl++) {
                        const uint32_t lo = query_part<E4>(y.x, y.y, finite, pl == P::QP - 1);
                        store(step, pl, lo, query_part<E4>(z.x, z.y, finite, pl == P::QP - 1));
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 2; e++) {
                top[nt][e] = -INFINITY;
                sum[nt][e] = 0.0f;
                row_scale[nt][e] = E4 ? p.scale * (1.0f / __shfl_sync(0xffffffffu, factor, 8 * t + 4 * e)) : P::WIDE ? p.scale * kBack : p.scale;
            }
        }
#pragma unroll
        for (int j = 0; j < kJ; j++)
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int e = 0; e < 4; e++) acc[j][nt][e] = 0.0f;
    };
    // one step of the first product: 16 positions' keys with every part of the queries.  The tensor cores cut what a sum
    // drops, always toward zero, so that a long chain of them is off by half a unit a step (2e-6 after 30): with all parts two
    // steps begin at zero, in `two`, and are added with a rounding.
    auto score = [&](float (&sums)[NT][4], float (&two)[NT][4], int step, const uint32_t (&a)[4]) {
        float(&c)[NT][4] = P::WIDE ? two : sums;
        if (P::WIDE && step % 2 == 0) {
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int e = 0; e < 4; e++) c[nt][e] = 0.0f;
        }
#pragma unroll
        for (int pl = 0; pl < P::QP; pl++)
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                constexpr int kE = P::kQInRegs ? P::kQEach : 1, kS = P::kQInRegs ? P::kSteps : 1;
                if (P::kQInRegs) {
                    mma<E4>(c[nt], a[0], a[1], a[2], a[3], qf[step % kS][2 * (pl * NT + nt) % kE], qf[step % kS][(2 * (pl * NT + nt) + 1) % kE]);
                } else {
                    const uint2 b = *reinterpret_cast<const uint2*>(q_shared + ((pl * NT + nt) * P::kSteps + step) * 256);
                    mma<E4>(c[nt], a[0], a[1], a[2], a[3], b.x, b.y);
                }
            }
        if (P::WIDE && step % 2 == 1) {
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int e = 0; e < 4; e++) sums[nt][e] += c[nt][e];
        }
    };
    // the rows' sums as a part: rows of kRow floats, then a maximum and a sum of weights a row
    auto put = [&](float* to) {
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int row = row_warp * P::kRows + nt * 8 + 2 * t + e;
                if (g == 0 && col_warp == 0) reinterpret_cast<float2*>(to + RT * P::kRow)[row] = make_float2(top[nt][e], sum[nt][e]);
                float* at = to + row * P::kRow + col_warp * P::kCols;
                if (E4) {
#pragma unroll
                    for (int j = 0; j < kJ; j += 2)
                        *reinterpret_cast<float4*>(at + col_of_value<E4>(j, 0)) = make_float4(acc[j][nt][e], acc[j][nt][2 + e], acc[j + 1][nt][e], acc[j + 1][nt][2 + e]);
                } else {
#pragma unroll
                    for (int j = 0; j < kJ; j++)
#pragma unroll
                        for (int h = 0; h < 2; h++) at[col_of_value<E4>(j, h)] = acc[j][nt][2 * h + e];
                }
            }
    };

    // ---- the pass over the run's tiles: tile i is consumed, tile i + ST - 1 copied, the one after it looked up
    int issued = 0, use = 0, fill = 0;
    for (int i = -ST; i < 0 || i < issued; i++) {
        const int stage = use;
        unsigned there = 0;
        if (i >= 0) {
            if (++use == ST) use = 0;
            __syncwarp();
            there = there_of[warp][stage];
            pos0 += TP;
            if (remain == 0) begin(item_of[warp][stage]);  // the queries are on their way with the tile
            remain--;
            cp_wait<ST - 2>();
            sync_warps(1 + team, P::kTeam);
        }
        if (i > -ST) {
            if (next.count > 0) {
                const unsigned found = __ballot_sync(0xffffffffu, ahead >= 0) & kAll;
                if (lane == 0) {
                    there_of[warp][fill] = found;
                    if (first) item_of[warp][fill] = entered;
                }
                first = false;
                const uint32_t to = key_to + fill * P::kStage;
                if (found == kAll && all_in) {
#pragma unroll
                    for (int k = 0; k < kPasses; k++) {
                        const int64_t offset = (int64_t)__shfl_sync(0xffffffffu, ahead, chunk_row + k * kStep) * p.places.unit;
                        cp16(to + k * kStep * P::kRowBytes + (key_piece ^ key_swap<E4, NC>(k * kStep) * 16), next.k + offset, true);
                        cp16(to + (TP + k * kStep) * P::kRowBytes + (value_piece ^ value_swap<E4, NC>(k * kStep) * 16), next.v + offset, true);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < kPasses; k++) {
                        const int at = __shfl_sync(0xffffffffu, ahead, chunk_row + k * kStep);
                        const bool ok = at >= 0 && chunk_in;
                        const int64_t offset = (int64_t)max(at, 0) * p.places.unit;
                        cp16(to + k * kStep * P::kRowBytes + (key_piece ^ key_swap<E4, NC>(k * kStep) * 16), next.k + offset, ok);
                        cp16(to + (TP + k * kStep) * P::kRowBytes + (value_piece ^ value_swap<E4, NC>(k * kStep) * 16), next.v + offset, ok);
                    }
                }
                if (E4 && warp % P::kTeam == 0 && lane < TP) {
                    const bool ok = ahead >= 0;
                    const int64_t offset = ok ? ahead_scale : 0;
                    const uint32_t scale_to = smem_u32(ring) + fill * P::kStage + 2 * TP * P::kRowBytes + lane * 4;
                    cp4(scale_to, next.k_scale + offset, ok);
                    cp4(scale_to + TP * 4, next.v_scale + offset, ok);
                }
                if (++fill == ST) fill = 0;
                issued++;
                next.left -= entered.weight;
                next.count--;
                next.pos += TP;
            }
            cp_commit();
        }
        while (next.count == 0 && next.left > 0) {  // an item is entered
            int at = entered.at + entered.tiles * entered.weight + P::kEnter, tile = 0;
            if (entered_one) {
                next.left -= P::kEnter;
                if (++next.item == next.items) {
                    next.item = 0;
                    next.seq++;
                }
            }
            Seq q;
            for (;; next.seq++) {
                next.seq = min(next.seq, p.seqs.n_seqs - 1);
                q = seq_of<P>(p, next.seq);
                if (q.tokens > 0 || next.seq + 1 >= p.seqs.n_seqs) break;
            }
            next.items = q.row_tiles * p.cache.n_kv;
            if (!entered_one) {  // the run's first, at any of its places
                const int64_t in = from - base;
                const int span = q.tiles * q.weight + P::kEnter;
                next.item = (int)div_of(in, span);
                const int place = (int)(in - (int64_t)next.item * span);
                tile = max(0, place - P::kEnter + q.weight - 1) / q.weight;  // the first that begins at or after it
                next.left -= tile * q.weight + P::kEnter - place;
                at = -place;
            }
            int kv = next.item, row0 = 0;
            if (q.row_tiles != 1) {
                kv = next.item / q.row_tiles;
                row0 = (next.item - kv * q.row_tiles) * RT;
            }
            next.count = max(0, min(q.tiles - tile, (next.left + q.weight - 1) / q.weight));
            next.pos = q.lo / TP * TP + tile * TP + lane % TP;
            entered_one = true;
            entered = Item{q.first_token, q.tokens * p.group, kv, row0, q.lo_base, q.hi_base, q.tiles, (tile == 0 ? kOpens : 0) | (tile + next.count == q.tiles ? kEnds : 0),
                           next.count, next.pos - lane % TP, at, q.weight};
            first = true;
            next.lo = lo_of(q.lo_base, row0);
            next.hi = lo_of(q.hi_base, min(row0 + RT, entered.rows) - 1);
            const int64_t head = kv * p.cache.head_stride + (chunk_in ? chunk * 16 : 0);
            next.k = p.cache.k + head;
            next.v = p.cache.v + head;
            next.table = p.seqs.table + next.seq * p.seqs.table_stride;
            if (E4) {
                next.k_scale = p.cache.k_scale + kv * p.cache.scale_head_stride;
                next.v_scale = p.cache.v_scale + kv * p.cache.scale_head_stride;
            }
        }
        ahead = -1;
        if (next.count > 0 && next.pos >= next.lo && next.pos < next.hi) {
            const int page_of = fast_div(next.pos, p.cache.page_div), slot = next.pos - page_of * p.cache.page_size, page = next.table[page_of];
            if ((unsigned)page < (unsigned)p.cache.n_pages) ahead = page * p.places.page + slot * p.places.slot;
            if (E4) ahead_scale = page * p.cache.scale_page_stride + slot * p.cache.scale_slot_stride;
        }
        if (i < 0) continue;

        uint8_t* const keys = ring + stage * P::kStage;
        uint8_t* const values = keys + TP * P::kRowBytes;
        const bool full = there == kAll && pos0 >= all_lo && pos0 + TP <= all_hi;
        // positions here that some of the item's rows see and others do not
        const bool mixed = !full && (min(pos0 + TP, tile_hi) > all_hi || max(pos0, tile_lo) < all_lo);
        // their values become zeros, once every row that sees one has added it by itself
        auto clear_mixed = [&]() {
            sync_warps(1 + team, P::kTeam);
#pragma unroll 1
            for (int y = team_tid; y < TP * NC; y += 32 * P::kTeam) {
                const int at = pos0 + y / NC;
                if (at < all_lo || at >= all_hi) reinterpret_cast<uint4*>(values)[y] = make_uint4(0, 0, 0, 0);
            }
            sync_warps(1 + team, P::kTeam);
        };
        if (!active) {
            if (mixed) clear_mixed();
        } else {
            const float* const scales = reinterpret_cast<const float*>(values + TP * P::kRowBytes);
            // S^T = K Q^T: 16 positions down, a warp's rows across.  With one block of positions two sums, of every second step: a
            // product waits three times its own length for the one before.
            constexpr int kB = TP / 16, kSums = kB == 1 && !P::WIDE ? 2 : 1;
            float sc[kSums * kB][NT][4];
#pragma unroll
            for (int b = 0; b < kSums * kB; b++)
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int e = 0; e < 4; e++) sc[b][nt][e] = 0.0f;
            float two[P::WIDE ? kB : 1][NT][4];
            if constexpr (E4) {
#pragma unroll
                for (int i4 = 0; i4 < NC / 4; i4++)
#pragma unroll
                    for (int b = 0; b < kB; b++) {
                        uint4 w[2];
#pragma unroll
                        for (int y = 0; y < 2; y++) {
                            const int row = 16 * b + 8 * y + g;
                            w[y] = *reinterpret_cast<const uint4*>(keys + row * P::kRowBytes + (((4 * i4 + t) ^ key_swap<E4, NC>(row)) * 16));
                        }
                        const uint32_t lo[4] = {w[0].x, w[0].y, w[0].z, w[0].w}, hi[4] = {w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
                        for (int h = 0; h < 4; h++) {
                            const uint32_t a[4] = {widen(lo[h]), widen(hi[h]), widen(lo[h] >> 16), widen(hi[h] >> 16)};
                            score(sc[b + h % kSums * kB], two[P::WIDE ? b : 0], 4 * i4 + h, a);
                        }
                    }
            } else {
                const int row = lane & 15;
                const uint32_t at = smem_u32(keys) + row * P::kRowBytes;
#pragma unroll
                for (int step = 0; step < P::kSteps; step++)
#pragma unroll
                    for (int b = 0; b < kB; b++) {
                        uint32_t a[4];
                        load_matrices<false>(a, at + 16 * b * P::kRowBytes + (((2 * step + (lane >> 4)) ^ key_swap<E4, NC>(row)) * 16));
                        score(sc[b + step % kSums * kB], two[P::WIDE ? b : 0], step, a);
                    }
            }
            // scores to weights.  A lane's are of rows 2 t + e at positions 16 b + 8 y + g, sc[b][nt][2 y + e].
            float by_key[kB][2], vs[kB][2], lv[kB][2];
#pragma unroll
            for (int b = 0; b < kB; b++)
#pragma unroll
                for (int y = 0; y < 2; y++) {
                    by_key[b][y] = 1.0f;
                    vs[b][y] = 1.0f;
                    lv[b][y] = 0.0f;
                    if (E4) {  // the values' scales count for the maximum
                        by_key[b][y] = scales[16 * b + 8 * y + g];
                        vs[b][y] = scales[TP + 16 * b + 8 * y + g];
                        lv[b][y] = fmaxf(lg2(vs[b][y]), kLeastScale);
                        // a position that some rows do not see counts for the maximum as any other, but it is left to its own sums
                        // below, with the scale as it is: here it has no weight, which may be beyond fp16 without its scale
                        if (mixed && (pos0 + 16 * b + 8 * y + g < all_lo || pos0 + 16 * b + 8 * y + g >= all_hi)) vs[b][y] = 0.0f;
                    }
                }
#pragma unroll
            for (int b = 0; b < kB; b++)
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        if (kSums == 2) sc[b][nt][e] += sc[(b + kB) % (kSums * kB)][nt][e];
                        sc[b][nt][e] *= E4 ? row_scale[nt][e % 2] * by_key[b][e / 2] : row_scale[nt][e % 2];
                    }
            if (!full) {
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const int row = w0 + nt * 8 + 2 * t + e;
                        const int lo = lo_of(item.lo_base, row) - pos0 - g, hi = lo_of(item.hi_base, row) - pos0 - g;
#pragma unroll
                        for (int y = 0; y < 2 * kB; y++)
                            if (!((there >> (8 * y + g)) & 1u) || 8 * y < lo || 8 * y >= hi) sc[y / 2][nt][y % 2 * 2 + e] = -INFINITY;
                    }
            }
            bool grown = false;
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float most = -INFINITY;
#pragma unroll
                    for (int b = 0; b < kB; b++) most = fmaxf(most, fmaxf(sc[b][nt][e] + lv[b][0], sc[b][nt][2 + e] + lv[b][1]));
                    grown |= most > top[nt][e] + (P::kUp + kSlack);
                }
            if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        float now = -INFINITY;
#pragma unroll
                        for (int b = 0; b < kB; b++) now = fmaxf(now, fmaxf(sc[b][nt][e] + lv[b][0], sc[b][nt][2 + e] + lv[b][1]));
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, o));
                        now = fmaxf(top[nt][e], now - P::kUp);
                        const float by = now == top[nt][e] ? 1.0f : ex2(top[nt][e] - now);
                        top[nt][e] = now;
                        sum[nt][e] *= by;
#pragma unroll
                        for (int j = 0; j < kJ; j++) {
                            acc[j][nt][e] *= by;
                            acc[j][nt][2 + e] *= by;
                        }
                    }
            }
            // weights, left in sc, and their parts (e4m3: with the value's scale), transposed to the second product's operand
            uint32_t pb[kB][NT][P::PP][2];
#pragma unroll
            for (int b = 0; b < kB; b++)
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int y = 0; y < 2; y++) {
                        float two[2];
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            const float z = sc[b][nt][2 * y + e], ref = top[nt][e] == -INFINITY ? 0.0f : top[nt][e];
                            two[e] = ex2(z - ref);
                            sum[nt][e] = E4 ? fmaf(two[e], kUnit, sum[nt][e]) : sum[nt][e] + two[e];
                            sc[b][nt][2 * y + e] = two[e];
                            if (E4) two[e] *= vs[b][y];
                        }
                        uint32_t parts[P::PP];
                        weight_parts<E4>(parts, two[0], two[1]);
#pragma unroll
                        for (int pl = 0; pl < P::PP; pl++) pb[b][nt][pl][y] = transposed(parts[pl]);
                    }
            if (mixed) {
                // positions that some of the rows see: one at a time, for those rows alone
#pragma unroll 1
                for (int at = max(pos0, tile_lo); at < min(pos0 + TP, tile_hi); at++) {
                    if (at >= all_lo && at < all_hi) {
                        at = all_hi - 1;
                        continue;
                    }
                    const int o = at - pos0;
                    if (!((there >> o) & 1u)) continue;
                    float by[NT][2];
                    bool sees[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            float mine = 0.0f;
#pragma unroll
                            for (int y = 0; y < 2 * kB; y++)
                                if (o / 8 == y) mine = sc[y / 2][nt][y % 2 * 2 + e];
                            by[nt][e] = __shfl_sync(0xffffffffu, mine, o % 8 * 4 + t) * (E4 ? scales[TP + o] : 1.0f);
                            const int row = w0 + nt * 8 + 2 * t + e;
                            sees[nt][e] = at >= lo_of(item.lo_base, row) && at < lo_of(item.hi_base, row);
                        }
                    const uint8_t* const value = values + o * P::kRowBytes;
                    const int swap = value_swap<E4, NC>(o);
#pragma unroll
                    for (int j = 0; j < kJ; j++) {
                        float2 v;
                        const int col = col_warp * P::kCols + col_of_value<E4>(j, 0);
                        if (E4) {
                            const uint32_t two = widen(*reinterpret_cast<const uint16_t*>(value + ((col / 16) ^ swap) * 16 + col % 16));
                            v = __half22float2(*reinterpret_cast<const __half2*>(&two));
                        } else {
                            v.x = bf16_lo(*reinterpret_cast<const uint16_t*>(value + ((col / 8) ^ swap) * 16 + g * 2));
                            v.y = bf16_lo(*reinterpret_cast<const uint16_t*>(value + ((col / 8 + 1) ^ swap) * 16 + g * 2));
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; nt++)
#pragma unroll
                            for (int e = 0; e < 2; e++)
                                if (sees[nt][e]) {
                                    acc[j][nt][e] = fmaf(by[nt][e], v.x, acc[j][nt][e]);
                                    acc[j][nt][2 + e] = fmaf(by[nt][e], v.y, acc[j][nt][2 + e]);
                                }
                    }
                }
                clear_mixed();
            }
            // O^T += V^T P^T: 16 columns down, a warp's rows across
            float tile[P::WIDE ? 4 : 1][NT][4];
#pragma unroll
            for (int bj = 0; bj < kB * kJ / 4; bj++) {
                // with all parts a tile's products begin at zero too: all of its positions for 64 columns, then the next
                const int b = P::WIDE ? bj % kB : bj / (kJ / 4), j4 = 4 * (P::WIDE ? bj / kB : bj % (kJ / 4));
                {
                    uint32_t w[4][2];  // e4m3: four positions' eight columns
                    if (E4) {
#pragma unroll
                        for (int r = 0; r < 4; r++) {
                            const int row = b * 16 + 2 * t + (r & 1) + (r >> 1) * 8;
                            const uint2 y = *reinterpret_cast<const uint2*>(values + row * P::kRowBytes + (((j4 + col_warp * kJ + g / 2) ^ value_swap<E4, NC>(row)) * 16) + (g & 1) * 8);
                            w[r][0] = y.x;
                            w[r][1] = y.y;
                        }
                    }
#pragma unroll
                    for (int m = 0; m < 4; m++) {
                        uint32_t a[4];
                        if (E4) {
                            const uint32_t y = __byte_perm(w[0][m / 2], w[1][m / 2], m % 2 ? 0x7362 : 0x5140);
                            const uint32_t z = __byte_perm(w[2][m / 2], w[3][m / 2], m % 2 ? 0x7362 : 0x5140);
                            a[0] = widen(y);
                            a[1] = widen(y >> 16);
                            a[2] = widen(z);
                            a[3] = widen(z >> 16);
                        } else {
                            const int row = (lane & 7) + (lane >> 4) * 8;
                            load_matrices<true>(a, smem_u32(values) + (b * 16 + row) * P::kRowBytes + (((2 * (j4 + m + col_warp * kJ) + (lane >> 3 & 1)) ^ value_swap<E4, NC>(row)) * 16));
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; nt++) {
                            float(&sums)[4] = P::WIDE ? tile[P::WIDE ? m : 0][nt] : acc[j4 + m][nt];
#pragma unroll
                            for (int e = 0; e < 4; e++)
                                if (P::WIDE && b == 0) sums[e] = 0.0f;
#pragma unroll
                            for (int pl = 0; pl < P::PP; pl++) mma<E4>(sums, a[0], a[1], a[2], a[3], pb[b][nt][pl][0], pb[b][nt][pl][1]);
#pragma unroll
                            for (int e = 0; e < 4; e++)
                                if (P::WIDE && b == kB - 1) acc[j4 + m][nt][e] += sums[e];
                        }
                    }
                }
            }
        }
        if (remain > 0) continue;

        // ---- the end of an item, or of the run inside one
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int e = 0; e < 2; e++)
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) sum[nt][e] += __shfl_xor_sync(0xffffffffu, sum[nt][e], o);
        const bool ends = item.marks & kEnds;
        if (item.marks == (kOpens | kEnds)) {
            if (active) finish_rows<P>(p, item, w0, col_warp * P::kCols, top, sum, acc);
            continue;
        }
        if (team_tid == 0) piece_of[2 * team + !ends] = Piece{from + item.at, item.first_token, item.rows, item.kv, item.row0, item.tiles, item.weight};
        if (!ends) break;  // the run's last; its sums wait for the ring to be free
        put(p.heads + (c * P::kTeams + team) * P::kPart);
    }
    cp_wait<0>();
    __syncthreads();  // the ring is free
    if (piece_of[2 * team + 1].at >= 0) put(red + team * P::kPart);
    __syncthreads();

    // ---- what the teams have of the same item, and then the CTAs: the warps are dealt to the items
    const int64_t my_at = lane < 2 * P::kTeams ? piece_of[lane].at : -1;
    const unsigned pieces = __ballot_sync(0xffffffffu, my_at >= 0);
    const unsigned before = pieces & ((1u << lane) - 1u);
    const int64_t at_before = __shfl_sync(0xffffffffu, my_at, before ? 31 - __clz(before) : 0);
    unsigned starts = __ballot_sync(0xffffffffu, my_at >= 0 && (!before || at_before != my_at));
    const int items = __popc(starts);
    if (items == 0) return;
    // (two of 64 rows one after the other: the last of an item's CTAs has every warp for it)
    const int crews = RT > 16 && items <= 2 ? 1 : min(items, kWarps), size = kWarps / crews, crew = warp / size, crew_tid = tid - crew * size * 32;
    if (crew >= crews) return;
    auto cta_of = [&](int64_t place) {  // the CTA whose run has it
        const int64_t split = longer * (each + 1);
        const bool low = place < split;
        return (int)((low ? 0 : longer) + div_of(low ? place : place - split, low ? each + 1 : each));
    };
#pragma unroll 1
    for (int n = 0; n < items; n++, starts &= starts - 1u) {
        if (n % crews != crew) continue;
        const int i0 = __ffs(starts) - 1;
        const unsigned later = starts & (starts - 1u), of_item = pieces & ~((1u << i0) - 1u) & (later ? (later & (0u - later)) - 1u : 0xffffffffu);
        const Piece q = piece_of[i0];
        const int64_t tiles0 = q.at + P::kEnter, last0 = tiles0 + (int64_t)(q.tiles - 1) * q.weight;
        const bool whole = tiles0 >= run0 && last0 < run1;
        int c0 = c, c1 = c;
        if (!whole) {
            c0 = cta_of(tiles0);
            c1 = cta_of(last0);
        }
        // CTAs c0 .. c1 have the item; the first kFan of them, the next kFan and so on are joined first
        const int sub = (c - c0) / kFan, first = c0 + sub * kFan, many = min(kFan, c1 - first + 1), subs = (c1 - c0) / kFan + 1;
#pragma unroll 1
        for (int level = 0;; level++) {
            // the parts: of the teams; of CTAs, of kFan CTAs, part i at base + i * step (+ shift, the first)
            const bool done = whole || level == 2 || (level == 1 && subs == 1);
            const float* const base = level == 1 ? p.parts + first * 2 * P::kPart : p.merged + c0 * 2 * P::kPart;
            const int step = level == 1 ? 2 * P::kPart : 2 * kFan * P::kPart, shift = level == 2 || first == c0 ? P::kPart : 0;
            float* const result = (level == 0 ? p.parts + (c * 2 + (c == c0)) * P::kPart : p.merged + (first * 2 + (first == c0)) * P::kPart);
            const int parts = level == 1 ? many : subs, n_real = min(RT, q.rows - q.row0);
            // four columns of a row a thread, of two such pieces at a time where the registers allow, seven parts of each on their way at once
            constexpr int kPer = kWarps <= 12 ? 2 : 1, kBatch = 7;
            const int pieces_end = (n_real * (DP / 4) + 31) / 32 * 32;
#pragma unroll 1
            for (int x0 = crew_tid; x0 < pieces_end; x0 += size * 32 * kPer) {
                float m[kPer], l[kPer], v[kPer][4];
#pragma unroll
                for (int k = 0; k < kPer; k++) {
                    m[k] = -INFINITY;
                    l[k] = v[k][0] = v[k][1] = v[k][2] = v[k][3] = 0.0f;
                }
                unsigned rest = level == 0 ? of_item : (1u << parts) - 1u;
#pragma unroll 1
                while (rest) {
                    float2 ml[kPer][kBatch];
                    float4 a[kPer][kBatch];
#pragma unroll
                    for (int y = 0; y < kBatch; y++) {
#pragma unroll
                        for (int k = 0; k < kPer; k++) {
                            ml[k][y] = make_float2(-INFINITY, 0.0f);
                            a[k][y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        }
                        if (!rest) continue;
                        const int i = __ffs(rest) - 1;
                        rest &= rest - 1u;
                        const bool shared = level == 0 && i % 2;
                        const float* const part = shared       ? red + i / 2 * P::kPart
                                                  : level == 0 ? p.heads + (c * P::kTeams + i / 2) * P::kPart
                                                               : base + (int64_t)i * step + (i == 0 ? shift : 0);
#pragma unroll
                        for (int k = 0; k < kPer; k++) {
                            const int x = x0 + k * size * 32, row = x / (DP / 4), col = x % (DP / 4) * 4;
                            if (x >= pieces_end) continue;
                            const float2* ml_at = reinterpret_cast<const float2*>(part + RT * P::kRow) + row;
                            const float4* a_at = reinterpret_cast<const float4*>(part + row * P::kRow + col);
                            ml[k][y] = shared ? *ml_at : __ldcg(ml_at);
                            a[k][y] = shared ? *a_at : __ldcg(a_at);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < kPer; k++) {
                        float now = m[k];
#pragma unroll
                        for (int y = 0; y < kBatch; y++) now = fmaxf(now, ml[k][y].x);
                        const float by = part_factor(make_float2(m[k], l[k]), now);
                        m[k] = now;
                        l[k] *= by;
#pragma unroll
                        for (int e = 0; e < 4; e++) v[k][e] *= by;
#pragma unroll
                        for (int y = 0; y < kBatch; y++) {
                            const float f = part_factor(ml[k][y], now);
                            l[k] += f * ml[k][y].y;
                            v[k][0] += f * a[k][y].x;
                            v[k][1] += f * a[k][y].y;
                            v[k][2] += f * a[k][y].z;
                            v[k][3] += f * a[k][y].w;
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < kPer; k++) {
                    const int x = x0 + k * size * 32, row = x / (DP / 4), col = x % (DP / 4) * 4;
                    if (x >= pieces_end) continue;
                    if (done) {
                        finish<E4, P::WIDE>(p, row_of(p, q, q.row0 + row), col, v[k], m[k], l[k]);
                    } else {
                        __stcg(reinterpret_cast<float4*>(result + row * P::kRow + col), make_float4(v[k][0], v[k][1], v[k][2], v[k][3]));
                        if (col == 0) __stcg(reinterpret_cast<float2*>(result + RT * P::kRow) + row, make_float2(m[k], l[k]));
                    }
                }
            }
            if (done) break;
            // the last of those that have parts goes on; it leaves the counter at zero.  One thread releases and acquires, the
            // barriers before and after it carry that from and to the others: fences in all threads cost 2 us.
            sync_warps(1 + crew, size);
            if (crew_tid == 0) {
                uint32_t* counter = p.joined + (level == 1 ? 2 * kAttnMaxCtas + c0 : sub == 0 ? c0 : kAttnMaxCtas + first);
                const bool last = atom_acq_rel_add(counter, 1u) == (uint32_t)((level == 0 ? many : subs) - 1);
                if (last) *counter = 0u;
                last_of[crew] = last;
            }
            sync_warps(1 + crew, size);
            const bool last = last_of[crew];
            sync_warps(1 + crew, size);
            if (!last) break;
        }
    }
}

// One CTA an SM of the current device, looked up once a kernel and device.
template <class P>
cudaError_t launch(AttnArgs p, cudaStream_t st) {
    static int ctas_of[64];  // 0: not known yet; written with the same value by whoever finds it
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int ctas = dev < 64 ? ctas_of[dev] : 0;
    if (ctas == 0) {
        int sms = 0, each = 0;
        if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        if ((e = cudaFuncSetAttribute(attn_kernel<P>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kSmem)) != cudaSuccess) return e;
        if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&each, attn_kernel<P>, 32 * P::kWarps, P::kSmem)) != cudaSuccess) return e;
        if (each < 1) return cudaErrorLaunchOutOfResources;
        ctas = std::min(kAttnMaxCtas, sms);  // equal runs: a second CTA on some SMs alone would end late
        if (dev < 64) ctas_of[dev] = ctas;
    }
    return launch_pdl(attn_kernel<P>, dim3((unsigned)ctas), 32 * P::kWarps, P::kSmem, st, p);
}

// Rows of an item: 8, 16 or 64, each with the plan that was fastest of those that fit.  Some of the others, us: 64 sequences
// of bf16, 8 rows a head: two column warps of 8, tiles of 32 178, one of 12, tiles of 16 179 (short sequences 43 and 49), one of 8
// 184, two of 16 196.  The same in e4m3: one of 8, tiles of 32 125, one of 12, tiles of 16 147, of 16 178.  131072 positions of
// e4m3, 256 columns: one of 8 46, two of 12 48, two of 16 60.  e4m3, 16 rows: one of 8 68, two of 12 109.  64 rows of bf16: 12
// warps 104, 8 113, 16 149, 8 of 32 rows each 139.
constexpr int padded_dim(int head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }
constexpr int item_rows(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 64; }
constexpr int most_teams(int rows) { return rows <= 16 ? 16 : 3; }

template <bool E4, int DP, bool WIDE>
cudaError_t launch_rows(const AttnArgs& p, cudaStream_t st) {
    constexpr int kBytes = DP * (E4 ? 1 : 2);
    const int rows = item_rows(p.n_heads / p.cache.n_kv * p.max_new);
    // a team's warps by columns, warps a CTA, positions a tile
    if (rows == 8) {
        constexpr int C = DP == 64 || E4 || (DP == 128 && WIDE) ? 1 : DP == 128 || WIDE ? 2 : 4;
        constexpr int W = DP == 64 ? 16 : DP == 128 || WIDE || E4 ? 8 : 16;
        return launch<Plan<E4, DP, 1, 1, C, W, kBytes <= 64 || (DP == 128 && (E4 || !WIDE)) ? 32 : 16, WIDE>>(p, st);
    }
    if (rows == 16) {
        constexpr int C = DP == 64 || (DP == 128 && (E4 || WIDE)) ? 1 : 2;
        constexpr int W = DP == 64 ? 12 : WIDE || (E4 && DP == 128) ? 8 : 12;
        return launch<Plan<E4, DP, DP == 256 ? 1 : 2, DP == 256 ? 2 : 1, C, W, kBytes <= 64 || (E4 && WIDE && DP == 128) ? 32 : 16, WIDE>>(p, st);
    }
    constexpr int C = DP == 256 && !E4 && !WIDE ? 2 : 1;
    constexpr int W = DP == 64 ? 12 : DP == 128 ? (WIDE && !E4 ? 8 : 12) : WIDE && !E4 ? 4 : 8;
    return launch<Plan<E4, DP, 2, 4, C, W, kBytes <= 256 ? 32 : 16, WIDE>>(p, st);
}

}  // namespace attn

// One translation unit each, for the time that they take to compile.
template <bool E4, int DP>
cudaError_t launch_attention(const AttnArgs& p, bool wide, cudaStream_t st) {
    return wide ? attn::launch_rows<E4, DP, true>(p, st) : attn::launch_rows<E4, DP, false>(p, st);
}
extern template cudaError_t launch_attention<false, 64>(const AttnArgs&, bool, cudaStream_t);
extern template cudaError_t launch_attention<false, 128>(const AttnArgs&, bool, cudaStream_t);
extern template cudaError_t launch_attention<false, 256>(const AttnArgs&, bool, cudaStream_t);
extern template cudaError_t launch_attention<true, 64>(const AttnArgs&, bool, cudaStream_t);
extern template cudaError_t launch_attention<true, 128>(const AttnArgs&, bool, cudaStream_t);
extern template cudaError_t launch_attention<true, 256>(const AttnArgs&, bool, cudaStream_t);

}  // namespace qs
