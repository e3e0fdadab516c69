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
// line keeps every SM busy to the end.  An item inside one team's run is written from its registers.  What a CTA's teams
// have of the same item is added up in shared memory when their runs end; what several CTAs have of one is joined by the
// last of them to finish (a counter an item, no waits), above kFan of them in two steps, always in the order of the
// positions, so the result does not depend on who was last.
//
// A team of R warps has a ring of ST tiles in shared memory filled by 16-byte asynchronous copies, which run ahead over the
// ends of items: pages of any size and order, one lookup a position a tile ahead of its copies; positions that are not
// there are filled with zeros, never read.  The warps of a team share the tile and have 8 NT rows each; with R = 1 no
// barrier wider than a warp is met before the run's end.
//
// Products.  mma.sync m16n8k16 in the cache's own 16-bit values: bf16, or e4m3 widened to fp16 (exact) in registers.
// tcgen05 would want 64 or 128 rows where there are 8, and the widened codes written back to shared memory first: here
// the codes pass from shared memory to registers once, and a lane's fragments are whole 16-byte pieces, since the order
// of the inner dimension is free as long as both operands have the same.  S = Q K^T has the queries down (rows 8..15
// are empty with NT = 1); its accumulator is, as it lies, the second operand of O^T = V^T P^T, whose first operand is
// made by interleaving the bytes of a lane's four positions.
//
// Roundings.  Scores, maxima, sums and O are fp32.  e4m3 scales stay out of the 16-bit operands: the key's multiplies
// the score, the value's the weight, and the running maximum is of s' + log2(value scale), so that weights stay below
// 2^kSlack whatever the scales are.  A weight goes into the product as PP 16-bit parts, each the rounding of what the
// ones before leave out: two of bf16 or one of fp16 for bf16 output (off by 2^-16, 2^-11 of the weight), three or two with fp32
// rows or codes (2^-24, 2^-22).  fp32 queries are QP such parts; for an fp16 product a row is scaled by a power of two.
//
// A position that a row does not see never touches it, NaN and infinity included: scores are replaced, and where a
// tile has positions that some rows see and others do not, the second product is formed for one token's rows at a time
// with the values that it does not see set to zero.
#pragma once

#include <algorithm>

#include "qs_cache.cuh"

namespace qs {

namespace attn {

constexpr float kSlack = 8.0f;    // a row's maximum may lag behind by this much (log2) before the sums are scaled
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kSmemMax = 227 * 1024;
constexpr int kFan = 12;          // parts of an item that one CTA joins at a time
constexpr int kMostTeams = 16;
constexpr int kStatic = 7 * 1024;  // shared memory for tables

// A kernel's sizes: cache type, columns (head_dim rounded up), 8 rows times NT a warp, teams of R warps with rows of their
// own times C with columns of their own, W warps a CTA, and whether queries and weights go into the products with all
// their parts.
template <bool E4_, int DP_, int NT_, int R_, int C_, int W_, bool WIDE_>
struct Plan {
    static constexpr bool E4 = E4_, WIDE = WIDE_;
    static constexpr int DP = DP_, NT = NT_, R = R_, C = C_, kWarps = W_;
    static constexpr int kRowBytes = DP * (E4 ? 1 : 2), kChunks = kRowBytes / 16;
    static constexpr int kTeam = R * C, kTeams = kWarps / kTeam, kRows = 8 * NT, RT = R * kRows, kCols = DP / C;
    static constexpr int TP = kRowBytes <= 64 || (R == 4 && kRowBytes <= 256) ? 32 : 16;
    static constexpr int kStage = 2 * TP * kRowBytes + (E4 ? 2 * TP * 4 : 0);  // keys, values, their scales
    static constexpr int QP = WIDE ? (E4 ? 2 : 3) : 1, PP = WIDE ? (E4 ? 2 : 3) : (E4 ? 1 : 2);
    static constexpr int kSteps = DP / 16;            // of the first product
    // The queries' fragments.  NT = 1: two parts share one, the second in the rows 8..15, which are empty.  In registers
    // where they fit beside the sums and about 80 others, else in shared memory.
    static constexpr int kQAll = NT == 1 ? (QP + 1) / 2 : QP;        // fragments of a step
    static constexpr int kQEach = NT == 1 ? 2 * QP : 4 * QP;         // registers of a step
    static constexpr bool kQInRegs = kQEach * kSteps <= 65536 / (32 * kWarps) - 80 - kCols * NT / 4;
    static constexpr int kQBytes = kQInRegs ? 0 : kWarps * kQAll * kSteps * 32 * 16;
    static constexpr int kRed = kTeams * RT * (DP + 4) * 4 + kTeams * RT * 8;  // the teams' results, over all of it
    static constexpr int kFit = (kSmemMax - kStatic - kQBytes) / (kTeams * kStage);
    static constexpr int ST = kFit > 6 ? 6 : kFit;
    static constexpr int kRing = kTeams * ST * kStage;
    static constexpr int kSmem = kQBytes + kRing > kRed ? kQBytes + kRing : kRed;
    static constexpr int kEnter = 2;
    static constexpr int kPart = RT * (DP + 2);       // floats of an item's part: sums, maxima and sums of weights
    static_assert(ST >= 2 && kSmem + kStatic <= kSmemMax, "shared memory");
    static_assert(kWarps % kTeam == 0 && 32 * kTeam % kChunks == 0 && TP * kChunks % (32 * kTeam) == 0, "copies");
    static_assert(kTeams <= kMostTeams && kTeams <= 16 && kCols % 64 == 0, "teams");
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
// Warps that wait for one another: `warps` of them at barrier `id` (1 .. 8).
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

// Two e4m3 codes as fp16.
__device__ __forceinline__ uint32_t widen(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)two));
    return r;
}

// Two values as their 16-bit roundings, and what these leave out.
template <bool E4>
__device__ __forceinline__ uint32_t part(float& lo, float& hi) {
    if (E4) {
        const __half2 h = __floats2half2_rn(lo, hi);
        const float2 f = __half22float2(h);
        lo -= f.x;
        hi -= f.y;
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const uint32_t w = pack_bf16(lo, hi);
    lo -= bf16_lo(w);
    hi -= bf16_hi(w);
    return w;
}

// One of a row's eight-element pieces as fp32; zeros past n.
__device__ __forceinline__ void load_q8(const HeadsView& x, bool aligned, const uint8_t* row, int i, int n, float (&v)[8]) {
    if (!row || i >= n) {
#pragma unroll
        for (int q = 0; q < 8; q++) v[q] = 0.0f;
    } else if (aligned) {
        load8_row<true>(row, x.dtype, i, n, v);
    } else {
#pragma unroll
        for (int q = 0; q < 8; q++)
            v[q] = x.dtype == QS_BF16 ? bf16_lo(reinterpret_cast<const uint16_t*>(row)[i + q]) : reinterpret_cast<const float*>(row)[i + q];
    }
}

// What a sequence has to do.  Positions are 32-bit numbers near enough to the table's (0 .. positions): a start far outside
// it is brought so near that its tokens see the same.
struct Seq {
    int first_token, tokens;  // the new tokens that are attended (max_new at most)
    int lo_base, hi_base;     // token j sees lo_base + j .. hi_base + j - 1, clipped to the table
    int lo;                   // the first position that any of them sees
    int tiles, row_tiles;     // of an item; row tiles of a head
};
// a / b, b > 0, a >= 0, in 32 bits where both fit.
__device__ __forceinline__ int64_t div_of(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}
__device__ __forceinline__ int near_pos(int64_t p, int n) { return (int)(p < -1024 ? -1024 : p > n ? n : p); }
__device__ __forceinline__ int clip_pos(int p, int n) { return min(max(p, 0), n); }

template <int TP, int RT>
__device__ __forceinline__ Seq seq_of(const AttnArgs& p, int s) {
    Seq q;
    q.first_token = s;
    q.tokens = 1;
    if (p.seqs.offsets) {
        q.first_token = min(max(p.seqs.offsets[s], 0), p.n_tokens);
        q.tokens = min(max(min(p.seqs.offsets[s + 1], p.n_tokens) - q.first_token, 0), p.max_new);
    }
    const int64_t start = p.seqs.starts ? p.seqs.starts[s] : 0;
    const int n = p.seqs.positions;
    q.lo_base = p.window ? near_pos(start - p.window + 1, n) : -1024;
    q.hi_base = near_pos(start + 1, n);
    q.lo = clip_pos(q.lo_base, n);
    q.tiles = max(1, (clip_pos(q.hi_base + q.tokens - 1, n) + TP - 1) / TP - q.lo / TP);  // one where nothing is seen: its rows are still written
    q.row_tiles = (q.tokens * p.group + RT - 1) / RT;
    return q;
}

// Four of an output row's columns from col: v is the sum of weighted values, l the sum of weights, m the maximum they are
// relative to.
__device__ __forceinline__ void finish(const AttnArgs& p, int token, int head, int col, float (&v)[4], float m, float l, bool real) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int q = 0; q < 4; q++) v[q] = l == 0.0f ? 0.0f : v[q] * inv;
    const int d = p.cache.head_dim;
    if (p.codes) {  // head_dim a multiple of 128: a warp has a scale's columns
        const BlockCode code(lanes_max(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))), 16), 1.0f, kMinAmax);
        if (real) {
            const int i = head * d + col;
            *reinterpret_cast<uint32_t*>(p.codes + token * p.codes_stride + i) = code.pair(v[0], v[1]) | (code.pair(v[2], v[3]) << 16);
            if (i % kScaleCols == 0) p.codes_scale[token * p.codes_scale_stride + i / kScaleCols] = code.scale;
        }
    }
    if (!real || col >= d) return;
    if (p.out.data) {
        uint8_t* row = p.out.data + token * p.out.token_stride + head * p.out.head_stride;
        if (!p.out_aligned) {
#pragma unroll
            for (int q = 0; q < 4; q++) {
                if (p.out.dtype == QS_BF16) reinterpret_cast<__nv_bfloat16*>(row)[col + q] = __float2bfloat16_rn(v[q]);
                else reinterpret_cast<float*>(row)[col + q] = v[q];
            }
        } else if (p.out.dtype == QS_BF16) {
            *reinterpret_cast<uint2*>(row + 2 * col) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        } else {
            *reinterpret_cast<float4*>(row + 4 * col) = make_float4(v[0], v[1], v[2], v[3]);
        }
    }
    if (p.lse && col == 0) p.lse[(int64_t)token * p.n_heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// The token of an item's row.
__device__ __forceinline__ int token_of(const AttnArgs& p, int row) { return fast_div(row, p.group_div); }

// An item's rows from the registers of the warps that have all their positions.  most: the warps' largest values by row, for
// the codes of 128 columns that two warps have.
template <class P>
__device__ __forceinline__ void finish_rows(const AttnArgs& p, const Seq& seq, int kv, int w0, int rows, const float (&top)[P::NT], const float (&sum)[P::NT],
                                            float (&acc)[P::kCols / 64][4][P::NT][4], float (*most)[8 * P::NT], int team) {
    constexpr int NT = P::NT, kJ = P::kCols / 64;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3, d = p.cache.head_dim;
    const int col0 = warp % P::C * P::kCols;
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
        const float inv = sum[nt] == 0.0f ? 0.0f : 1.0f / sum[nt];
        const int own = w0 + nt * 8 + g;
        if (p.lse && t == 0 && col0 == 0 && own < rows)
            p.lse[(int64_t)(seq.first_token + token_of(p, own)) * p.n_heads + kv * p.group + (own - token_of(p, own) * p.group)] = sum[nt] == 0.0f ? -INFINITY : (top[nt] + log2f(sum[nt])) * kLn2;
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const float by = __shfl_sync(0xffffffffu, inv, 8 * t + 4 * e);
#pragma unroll
            for (int jj = 0; jj < kJ; jj++)
#pragma unroll
                for (int q = 0; q < 8; q++) {
                    float& x = acc[jj][q / 2][nt][q % 2 * 2 + e];
                    x = by == 0.0f ? 0.0f : x * by;
                }
        }
    }
    const bool shared_scale = P::kCols < kScaleCols && P::C > 1 && p.codes;
    if (shared_scale) {
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                float a = 0.0f;
#pragma unroll
                for (int q = 0; q < 8; q++) a = fmaxf(a, fabsf(acc[0][q / 2][nt][q % 2 * 2 + e]));
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
                if (g == 0) most[warp][nt * 8 + 2 * t + e] = a;
            }
        sync_warps(1 + team, P::kTeam);
    }
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const int row = w0 + nt * 8 + 2 * t + e;
            const bool real = row < rows;
            const int at = token_of(p, row), head = kv * p.group + row - at * p.group;
            const int64_t token = seq.first_token + at;
            auto columns = [&](int jj, float (&v)[8]) {
#pragma unroll
                for (int q = 0; q < 8; q++) v[q] = acc[jj][q / 2][nt][q % 2 * 2 + e];
            };
            if (P::DP >= kScaleCols && p.codes) {  // a scale's columns are in the eight lanes of the same t, eight or twice eight each
                constexpr int kEach = kJ >= 2 ? 2 : 1;
#pragma unroll
                for (int b = 0; b < kJ; b += kEach) {
                    float a = 0.0f;
                    if (shared_scale) {
                        a = fmaxf(most[warp][nt * 8 + 2 * t + e], most[warp ^ 1][nt * 8 + 2 * t + e]);
                    } else {
#pragma unroll
                        for (int k = 0; k < kEach; k++)
#pragma unroll
                            for (int q = 0; q < 8; q++) a = fmaxf(a, fabsf(acc[(b + k) % kJ][q / 2][nt][q % 2 * 2 + e]));
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
                    }
                    const BlockCode code(a, 1.0f, kMinAmax);
                    if (!real || col0 + 64 * b >= d) continue;
                    if (g == 0 && (col0 + 64 * b) % kScaleCols == 0) p.codes_scale[token * p.codes_scale_stride + (head * d + col0 + 64 * b) / kScaleCols] = code.scale;
#pragma unroll
                    for (int k = 0; k < kEach; k++) {
                        float x[8];
                        columns((b + k) % kJ, x);
                        *reinterpret_cast<uint2*>(p.codes + token * p.codes_stride + head * d + col0 + 64 * (b + k) + 8 * g) =
                            make_uint2(code.pair(x[0], x[1]) | (code.pair(x[2], x[3]) << 16), code.pair(x[4], x[5]) | (code.pair(x[6], x[7]) << 16));
                    }
                }
            }
            if (!real || !p.out.data) continue;
            uint8_t* to = p.out.data + token * p.out.token_stride + head * p.out.head_stride;
#pragma unroll
            for (int jj = 0; jj < kJ; jj++) {
                const int col = col0 + 64 * jj + 8 * g;
                if (col >= d) continue;
                float v[8];
                columns(jj, v);
                if (p.out_aligned) {
                    store8_row<true>(to, p.out.dtype, col, d, v);
                } else {
#pragma unroll
                    for (int q = 0; q < 8; q++) {
                        if (p.out.dtype == QS_BF16) reinterpret_cast<__nv_bfloat16*>(to)[col + q] = __float2bfloat16_rn(v[q]);
                        else reinterpret_cast<float*>(to)[col + q] = v[q];
                    }
                }
            }
        }
}

// What a team has of an item that is not whole in its run: where the item begins in the line (-1: nothing), and which.
struct Piece {
    int64_t at;
    int seq, item;
};
// A tile in the ring: positions that are there, the first one, and whether it is the first or last of a stretch (the item's
// or the run's); the item, the tile's number in it, and where it begins in the line, from the run's start.
struct Tile {
    unsigned there;
    int pos0, first, last;
    int seq, item, tile, at;
};

// What a part with maximum ml.x counts beside the maximum m; one of no positions (-infinity, 0) nothing.
__device__ __forceinline__ float part_factor(float2 ml, float m) { return ml.x == -INFINITY ? (ml.y == 0.0f ? 0.0f : 1.0f) : ex2(ml.x - m); }

template <class P>
__global__ void __launch_bounds__(32 * P::kWarps, 1) attn_kernel(const AttnArgs p) {
    constexpr bool E4 = P::E4;
    constexpr int DP = P::DP, NT = P::NT, RT = P::RT, TP = P::TP, ST = P::ST, NC = P::kChunks, kJ = P::kCols / 64;
    constexpr int kWarps = P::kWarps, kThreads = 32 * kWarps;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t scan[kWarps], found_base[P::kTeams];
    __shared__ int found_seq[P::kTeams];
    __shared__ Tile tile_of[kWarps][ST];
    __shared__ Piece piece_of[2 * P::kTeams];  // of each team: the stretch that begins inside an item and ends with it; the run's last
    __shared__ float most_of[kWarps][8 * NT];
    __shared__ bool last_of[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int team = warp / P::kTeam, team_tid = tid % (32 * P::kTeam), row_warp = warp % P::kTeam / P::C, col_warp = warp % P::C;
    const int d = p.cache.head_dim;
    uint8_t* const q_shared = smem + warp * (P::kQBytes / kWarps) + lane * 16;
    uint8_t* const ring = smem + P::kQBytes + team * ST * P::kStage;
    float* const red = reinterpret_cast<float*>(smem);
    float2* const red_ml = reinterpret_cast<float2*>(red + P::kTeams * RT * (DP + 4));
    pdl_wait();
    pdl_launch_next();

    // ---- the CTA's run of the line [run0, run1), the team's share of it, and the sequence that this begins in.  An item
    // takes kEnter places before its tiles', about what entering and leaving it costs.
    const int per = (p.seqs.n_seqs + kThreads - 1) / kThreads;
    const int s0 = min(tid * per, p.seqs.n_seqs), s1 = min(s0 + per, p.seqs.n_seqs);
    auto places_of = [&](const Seq& q) { return (int64_t)(q.tiles + P::kEnter) * (q.row_tiles * p.cache.n_kv); };
    int64_t mine = 0;
    for (int s = s0; s < s1; s++) mine += places_of(seq_of<TP, RT>(p, s));
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) scan[warp] = upto;
    if (tid < 2 * P::kTeams) piece_of[tid].at = -1;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
        if (w < warp) upto += scan[w];
        total += scan[w];
    }
    // as many CTAs as have an item's first tile for each team
    const int64_t workers = min((int64_t)gridDim.x, div_of(total - 1, P::kTeams * (P::kEnter + 1)) + 1);
    const int c = blockIdx.x;
    if (total == 0 || c >= workers) return;
    // equal runs, the first of them a place longer
    const int64_t each = div_of(total, workers), longer = total - each * workers;
    const int64_t run0 = c * each + min((int64_t)c, longer), run1 = run0 + each + (c < longer);
    auto cta_of = [&](int64_t place) {  // the CTA whose run has it
        const int64_t split = longer * (each + 1);
        return (int)(place < split ? div_of(place, each + 1) : longer + div_of(place - split, each));
    };
    const unsigned length = (unsigned)(run1 - run0);
    auto begin_of = [&](unsigned x) { return length / P::kTeams * x + length % P::kTeams * x / P::kTeams; };
    // the threads whose sequences the teams begin in say so
    if (upto > run0 && upto - mine < run1) {
        for (unsigned w = 0; w < P::kTeams; w++) {
            const int64_t from = run0 + begin_of(w);
            if (from < upto - mine || from >= upto) continue;
            int64_t base = upto - mine;
            int s = s0;
            for (; s + 1 < s1; s++) {
                const int64_t x = places_of(seq_of<TP, RT>(p, s));
                if (from < base + x) break;
                base += x;
            }
            found_base[w] = base;
            found_seq[w] = s;
        }
    }
    __syncthreads();
    const int64_t from = run0 + begin_of(team);

    // ---- copies: the next tile's place, kept by all warps of a team alike
    struct {
        int seq, item, items, kv, tile, tiles, left, base_pos, lo, hi, at;
        bool first;
        const uint8_t *k, *v;
    } next = {};
    int issued = 0;
    Place ahead = {-1, -1};
    auto hi_of = [&](const Seq& q, int token) { return clip_pos(q.hi_base + token, p.seqs.positions); };
    auto lo_of = [&](const Seq& q, int token) { return clip_pos(q.lo_base + token, p.seqs.positions); };
    // an item's key-value head and first row
    auto rows_of = [&](const Seq& q, int item, int& kv, int& row0) {
        kv = item;
        row0 = 0;
        if (q.row_tiles != 1) {
            kv = item / q.row_tiles;
            row0 = (item - kv * q.row_tiles) * RT;
        }
    };
    const int chunk = team_tid % NC, chunk_row = team_tid / NC;
    const bool chunk_in = chunk * 16 < d * (E4 ? 1 : 2);
    auto enter = [&](const Seq& q) {
        int row0;
        rows_of(q, next.item, next.kv, row0);
        next.items = q.row_tiles * p.cache.n_kv;
        next.tiles = q.tiles;
        next.base_pos = q.lo / TP * TP;
        next.lo = lo_of(q, token_of(p, row0));
        next.hi = hi_of(q, token_of(p, min(row0 + RT, q.tokens * p.group) - 1));
        next.k = p.cache.k + next.kv * p.cache.head_stride + (chunk_in ? chunk * 16 : 0);
        next.v = p.cache.v + next.kv * p.cache.head_stride + (chunk_in ? chunk * 16 : 0);
    };
    auto look = [&]() {
        const int pos = next.base_pos + next.tile * TP + lane % TP;
        ahead = Place{-1, -1};
        if (next.left > 0 && pos >= next.lo && pos < next.hi) ahead = place_of(p.cache, p.seqs, next.seq, pos);
    };
    const int run = (int)(begin_of(team + 1) - begin_of(team));
    if (run > 0) {
        next.seq = found_seq[team];
        const Seq q = seq_of<TP, RT>(p, next.seq);
        const int64_t in = from - found_base[team];
        next.item = (int)div_of(in, q.tiles + P::kEnter);
        const int place = (int)(in - (int64_t)next.item * (q.tiles + P::kEnter));
        next.tile = max(0, place - P::kEnter);
        next.left = run - max(0, P::kEnter - place);
        next.at = -place;
        next.first = true;
        enter(q);
        look();
    }
    auto issue = [&](int i) {
        if (next.left > 0) {
            const int stage = i % ST;
            const unsigned there = __ballot_sync(0xffffffffu, ahead.at >= 0);
            const bool ends = next.tile + 1 == next.tiles;
            if (lane == 0) tile_of[warp][stage] = Tile{there, next.base_pos + next.tile * TP, next.first, ends || next.left == 1, next.seq, next.item, ends ? -1 - next.tile : next.tile, next.at};
            const uint32_t to = smem_u32(ring + stage * P::kStage);
#pragma unroll
            for (int k = 0; k < TP * NC / (32 * P::kTeam); k++) {
                const int row = chunk_row + k * (32 * P::kTeam / NC);
                const int64_t at = __shfl_sync(0xffffffffu, ahead.at, row);
                const bool ok = at >= 0 && chunk_in;
                const int64_t from_base = ok ? at : 0;
                cp16(to + row * P::kRowBytes + ((chunk ^ (NC >= 8 ? (row & 1) * 4 : 0)) * 16), next.k + from_base, ok);
                cp16(to + (TP + row) * P::kRowBytes + ((chunk ^ (((row >> 1) & 3) * 2 & (NC - 1))) * 16), next.v + from_base, ok);
            }
            if (E4 && warp % P::kTeam == 0 && lane < TP) {
                const bool ok = ahead.at >= 0;
                const int64_t from_base = ok ? ahead.scale_at + next.kv * p.cache.scale_head_stride : 0;
                cp4(to + 2 * TP * P::kRowBytes + lane * 4, p.cache.k_scale + from_base, ok);
                cp4(to + 2 * TP * P::kRowBytes + (TP + lane) * 4, p.cache.v_scale + from_base, ok);
            }
            issued++;
            next.left--;
            next.tile++;
            next.first = ends;
            if (ends) {
                next.left -= P::kEnter;
                if (next.left > 0) {
                    next.at += next.tiles + P::kEnter;
                    next.tile = 0;
                    Seq q;
                    if (++next.item == next.items) {
                        next.item = 0;
                        do {
                            next.seq = min(next.seq + 1, p.seqs.n_seqs - 1);
                            q = seq_of<TP, RT>(p, next.seq);
                        } while (q.tokens == 0 && next.seq + 1 < p.seqs.n_seqs);
                    } else {
                        q = seq_of<TP, RT>(p, next.seq);
                    }
                    enter(q);
                }
            }
            look();
        }
        cp_commit();
    };

    // ---- the pass over the run's tiles
    Seq seq = {};
    int kv = 0, w0 = 0, rows = 0, token0 = 0, token1 = 0, all_lo = 0, all_hi = 0, tile_lo = 0, tile_hi = 0, tile0 = 0;
    bool active = false;
    uint32_t qf[P::kQInRegs ? P::kSteps : 1][P::kQInRegs ? P::kQEach : 1];
    float row_scale[NT];
    float acc[kJ][4][NT][4];  // [64 columns][their pair][rows]: columns 64 jj + 8 g + 2 m (+ 1), rows 2 t, 2 t + 1
    float top[NT], sum[NT];

    // an item's rows: queries as fragments in the order in which the keys' pieces lie
    auto begin = [&](const Tile& x) {
        seq = seq_of<TP, RT>(p, x.seq);
        tile0 = x.tile < 0 ? -1 - x.tile : x.tile;
        int row0;
        rows_of(seq, x.item, kv, row0);
        rows = seq.tokens * p.group;
        tile_lo = lo_of(seq, token_of(p, row0));
        tile_hi = hi_of(seq, token_of(p, min(row0 + RT, rows) - 1));
        w0 = row0 + row_warp * P::kRows;
        active = w0 < rows;
        token0 = token_of(p, w0);
        token1 = max(token_of(p, max(min(w0 + P::kRows, rows) - 1, 0)), token0);
        all_lo = lo_of(seq, token1);
        all_hi = hi_of(seq, token0);
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            top[nt] = -INFINITY;
            sum[nt] = 0.0f;
            const int row = w0 + nt * 8 + g;
            const int at = token_of(p, row);
            const uint8_t* q = row < rows ? p.q.data + (seq.first_token + at) * p.q.token_stride + (kv * p.group + row - at * p.group) * p.q.head_stride : nullptr;
            row_scale[nt] = p.scale;
            if constexpr (!E4 && !P::WIDE) {  // bf16 as it lies, by the rule below
                uint4 raw[DP / 32];
#pragma unroll
                for (int i = 0; i < DP / 32; i++) {
                    const int col = 32 * i + 8 * t;
                    raw[i] = make_uint4(0, 0, 0, 0);
                    if (!q || col >= d) continue;
                    if (p.q_aligned) {
                        raw[i] = *reinterpret_cast<const uint4*>(q + 2 * col);
                    } else {
                        const uint16_t* e = reinterpret_cast<const uint16_t*>(q) + col;
                        raw[i] = make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16, e[4] | (uint32_t)e[5] << 16, e[6] | (uint32_t)e[7] << 16);
                    }
                }
#pragma unroll
                for (int i = 0; i < DP / 32; i++)
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const uint32_t x0 = h ? raw[i].z : raw[i].x, x1 = h ? raw[i].w : raw[i].y;
                        constexpr int kE = P::kQInRegs ? P::kQEach : 1;
                        if (P::kQInRegs) {
                            uint32_t(&to)[kE] = qf[(2 * i + h) % (P::kQInRegs ? P::kSteps : 1)];
                            to[nt % kE] = x0;
                            to[(NT + nt) % kE] = x1;
                        } else {
                            uint32_t* shared = reinterpret_cast<uint32_t*>(q_shared + (2 * i + h) * 512);
                            if (NT == 1) {
                                *reinterpret_cast<uint4*>(shared) = make_uint4(x0, 0u, x1, 0u);
                            } else {
                                shared[nt] = x0;
                                shared[2 + nt] = x1;
                            }
                        }
                    }
            } else {
            // bf16: piece i is columns 32 i + 8 t .. + 7, two steps of four; e4m3: 64 i + 16 t .. + 15, four steps
            float v[DP / 32][8];
#pragma unroll
            for (int i = 0; i < DP / 32; i++) load_q8(p.q, p.q_aligned, q, E4 ? 64 * (i / 2) + 16 * t + 8 * (i % 2) : 32 * i + 8 * t, d, v[i]);
            float factor = 1.0f;
            if (E4) {  // a power of two that brings the row's largest into fp16's upper range
                float a = 0.0f;
#pragma unroll
                for (int i = 0; i < DP / 32; i++)
#pragma unroll
                    for (int e = 0; e < 8; e++) a = fmaxf(a, fabsf(v[i][e]));
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
                const int e = min(max(14 - ((int)(__float_as_uint(a) >> 23) - 127), -100), 100);
                factor = __uint_as_float((uint32_t)(127 + e) << 23);
                row_scale[nt] = p.scale * __uint_as_float((uint32_t)(127 - e) << 23);
            }
#pragma unroll
            for (int i = 0; i < DP / 32; i++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int step = 2 * i + h;
                    float* x = v[i] + 4 * h;
#pragma unroll
                    for (int e = 0; e < 4; e++) x[e] *= factor;
#pragma unroll
                    for (int f = 0; f < P::kQAll; f++) {  // a fragment: rows g, g + 8, the same of the upper columns
                        uint32_t lo[2] = {0u, 0u}, hi[2] = {0u, 0u};
#pragma unroll
                        for (int y = 0; y < (NT == 1 ? 2 : 1); y++)
                            if (NT == 2 || 2 * f + y < P::QP) {
                                lo[y] = part<E4>(x[0], x[1]);
                                hi[y] = part<E4>(x[2], x[3]);
                            }
                        constexpr int kE = P::kQInRegs ? P::kQEach : 1;
                        uint32_t(&to)[kE] = qf[step % (P::kQInRegs ? P::kSteps : 1)];
                        uint32_t* shared = reinterpret_cast<uint32_t*>(q_shared + (f * P::kSteps + step) * 512);
                        if (P::kQInRegs) {
                            // NT = 1: a part's two; NT = 2: the four of a part for both rows
                            if (NT == 1) {
#pragma unroll
                                for (int y = 0; y < 2; y++)
                                    if (2 * f + y < P::QP) {
                                        to[(4 * f + 2 * y) % kE] = lo[y];
                                        to[(4 * f + 2 * y + 1) % kE] = hi[y];
                                    }
                            } else {
                                to[(4 * f + nt) % kE] = lo[0];
                                to[(4 * f + 2 + nt) % kE] = hi[0];
                            }
                        } else if (NT == 1) {
                            *reinterpret_cast<uint4*>(shared) = make_uint4(lo[0], lo[1], hi[0], hi[1]);
                        } else {
                            shared[nt] = lo[0];
                            shared[2 + nt] = hi[0];
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int jj = 0; jj < kJ; jj++)
#pragma unroll
            for (int m = 0; m < 4; m++)
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int e = 0; e < 4; e++) acc[jj][m][nt][e] = 0.0f;
    };
    // one step of the first product: a key's piece with every part of the queries
    auto score = [&](float (&c4)[4], int step, uint32_t b0, uint32_t b1) {
#pragma unroll
        for (int f = 0; f < P::kQAll; f++) {
            if (P::kQInRegs) {
                constexpr int kE = P::kQInRegs ? P::kQEach : 1;
                const uint32_t(&q)[kE] = qf[step % (P::kQInRegs ? P::kSteps : 1)];
                if (NT == 2) mma<E4>(c4, q[4 * f % kE], q[(4 * f + 1) % kE], q[(4 * f + 2) % kE], q[(4 * f + 3) % kE], b0, b1);
                else if (2 * f + 1 < P::QP) mma<E4>(c4, q[4 * f % kE], q[(4 * f + 2) % kE], q[(4 * f + 1) % kE], q[(4 * f + 3) % kE], b0, b1);
                else mma<E4>(c4, q[4 * f % kE], 0u, q[(4 * f + 1) % kE], 0u, b0, b1);
            } else {
                const uint4 x = *reinterpret_cast<const uint4*>(q_shared + (f * P::kSteps + step) * 512);
                mma<E4>(c4, x.x, x.y, x.z, x.w, b0, b1);
            }
        }
    };
    // the rows' sums to where they are joined: [rows x stride], maxima and sums of weights at ml
    auto put = [&](float* to, int stride, float2* ml) {
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            const int row = row_warp * P::kRows + nt * 8;
            if (t == 0 && col_warp == 0) ml[row + g] = make_float2(top[nt], sum[nt]);
#pragma unroll
            for (int jj = 0; jj < kJ; jj++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float4* at = reinterpret_cast<float4*>(to + (row + 2 * t + e) * stride + col_warp * P::kCols + 64 * jj + 8 * g);
                    at[0] = make_float4(acc[jj][0][nt][e], acc[jj][0][nt][e + 2], acc[jj][1][nt][e], acc[jj][1][nt][e + 2]);
                    at[1] = make_float4(acc[jj][2][nt][e], acc[jj][2][nt][e + 2], acc[jj][3][nt][e], acc[jj][3][nt][e + 2]);
                }
        }
    };

    for (int i = 1 - ST; i < 0 || i < issued; i++) {  // tile i is consumed, tile i + ST - 1 copied
        const int stage = i < 0 ? 0 : i % ST;
        const Tile& x = tile_of[warp][stage];
        if (i >= 0) {
            __syncwarp();
            if (x.first) begin(x);  // the queries are on their way with the tile
            cp_wait<ST - 2>();
            sync_warps(1 + team, P::kTeam);
        }
        issue(i + ST - 1);
        if (i < 0) continue;
        const unsigned there = x.there;
        const int pos0 = x.pos0;
        if (active) {
            const uint8_t* const keys = ring + stage * P::kStage;
            const uint8_t* const values = keys + TP * P::kRowBytes;
            const float* const scales = reinterpret_cast<const float*>(values + TP * P::kRowBytes);
            const unsigned whole = TP == 32 ? 0xffffffffu : (1u << (TP & 31)) - 1u;
            const bool full = (there & whole) == whole && pos0 >= all_lo && pos0 + TP <= all_hi;

            float sc[TP / 8][4];
#pragma unroll
            for (int n8 = 0; n8 < TP / 8; n8++)
#pragma unroll
                for (int e = 0; e < 4; e++) sc[n8][e] = 0.0f;
#pragma unroll
            for (int i4 = 0; i4 < NC / 4; i4++)
#pragma unroll
                for (int n8 = 0; n8 < TP / 8; n8++) {
                    const int row = n8 * 8 + g;
                    const uint4 w = *reinterpret_cast<const uint4*>(keys + row * P::kRowBytes + (((4 * i4 + t) ^ (NC >= 8 ? (row & 1) * 4 : 0)) * 16));
                    const uint32_t r4[4] = {w.x, w.y, w.z, w.w};
                    if (E4) {
#pragma unroll
                        for (int h = 0; h < 4; h++) score(sc[n8], 4 * i4 + h, widen(r4[h]), widen(r4[h] >> 16));
                    } else {
                        score(sc[n8], 2 * i4, r4[0], r4[1]);
                        score(sc[n8], 2 * i4 + 1, r4[2], r4[3]);
                    }
                }
            float2 vs[TP / 8];
#pragma unroll
            for (int n8 = 0; n8 < TP / 8; n8++) {
                if (NT == 1 && P::QP > 1) {  // the second part's rows
                    sc[n8][0] += sc[n8][2];
                    sc[n8][1] += sc[n8][3];
                }
#pragma unroll
                for (int e = 0; e < 2 * NT; e++) sc[n8][e] *= row_scale[e / 2];
                if (E4) {
                    const float2 ks = *reinterpret_cast<const float2*>(scales + n8 * 8 + 2 * t);
                    vs[n8] = *reinterpret_cast<const float2*>(scales + TP + n8 * 8 + 2 * t);
#pragma unroll
                    for (int e = 0; e < 2 * NT; e++) sc[n8][e] *= e % 2 ? ks.y : ks.x;
                }
            }
            if (!full) {
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    const int token = token_of(p, w0 + nt * 8 + g);
                    const int lo = lo_of(seq, token), hi = hi_of(seq, token);
#pragma unroll
                    for (int n8 = 0; n8 < TP / 8; n8++)
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            const int at = n8 * 8 + 2 * t + e;
                            if (!((there >> at) & 1u) || pos0 + at < lo || pos0 + at >= hi) sc[n8][2 * nt + e] = -INFINITY;
                        }
                }
            }
            // the values' scales count for the maximum, as within 2^-100 .. 2^118: the weight's two factors stay in fp32's range
            float2 lv[TP / 8];
#pragma unroll
            for (int n8 = 0; n8 < TP / 8; n8++) {
                lv[n8] = make_float2(0.0f, 0.0f);
                if (E4) lv[n8] = make_float2(fminf(fmaxf(lg2(vs[n8].x), -100.0f), 118.0f), fminf(fmaxf(lg2(vs[n8].y), -100.0f), 118.0f));
            }
            bool grown = false;
            float most[NT];
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                float a = -INFINITY;
#pragma unroll
                for (int n8 = 0; n8 < TP / 8; n8++) a = fmaxf(a, fmaxf(sc[n8][2 * nt] + lv[n8].x, sc[n8][2 * nt + 1] + lv[n8].y));
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
                most[nt] = a;
                grown |= a > top[nt] + kSlack;
            }
            if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    const float now = fmaxf(top[nt], most[nt]);
                    const float by = now == top[nt] ? 1.0f : ex2(top[nt] - now);
                    top[nt] = now;
                    sum[nt] *= by;
                    const float b0 = __shfl_sync(0xffffffffu, by, 8 * t), b1 = __shfl_sync(0xffffffffu, by, 8 * t + 4);
#pragma unroll
                    for (int jj = 0; jj < kJ; jj++)
#pragma unroll
                        for (int m = 0; m < 4; m++) {
                            acc[jj][m][nt][0] *= b0;
                            acc[jj][m][nt][1] *= b1;
                            acc[jj][m][nt][2] *= b0;
                            acc[jj][m][nt][3] *= b1;
                        }
                }
            }
            uint32_t pb[TP / 16][NT][P::PP][2];
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                const float ref = top[nt] == -INFINITY ? 0.0f : top[nt];
#pragma unroll
                for (int n8 = 0; n8 < TP / 8; n8++) {
                    float a = ex2(sc[n8][2 * nt] - ref), b = ex2(sc[n8][2 * nt + 1] - ref);
                    sum[nt] += a + b;
                    if (E4) {  // a weight of 0 stays 0 beside whatever scale a position has that is not seen
                        a = sc[n8][2 * nt] == -INFINITY ? 0.0f : a * vs[n8].x;
                        b = sc[n8][2 * nt + 1] == -INFINITY ? 0.0f : b * vs[n8].y;
                    }
#pragma unroll
                    for (int pl = 0; pl < P::PP; pl++) pb[n8 / 2][nt][pl][n8 % 2] = part<E4>(a, b);
                }
            }
            // positions here that one of the warp's rows does not see and that were copied for another
            const bool mixed = !full && (min(pos0 + TP, tile_hi) > all_hi || max(pos0, tile_lo) < all_lo);
            // four positions' eight columns, and a pair of these as the product's operand
            constexpr int kW = E4 ? 2 : 4;
            auto load_values = [&](int kk, int jj, uint32_t (&w)[4][kW]) {
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const int row = kk * 16 + 2 * t + (r & 1) + (r >> 1) * 8;
                    if (E4) {
                        const uint2 y = *reinterpret_cast<const uint2*>(values + row * P::kRowBytes + (((4 * (jj + col_warp * kJ) + g / 2) ^ (((row >> 1) & 3) * 2 & (NC - 1))) * 16) + (g & 1) * 8);
                        w[r][0] = y.x;
                        w[r][1] = y.y;
                    } else {
                        const uint4 y = *reinterpret_cast<const uint4*>(values + row * P::kRowBytes + (((8 * (jj + col_warp * kJ) + g) ^ (((row >> 1) & 3) * 2)) * 16));
                        w[r][0] = y.x;
                        w[r][1] = y.y;
                        w[r][2 % kW] = y.z;
                        w[r][3 % kW] = y.w;
                    }
                }
            };
            auto pair_of = [&](const uint32_t (&w)[4][kW], int m, uint32_t (&a)[4]) {
                if (E4) {
                    const uint32_t y = __byte_perm(w[0][m / 2], w[1][m / 2], m % 2 ? 0x7362 : 0x5140);
                    const uint32_t z = __byte_perm(w[2][m / 2], w[3][m / 2], m % 2 ? 0x7362 : 0x5140);
                    a[0] = widen(y);
                    a[1] = widen(y >> 16);
                    a[2] = widen(z);
                    a[3] = widen(z >> 16);
                } else {
                    a[0] = __byte_perm(w[0][m % kW], w[1][m % kW], 0x5410);
                    a[1] = __byte_perm(w[0][m % kW], w[1][m % kW], 0x7632);
                    a[2] = __byte_perm(w[2][m % kW], w[3][m % kW], 0x5410);
                    a[3] = __byte_perm(w[2][m % kW], w[3][m % kW], 0x7632);
                }
            };
            if (!mixed) {
#pragma unroll
                for (int kk = 0; kk < TP / 16; kk++)
#pragma unroll
                    for (int jj = 0; jj < kJ; jj++) {
                        uint32_t w[4][kW];
                        load_values(kk, jj, w);
#pragma unroll
                        for (int m = 0; m < 4; m++) {
                            uint32_t a[4];
                            pair_of(w, m, a);
#pragma unroll
                            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                                for (int pl = 0; pl < P::PP; pl++) mma<E4>(acc[jj][m][nt], a[0], a[1], a[2], a[3], pb[kk][nt][pl][0], pb[kk][nt][pl][1]);
                        }
                    }
            } else {
#pragma unroll 1
                for (int token = token0; token <= token1; token++) {
                    const int lo = lo_of(seq, token), hi = hi_of(seq, token);
#pragma unroll
                    for (int kk = 0; kk < TP / 16; kk++)
#pragma unroll
                        for (int jj = 0; jj < kJ; jj++) {
                            uint32_t w[4][kW];
                            load_values(kk, jj, w);
#pragma unroll
                            for (int r = 0; r < 4; r++) {
                                const int at = pos0 + kk * 16 + 2 * t + (r & 1) + (r >> 1) * 8;
#pragma unroll
                                for (int y = 0; y < kW; y++)
                                    if (at < lo || at >= hi) w[r][y] = 0u;
                            }
#pragma unroll
                            for (int m = 0; m < 4; m++) {
                                uint32_t a[4];
                                pair_of(w, m, a);
#pragma unroll
                                for (int nt = 0; nt < NT; nt++) {
                                    float one[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                                    for (int pl = 0; pl < P::PP; pl++) mma<E4>(one, a[0], a[1], a[2], a[3], pb[kk][nt][pl][0], pb[kk][nt][pl][1]);
                                    const int row = w0 + nt * 8 + 2 * t;
                                    if (token_of(p, row) == token) {
                                        acc[jj][m][nt][0] += one[0];
                                        acc[jj][m][nt][2] += one[2];
                                    }
                                    if (token_of(p, row + 1) == token) {
                                        acc[jj][m][nt][1] += one[1];
                                        acc[jj][m][nt][3] += one[3];
                                    }
                                }
                            }
                        }
                }
            }
        }
        if (!x.last) continue;

        // ---- the end of an item, or of the run inside one
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            sum[nt] += __shfl_xor_sync(0xffffffffu, sum[nt], 1);
            sum[nt] += __shfl_xor_sync(0xffffffffu, sum[nt], 2);
        }
        const bool ends = x.tile < 0;
        if (tile0 == 0 && ends) {
            finish_rows<P>(p, seq, kv, w0, rows, top, sum, acc, most_of, team);
            continue;
        }
        if (team_tid == 0) piece_of[2 * team + !ends] = Piece{from + x.at, x.seq, x.item};
        if (ends) {
            float* to = p.heads + (c * P::kTeams + team) * P::kPart;
            put(to, DP, reinterpret_cast<float2*>(to + RT * DP));
        }
    }
    cp_wait<0>();
    __syncthreads();  // the ring is free
    if (piece_of[2 * team + 1].at >= 0) put(red + team * RT * (DP + 4), DP + 4, red_ml + team * RT);
    __syncthreads();

    // ---- what the teams have of the same item, and then the CTAs: the warps are dealt to the items
    const int64_t my_at = lane < 2 * P::kTeams ? piece_of[lane].at : -1;
    const unsigned pieces = __ballot_sync(0xffffffffu, my_at >= 0);
    const unsigned before = pieces & ((1u << lane) - 1u);
    const int64_t at_before = __shfl_sync(0xffffffffu, my_at, before ? 31 - __clz(before) : 0);
    unsigned starts = __ballot_sync(0xffffffffu, my_at >= 0 && (!before || at_before != my_at));
    const int items = __popc(starts);
    if (items == 0) return;
    const int crews = min(items, kWarps), size = kWarps / crews, crew = warp / size, crew_tid = tid - crew * size * 32;
    if (crew >= crews) return;
    for (int n = 0; n < items; n++, starts &= starts - 1u) {
        if (n % crews != crew) continue;
        const int i0 = __ffs(starts) - 1;
        const unsigned later = starts & (starts - 1u), of_item = pieces & ~((1u << i0) - 1u) & (later ? (later & (0u - later)) - 1u : 0xffffffffu);
        const Seq q = seq_of<TP, RT>(p, piece_of[i0].seq);
        int kv, row0;
        rows_of(q, piece_of[i0].item, kv, row0);
        const int n_rows = q.tokens * p.group;
        const int64_t tiles0 = piece_of[i0].at + P::kEnter, tiles1 = tiles0 + q.tiles;
        const bool whole = tiles0 >= run0 && tiles1 <= run1;
        const int c0 = whole ? c : cta_of(tiles0), c1 = whole ? c : cta_of(tiles1 - 1);
        // CTAs c0 .. c1 have the item; the first kFan of them, the next kFan and so on are joined first
        const int sub = (c - c0) / kFan, first = c0 + sub * kFan, many = min(kFan, c1 - first + 1), subs = (c1 - c0) / kFan + 1;
        for (int level = 0;; level++) {
            // the parts: of the teams, of CTAs, of kFan CTAs
            const bool done = whole || level == 2 || (level == 1 && subs == 1);
            for (int x = crew_tid; x < RT * DP / 4; x += size * 32) {  // four columns of a row a thread
                const int row = x / (DP / 4), col = x % (DP / 4) * 4;
                unsigned rest = level == 0 ? of_item : (1u << (level == 1 ? many : subs)) - 1u;
                float m = -INFINITY, l = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                constexpr int kBatch = 6;  // parts on their way at once
                while (rest) {
                    float2 ml[kBatch];
                    float4 a[kBatch];
#pragma unroll
                    for (int y = 0; y < kBatch; y++) {
                        const int i = __ffs(rest) - 1;
                        rest &= rest - 1u;
                        ml[y] = make_float2(-INFINITY, 0.0f);
                        a[y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (i < 0) continue;
                        if (level == 0 && i % 2) {
                            ml[y] = red_ml[i / 2 * RT + row];
                            a[y] = *reinterpret_cast<const float4*>(red + (i / 2 * RT + row) * (DP + 4) + col);
                        } else {
                            const float* part = level == 0   ? p.heads + (c * P::kTeams + i / 2) * P::kPart
                                                : level == 1 ? p.parts + ((first + i) * 2 + (first + i == c0)) * P::kPart
                                                             : p.merged + ((c0 + i * kFan) * 2 + (i == 0)) * P::kPart;
                            ml[y] = __ldcg(reinterpret_cast<const float2*>(part + RT * DP) + row);
                            a[y] = __ldcg(reinterpret_cast<const float4*>(part + row * DP + col));
                        }
                    }
                    float now = m;
#pragma unroll
                    for (int y = 0; y < kBatch; y++) now = fmaxf(now, ml[y].x);
                    const float by = part_factor(make_float2(m, l), now);
                    m = now;
                    l *= by;
#pragma unroll
                    for (int e = 0; e < 4; e++) v[e] *= by;
#pragma unroll
                    for (int y = 0; y < kBatch; y++) {
                        const float f = part_factor(ml[y], m);
                        l += f * ml[y].y;
                        v[0] += f * a[y].x;
                        v[1] += f * a[y].y;
                        v[2] += f * a[y].z;
                        v[3] += f * a[y].w;
                    }
                }
                if (done) {
                    const int r = row0 + row, token = token_of(p, r);
                    finish(p, q.first_token + token, kv * p.group + r - token * p.group, col, v, m, l, r < n_rows);
                } else {
                    float* to = level == 0 ? p.parts + (c * 2 + (c == c0)) * P::kPart : p.merged + (first * 2 + (first == c0)) * P::kPart;
                    __stcg(reinterpret_cast<float4*>(to + row * DP + col), make_float4(v[0], v[1], v[2], v[3]));
                    if (col == 0) __stcg(reinterpret_cast<float2*>(to + RT * DP) + row, make_float2(m, l));
                }
            }
            if (done) break;
            // the last of those that have parts goes on; it leaves the counter at zero
            __threadfence();
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
            __threadfence();
        }
    }
}

// CTAs that fit the current device, looked up once a kernel and device.
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
        ctas = std::min(kAttnMaxCtas, sms * each);
        if (dev < 64) ctas_of[dev] = ctas;
    }
    return launch_pdl(attn_kernel<P>, dim3((unsigned)ctas), 32 * P::kWarps, P::kSmem, st, p);
}

// Rows of an item: 8, 16 or 64, each with the plan that was fastest of those that fit the registers and three tiles a team.
constexpr int padded_dim(int head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }
constexpr int item_rows(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 64; }
constexpr int most_teams(int rows) { return rows <= 16 ? 16 : 4; }

template <bool E4, int DP, bool WIDE>
cudaError_t launch_rows(const AttnArgs& p, cudaStream_t st) {
    const int rows = item_rows(p.n_heads / p.cache.n_kv * p.max_new);
    // columns of a team's warps and warps a CTA
    if (rows == 8) {
        constexpr int C = DP == 64 ? 1 : DP == 128 ? (E4 || WIDE ? 1 : 2) : E4 ? (WIDE ? 1 : 2) : WIDE ? 2 : 4;
        constexpr int W = DP == 64 ? 16 : DP == 128 ? (E4 ? 12 : WIDE ? 8 : 16) : WIDE ? 8 : E4 ? 12 : 16;
        return launch<Plan<E4, DP, 1, 1, C, W, WIDE>>(p, st);
    }
    if (rows == 16) {
        constexpr int C = DP == 64 || (DP == 128 && WIDE) ? 1 : 2;
        return launch<Plan<E4, DP, DP == 256 ? 1 : 2, DP == 256 ? 2 : 1, C, (DP > 64 && WIDE ? 8 : 12), WIDE>>(p, st);
    }
    constexpr int C = DP == 256 && (E4 || !WIDE) ? 2 : 1;
    constexpr int W = DP == 64 ? 12 : DP == 128 ? (WIDE && !E4 ? 8 : 12) : WIDE && !E4 ? 4 : 8;
    return launch<Plan<E4, DP, 2, 4, C, W, WIDE>>(p, st);
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
