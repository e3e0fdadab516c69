// qs_attn.cuh -- attention of the newest tokens of each sequence over the paged key-value cache (sm_103a).
//
// Per token at position p and head h (key-value head h / group), over the positions i that it sees:
//   s_i = scale q . k_i,  out = sum_i 2^(s_i' - m) v_i / sum_i 2^(s_i' - m),  s' = s log2(e),  m the running maximum
// in one pass over keys and values.  Bound: HBM, each key and value once; at 8 rows (heads of a group, drafted tokens) to
// a key the products are 8 to 16 operations a byte.
//
// Work.  An item is a sequence, a key-value head and a tile of RT rows (a row: a new token and one of the group's
// heads).  Its positions are cut into tiles of TP.  All items' tiles in one line are dealt to the CTAs in equal runs,
// wherever an item begins or ends: lengths are known on the device alone and may be uneven, and the line's share keeps
// every SM busy to the end.  An item that several CTAs have parts of is joined by the last of them to finish (a counter
// an item, no waits), in the order of the positions, so the result does not depend on who was last.
//
// A team of R warps goes through tiles of its own, with a ring of ST tiles in shared memory filled by 16-byte
// asynchronous copies: pages of any size and order, one lookup a position a tile ahead of its copies; positions that are
// not there are filled with zeros, never read.  The warps of a team share the tile and have 8 NT rows each; with R = 1
// no barrier wider than a warp is met inside an item.
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

constexpr int kWarps = 4;         // of a CTA
constexpr float kSlack = 8.0f;    // a row's maximum may lag behind by this much (log2) before the sums are scaled
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kSmemMax = 227 * 1024;

// A kernel's sizes: cache type, columns (head_dim rounded up), 8 rows times NT a warp, R warps a team, and whether queries
// and weights go into the products with all their parts.
template <bool E4_, int DP_, int NT_, int R_, bool WIDE_>
struct Plan {
    static constexpr bool E4 = E4_, WIDE = WIDE_;
    static constexpr int DP = DP_, NT = NT_, R = R_;
    static constexpr int kTeams = kWarps / R, kRows = 8 * NT, RT = R * kRows;
    static constexpr int kRowBytes = DP * (E4 ? 1 : 2), kChunks = kRowBytes / 16;
    static constexpr int TP = kRowBytes >= 256 && (R == 1 || kRowBytes >= 512) ? 16 : 32;
    static constexpr int kStage = 2 * TP * kRowBytes + (E4 ? 2 * TP * 4 : 0);  // keys, values, their scales
    static constexpr int QP = WIDE ? (E4 ? 2 : 3) : 1, PP = WIDE ? (E4 ? 2 : 3) : (E4 ? 1 : 2);
    static constexpr int kSteps = DP / 16;            // of the first product
    static constexpr bool kQShared = WIDE || NT * DP > 256;  // query fragments: in shared memory, else in registers
    static constexpr int kQBytes = kQShared ? kWarps * QP * kSteps * 32 * 8 * NT : 0;
    static constexpr int kRed = kTeams * RT * (DP + 4) * 4 + kTeams * RT * 8;  // the teams' results, over the ring
    static constexpr int kFit = (kSmemMax - 1024 - kQBytes) / (kTeams * kStage);
    static constexpr int kGoal = 108 * 1024 / (kTeams * kStage);  // two CTAs an SM
    static constexpr int ST = kGoal >= 3 ? (kGoal > 6 ? 6 : kGoal) : (kFit >= 3 ? 3 : kFit);
    static constexpr int kRing = kTeams * ST * kStage;
    static constexpr int kSmem = kQBytes + (kRing > kRed ? kRing : kRed);
    static_assert(ST >= 2 && kSmem + 1024 <= kSmemMax, "shared memory");
    static_assert(kWarps % R == 0 && 32 * R % kChunks == 0 && TP * kChunks % (32 * R) == 0, "copies");
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
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ float2 lds_f2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts_f2(uint32_t a, float x, float y) {
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(x), "f"(y) : "memory");
}
template <int R>
__device__ __forceinline__ void team_sync(int team) {
    if (R == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * R) : "memory");
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

// What a sequence has to do.
struct Seq {
    int first_token, tokens;  // the new tokens that are attended (max_new at most)
    int64_t start;            // the first one's position
    int lo, hi;               // positions that any of them sees
    int tiles, row_tiles;     // of an item; row tiles of a head
    int64_t work;             // tiles of the whole sequence
};
__device__ __forceinline__ int clip_pos(int64_t p, int n) { return (int)(p < 0 ? 0 : p > n ? n : p); }

template <int TP, int RT>
__device__ __forceinline__ Seq seq_of(const AttnArgs& p, int s, int group) {
    Seq q;
    q.first_token = s;
    int end = s + 1;
    if (p.seqs.offsets) {
        q.first_token = min(max(p.seqs.offsets[s], 0), p.n_tokens);
        end = min(max(p.seqs.offsets[s + 1], 0), p.n_tokens);
    }
    q.tokens = min(max(end - q.first_token, 0), p.max_new);
    q.start = p.seqs.starts ? p.seqs.starts[s] : 0;
    q.lo = p.window ? clip_pos(q.start - p.window + 1, p.seqs.positions) : 0;
    q.hi = clip_pos(q.start + q.tokens, p.seqs.positions);
    q.tiles = max(1, (q.hi + TP - 1) / TP - q.lo / TP);  // one where nothing is seen: its rows are still written
    q.row_tiles = (q.tokens * group + RT - 1) / RT;
    q.work = (int64_t)q.tiles * q.row_tiles * p.cache.n_kv;
    return q;
}

// An output row's eight columns from col: v is the sum of weighted values, l the sum of weights, m the maximum
// they are relative to.
template <int DP>
__device__ __forceinline__ void finish(const AttnArgs& p, int token, int head, int col, float (&v)[8], float m, float l, bool real) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int q = 0; q < 8; q++) v[q] = l == 0.0f ? 0.0f : v[q] * inv;
    const int d = p.cache.head_dim;
    if (p.codes) {  // head_dim a multiple of 128: the 16 lanes of a scale's columns are all here
        float w[1][8];
#pragma unroll
        for (int q = 0; q < 8; q++) w[0][q] = v[q];
        const int i = head * d + col;
        quant_vec<1>(w, 1.0f, kMinAmax, p.codes + token * p.codes_stride, p.codes_scale + token * p.codes_scale_stride, i, real ? p.n_heads * d : 0);
    }
    if (!real || col >= d) return;
    if (p.out.data) {
        uint8_t* row = p.out.data + token * p.out.token_stride + head * p.out.head_stride;
        if (p.out_aligned) {
            store8_row<true>(row, p.out.dtype, col, d, v);
        } else {
#pragma unroll
            for (int q = 0; q < 8; q++) {
                if (p.out.dtype == QS_BF16) reinterpret_cast<__nv_bfloat16*>(row)[col + q] = __float2bfloat16_rn(v[q]);
                else reinterpret_cast<float*>(row)[col + q] = v[q];
            }
        }
    }
    if (p.lse && col == 0) p.lse[(int64_t)token * p.n_heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <class P>
__global__ void __launch_bounds__(32 * kWarps, 1) attn_kernel(const AttnArgs p) {
    constexpr bool E4 = P::E4;
    constexpr int DP = P::DP, NT = P::NT, R = P::R, RT = P::RT, TP = P::TP, ST = P::ST, NC = P::kChunks;
    constexpr int kThreads = 32 * kWarps;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t scan[kWarps];
    __shared__ int64_t found_base;
    __shared__ int found_seq;
    __shared__ unsigned there_of[kWarps][ST];
    __shared__ bool is_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int team = warp / R, team_tid = tid % (32 * R);
    const int group = p.n_heads / p.cache.n_kv, d = p.cache.head_dim;
    uint8_t* ring_at = smem + P::kQBytes;
    const uint32_t q_smem = smem_u32(smem) + warp * (P::kQBytes / kWarps), ring = smem_u32(ring_at) + team * ST * P::kStage, red = smem_u32(ring_at);
    pdl_wait();
    pdl_launch_next();

    // ---- this CTA's run of tiles [a, b), and the sequence that it begins in
    const int per = (p.seqs.n_seqs + kThreads - 1) / kThreads;
    const int s0 = min(tid * per, p.seqs.n_seqs), s1 = min(s0 + per, p.seqs.n_seqs);
    int64_t mine = 0;
    for (int s = s0; s < s1; s++) mine += seq_of<TP, RT>(p, s, group).work;
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) scan[warp] = upto;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
        if (w < warp) upto += scan[w];
        total += scan[w];
    }
    // as many CTAs as have a tile for each team
    const int64_t workers = min((int64_t)gridDim.x, (total + P::kTeams - 1) / P::kTeams);
    const int64_t c = blockIdx.x;
    if (c >= workers) return;
    auto begin_of = [&](int64_t x) { return x * total / workers; };
    auto cta_of = [&](int64_t tile) { return ((tile + 1) * workers - 1) / total; };  // the CTA whose run has it
    int64_t cur = begin_of(c);
    const int64_t end = begin_of(c + 1);
    if (cur >= upto - mine && cur < upto) {
        int64_t base = upto - mine;
        int s = s0;
        for (; s + 1 < s1; s++) {
            const int64_t w = seq_of<TP, RT>(p, s, group).work;
            if (cur < base + w) break;
            base += w;
        }
        found_base = base;
        found_seq = s;
    }
    __syncthreads();
    int64_t base = found_base;
    int s = found_seq;
    Seq seq = seq_of<TP, RT>(p, s, group);

    while (cur < end) {
        while (cur >= base + seq.work && s + 1 < p.seqs.n_seqs) {
            base += seq.work;
            seq = seq_of<TP, RT>(p, ++s, group);
        }
        const int item = (int)((cur - base) / seq.tiles), tile0 = (int)((cur - base) % seq.tiles);
        const int tile1 = (int)min((int64_t)seq.tiles, tile0 + (end - cur));
        const int kv = item / seq.row_tiles, row0 = item % seq.row_tiles * RT, rows = seq.tokens * group;
        const int64_t item0 = cur - tile0;  // the item's first tile in the line
        cur += tile1 - tile0;

        // positions that the row tile sees, and that all this warp's rows see
        auto hi_of = [&](int token) { return clip_pos(seq.start + token + 1, p.seqs.positions); };
        auto lo_of = [&](int token) { return p.window ? clip_pos(seq.start + token + 1 - p.window, p.seqs.positions) : 0; };
        const int tile_lo = lo_of(row0 / group), tile_hi = hi_of((min(row0 + RT, rows) - 1) / group);
        const int w0 = row0 + (warp % R) * P::kRows, w1 = min(w0 + P::kRows, rows);
        const bool active = w0 < rows;
        const int token0 = w0 / group, token1 = max(w1 - 1, w0) / group;
        const int all_lo = lo_of(token1), all_hi = hi_of(token0);

        // ---- copies
        const int n = max(0, (tile1 - tile0 - team + P::kTeams - 1) / P::kTeams);  // this team's tiles
        const int first_pos = (seq.lo / TP + tile0 + team) * TP;
        const uint8_t* k_base = p.cache.k + kv * p.cache.head_stride;
        const uint8_t* v_base = p.cache.v + kv * p.cache.head_stride;
        Place ahead = {-1, -1};
        auto look = [&](int i) {
            const int pos = first_pos + i * P::kTeams * TP + lane % TP;
            ahead = i < n && pos >= tile_lo && pos < tile_hi ? place_of(p.cache, p.seqs, s, pos) : Place{-1, -1};
        };
        auto issue = [&](int i) {
            if (i < n) {
                const int stage = i % ST;
                const uint32_t keys = ring + stage * P::kStage, values = keys + TP * P::kRowBytes;
                const unsigned there = __ballot_sync(0xffffffffu, ahead.at >= 0);
                if (lane == 0) there_of[warp][stage] = there;
                const int chunk = team_tid % NC;
                const bool in = chunk * 16 < d * (E4 ? 1 : 2);
#pragma unroll
                for (int k = 0; k < TP * NC / (32 * R); k++) {
                    const int row = team_tid / NC + k * (32 * R / NC);
                    const int64_t at = __shfl_sync(0xffffffffu, ahead.at, row);
                    const bool ok = at >= 0 && in;
                    const int64_t from = ok ? at + chunk * 16 : 0;
                    cp16(keys + row * P::kRowBytes + ((chunk ^ (NC >= 8 ? (row & 1) * 4 : 0)) * 16), ok ? k_base + from : p.cache.k, ok);
                    cp16(values + row * P::kRowBytes + ((chunk ^ (((row >> 1) & 3) * 2 & (NC - 1))) * 16), ok ? v_base + from : p.cache.v, ok);
                }
                if (E4 && warp % R == 0 && lane < TP) {
                    const bool ok = ahead.at >= 0;
                    const int64_t from = ok ? ahead.scale_at + kv * p.cache.scale_head_stride : 0;
                    cp4(values + TP * P::kRowBytes + lane * 4, p.cache.k_scale + from, ok);
                    cp4(values + TP * P::kRowBytes + (TP + lane) * 4, p.cache.v_scale + from, ok);
                }
            }
            cp_commit();
            look(i + 1);
        };
        look(0);
#pragma unroll
        for (int i = 0; i < ST - 1; i++) issue(i);

        // ---- queries: fragments in the order in which the keys' pieces lie
        constexpr int kEach = NT == 1 ? 2 : 4;  // registers of a step: rows g, and g + 8 with NT = 2
        uint32_t qf[P::kQShared ? 1 : P::kSteps][kEach];
        float row_scale[NT];
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            const int row = w0 + nt * 8 + g;
            const uint8_t* q = row < rows ? p.q.data + (seq.first_token + row / group) * p.q.token_stride + (kv * group + row % group) * p.q.head_stride : nullptr;
            float factor = 1.0f;
            if (E4) {  // a power of two that brings the row's largest into fp16's upper range
                float a = 0.0f;
#pragma unroll
                for (int i = 0; i < DP / 32; i++) {
                    float v[8];
                    load_q8(p.q, p.q_aligned, q, 32 * i + 8 * t, d, v);
#pragma unroll
                    for (int e = 0; e < 8; e++) a = fmaxf(a, fabsf(v[e]));
                }
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
                const int e = min(max(14 - ((int)(__float_as_uint(a) >> 23) - 127), -100), 100);
                factor = __uint_as_float((uint32_t)(127 + e) << 23);
                row_scale[nt] = p.scale * __uint_as_float((uint32_t)(127 - e) << 23);
            } else {
                row_scale[nt] = p.scale;
            }
            // bf16: piece i is columns 32 i + 8 t .. + 7, two steps of four; e4m3: 64 i + 16 t .. + 15, four steps
#pragma unroll
            for (int i = 0; i < DP / 32; i++) {
                float v[8];
                const int col = E4 ? 64 * (i / 2) + 16 * t + 8 * (i % 2) : 32 * i + 8 * t;
                load_q8(p.q, p.q_aligned, q, col, d, v);
#pragma unroll
                for (int e = 0; e < 8; e++) v[e] *= factor;
#pragma unroll
                for (int pl = 0; pl < P::QP; pl++) {
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const int step = 2 * i + h;
                        const uint32_t x = part<E4>(v[4 * h], v[4 * h + 1]), y = part<E4>(v[4 * h + 2], v[4 * h + 3]);
                        if (P::kQShared) {
                            const uint32_t at = q_smem + ((pl * P::kSteps + step) * 32 + lane) * (8 * NT) + 4 * nt;
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 4 * NT), "r"(y) : "memory");
                        } else {
                            qf[step][nt] = x;
                            qf[step][kEach / 2 + nt] = y;
                        }
                    }
                }
            }
        }
        // one step of the first product: b of a key's piece with every part of the queries
        auto score = [&](float (&c4)[4], int step, uint32_t b0, uint32_t b1) {
#pragma unroll
            for (int pl = 0; pl < P::QP; pl++) {
                uint32_t a[4];
                if (P::kQShared) {
                    const uint32_t at = q_smem + ((pl * P::kSteps + step) * 32 + lane) * (8 * NT);
                    if (NT == 1) {
                        const uint2 x = lds8(at);
                        a[0] = x.x; a[1] = 0; a[2] = x.y; a[3] = 0;
                    } else {
                        const uint4 x = lds16(at);
                        a[0] = x.x; a[1] = x.y; a[2] = x.z; a[3] = x.w;
                    }
                } else {
                    constexpr int kS = P::kQShared ? 0 : 1;
                    a[0] = qf[step * kS][0];
                    a[1] = NT == 1 ? 0u : qf[step * kS][1 % kEach];
                    a[2] = qf[step * kS][kEach / 2];
                    a[3] = NT == 1 ? 0u : qf[step * kS][kEach - 1];
                }
                mma<E4>(c4, a[0], a[1], a[2], a[3], b0, b1);
            }
        };

        // ---- the pass over the positions
        float acc[DP / 64][4][NT][4];  // [64 columns][their pair][rows]: columns 64 jj + 8 g + 2 m (+ 1), rows 2 t, 2 t + 1
        float top[NT], sum[NT];
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            top[nt] = -INFINITY;
            sum[nt] = 0.0f;
        }
#pragma unroll
        for (int jj = 0; jj < DP / 64; jj++)
#pragma unroll
            for (int m = 0; m < 4; m++)
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int e = 0; e < 4; e++) acc[jj][m][nt][e] = 0.0f;

        for (int i = 0; i < n; i++) {
            cp_wait<ST - 2>();
            team_sync<R>(team);
            issue(i + ST - 1);
            if (!active) continue;
            const int stage = i % ST, pos0 = first_pos + i * P::kTeams * TP;
            const uint32_t keys = ring + stage * P::kStage, values = keys + TP * P::kRowBytes, scales = values + TP * P::kRowBytes;
            const unsigned there = there_of[warp][stage];
            const unsigned whole = TP == 32 ? 0xffffffffu : (1u << (TP & 31)) - 1u;
            const bool full = (there & whole) == whole && pos0 >= all_lo && pos0 + TP <= all_hi;

            float sc[TP / 8][4];
#pragma unroll
            for (int nt8 = 0; nt8 < TP / 8; nt8++) {
#pragma unroll
                for (int e = 0; e < 4; e++) sc[nt8][e] = 0.0f;
                const int row = nt8 * 8 + g;
#pragma unroll
                for (int i4 = 0; i4 < NC / 4; i4++) {
                    const uint4 w = lds16(keys + row * P::kRowBytes + (((4 * i4 + t) ^ (NC >= 8 ? (row & 1) * 4 : 0)) * 16));
                    const uint32_t r4[4] = {w.x, w.y, w.z, w.w};
                    if (E4) {
#pragma unroll
                        for (int h = 0; h < 4; h++) score(sc[nt8], 4 * i4 + h, widen(r4[h]), widen(r4[h] >> 16));
                    } else {
                        score(sc[nt8], 2 * i4, r4[0], r4[1]);
                        score(sc[nt8], 2 * i4 + 1, r4[2], r4[3]);
                    }
                }
            }
            float2 vs[TP / 8];
#pragma unroll
            for (int nt8 = 0; nt8 < TP / 8; nt8++) {
#pragma unroll
                for (int e = 0; e < 2 * NT; e++) sc[nt8][e] *= row_scale[e / 2];
                if (E4) {
                    const float2 ks = lds_f2(scales + (nt8 * 8 + 2 * t) * 4);
                    vs[nt8] = lds_f2(scales + (TP + nt8 * 8 + 2 * t) * 4);
#pragma unroll
                    for (int e = 0; e < 2 * NT; e++) sc[nt8][e] *= e % 2 ? ks.y : ks.x;
                }
            }
            if (!full) {
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    const int token = (w0 + nt * 8 + g) / group;
                    const int lo = lo_of(token), hi = hi_of(token);
#pragma unroll
                    for (int nt8 = 0; nt8 < TP / 8; nt8++)
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            const int at = nt8 * 8 + 2 * t + e;
                            if (!((there >> at) & 1u) || pos0 + at < lo || pos0 + at >= hi) sc[nt8][2 * nt + e] = -INFINITY;
                        }
                }
            }
            // the values' scales count for the maximum, as within 2^-100 .. 2^118: the weight's two factors stay in fp32's range
            float2 lv[TP / 8];
#pragma unroll
            for (int nt8 = 0; nt8 < TP / 8; nt8++) {
                lv[nt8] = make_float2(0.0f, 0.0f);
                if (E4) lv[nt8] = make_float2(fminf(fmaxf(lg2(vs[nt8].x), -100.0f), 118.0f), fminf(fmaxf(lg2(vs[nt8].y), -100.0f), 118.0f));
            }
            bool grown = false;
            float most[NT];
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                float a = -INFINITY;
#pragma unroll
                for (int nt8 = 0; nt8 < TP / 8; nt8++) a = fmaxf(a, fmaxf(sc[nt8][2 * nt] + lv[nt8].x, sc[nt8][2 * nt + 1] + lv[nt8].y));
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
                    for (int jj = 0; jj < DP / 64; jj++)
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
                for (int nt8 = 0; nt8 < TP / 8; nt8++) {
                    float x = ex2(sc[nt8][2 * nt] - ref), y = ex2(sc[nt8][2 * nt + 1] - ref);
                    sum[nt] += x + y;
                    if (E4) {  // a weight of 0 stays 0 beside whatever scale a position has that is not seen
                        x = sc[nt8][2 * nt] == -INFINITY ? 0.0f : x * vs[nt8].x;
                        y = sc[nt8][2 * nt + 1] == -INFINITY ? 0.0f : y * vs[nt8].y;
                    }
#pragma unroll
                    for (int pl = 0; pl < P::PP; pl++) pb[nt8 / 2][nt][pl][nt8 % 2] = part<E4>(x, y);
                }
            }
            // positions here that one of the warp's rows does not see and that were copied for another
            const bool mixed = !full && (min(pos0 + TP, tile_hi) > all_hi || max(pos0, tile_lo) < all_lo);
#pragma unroll
            for (int kk = 0; kk < TP / 16; kk++) {
#pragma unroll
                for (int jj = 0; jj < DP / 64; jj++) {
                    // four positions' eight columns
                    uint32_t w[4][E4 ? 2 : 4];
#pragma unroll
                    for (int r = 0; r < 4; r++) {
                        const int row = kk * 16 + 2 * t + (r & 1) + (r >> 1) * 8;
                        if (E4) {
                            const int chunk = 4 * jj + g / 2;
                            const uint2 x = lds8(values + row * P::kRowBytes + ((chunk ^ (((row >> 1) & 3) * 2 & (NC - 1))) * 16) + (g & 1) * 8);
                            w[r][0] = x.x;
                            w[r][1] = x.y;
                        } else {
                            const int chunk = 8 * jj + g;
                            const uint4 x = lds16(values + row * P::kRowBytes + ((chunk ^ (((row >> 1) & 3) * 2)) * 16));
                            w[r][0] = x.x; w[r][1] = x.y; w[r][E4 ? 0 : 2] = x.z; w[r][E4 ? 0 : 3] = x.w;
                        }
                    }
                    auto values_of = [&](int m, uint32_t (&a)[4]) {
                        if (E4) {
                            const uint32_t x = __byte_perm(w[0][m / 2], w[1][m / 2], m % 2 ? 0x7362 : 0x5140);
                            const uint32_t y = __byte_perm(w[2][m / 2], w[3][m / 2], m % 2 ? 0x7362 : 0x5140);
                            a[0] = widen(x);
                            a[1] = widen(x >> 16);
                            a[2] = widen(y);
                            a[3] = widen(y >> 16);
                        } else {
                            constexpr int kM = E4 ? 0 : 1;
                            a[0] = __byte_perm(w[0][m * kM], w[1][m * kM], 0x5410);
                            a[1] = __byte_perm(w[0][m * kM], w[1][m * kM], 0x7632);
                            a[2] = __byte_perm(w[2][m * kM], w[3][m * kM], 0x5410);
                            a[3] = __byte_perm(w[2][m * kM], w[3][m * kM], 0x7632);
                        }
                    };
                    if (!mixed) {
#pragma unroll
                        for (int m = 0; m < 4; m++) {
                            uint32_t a[4];
                            values_of(m, a);
#pragma unroll
                            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                                for (int pl = 0; pl < P::PP; pl++) mma<E4>(acc[jj][m][nt], a[0], a[1], a[2], a[3], pb[kk][nt][pl][0], pb[kk][nt][pl][1]);
                        }
                    } else {
                        uint32_t all[4][E4 ? 2 : 4];
#pragma unroll
                        for (int r = 0; r < 4; r++)
#pragma unroll
                            for (int x = 0; x < (E4 ? 2 : 4); x++) all[r][x] = w[r][x];
                        for (int token = token0; token <= token1; token++) {
                            const int lo = lo_of(token), hi = hi_of(token);
#pragma unroll
                            for (int r = 0; r < 4; r++) {
                                const int at = pos0 + kk * 16 + 2 * t + (r & 1) + (r >> 1) * 8;
#pragma unroll
                                for (int x = 0; x < (E4 ? 2 : 4); x++) w[r][x] = at >= lo && at < hi ? all[r][x] : 0u;
                            }
#pragma unroll
                            for (int m = 0; m < 4; m++) {
                                uint32_t a[4];
                                values_of(m, a);
#pragma unroll
                                for (int nt = 0; nt < NT; nt++) {
                                    float one[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                                    for (int pl = 0; pl < P::PP; pl++) mma<E4>(one, a[0], a[1], a[2], a[3], pb[kk][nt][pl][0], pb[kk][nt][pl][1]);
                                    const int row = w0 + nt * 8 + 2 * t;
                                    const bool x0 = row / group == token, x1 = (row + 1) / group == token;
                                    if (x0) {
                                        acc[jj][m][nt][0] += one[0];
                                        acc[jj][m][nt][2] += one[2];
                                    }
                                    if (x1) {
                                        acc[jj][m][nt][1] += one[1];
                                        acc[jj][m][nt][3] += one[3];
                                    }
                                }
                            }
                        }
                    }
                }
            }
        }
        cp_wait<0>();
        __syncthreads();

        // ---- the teams' results, through shared memory
        const uint32_t red_ml = red + P::kTeams * RT * (DP + 4) * 4;
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            sum[nt] += __shfl_xor_sync(0xffffffffu, sum[nt], 1);
            sum[nt] += __shfl_xor_sync(0xffffffffu, sum[nt], 2);
            const int row = team * RT + (warp % R) * P::kRows + nt * 8;
            if (t == 0) sts_f2(red_ml + (row + g) * 8, top[nt], sum[nt]);
#pragma unroll
            for (int jj = 0; jj < DP / 64; jj++)
#pragma unroll
                for (int m = 0; m < 4; m++) {
                    const uint32_t at = red + ((row + 2 * t) * (DP + 4) + 64 * jj + 8 * g + 2 * m) * 4;
                    sts_f2(at, acc[jj][m][nt][0], acc[jj][m][nt][2]);
                    sts_f2(at + (DP + 4) * 4, acc[jj][m][nt][1], acc[jj][m][nt][3]);
                }
        }
        __syncthreads();
        const int64_t c0 = cta_of(item0), c1 = cta_of(item0 + seq.tiles - 1);
        // 8 columns of a row a thread; whole warps, as the codes' maxima are found by shuffles
        constexpr int kPieces = RT * DP / 8;
        for (int x = tid; x < (kPieces + 31) / 32 * 32; x += kThreads) {
            const int row = x / (DP / 8), col = x % (DP / 8) * 8;
            float m = -INFINITY, l = 0.0f, v[8];
#pragma unroll
            for (int e = 0; e < 8; e++) v[e] = 0.0f;
#pragma unroll
            for (int w = 0; w < P::kTeams; w++) m = fmaxf(m, lds_f2(red_ml + (w * RT + row) * 8).x);
#pragma unroll
            for (int w = 0; w < P::kTeams; w++) {
                const float2 ml = lds_f2(red_ml + (w * RT + row) * 8);
                const float by = ml.x == -INFINITY ? (ml.y == 0.0f ? 0.0f : 1.0f) : ex2(ml.x - m);
                const uint32_t at = red + ((w * RT + row) * (DP + 4) + col) * 4;
                l += by * ml.y;
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 o = lds_f2(at + 4 * e);
                    v[e] += by * o.x;
                    v[e + 1] += by * o.y;
                }
            }
            if (c0 == c1) {
                const int r = row0 + row;
                finish<DP>(p, seq.first_token + r / group, kv * group + r % group, col, v, m, l, r < rows);
            } else {
                float* to = p.parts + (c * 2 + (c == c0)) * (RT * (DP + 2));
                float4* o = reinterpret_cast<float4*>(to + row * DP + col);
                __stcg(o, make_float4(v[0], v[1], v[2], v[3]));
                __stcg(o + 1, make_float4(v[4], v[5], v[6], v[7]));
                if (col == 0) __stcg(reinterpret_cast<float2*>(to + RT * DP) + row, make_float2(m, l));
            }
        }
        if (c0 != c1) {
            __threadfence();
            __syncthreads();
            if (tid == 0) is_last = atom_acq_rel_add(p.joined + c0, 1u) == (uint32_t)(c1 - c0);
            __syncthreads();
            if (is_last) {
                __threadfence();
                for (int x = tid; x < (kPieces + 31) / 32 * 32; x += kThreads) {
                    const int row = x / (DP / 8), col = x % (DP / 8) * 8;
                    auto part_at = [&](int64_t w) { return p.parts + (w * 2 + (w == c0)) * (RT * (DP + 2)); };
                    float m = -INFINITY, l = 0.0f, v[8];
#pragma unroll
                    for (int e = 0; e < 8; e++) v[e] = 0.0f;
                    for (int64_t w = c0; w <= c1; w++) m = fmaxf(m, __ldcg(reinterpret_cast<const float2*>(part_at(w) + RT * DP) + row).x);
                    for (int64_t w = c0; w <= c1; w++) {
                        const float* from = part_at(w);
                        const float2 ml = __ldcg(reinterpret_cast<const float2*>(from + RT * DP) + row);
                        const float by = ml.x == -INFINITY ? (ml.y == 0.0f ? 0.0f : 1.0f) : ex2(ml.x - m);
                        l += by * ml.y;
                        const float4 a = __ldcg(reinterpret_cast<const float4*>(from + row * DP + col));
                        const float4 b = __ldcg(reinterpret_cast<const float4*>(from + row * DP + col) + 1);
                        v[0] += by * a.x; v[1] += by * a.y; v[2] += by * a.z; v[3] += by * a.w;
                        v[4] += by * b.x; v[5] += by * b.y; v[6] += by * b.z; v[7] += by * b.w;
                    }
                    const int r = row0 + row;
                    finish<DP>(p, seq.first_token + r / group, kv * group + r % group, col, v, m, l, r < rows);
                }
                if (tid == 0) p.joined[c0] = 0u;
            }
        }
        __syncthreads();  // the ring is free for the next item
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
        if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&each, attn_kernel<P>, 32 * kWarps, P::kSmem)) != cudaSuccess) return e;
        if (each < 1) return cudaErrorLaunchOutOfResources;
        ctas = std::min(kAttnMaxCtas, sms * each);
        if (dev < 64) ctas_of[dev] = ctas;
    }
    return launch_pdl(attn_kernel<P>, dim3((unsigned)ctas), 32 * kWarps, P::kSmem, st, p);
}

// Rows of an item: 8 of one warp, 16 of one (two with 256 columns, whose sums fill the registers), else 64 of four.
constexpr int padded_dim(int head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }
constexpr int item_rows(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 64; }

template <bool E4, int DP, bool WIDE>
cudaError_t launch_rows(const AttnArgs& p, cudaStream_t st) {
    const int rows = item_rows(p.n_heads / p.cache.n_kv * p.max_new);
    if (rows == 8) return launch<Plan<E4, DP, 1, 1, WIDE>>(p, st);
    if (rows == 16) return launch<Plan<E4, DP, DP == 256 ? 1 : 2, DP == 256 ? 2 : 1, WIDE>>(p, st);
    return launch<Plan<E4, DP, 2, 4, WIDE>>(p, st);
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
