// qs_tokens.cu -- token rows sorted by expert and back, with weights, and their gradients (sm_103a).
//
// Dispatch.  A stable counting sort of the n = n_tokens * top_k entries by expert, then the rows.
// Up to kSmallN entries it is one launch: an entry's position is the number of entries with a lower
// expert plus the number of earlier ones with the same, which a warp counts over all ids (n / 32
// comparisons a lane, the ids in L2) -- less than the launch of a second kernel costs.  Above that
// three: a histogram of every chunk of entries, the positions (each CTA adds the chunks before its
// own), and the rows, one token a CTA, so that a token's row is read once for its k copies.
// Combine.  One token a CTA row: sum of w * y[pos] over the slots in ascending order, k loads in
// flight a thread.  Its gradient reads dout once a token and y once, and writes dy once.
// All of them move bytes once: the bound is HBM.  8192 tokens to 8 of 256 experts, bf16 rows of 2048: rows out 46 us
// (302 MB), back 49 us (302 MB), the gradient of that 94 us (570 MB); the positions 12 us before.
#include "qs_internal.h"
#include "qs_rows.cuh"

#include <algorithm>

namespace qs {

namespace {

constexpr int kSmallN = 4096;   // entries of the one-launch form: with 8 a token, 256 tokens 5.3 us against 8.8 in three
                                // launches, 512 9.9 against 10.2, 1024 28.5 against 12.8 (bf16 rows of 2048)
constexpr int kChunk = 1024;    // least entries of a chunk of the sort
constexpr int kMaxChunks = 256; // most chunks
constexpr int kSortThreads = 256;
constexpr int kPlaceThreads = 1024;

int chunk_entries(int64_t n) {
    const int64_t c = (n + kMaxChunks - 1) / kMaxChunks;
    return (int)std::max<int64_t>(kChunk, (c + 31) / 32 * 32);
}
int chunk_count(int64_t n) { return (int)((n + chunk_entries(n) - 1) / chunk_entries(n)); }

// Rows are copied by words of 16 bytes where base addresses and strides allow, else of 4, 2 or 1; what is left of a
// row behind its last whole word, byte by byte.
template <int W>
struct Word;
template <> struct Word<16> { using T = uint4; };
template <> struct Word<4> { using T = uint32_t; };
template <> struct Word<2> { using T = uint16_t; };
template <> struct Word<1> { using T = uint8_t; };

// off[e] = the sum of cnt[0 .. e - 1], off[E] the sum of all.  One warp calls it; the caller's barriers stand before and after.
__device__ void scan_counts(const int32_t* cnt, int32_t* off, int E) {
    const int lane = threadIdx.x & 31;
    int carry = 0;
    for (int b = 0; b < E; b += 32) {
        const int c = b + lane < E ? cnt[b + lane] : 0;
        int s = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += v;
        }
        if (b + lane < E) off[b + lane] = carry + s - c;
        carry += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) off[E] = carry;
}

// ------------------------------------------------------------------ one launch

// CTA t < n_tokens: its token's positions and rows (a warp an entry).  The last CTA: counts, offsets
// and the -1 entries of perm.
template <int W>
__global__ void __launch_bounds__(256) dispatch_small_kernel(const DispatchArgs p) {
    extern __shared__ int32_t sm[];
    pdl_wait();
    pdl_launch_next();
    const int n = p.n_tokens * p.top_k;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if ((int)blockIdx.x == p.n_tokens) {
        int32_t *cnt = sm, *off = sm + p.n_experts;
        for (int e = threadIdx.x; e < p.n_experts; e += blockDim.x) cnt[e] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            const int e = p.ids[i];
            if ((unsigned)e < (unsigned)p.n_experts) atomicAdd(&cnt[e], 1);
        }
        __syncthreads();
        if (warp == 0) scan_counts(cnt, off, p.n_experts);
        __syncthreads();
        for (int e = threadIdx.x; e < p.n_experts; e += blockDim.x) p.counts[e] = cnt[e];
        for (int e = threadIdx.x; e <= p.n_experts; e += blockDim.x) p.offsets[e] = off[e];
        for (int i = off[p.n_experts] + threadIdx.x; i < n; i += blockDim.x) p.perm[i] = -1;
        return;
    }
    using T = typename Word<W>::T;
    const int t = blockIdx.x;
    for (int j = warp; j < p.top_k; j += 8) {
        const int i = t * p.top_k + j;
        const int e = p.ids[i];
        if ((unsigned)e >= (unsigned)p.n_experts) {
            if (lane == 0) p.pos[i] = -1;
            continue;
        }
        int before = 0;
#pragma unroll 8
        for (int b = lane; b < n; b += 32) {
            const int o = p.ids[b];
            before += (o >= 0 && o < e) || (o == e && b < i);
        }
        const int at = __reduce_add_sync(0xffffffffu, before);
        if (lane == 0) {
            p.pos[i] = at;
            p.perm[at] = i;
        }
        if (!p.xs) continue;
        const T* src = reinterpret_cast<const T*>(static_cast<const uint8_t*>(p.x) + t * p.x_stride);
        T* dst = reinterpret_cast<T*>(static_cast<uint8_t*>(p.xs) + at * p.xs_stride);
#pragma unroll 4
        for (int c = lane; c < p.row_bytes / W; c += 32) dst[c] = src[c];
        if (W > 1 && lane < p.row_bytes % W) {
            const int c = p.row_bytes / W * W + lane;
            reinterpret_cast<uint8_t*>(dst)[c] = reinterpret_cast<const uint8_t*>(src)[c];
        }
        for (int c = lane; c < p.n_scales; c += 32)
            p.xs_scale[at * p.xs_scale_stride + c] = p.x_scale[t * p.x_scale_stride + c];
    }
}

// ------------------------------------------------------------------ three launches

__global__ void __launch_bounds__(kSortThreads) dispatch_hist_kernel(const int32_t* __restrict__ ids, int n, int E,
                                                                     int chunk, int32_t* hist) {
    extern __shared__ int32_t sm[];
    pdl_wait();
    pdl_launch_next();
    for (int e = threadIdx.x; e < E; e += blockDim.x) sm[e] = 0;
    __syncthreads();
    const int64_t i0 = (int64_t)blockIdx.x * chunk, i1 = min((int64_t)n, i0 + chunk);
#pragma unroll 4
    for (int64_t i = i0 + threadIdx.x; i < i1; i += blockDim.x) {
        const int e = ids[i];
        if ((unsigned)e < (unsigned)E) atomicAdd(&sm[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[(size_t)blockIdx.x * E + e] = sm[e];
}

// A chunk a CTA, 1024 entries at a time.  An entry's position: its expert's offset, the entries of that expert in
// earlier chunks and earlier in this one -- those of earlier warps from the warps' counts (a byte each: a warp
// has 32 entries), those of its own warp from a match.  sm: total[E], off[E + 1], base[E], then cnt[32][E] bytes.
__global__ void __launch_bounds__(kPlaceThreads) dispatch_place_kernel(const DispatchArgs p, int n, int chunk, int chunks) {
    extern __shared__ int32_t sm[];
    const int E = p.n_experts, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t *total = sm, *off = sm + E, *base = off + E + 1;
    uint8_t* cnt = reinterpret_cast<uint8_t*>(base + E);
    pdl_wait();
    pdl_launch_next();
    for (int e = threadIdx.x; e < E; e += kPlaceThreads) total[e] = base[e] = 0;
    __syncthreads();
    // all chunks, and those before this one: four threads an expert, each a quarter of the chunks, so that the
    // loads of a thread are in flight together (one thread an expert took 9 us of 15)
    const int per = (chunks + 3) / 4, c0 = threadIdx.x / (kPlaceThreads / 4) * per, c1 = min(chunks, c0 + per);
    for (int e = threadIdx.x % (kPlaceThreads / 4); e < E; e += kPlaceThreads / 4) {
        int before = 0, all = 0;
#pragma unroll 16
        for (int c = c0; c < c1; c++) {
            const int h = p.hist[(size_t)c * E + e];
            all += h;
            before += c < (int)blockIdx.x ? h : 0;
        }
        if (all) atomicAdd(&total[e], all);
        if (before) atomicAdd(&base[e], before);
    }
    __syncthreads();
    if (warp == 0) scan_counts(total, off, E);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kPlaceThreads) base[e] += off[e];
    if (blockIdx.x == 0) {
        for (int e = threadIdx.x; e < E; e += kPlaceThreads) p.counts[e] = total[e];
        for (int e = threadIdx.x; e <= E; e += kPlaceThreads) p.offsets[e] = off[e];
    }
    const int64_t i0 = (int64_t)blockIdx.x * chunk, i1 = min((int64_t)n, i0 + chunk);
    // this chunk's share of perm's tail
    for (int64_t i = max(i0, (int64_t)off[E]) + threadIdx.x; i < i1; i += kPlaceThreads) p.perm[i] = -1;
    for (int64_t b = i0; b < i1; b += kPlaceThreads) {
        const int64_t i = b + threadIdx.x;
        const int e = i < i1 ? p.ids[i] : -1;
        const bool valid = (unsigned)e < (unsigned)E;
        for (int k = threadIdx.x; k < 8 * E; k += kPlaceThreads) reinterpret_cast<uint32_t*>(cnt)[k] = 0;  // 32 E bytes
        __syncthreads();
        const unsigned peers = __match_any_sync(0xffffffffu, valid ? e : -1);
        const bool lead = valid && lane == __ffs(peers) - 1;
        if (lead) cnt[warp * E + e] = (uint8_t)__popc(peers);
        __syncthreads();
        int at = -1;
        if (valid) {
            at = base[e] + __popc(peers & ((1u << lane) - 1u));
            for (int w = 0; w < warp; w++) at += cnt[w * E + e];
            p.perm[at] = (int32_t)i;
        }
        if (i < i1) p.pos[i] = at;
        __syncthreads();
        if (lead) atomicAdd(&base[e], __popc(peers));  // for the next 1024
    }
}

// One token a CTA: its row is read once and written to its k positions.
template <int W>
__global__ void __launch_bounds__(256) dispatch_rows_kernel(const DispatchArgs p) {
    __shared__ int32_t at[32];
    using T = typename Word<W>::T;
    const int64_t t = blockIdx.x;
    pdl_wait();
    pdl_launch_next();
    if (threadIdx.x < p.top_k) at[threadIdx.x] = p.pos[t * p.top_k + threadIdx.x];
    __syncthreads();
    const T* src = reinterpret_cast<const T*>(static_cast<const uint8_t*>(p.x) + t * p.x_stride);
    uint8_t* xs = static_cast<uint8_t*>(p.xs);
    for (int c = threadIdx.x; c < p.row_bytes / W; c += blockDim.x) {
        const T v = src[c];
        for (int j = 0; j < p.top_k; j++)
            if (at[j] >= 0) reinterpret_cast<T*>(xs + at[j] * p.xs_stride)[c] = v;
    }
    if (W > 1 && threadIdx.x < p.row_bytes % W) {
        const int c = p.row_bytes / W * W + threadIdx.x;
        const uint8_t v = reinterpret_cast<const uint8_t*>(src)[c];
        for (int j = 0; j < p.top_k; j++)
            if (at[j] >= 0) xs[at[j] * p.xs_stride + c] = v;
    }
    for (int c = threadIdx.x; c < p.n_scales * p.top_k; c += blockDim.x) {
        const int j = c / p.n_scales, b = c - j * p.n_scales;
        if (at[j] >= 0) p.xs_scale[at[j] * p.xs_scale_stride + b] = p.x_scale[t * p.x_scale_stride + b];
    }
}

// ------------------------------------------------------------------ combine and its gradient

constexpr int kBatch = 8;  // slots whose rows are in flight together

// Rows in flight are held as they come (bf16: four registers each), half as many where they are fp32:
// widened at once they took 86 registers, a quarter of the threads, and twice the time.
template <bool VEC, bool B16>
__global__ void __launch_bounds__(256) combine_kernel(const CombineArgs p) {
    constexpr int kHeld = B16 ? kBatch : kBatch / 2;
    __shared__ int32_t at[32];
    __shared__ float w[32];
    const int64_t t = blockIdx.x;
    pdl_wait();
    pdl_launch_next();
    if (threadIdx.x < 32) {
        int a = -1;
        float f = 0.0f;
        if (threadIdx.x < p.top_k) {
            const int64_t i = t * p.top_k + threadIdx.x;
            a = p.pos[i];
            // a position outside the rows is not read
            if ((unsigned)a >= (unsigned)(p.n_tokens * p.top_k)) a = -1;
            f = p.w ? p.w[i] : 1.0f;
        }
        at[threadIdx.x] = a;
        w[threadIdx.x] = f;
    }
    __syncthreads();
    void* out = row_at(p.out, p.out_stride, type_size(p.out_dtype), t);
    for (int i = (blockIdx.y * blockDim.x + threadIdx.x) * 8; cols_left<VEC>(i, p.hidden); i += gridDim.y * blockDim.x * 8) {
        float acc[8];
#pragma unroll
        for (int q = 0; q < 8; q++) acc[q] = 0.0f;
        for (int j0 = 0; j0 < p.top_k; j0 += kHeld) {
            Held8<VEC, B16> v[kHeld];
#pragma unroll
            for (int j = 0; j < kHeld; j++) {
                const int a = at[j0 + j];
                v[j].load(row_at(p.y, p.y_stride, type_size(p.y_dtype), max(a, 0)), p.y_dtype, i, a >= 0 ? p.hidden : 0);
            }
#pragma unroll
            for (int j = 0; j < kHeld; j++) {
                if (at[j0 + j] < 0) continue;  // a dropped entry adds nothing, whatever its weight is
                const float f = w[j0 + j];
                float x[8];
                v[j].get(p.y_dtype, x);
#pragma unroll
                for (int q = 0; q < 8; q++) acc[q] = fmaf(f, x[q], acc[q]);
            }
        }
        store8_row<VEC>(out, p.out_dtype, i, p.hidden, acc);
    }
}

// The rows of y are read, held as they come, before rows of dy are written: the compiler may not move a read
// across a write that could be to the same place (one row's read at a time: 98 us instead of 94 at the size above).
template <bool VEC, bool B16>
__global__ void __launch_bounds__(256) combine_backward_kernel(const CombineBwdArgs p) {
    constexpr int kHeld = B16 ? kBatch : kBatch / 2;
    __shared__ int32_t at[32];
    __shared__ float w[32];
    __shared__ float red[8][kHeld];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    pdl_wait();
    pdl_launch_next();
    if (threadIdx.x < 32) {
        int a = -1;
        float f = 0.0f;
        if (threadIdx.x < p.top_k) {
            const int64_t i = t * p.top_k + threadIdx.x;
            a = p.pos[i];
            if ((unsigned)a >= (unsigned)(p.n_tokens * p.top_k)) a = -1;
            f = p.w ? p.w[i] : 1.0f;
        }
        at[threadIdx.x] = a;
        w[threadIdx.x] = f;
    }
    __syncthreads();
    const void* dr = row_at(p.dout, p.dout_stride, type_size(p.dout_dtype), t);
    for (int j0 = 0; j0 < p.top_k; j0 += kHeld) {
        float dot[kHeld];
#pragma unroll
        for (int j = 0; j < kHeld; j++) dot[j] = 0.0f;
        for (int i = threadIdx.x * 8; cols_left<VEC>(i, p.hidden); i += blockDim.x * 8) {
            float d[8];
            load8_row<VEC>(dr, p.dout_dtype, i, p.hidden, d);
            Held8<VEC, B16> y[kHeld];
            if (p.dw) {
#pragma unroll
                for (int j = 0; j < kHeld; j++) {
                    const int a = at[j0 + j];
                    y[j].load(row_at(p.y, p.y_stride, type_size(p.y_dtype), max(a, 0)), p.y_dtype, i, a >= 0 ? p.hidden : 0);
                }
            }
#pragma unroll
            for (int j = 0; j < kHeld; j++) {
                const int a = at[j0 + j];
                if (a < 0) continue;
                float v[8];
                if (p.dw) {
                    y[j].get(p.y_dtype, v);
#pragma unroll
                    for (int q = 0; q < 8; q++) dot[j] = fmaf(d[q], v[q], dot[j]);
                }
                const float f = w[j0 + j];
#pragma unroll
                for (int q = 0; q < 8; q++) v[q] = f * d[q];
                store8_row<VEC>(row_at(p.dy, p.dy_stride, type_size(p.dy_dtype), a), p.dy_dtype, i, p.hidden, v);
            }
        }
        if (!p.dw) continue;
#pragma unroll
        for (int j = 0; j < kHeld; j++) {
            const float v = warp_sum(dot[j]);
            if (lane == 0) red[warp][j] = v;
        }
        __syncthreads();
        if (threadIdx.x < kHeld && j0 + threadIdx.x < p.top_k) {
            float v = 0.0f;
            for (int q = 0; q < nw; q++) v += red[q][threadIdx.x];
            p.dw[t * p.top_k + j0 + threadIdx.x] = v;
        }
        __syncthreads();
    }
}

// Threads for a row of `units` units: whole warps, at most 256.
unsigned row_threads(int units) { return (unsigned)std::min(256, (std::max(units, 1) + 31) / 32 * 32); }

template <int W>
cudaError_t dispatch_run(const DispatchArgs& p, cudaStream_t st) {
    const int64_t n = (int64_t)p.n_tokens * p.top_k;
    if (n <= kSmallN)
        return launch_pdl(dispatch_small_kernel<W>, dim3(p.n_tokens + 1), 256, (2 * p.n_experts + 1) * 4, st, p);
    const int chunk = chunk_entries(n), chunks = chunk_count(n);
    cudaError_t e = launch_pdl(dispatch_hist_kernel, dim3(chunks), kSortThreads, p.n_experts * 4, st, p.ids, (int)n,
                               p.n_experts, chunk, p.hist);
    if (e != cudaSuccess) return e;
    e = launch_pdl(dispatch_place_kernel, dim3(chunks), kPlaceThreads, (3 * p.n_experts + 1) * 4 + 32 * p.n_experts, st, p,
                   (int)n, chunk, chunks);
    if (e != cudaSuccess || !p.xs) return e;
    return launch_pdl(dispatch_rows_kernel<W>, dim3(p.n_tokens), row_threads(p.row_bytes / W), 0, st, p);
}

}  // namespace

size_t dispatch_workspace(int n_tokens, int top_k, int n_experts) {
    // a histogram a chunk, for the most chunks that n entries or fewer have: past 262144 entries chunks grow by 32 at a
    // time and their number falls, but a workspace is for calls of up to its size
    const int64_t n = (int64_t)n_tokens * top_k, most = std::min<int64_t>((n + kChunk - 1) / kChunk, kMaxChunks);
    return n <= kSmallN ? 256 : ((size_t)most * n_experts * 4 + 255) / 256 * 256;
}

cudaError_t launch_dispatch(const DispatchArgs& p, cudaStream_t st) {
    // bits that every row's address has in common
    const uintptr_t all =
        p.xs ? ((uintptr_t)p.x | (uintptr_t)p.xs | (uintptr_t)p.x_stride | (uintptr_t)p.xs_stride) : 0;
    if (all % 16 == 0) return dispatch_run<16>(p, st);
    if (all % 4 == 0) return dispatch_run<4>(p, st);
    if (all % 2 == 0) return dispatch_run<2>(p, st);
    return dispatch_run<1>(p, st);
}

cudaError_t launch_combine(const CombineArgs& p, cudaStream_t st) {
    if (p.n_tokens == 0) return cudaSuccess;
    const bool vec = p.hidden % 8 == 0 && al16(p.y, p.y_stride, p.y_dtype) && al16(p.out, p.out_stride, p.out_dtype);
    // few tokens: a row is split over CTAs of 64 threads so that more SMs load
    const int units = (p.hidden + 7) / 8;
    const unsigned block = p.n_tokens < 256 ? std::min(64u, row_threads(units)) : row_threads(units);
    const unsigned split = p.n_tokens < 256 ? (units + block - 1) / block : 1;
    const dim3 grid(p.n_tokens, split);
    if (!vec) return launch_pdl(combine_kernel<false, false>, grid, block, 0, st, p);
    return p.y_dtype == QS_BF16 ? launch_pdl(combine_kernel<true, true>, grid, block, 0, st, p)
                                : launch_pdl(combine_kernel<true, false>, grid, block, 0, st, p);
}

cudaError_t launch_combine_backward(const CombineBwdArgs& p, cudaStream_t st) {
    if (p.n_tokens == 0) return cudaSuccess;
    const bool vec = p.hidden % 8 == 0 && al16(p.dout, p.dout_stride, p.dout_dtype) &&
                     (!p.dw || al16(p.y, p.y_stride, p.y_dtype)) && al16(p.dy, p.dy_stride, p.dy_dtype);
    const unsigned block = row_threads((p.hidden + 7) / 8);
    if (!vec) return launch_pdl(combine_backward_kernel<false, false>, dim3(p.n_tokens), block, 0, st, p);
    return p.y_dtype == QS_BF16 || !p.dw ? launch_pdl(combine_backward_kernel<true, true>, dim3(p.n_tokens), block, 0, st, p)
                                         : launch_pdl(combine_backward_kernel<true, false>, dim3(p.n_tokens), block, 0, st, p);
}

}  // namespace qs
