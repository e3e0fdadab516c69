// qs_cache.cu -- rows of new keys and values into the paged cache, and cached rows back (sm_103a).
//
// Writing.  bf16: the value rounded.  e4m3: one scale per token and head, scale = max(amax, 2^-100) / 448, code =
// v / scale rounded to nearest, ties to even (BlockCode: 448 / amax in two parts, so a code has one rounding before
// its own).  Reading: code * scale (one fp32 product) or the bf16 value, rounded to the output's type.
//
// Bound: HBM, each row in once and out once.  A head row is held by the lanes that take eight elements each (2 to 32 of
// them, a power of two), so a warp has one to 16 rows side by side and a row's maximum is at most five shuffles.  A
// warp takes kPasses such steps of one token, all their loads before the first use: at one row a warp in flight the
// copy was bound by latency.  The sequence of a token is looked up once a warp.
#include "qs_cache.cuh"

namespace qs {

namespace {

constexpr int kPasses = 4;   // steps of a warp
constexpr int kWarps = 4;    // of a CTA

// One of a token's 2 * n_kv head rows, keys first.
struct HeadRow {
    int which, head;
    bool there;
};
__device__ __forceinline__ HeadRow head_row(int r, int n_kv) {
    HeadRow h;
    h.which = r >= n_kv;
    h.head = r - (h.which ? n_kv : 0);
    h.there = r < 2 * n_kv;
    return h;
}

// Eight elements of a row from column i; VEC: 16-byte aligned rows.
template <bool VEC>
__device__ __forceinline__ void load8_at(const void* row, int dtype, int i, float (&v)[8]) {
    if (VEC) {
        load8_row<true>(row, dtype, i, i + 8, v);
    } else {
#pragma unroll
        for (int q = 0; q < 8; q++)
            v[q] = dtype == QS_BF16 ? bf16_lo(static_cast<const uint16_t*>(row)[i + q]) : static_cast<const float*>(row)[i + q];
    }
}
template <bool VEC>
__device__ __forceinline__ void store8_at(void* row, int dtype, int i, const float (&v)[8]) {
    if (VEC) {
        store8_row<true>(row, dtype, i, i + 8, v);
    } else {
#pragma unroll
        for (int q = 0; q < 8; q++) {
            if (dtype == QS_BF16) static_cast<__nv_bfloat16*>(row)[i + q] = __float2bfloat16_rn(v[q]);
            else static_cast<float*>(row)[i + q] = v[q];
        }
    }
}

template <bool E4, bool VEC>
__global__ void __launch_bounds__(32 * kWarps) cache_write_kernel(const CacheRowsArgs p) {
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_next();
    const int t = (int)(item / p.units), unit = (int)(item % p.units);
    if (t >= p.n_tokens) return;
    const int rows = 32 / p.lanes, col = (lane % p.lanes) * 8, first = (unit * kPasses) * rows + lane / p.lanes;
    const bool in = col < p.cache.head_dim;
    float v[kPasses][8];
#pragma unroll
    for (int k = 0; k < kPasses; k++) {
        const HeadRow h = head_row(first + k * rows, p.cache.n_kv);
#pragma unroll
        for (int q = 0; q < 8; q++) v[k][q] = 0.0f;
        if (h.there && in) {
            const HeadsView& x = h.which ? p.v : p.k;
            load8_at<VEC>(x.data + t * x.token_stride + h.head * x.head_stride, x.dtype, col, v[k]);
        }
    }
    int seq;
    int64_t pos;
    if (!token_at(p.seqs, t, seq, pos)) return;
    const Place at = place_of(p.cache, p.seqs, seq, pos);
    if (at.at < 0) return;
#pragma unroll
    for (int k = 0; k < kPasses; k++) {
        const HeadRow h = head_row(first + k * rows, p.cache.n_kv);
        uint8_t* row = (h.which ? p.cache.v : p.cache.k) + at.at + h.head * p.cache.head_stride;
        if (E4) {
            float a = 0.0f;
#pragma unroll
            for (int q = 0; q < 8; q++) a = fmaxf(a, fabsf(v[k][q]));
            const BlockCode code(lanes_max(a, p.lanes / 2), 1.0f, kMinAmax);
            if (!h.there || !in) continue;
            const float* x = v[k];
            *reinterpret_cast<uint2*>(row + col) =
                make_uint2(code.pair(x[0], x[1]) | (code.pair(x[2], x[3]) << 16), code.pair(x[4], x[5]) | (code.pair(x[6], x[7]) << 16));
            if (col == 0) (h.which ? p.cache.v_scale : p.cache.k_scale)[at.scale_at + h.head * p.cache.scale_head_stride] = code.scale;
        } else if (h.there && in) {
            store8_row<true>(row, QS_BF16, col, col + 8, v[k]);
        }
    }
}

template <bool E4, bool VEC>
__global__ void __launch_bounds__(32 * kWarps) cache_read_kernel(const CacheRowsArgs p) {
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_next();
    const int t = (int)(item / p.units), unit = (int)(item % p.units);
    if (t >= p.n_tokens) return;
    int seq;
    int64_t pos;
    if (!token_at(p.seqs, t, seq, pos)) return;
    const Place at = place_of(p.cache, p.seqs, seq, pos);
    const int rows = 32 / p.lanes, col = (lane % p.lanes) * 8, first = (unit * kPasses) * rows + lane / p.lanes;
    if (col >= p.cache.head_dim) return;
    uint4 raw[kPasses];
    float scale[kPasses];
#pragma unroll
    for (int k = 0; k < kPasses; k++) {
        const HeadRow h = head_row(first + k * rows, p.cache.n_kv);
        raw[k] = make_uint4(0, 0, 0, 0);
        scale[k] = 0.0f;
        if (!h.there || at.at < 0) continue;
        const uint8_t* row = (h.which ? p.cache.v : p.cache.k) + at.at + h.head * p.cache.head_stride;
        if (E4) {
            const uint2 w = *reinterpret_cast<const uint2*>(row + col);
            raw[k].x = w.x;
            raw[k].y = w.y;
            scale[k] = (h.which ? p.cache.v_scale : p.cache.k_scale)[at.scale_at + h.head * p.cache.scale_head_stride];
        } else {
            raw[k] = *reinterpret_cast<const uint4*>(row + 2 * col);
        }
    }
#pragma unroll
    for (int k = 0; k < kPasses; k++) {
        const HeadRow h = head_row(first + k * rows, p.cache.n_kv);
        if (!h.there) continue;
        float v[8];
        if (E4) {
            const uint32_t w[2] = {raw[k].x, raw[k].y};
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[q / 2] >> (16 * (q % 2))), __NV_E4M3)));
                v[2 * q] = f.x * scale[k];
                v[2 * q + 1] = f.y * scale[k];
            }
        } else {
            const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
            for (int q = 0; q < 4; q++) {
                v[2 * q] = bf16_lo(w[q]);
                v[2 * q + 1] = bf16_hi(w[q]);
            }
        }
        const HeadsView& x = h.which ? p.v : p.k;
        store8_at<VEC>(x.data + t * x.token_stride + h.head * x.head_stride, x.dtype, col, v);
    }
}

template <class K>
cudaError_t launch_rows(K kernel, CacheRowsArgs p, cudaStream_t st) {
    if (p.n_tokens == 0 || p.seqs.n_seqs == 0) return cudaSuccess;
    p.lanes = 2;
    while (p.lanes * 8 < p.cache.head_dim) p.lanes *= 2;
    const int rows = 32 / p.lanes * kPasses;  // of a unit
    p.units = (2 * p.cache.n_kv + rows - 1) / rows;
    const int64_t ctas = ((int64_t)p.n_tokens * p.units + kWarps - 1) / kWarps;
    return launch_pdl(kernel, dim3((unsigned)ctas), 32 * kWarps, 0, st, p);
}

}  // namespace

cudaError_t launch_cache_write(const CacheRowsArgs& p, cudaStream_t st) {
    if (p.cache.dtype == QS_E4M3) return p.aligned ? launch_rows(cache_write_kernel<true, true>, p, st) : launch_rows(cache_write_kernel<true, false>, p, st);
    return p.aligned ? launch_rows(cache_write_kernel<false, true>, p, st) : launch_rows(cache_write_kernel<false, false>, p, st);
}

cudaError_t launch_cache_read(const CacheRowsArgs& p, cudaStream_t st) {
    if (p.cache.dtype == QS_E4M3) return p.aligned ? launch_rows(cache_read_kernel<true, true>, p, st) : launch_rows(cache_read_kernel<true, false>, p, st);
    return p.aligned ? launch_rows(cache_read_kernel<false, true>, p, st) : launch_rows(cache_read_kernel<false, false>, p, st);
}

}  // namespace qs
