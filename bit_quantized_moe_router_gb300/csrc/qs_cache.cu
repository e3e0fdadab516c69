// qs_cache.cu -- rows of new keys and values into the paged cache, and cached rows back (sm_103a).
//
// Writing.  bf16: the value rounded.  e4m3: one scale per token and head, scale = max(amax, 2^-100) / 448, code =
// v / scale rounded to nearest, ties to even (BlockCode: 448 / amax in two parts, so a code has one rounding before
// its own).  Reading: code * scale (one fp32 product) or the bf16 value, rounded to the output's type.
//
// Bound: HBM, each row in once and out once, and nearly as much the instructions of a row (its maximum, the codes' own
// rounding, addresses).  A head row is held by the lanes that take eight elements each (2 to 32 of them, a power of two),
// so a warp has one to 16 rows side by side.  A warp takes kPasses such steps of one token, all their loads before the first
// use and held as they came: eight steps where there are many rows (16384 tokens of 8 heads of 128 into e4m3, with a
// butterfly and a reciprocal a row: 25.1 us with eight, 26.4 with four, 31.7 with two), two where all warps have a place
// at once (one token of 2 heads of 256: 2.2 us, 3.8 with eight).  Of eight steps' rows each is one group of lanes' to reduce and
// to take the reciprocal of (23.7 -> 20.7 us; addresses added up, not multiplied, were 25.1 -> 23.7).  The place of a token is
// looked up once a warp, while its rows are on their way.  On one GB300, cold: that write 20.7 us (4.9 TB/s), 32768 e4m3 tokens of
// 8 heads of 128 read into bf16 33.2 us (6.1 TB/s).
#include "qs_cache.cuh"

namespace qs {

namespace {

constexpr int kWarps = 4;    // of a CTA

// A lane's head rows of a token, keys' first: r, r + rows, ... of 2 * n_kv.  Addresses go along by additions (as integers:
// those of the half that a row is not in are never used).
template <class T>
struct Walk {
    T *k, *v;
    int64_t k_step, v_step;
    __device__ __forceinline__ Walk(T* keys, T* values, int64_t k_stride, int64_t v_stride, int r, int n_kv, int rows)
        : k(reinterpret_cast<T*>((uintptr_t)keys + r * k_stride * (int64_t)sizeof(T))),
          v(reinterpret_cast<T*>((uintptr_t)values + (r - n_kv) * v_stride * (int64_t)sizeof(T))),
          k_step(rows * k_stride * (int64_t)sizeof(T)), v_step(rows * v_stride * (int64_t)sizeof(T)) {}
    __device__ __forceinline__ T* row(bool which) const { return which ? v : k; }
    __device__ __forceinline__ void next() {
        k = reinterpret_cast<T*>((uintptr_t)k + k_step);
        v = reinterpret_cast<T*>((uintptr_t)v + v_step);
    }
};

// Eight elements of a row from column i, as they are and widened.  VEC: 16-byte aligned rows; B16: bf16, else fp32.
template <bool VEC, bool B16>
struct Eight {
    uint4 a, b;
    __device__ __forceinline__ void clear() {
        a = make_uint4(0, 0, 0, 0);
        if (!B16) b = a;
    }
    __device__ __forceinline__ void load(const void* row, int i) {
        if (VEC) {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + i * (B16 ? 2 : 4));
            a = p[0];
            if (!B16) b = p[1];
        } else if (B16) {
            const uint16_t* p = static_cast<const uint16_t*>(row) + i;
            a = make_uint4(p[0] | (uint32_t)p[1] << 16, p[2] | (uint32_t)p[3] << 16, p[4] | (uint32_t)p[5] << 16, p[6] | (uint32_t)p[7] << 16);
        } else {
            const uint32_t* p = static_cast<const uint32_t*>(row) + i;
            a = make_uint4(p[0], p[1], p[2], p[3]);
            b = make_uint4(p[4], p[5], p[6], p[7]);
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        if (B16) {
            v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x);
            v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
            v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z);
            v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
        } else {
            v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
            v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
        }
    }
    // The largest |v|, a NaN left out; bf16 two at a time.
    __device__ __forceinline__ float largest() const {
        if (B16) {
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
            __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[0]));
#pragma unroll
            for (int q = 1; q < 4; q++) m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[q])));
            return fmaxf(__low2float(m), __high2float(m));
        }
        float v[8], m = 0.0f;
        get(v);
#pragma unroll
        for (int q = 0; q < 8; q++) m = fmaxf(m, fabsf(v[q]));
        return m;
    }
};

// The maxima of eight rows over the lanes that hold them (8 or more, a power of two): a lane's a[] are its own columns' of
// each, and it ends with that of the row returned.  Halves are swapped, so that a lane keeps half of the rows at a step: 8
// shuffles where a butterfly a row takes 24 to 40.
__device__ __forceinline__ int max_of_rows(float (&a)[8], int lanes, float& most) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int half = 4; half > 0; half >>= 1) {
        lanes >>= 1;
        const bool upper = lane & lanes;
#pragma unroll
        for (int k = 0; k < half; k++) {
            const float other = __shfl_xor_sync(0xffffffffu, upper ? a[k] : a[k + half], lanes);
            a[k] = fmaxf(upper ? a[k + half] : a[k], other);
        }
    }
    const int row = lane / lanes & 7;
    most = a[0];
#pragma unroll 1
    for (int o = lanes >> 1; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    return row;
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

template <int kPasses, bool E4, bool VEC, bool B16>
__global__ void __launch_bounds__(32 * kWarps) cache_write_kernel(const CacheRowsArgs p) {
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_next();
    if (t >= p.n_tokens) return;
    const int lanes = 1 << p.lane_bits, rows = 32 >> p.lane_bits, col = (lane & (lanes - 1)) * 8, first = blockIdx.y * kPasses * rows + (lane >> p.lane_bits);
    const bool in = col < p.cache.head_dim;
    const int n_kv = p.cache.n_kv;
    Eight<VEC, B16> x[kPasses];
    Walk<uint8_t> from(p.k.data + t * p.k.token_stride, p.v.data + t * p.v.token_stride, p.k.head_stride, p.v.head_stride, first, n_kv, rows);
#pragma unroll
    for (int k = 0; k < kPasses; k++) {
        const int r = first + k * rows;
        x[k].clear();
        if (in && r < 2 * n_kv) x[k].load(from.row(r >= n_kv), col);
        from.next();
    }
    int seq;
    int64_t pos;
    if (!token_at(p.seqs, t, seq, pos)) return;
    const Place at = place_of(p.cache, p.seqs, seq, pos);
    if (at.at < 0) return;
    Walk<uint8_t> to(p.cache.k + at.at, p.cache.v + at.at, p.cache.head_stride, p.cache.head_stride, first, n_kv, rows);
    float* const k_scale = p.cache.k_scale + at.scale_at;
    float* const v_scale = p.cache.v_scale + at.scale_at;
    const auto scale_to = [&](int r) { return r < n_kv ? k_scale + r * p.cache.scale_head_stride : v_scale + (r - n_kv) * p.cache.scale_head_stride; };
    // The rows' factors: with eight rows a group of lanes each has one of them to compute, and all get them from shared memory.
    __shared__ float2 factor_of[E4 && kPasses == 8 ? kWarps : 1][8][4];
    const bool dealt = E4 && kPasses == 8 && lanes >= 8;
    if (dealt) {
        float a[8], most;
#pragma unroll
        for (int k = 0; k < 8; k++) a[k] = x[k % kPasses].largest();
        const int k = max_of_rows(a, lanes, most), r = first + k * rows;
        const BlockCode code(most, 1.0f, kMinAmax);
        if ((lane & (lanes / 8 - 1)) == 0) {
            factor_of[threadIdx.x >> 5][k][lane >> p.lane_bits] = make_float2(code.inv, code.rest);
            if (r < 2 * n_kv) *scale_to(r) = code.scale;
        }
        __syncwarp();
    }
#pragma unroll
    for (int k = 0; k < kPasses; k++, to.next()) {
        const int r = first + k * rows;
        const bool there = in && r < 2 * n_kv;
        uint8_t* row = to.row(r >= n_kv);
        float v[8];
        x[k].get(v);
        if (E4) {
            BlockCode code;
            if (dealt) {
                const float2 f = factor_of[threadIdx.x >> 5][k][lane >> p.lane_bits];
                code.inv = f.x;
                code.rest = f.y;
            } else {
                code = BlockCode(lanes_max(x[k].largest(), lanes / 2), 1.0f, kMinAmax);
                if (there && col == 0) *scale_to(r) = code.scale;
            }
            if (!there) continue;
            *reinterpret_cast<uint2*>(row + col) =
                make_uint2(code.pair(v[0], v[1]) | (code.pair(v[2], v[3]) << 16), code.pair(v[4], v[5]) | (code.pair(v[6], v[7]) << 16));
        } else if (there) {
            store8_row<true>(row, QS_BF16, col, col + 8, v);
        }
    }
}

template <int kPasses, bool E4, bool VEC>
__global__ void __launch_bounds__(32 * kWarps) cache_read_kernel(const CacheRowsArgs p) {
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_next();
    if (t >= p.n_tokens) return;
    int seq;
    int64_t pos;
    if (!token_at(p.seqs, t, seq, pos)) return;
    const Place at = place_of(p.cache, p.seqs, seq, pos);
    const int lanes = 1 << p.lane_bits, rows = 32 >> p.lane_bits, col = (lane & (lanes - 1)) * 8, first = blockIdx.y * kPasses * rows + (lane >> p.lane_bits);
    if (col >= p.cache.head_dim) return;
    const int n_kv = p.cache.n_kv;
    uint4 raw[kPasses];
    float scale[kPasses];
    Walk<uint8_t> from(p.cache.k + at.at, p.cache.v + at.at, p.cache.head_stride, p.cache.head_stride, first, n_kv, rows);
    Walk<float> scale_from(p.cache.k_scale + at.scale_at, p.cache.v_scale + at.scale_at, p.cache.scale_head_stride, p.cache.scale_head_stride, first, n_kv, rows);
#pragma unroll
    for (int k = 0; k < kPasses; k++, from.next(), scale_from.next()) {
        const int r = first + k * rows;
        raw[k] = make_uint4(0, 0, 0, 0);
        scale[k] = 0.0f;
        if (r >= 2 * n_kv || at.at < 0) continue;
        const uint8_t* row = from.row(r >= n_kv);
        if (E4) {
            const uint2 w = *reinterpret_cast<const uint2*>(row + col);
            raw[k].x = w.x;
            raw[k].y = w.y;
            scale[k] = *scale_from.row(r >= n_kv);
        } else {
            raw[k] = *reinterpret_cast<const uint4*>(row + 2 * col);
        }
    }
    Walk<uint8_t> to(p.k.data + t * p.k.token_stride, p.v.data + t * p.v.token_stride, p.k.head_stride, p.v.head_stride, first, n_kv, rows);
#pragma unroll
    for (int k = 0; k < kPasses; k++, to.next()) {
        const int r = first + k * rows;
        if (r >= 2 * n_kv) continue;
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
        store8_at<VEC>(to.row(r >= n_kv), p.k.dtype, col, v);
    }
}

// few and many: the kernel with two and with eight steps a warp.
template <class K>
cudaError_t launch_rows(K few, K many, CacheRowsArgs p, cudaStream_t st) {
    if (p.n_tokens == 0 || p.seqs.n_seqs == 0) return cudaSuccess;
    p.lane_bits = 1;
    while ((8 << p.lane_bits) < p.cache.head_dim) p.lane_bits++;
    const int head_rows = 2 * p.cache.n_kv, rows = 32 >> p.lane_bits;  // of a token, of a step
    const int units = (head_rows + 2 * rows - 1) / (2 * rows);
    const bool small = (int64_t)p.n_tokens * units <= 152 * 32;        // warps that run at once
    const dim3 grid((p.n_tokens + kWarps - 1) / kWarps, small ? units : (head_rows + 8 * rows - 1) / (8 * rows));
    return launch_pdl(small ? few : many, grid, 32 * kWarps, 0, st, p);
}

template <bool E4, bool VEC, bool B16>
cudaError_t launch_write(const CacheRowsArgs& p, cudaStream_t st) {
    return launch_rows(cache_write_kernel<2, E4, VEC, B16>, cache_write_kernel<8, E4, VEC, B16>, p, st);
}
template <bool E4, bool VEC>
cudaError_t launch_read(const CacheRowsArgs& p, cudaStream_t st) {
    return launch_rows(cache_read_kernel<2, E4, VEC>, cache_read_kernel<8, E4, VEC>, p, st);
}

}  // namespace

cudaError_t launch_cache_write(const CacheRowsArgs& p, cudaStream_t st) {
    const bool e4 = p.cache.dtype == QS_E4M3, b16 = p.k.dtype == QS_BF16;  // v's type too
    if (p.aligned) {
        if (e4) return b16 ? launch_write<true, true, true>(p, st) : launch_write<true, true, false>(p, st);
        return b16 ? launch_write<false, true, true>(p, st) : launch_write<false, true, false>(p, st);
    }
    if (e4) return b16 ? launch_write<true, false, true>(p, st) : launch_write<true, false, false>(p, st);
    return b16 ? launch_write<false, false, true>(p, st) : launch_write<false, false, false>(p, st);
}

cudaError_t launch_cache_read(const CacheRowsArgs& p, cudaStream_t st) {
    if (p.cache.dtype == QS_E4M3) return p.aligned ? launch_read<true, true>(p, st) : launch_read<true, false>(p, st);
    return p.aligned ? launch_read<false, true>(p, st) : launch_read<false, false>(p, st);
}

}  // namespace qs
