// qs_rows.cuh -- device helpers of the row operators: eight consecutive elements of a row read
// and written as fp32 / bf16 / e4m3, and the e4m3 encoding with one scale per 128 columns.
#pragma once

#include <cuda_fp8.h>

#include "qs_common.cuh"

namespace qs {

constexpr int kScaleCols = 128;                       // columns that share a scale
constexpr float kE4m3Max = 448.0f;                    // largest e4m3 value
constexpr float kMinAmax = 7.888609052210118e-31f;    // 2^-100: an all-zero block keeps a finite scale

__host__ __device__ constexpr int scale_blocks(int cols) { return (cols + kScaleCols - 1) / kScaleCols; }

// Wait for the kernels before this one in the stream (programmatic dependent launch); nothing is
// read or written before it.  The launch of the kernel after this one may then begin: it waits in
// the same way for this grid to end.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A warp takes 256 columns of a row at a time, a lane eight of them: i is the warp's first plus 8 * lane.
// VEC (the row 16-byte aligned, its length a multiple of 8): columns i .. i+7, one or two vectors, there or not
// as one.  Else every 32nd column from the warp's first plus lane, so that the lanes' single elements are neighbours.
template <bool VEC>
__device__ __forceinline__ int col_of(int i, int q) {
    const int lane = threadIdx.x & 31;
    return VEC ? i + q : i - 7 * lane + 32 * q;
}
// Whether a warp at i has a column below n.
template <bool VEC>
__device__ __forceinline__ bool cols_left(int i, int n) { return (VEC ? i : i - 8 * (int)(threadIdx.x & 31)) < n; }

// A lane's eight elements as fp32; those at and past n are 0.
template <bool VEC>
__device__ __forceinline__ void load8_row(const void* row, int dtype, int i, int n, float (&v)[8]) {
    if (VEC) {
        if (i >= n) {
#pragma unroll
            for (int q = 0; q < 8; q++) v[q] = 0.0f;
        } else if (dtype == QS_BF16) {
            const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + i);
            v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x);
            v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
            v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z);
            v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
        } else {
            const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(row) + i);
            const float4 a = p[0], b = p[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        }
    } else {
        if (dtype == QS_BF16) {
#pragma unroll
            for (int q = 0; q < 8; q++) {
                const int c = col_of<false>(i, q);
                v[q] = c < n ? bf16_lo(static_cast<const uint16_t*>(row)[c]) : 0.0f;
            }
        } else {
#pragma unroll
            for (int q = 0; q < 8; q++) {
                const int c = col_of<false>(i, q);
                v[q] = c < n ? static_cast<const float*>(row)[c] : 0.0f;
            }
        }
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// The same eight elements written, rounded once to the row's type.
template <bool VEC>
__device__ __forceinline__ void store8_row(void* row, int dtype, int i, int n, const float (&v)[8]) {
    if (VEC) {
        if (i >= n) return;
        if (dtype == QS_BF16) {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + i) =
                make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        } else {
            float4* p = reinterpret_cast<float4*>(static_cast<float*>(row) + i);
            p[0] = make_float4(v[0], v[1], v[2], v[3]);
            p[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
        if (dtype == QS_BF16) {
#pragma unroll
            for (int q = 0; q < 8; q++) {
                const int c = col_of<false>(i, q);
                if (c < n) static_cast<__nv_bfloat16*>(row)[c] = __float2bfloat16_rn(v[q]);
            }
        } else {
#pragma unroll
            for (int q = 0; q < 8; q++) {
                const int c = col_of<false>(i, q);
                if (c < n) static_cast<float*>(row)[c] = v[q];
            }
        }
    }
}

// Address of row r: stride in elements of `size` bytes, offsets in 64 bits.
__device__ __forceinline__ const void* row_at(const void* base, int64_t stride, int size, int64_t r) {
    return static_cast<const uint8_t*>(base) + r * stride * size;
}
__device__ __forceinline__ void* row_at(void* base, int64_t stride, int size, int64_t r) {
    return static_cast<uint8_t*>(base) + r * stride * size;
}
__host__ __device__ constexpr int type_size(int dtype) { return dtype == QS_F32 ? 4 : dtype == QS_BF16 ? 2 : 1; }

// How a scale block's values v * factor (one factor for the row) become codes, from a, the largest |v|.  The factor
// drops out of a code, v * factor * (448 / (a * factor)), so it is left out of it; 448 / a is held in two parts (its
// fp32 value and what that rounding left out), and a code's product has one rounding.  least: kMinAmax / factor.
// An infinite a leaves no remainder: all codes of the block are NaNs.
struct BlockCode {
    float inv, rest, scale;
    __device__ __forceinline__ BlockCode(float a, float factor, float least) {
        a = fmaxf(a, least);
        const float part = __frcp_rn(a);
        inv = kE4m3Max * part;
        rest = fmaf(-inv, a, kE4m3Max) * part;
        scale = a * factor * (1.0f / kE4m3Max);
    }
    __device__ __forceinline__ float scaled(float v) const { return fmaf(v, inv, v * rest); }
    __device__ __forceinline__ uint32_t pair(float lo, float hi) const {
        return __nv_cvt_float2_to_fp8x2(make_float2(scaled(lo), scaled(hi)), __NV_SATFINITE, __NV_E4M3);
    }
    __device__ __forceinline__ uint8_t one(float v) const { return __nv_cvt_float_to_fp8(scaled(v), __NV_SATFINITE, __NV_E4M3); }
};

// Largest |v| of the lanes that differ in the bits below 2 * first.  fmaxf drops a NaN: its own code is a NaN and
// the others of its block keep their scale.
__device__ __forceinline__ float lanes_max(float a, int first) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o <= first) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    return a;
}

// The 16 / N lanes that hold the 128 columns of one scale block, 8 N neighbours each (columns i .. i + 8 N - 1;
// those past n hold 0; n a multiple of 8): the block's scale, and the lane's codes.
template <int N>
__device__ __forceinline__ void quant_vec(const float (&v)[N][8], float factor, float least, uint8_t* q_row, float* scale_row,
                                          int i, int n) {
    float a = 0.0f;
#pragma unroll
    for (int k = 0; k < N; k++)
#pragma unroll
        for (int q = 0; q < 8; q++) a = fmaxf(a, fabsf(v[k][q]));
    const BlockCode code(lanes_max(a, kScaleCols / (16 * N)), factor, least);
    if (i >= n) return;
    if (i % kScaleCols == 0) scale_row[i / kScaleCols] = code.scale;
#pragma unroll
    for (int k = 0; k < N; k++) {
        const float* x = v[k];
        if (i + 8 * k < n)
            *reinterpret_cast<uint2*>(q_row + i + 8 * k) =
                make_uint2(code.pair(x[0], x[1]) | (code.pair(x[2], x[3]) << 16), code.pair(x[4], x[5]) | (code.pair(x[6], x[7]) << 16));
    }
}

// The same for a warp's 256 columns as col_of<false> has them: two scale blocks, four elements a lane of each.
__device__ __forceinline__ void quant_any(const float (&v)[8], float factor, float least, uint8_t* q_row, float* scale_row,
                                          int i, int n) {
    const int lane = threadIdx.x & 31, first = i - 8 * lane;
#pragma unroll
    for (int h = 0; h < 2; h++) {
        float a = 0.0f;
#pragma unroll
        for (int q = 4 * h; q < 4 * h + 4; q++) a = fmaxf(a, fabsf(v[q]));
        const BlockCode code(lanes_max(a, 16), factor, least);
        const int block = first / kScaleCols + h;
        if (lane == 0 && block * kScaleCols < n) scale_row[block] = code.scale;
#pragma unroll
        for (int q = 4 * h; q < 4 * h + 4; q++) {
            const int c = col_of<false>(i, q);
            if (c < n) q_row[c] = code.one(v[q]);
        }
    }
}

// Eight elements of a row as they were loaded, to be widened later: loads of the next row or slot stay
// in flight in half the registers (bf16).  B16: the row is known to be bf16.
template <bool VEC, bool B16>
struct Held8 {
    uint4 a, b;
    __device__ __forceinline__ void load(const void* row, int dtype, int i, int n) {
        static_assert(VEC, "whole vectors");
        if (i >= n) {
            a = make_uint4(0, 0, 0, 0);
            if (!B16) b = a;
        } else if (B16 || dtype == QS_BF16) {
            a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + i);
        } else {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(row) + i);
            a = p[0];
            b = p[1];
        }
    }
    __device__ __forceinline__ void get(int dtype, float (&v)[8]) const {
        if (B16 || dtype == QS_BF16) {
            v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x);
            v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
            v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z);
            v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
        } else {
            v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
            v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
        }
    }
};
template <>
struct Held8<false, false> {  // any alignment: single elements, as load8_row has them
    float f[8];
    __device__ __forceinline__ void load(const void* row, int dtype, int i, int n) { load8_row<false>(row, dtype, i, n, f); }
    __device__ __forceinline__ void get(int, float (&v)[8]) const {
#pragma unroll
        for (int q = 0; q < 8; q++) v[q] = f[q];
    }
};

// ------------------------------------------------------------------ host side

// Every row at 16-byte boundaries.
inline bool al16(const void* p, int64_t stride, int dtype) {
    return ((uintptr_t)p & 15u) == 0 && (stride * type_size(dtype)) % 16 == 0;
}

// A programmatic dependent launch: the kernel may start while the one before it in the stream ends, and waits for
// it (pdl_wait) before it reads or writes anything.
template <class K, class... A>
cudaError_t launch_pdl(K kernel, dim3 grid, unsigned block, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace qs
