// qs_norm.cu -- root-mean-square norm with the residual's addition, its gradient, and the SwiGLU
// activation, each with e4m3 output rows where asked (sm_103a).
//
// Norm.  s = x + residual, rho = 1 / sqrt(mean(s^2) + eps), v = s * rho * weight.  Bound: HBM (x
// and residual in once, the sum, y and codes out once).  A row is held in the registers of a group
// of G warps, eight consecutive elements a thread and step, so it is read once; the sum of squares
// is a fixed-order tree over the group.  Sixteen neighbouring threads hold the 128 columns of a
// scale, so a block's maximum is four shuffles and nothing is staged in shared memory.  16384 x 4096 in bf16 with
// the sum and the codes: 77 us, 6.1 TB/s; in fp32 without them 78 us, 6.9 TB/s.
//
// Gradient.  With g = weight * dy: dx = rho * (g - s * rho * (rho * mean(g * s))) + dsum.  Both sums over a
// row (s^2 and g * s) are formed in one pass; a group keeps its columns' share of dweight in
// registers over all its rows, a CTA writes one partial row, and a second launch adds the partial
// rows in a fixed order (no atomics: the same bits every run).  8192 x 2048 in bf16: 28 us, 4.8 TB/s; three CTAs an SM
// with two rows each in registers, 8 bytes a thread of them spilled (four CTAs with more spills 32 us, two 31).  In fp32
// 52 us, 5.1 TB/s.  Rows of more than 4096 columns in fp32 or 8192 in bf16 hold more than there are registers: 2048 x 8192
// in fp32 68 us, in bf16 35; 1024 x 16384 149 and 62.
#include "qs_internal.h"
#include "qs_rows.cuh"

#include <algorithm>

namespace qs {

namespace {

// Sum over a group of G warps, the same in every thread; red: G floats of the group's own, free
// again after the next call's first barrier.  bar: the group's named barrier.
template <int G, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* red, int wg, int lane, int bar) {
#pragma unroll
    for (int j = 0; j < N; j++) v[j] = warp_sum(v[j]);
    if (G == 1) return;
    if (lane == 0) {
#pragma unroll
        for (int j = 0; j < N; j++) red[j * G + wg] = v[j];
    }
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(32 * G) : "memory");
#pragma unroll
    for (int j = 0; j < N; j++) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < G; w++) t += red[j * G + w];
        v[j] = t;
    }
}

constexpr int cta_warps(int G) { return G < 8 ? 8 : G; }

// G warps a row, NV steps of eight elements a thread: rows of up to 256 * G * NV elements.  B16: every row that is
// there is known to be bf16 (2 to 4 % less time than with the types looked up).
template <bool VEC, bool B16, int G, int NV>
__global__ void __launch_bounds__(32 * cta_warps(G)) rmsnorm_kernel(const NormArgs p) {
    constexpr int kGroups = cta_warps(G) / G;
    __shared__ float red[kGroups][G];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = warp / G, wg = warp % G;
    const int64_t t = (int64_t)blockIdx.x * kGroups + group;
    auto col = [&](int j) { return (j * 32 * G + wg * 32 + lane) * 8; };
    const int x_type = B16 ? QS_BF16 : p.x_dtype, r_type = B16 ? QS_BF16 : p.residual_dtype;
    const int s_type = B16 ? QS_BF16 : p.sum_dtype, y_type = B16 ? QS_BF16 : p.y_dtype;
    pdl_wait();
    pdl_launch_next();
    if (t >= p.n_rows) return;
    const void* xr = row_at(p.x, p.x_stride, type_size(x_type), t);
    const void* rr = p.residual ? row_at(p.residual, p.residual_stride, type_size(r_type), t) : nullptr;
    float s[NV][1][8];
#pragma unroll
    for (int j = 0; j < NV; j++) load8_row<VEC>(xr, x_type, col(j), p.hidden, s[j][0]);
    if (rr) {
#pragma unroll
        for (int j = 0; j < NV; j++) {
            float r[8];
            load8_row<VEC>(rr, r_type, col(j), p.hidden, r);
#pragma unroll
            for (int q = 0; q < 8; q++) s[j][0][q] += r[q];
        }
    }
    float ss[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; j++)
#pragma unroll
        for (int q = 0; q < 8; q++) ss[0] = fmaf(s[j][0][q], s[j][0][q], ss[0]);
    if (p.sum_out) {
        void* o = row_at(p.sum_out, p.sum_stride, type_size(s_type), t);
#pragma unroll
        for (int j = 0; j < NV; j++) store8_row<VEC>(o, s_type, col(j), p.hidden, s[j][0]);
    }
    if (!p.y && !p.q) return;
    group_sum<G, 1>(ss, red[group], wg, lane, 1 + group);
    const float rho = rsqrtf(ss[0] / (float)p.hidden + p.eps);
    void* yr = p.y ? row_at(p.y, p.y_stride, type_size(y_type), t) : nullptr;
    // rho is left to the end, where it costs the codes no rounding; rows so small that it is large take it at once, and
    // so do those whose sum of squares is infinite, since kMinAmax over their rho of 0 made every block's scale a NaN
    const float factor = rho > 65536.0f || rho == 0.0f ? 1.0f : rho, least = kMinAmax / factor;
#pragma unroll
    for (int j = 0; j < NV; j++) {
        float w[8];  // read here, not before the barrier: early, it took 10 % more at 8192 fp32 columns and gave decode 0.15 us
        load8_row<VEC>(p.weight, QS_F32, col(j), p.hidden, w);
        if (rho != factor) {
#pragma unroll
            for (int q = 0; q < 8; q++) s[j][0][q] *= rho;
        }
#pragma unroll
        for (int q = 0; q < 8; q++) s[j][0][q] *= w[q];
        if (p.q) {
            uint8_t* q_row = p.q + t * p.q_stride;
            float* scale_row = p.q_scale + t * p.q_scale_stride;
            if (VEC) quant_vec<1>(s[j], factor, least, q_row, scale_row, col(j), p.hidden);
            else quant_any(s[j][0], factor, least, q_row, scale_row, col(j), p.hidden);
        }
        if (yr) {
#pragma unroll
            for (int q = 0; q < 8; q++) s[j][0][q] *= factor;
            store8_row<VEC>(yr, y_type, col(j), p.hidden, s[j][0]);
        }
    }
}

// Rows r = group, group + (number of groups), ...; row blockIdx.x of `partial` gets the CTA's dweight.  The
// next row is on its way while a row's sums cross the group: without that a row cost its whole latency.
template <bool VEC, bool B16, int G, int NV>
__global__ void __launch_bounds__(32 * cta_warps(G), B16 && NV == 1 && G <= 8 ? 3 : 1) rmsnorm_backward_kernel(const NormBwdArgs p) {
    constexpr int kGroups = cta_warps(G) / G, kCols = 256 * G * NV;
    __shared__ float red[kGroups][2][2 * G];
    __shared__ float part[kGroups > 1 ? kGroups : 1][kGroups > 1 ? kCols : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = warp / G, wg = warp % G;
    const int64_t first = (int64_t)blockIdx.x * kGroups + group, step = (int64_t)gridDim.x * kGroups;
    auto col = [&](int j) { return (j * 32 * G + wg * 32 + lane) * 8; };
    pdl_wait();
    pdl_launch_next();
    struct Row {
        Held8<VEC, B16> s[NV], g[NV], d[NV];
    };
    Row here, next;
    auto load = [&](Row& r, int64_t t) {
#pragma unroll
        for (int j = 0; j < NV; j++) {
            r.s[j].load(row_at(p.sum, p.sum_stride, type_size(p.sum_dtype), t), p.sum_dtype, col(j), p.hidden);
            r.g[j].load(row_at(p.dy, p.dy_stride, type_size(p.dy_dtype), t), p.dy_dtype, col(j), p.hidden);
            if (p.dsum) r.d[j].load(row_at(p.dsum, p.dsum_stride, type_size(p.dsum_dtype), t), p.dsum_dtype, col(j), p.hidden);
        }
    };
    float dw[NV][8], w0[8];
#pragma unroll
    for (int j = 0; j < NV; j++)
#pragma unroll
        for (int q = 0; q < 8; q++) dw[j][q] = 0.0f;
    if (NV == 1) load8_row<VEC>(p.weight, QS_F32, col(0), p.hidden, w0);
    if (VEC && first < p.n_rows) load(next, first);
    int flip = 0;
    for (int64_t t = first; t < p.n_rows; t += step, flip ^= 1) {
        if (VEC) {
            here = next;
            if (t + step < p.n_rows) load(next, t + step);
        } else {  // single elements are held widened: no room for two rows
            load(here, t);
        }
        float a[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < NV; j++) {
            float w[8], s[8], g[8];
            if (NV > 1) load8_row<VEC>(p.weight, QS_F32, col(j), p.hidden, w);
            here.s[j].get(p.sum_dtype, s);
            here.g[j].get(p.dy_dtype, g);
#pragma unroll
            for (int q = 0; q < 8; q++) {
                a[0] = fmaf(s[q], s[q], a[0]);
                a[1] = fmaf((NV > 1 ? w[q] : w0[q]) * g[q], s[q], a[1]);
            }
        }
        group_sum<G, 2>(a, red[group][flip], wg, lane, 1 + group);
        const float rho = rsqrtf(a[0] / (float)p.hidden + p.eps);
        // rho^3 alone leaves fp32 for rows of an rms under 1e-13 or over 1e12, rho * mean(g * s) does not
        const float c = rho * (a[1] / (float)p.hidden);
        void* o = row_at(p.dx, p.dx_stride, type_size(p.dx_dtype), t);
#pragma unroll
        for (int j = 0; j < NV; j++) {
            float w[8], s[8], g[8], d[8];
            if (NV > 1) load8_row<VEC>(p.weight, QS_F32, col(j), p.hidden, w);
            here.s[j].get(p.sum_dtype, s);
            here.g[j].get(p.dy_dtype, g);
            if (p.dsum) {
                here.d[j].get(p.dsum_dtype, d);
            } else {
#pragma unroll
                for (int q = 0; q < 8; q++) d[q] = 0.0f;
            }
#pragma unroll
            for (int q = 0; q < 8; q++) {
                const float unit = s[q] * rho;
                dw[j][q] = fmaf(g[q], unit, dw[j][q]);
                d[q] = fmaf(rho, fmaf(-c, unit, (NV > 1 ? w[q] : w0[q]) * g[q]), d[q]);
            }
            store8_row<VEC>(o, p.dx_dtype, col(j), p.hidden, d);
        }
    }
    if (!p.partial) return;
    // the CTA's groups in ascending order
    float* row = p.partial + (int64_t)blockIdx.x * p.part_stride;
    if (kGroups == 1) {
#pragma unroll
        for (int j = 0; j < NV; j++) store8_row<VEC>(row, QS_F32, col(j), p.part_stride, dw[j]);  // hidden rounded up to 8
    } else {
#pragma unroll
        for (int j = 0; j < NV; j++)
#pragma unroll
            for (int q = 0; q < 8; q++) part[group][col_of<VEC>(col(j), q)] = dw[j][q];
        __syncthreads();
        for (int i = threadIdx.x; i < p.part_stride; i += blockDim.x) {
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < kGroups; k++) v += part[k][i];
            row[i] = v;
        }
    }
}

// dweight[h] = sum of partial[r][h], r ascending within each of 32 slices of the rows, then the
// slices ascending.  32 columns a CTA (lanes: neighbouring columns), 32 slices (warps).
__global__ void __launch_bounds__(1024) rmsnorm_dweight_kernel(const float* __restrict__ partial, int n_parts,
                                                               int stride, int hidden, float* __restrict__ dweight) {
    __shared__ float sm[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.x * 32 + lane;
    pdl_wait();
    pdl_launch_next();
    float a = 0.0f;
    if (h < hidden) {
#pragma unroll 10
        for (int r = warp; r < n_parts; r += 32) a += partial[(size_t)r * stride + h];
    }
    sm[warp][lane] = a;
    __syncthreads();
    const float v = warp_sum(sm[lane][warp]);  // column `warp` of this CTA
    const int c = blockIdx.x * 32 + warp;
    if (lane == 0 && c < hidden) dweight[c] = v;
}

// silu(g) * u = g u / (1 + exp(-g)).  exp(-g) = 2^h (1 + r) with h the fp32 value next to -g / ln 2 and r = -g - h ln 2,
// what its rounding left out: without r the value is off by up to |g| 2^-24, which a block's scale shows where all its
// gates are far below zero (65536 x 512: 30.0 us without r, 31.2 with it, 37.0 with expf and __fdividef).  ex2.approx is off
// by 2^-22 at most, r by 2^-29 |h| (ln 2 in fp32), rcp.approx by 2^-23: with the other roundings under 2^-20 of the value.
// Below g = -87.3, where 1 / (1 + exp(-g)) is no normal number, the value is 0.
__device__ __forceinline__ float silu_mul(float g, float u) {
    constexpr double kLn2 = 0.69314718055994531;
    const float t = fminf(fmaxf(g, -88.0f), 88.0f), h = t * (float)(-1.0 / kLn2), r = fmaf(h, -(float)kLn2, -t);
    float e, d;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(h));
    e = fmaf(e, r, e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(1.0f + e));
    return g * d * u;
}

// Eight lanes a (row, 128 columns): sixteen elements of gate and of up each.
template <bool VEC>
__global__ void __launch_bounds__(256) silu_mul_quant_kernel(const SiluArgs p) {
    pdl_wait();
    pdl_launch_next();
    const unsigned nb = scale_blocks(p.ffn);
    const unsigned part = threadIdx.x >> 3, l = threadIdx.x & 7;
    int64_t rows = p.n_rows;
    if (p.n_rows_dev) rows = min(rows, (int64_t)max(*p.n_rows_dev, 0));
    // (row, block) of these eight lanes, and the step to their next: the grid is small enough for 32 bits
    const unsigned u0 = blockIdx.x * 32 + part, du = gridDim.x * 32;
    int64_t t = u0 / nb;
    unsigned b = u0 % nb;
    const unsigned dt = du / nb, db = du % nb;
    // a warp's four parts all run the shuffles as long as one has work
    while (__any_sync(0xffffffffu, t < rows)) {
        const bool on = t < rows;
        const int64_t r = on ? t : 0;
        const uint8_t* row = static_cast<const uint8_t*>(row_at(p.gate_up, p.gate_up_stride, type_size(p.dtype), r));
        const uint8_t* up = row + (size_t)p.ffn * type_size(p.dtype);
        uint8_t* q_row = p.q + r * p.q_stride;
        float* scale_row = p.q_scale + r * p.q_scale_stride;
        const int first = (int)(b * kScaleCols), n = on ? p.ffn : 0;
        if (VEC) {  // sixteen neighbours a lane
            const int i = first + l * 16;
            float g[2][8], v[2][8];
#pragma unroll
            for (int k = 0; k < 2; k++) {
                load8_row<true>(row, p.dtype, i + 8 * k, n, g[k]);
                load8_row<true>(up, p.dtype, i + 8 * k, n, v[k]);
            }
#pragma unroll
            for (int k = 0; k < 2; k++)
#pragma unroll
                for (int q = 0; q < 8; q++) v[k][q] = silu_mul(g[k][q], v[k][q]);
            quant_vec<2>(v, 1.0f, kMinAmax, q_row, scale_row, i, n);
        } else {  // every eighth
            float v[16], a = 0.0f;
#pragma unroll
            for (int q = 0; q < 16; q++) {
                const int c = first + l + 8 * q;
                v[q] = c < n ? silu_mul(load_x(row, p.dtype, (size_t)c), load_x(up, p.dtype, (size_t)c)) : 0.0f;
                a = fmaxf(a, fabsf(v[q]));
            }
            const BlockCode code(lanes_max(a, 4), 1.0f, kMinAmax);
            if (l == 0 && first < n) scale_row[b] = code.scale;
#pragma unroll
            for (int q = 0; q < 16; q++)
                if (first + (int)l + 8 * q < n) q_row[first + l + 8 * q] = code.one(v[q]);
        }
        t += dt;
        b += db;
        if (b >= nb) {
            b -= nb;
            t++;
        }
    }
}

template <bool VEC, bool B16, int G, int NV>
cudaError_t norm_run(const NormArgs& p, cudaStream_t st) {
    constexpr int groups = cta_warps(G) / G;
    return launch_pdl(rmsnorm_kernel<VEC, B16, G, NV>, dim3((unsigned)(((int64_t)p.n_rows + groups - 1) / groups)), 32 * cta_warps(G), 0, st, p);
}

template <bool VEC, bool B16>
cudaError_t norm_pick(const NormArgs& p, cudaStream_t st) {
    // Few rows: as many threads a row as have a load, for the least latency (32 x 2048: 2.1 us, with two warps
    // a row 4.0).  Many: a warp a row where its registers hold it, which needs no barrier, else eight.  32768 rows of
    // 1024: 43 us; with the types looked up 46, with two warps 53, with four 64.  Of 2048: 85; with the types looked up
    // 91, with four warps 90, with two 89.  16384 of 4096: 77; with the types looked up 85, with sixteen warps 94, with four 84.
    const bool few = p.n_rows <= 304;  // two a SM
    if (p.hidden <= 256) return norm_run<VEC, B16, 1, 1>(p, st);
    if (p.hidden <= 512) return norm_run<VEC, B16, 1, 2>(p, st);
    if (p.hidden <= 1024) return few ? norm_run<VEC, B16, 4, 1>(p, st) : norm_run<VEC, B16, 1, 4>(p, st);
    if (p.hidden <= 2048) return norm_run<VEC, B16, 8, 1>(p, st);
    if (p.hidden <= 4096) return few ? norm_run<VEC, B16, 16, 1>(p, st) : norm_run<VEC, B16, 8, 2>(p, st);
    if (p.hidden <= 8192) return norm_run<VEC, false, 16, 2>(p, st);
    return norm_run<VEC, false, 16, 4>(p, st);
}

template <bool VEC, bool B16, int G, int NV>
cudaError_t norm_bwd_run(NormBwdArgs p, float* dweight, cudaStream_t st) {
    constexpr int groups = cta_warps(G) / G;
    const int64_t ctas = ((int64_t)p.n_rows + groups - 1) / groups;
    const unsigned grid = (unsigned)std::min<int64_t>(ctas, kNormParts);
    if (grid > 0) {
        const cudaError_t e = launch_pdl(rmsnorm_backward_kernel<VEC, B16, G, NV>, dim3(grid), 32 * cta_warps(G), 0, st, p);
        if (e != cudaSuccess) return e;
    }
    if (!dweight) return cudaSuccess;
    return launch_pdl(rmsnorm_dweight_kernel, dim3((unsigned)((p.hidden + 31) / 32)), 1024, 0, st, (const float*)p.partial,
                      (int)grid, p.part_stride, p.hidden, dweight);
}

template <bool VEC, bool B16>
cudaError_t norm_bwd_pick(const NormBwdArgs& p, float* dweight, cudaStream_t st) {
    if (p.hidden <= 256) return norm_bwd_run<VEC, B16, 1, 1>(p, dweight, st);
    if (p.hidden <= 512) return norm_bwd_run<VEC, B16, 2, 1>(p, dweight, st);
    if (p.hidden <= 1024) return norm_bwd_run<VEC, B16, 4, 1>(p, dweight, st);
    if (p.hidden <= 2048) return norm_bwd_run<VEC, B16, 8, 1>(p, dweight, st);
    if (p.hidden <= 4096) return norm_bwd_run<VEC, B16, 16, 1>(p, dweight, st);
    if (p.hidden <= 8192) return norm_bwd_run<VEC, B16, 16, 2>(p, dweight, st);
    return norm_bwd_run<VEC, B16, 16, 4>(p, dweight, st);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs& p, cudaStream_t st) {
    if (p.n_rows == 0) return cudaSuccess;
    const bool vec = p.hidden % 8 == 0 && al16(p.x, p.x_stride, p.x_dtype) &&
                     (!p.residual || al16(p.residual, p.residual_stride, p.residual_dtype)) &&
                     al16(p.weight, 0, QS_F32) && (!p.sum_out || al16(p.sum_out, p.sum_stride, p.sum_dtype)) &&
                     (!p.y || al16(p.y, p.y_stride, p.y_dtype)) &&
                     (!p.q || (((uintptr_t)p.q & 7u) == 0 && p.q_stride % 8 == 0));
    const bool b16 = p.x_dtype == QS_BF16 && (!p.residual || p.residual_dtype == QS_BF16) &&
                     (!p.sum_out || p.sum_dtype == QS_BF16) && (!p.y || p.y_dtype == QS_BF16);
    if (!vec) return norm_pick<false, false>(p, st);
    return b16 ? norm_pick<true, true>(p, st) : norm_pick<true, false>(p, st);
}

cudaError_t launch_rmsnorm_backward(const NormBwdArgs& p, float* dweight, cudaStream_t st) {
    const bool vec = p.hidden % 8 == 0 && al16(p.sum, p.sum_stride, p.sum_dtype) &&
                     al16(p.dy, p.dy_stride, p.dy_dtype) && al16(p.weight, 0, QS_F32) &&
                     (!p.dsum || al16(p.dsum, p.dsum_stride, p.dsum_dtype)) && al16(p.dx, p.dx_stride, p.dx_dtype);
    const bool b16 = p.sum_dtype == QS_BF16 && p.dy_dtype == QS_BF16 && (!p.dsum || p.dsum_dtype == QS_BF16);
    if (!vec) return norm_bwd_pick<false, false>(p, dweight, st);
    return b16 ? norm_bwd_pick<true, true>(p, dweight, st) : norm_bwd_pick<true, false>(p, dweight, st);
}

cudaError_t launch_silu_mul_quant(const SiluArgs& p, cudaStream_t st) {
    if (p.n_rows == 0) return cudaSuccess;
    const bool vec = p.ffn % 8 == 0 && al16(p.gate_up, p.gate_up_stride, p.dtype) &&
                     (p.ffn * type_size(p.dtype)) % 16 == 0 && ((uintptr_t)p.q & 7u) == 0 && p.q_stride % 8 == 0;
    const int64_t work = (int64_t)p.n_rows * scale_blocks(p.ffn);
    const unsigned grid = (unsigned)std::min<int64_t>((work + 31) / 32, 1216);  // eight CTAs an SM walk on: 31.2 us at 65536 x 512; with one step each 12 % more
    return vec ? launch_pdl(silu_mul_quant_kernel<true>, dim3(grid), 256, 0, st, p)
               : launch_pdl(silu_mul_quant_kernel<false>, dim3(grid), 256, 0, st, p);
}

}  // namespace qs
