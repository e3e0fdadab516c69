// qs_rows_api.cu -- C ABI of the row operators: argument checks, then the kernels.
#include "qs_internal.h"
#include "qs_rows.cuh"

using namespace qs;

namespace {

bool wide_type(int dtype) { return dtype == QS_F32 || dtype == QS_BF16; }

// A matrix of fp32 or bf16 rows: there, aligned to its elements, rows not longer than their stride
// (one row may have any stride).  A matrix without rows may have no address.
bool rows_ok(const void* p, int64_t stride, int dtype, int n_rows, int cols) {
    return (p || n_rows == 0) && wide_type(dtype) && ((uintptr_t)p % type_size(dtype)) == 0 && (stride >= cols || (n_rows <= 1 && stride >= 0));
}
bool codes_ok(const void* q, int64_t stride, const float* scale, int64_t scale_stride, int n_rows, int cols) {
    const bool one = n_rows <= 1;
    return ((q && scale) || n_rows == 0) && ((uintptr_t)scale & 3u) == 0 && (stride >= cols || (one && stride >= 0)) &&
           (scale_stride >= scale_blocks(cols) || (one && scale_stride >= 0));
}
bool eps_ok(float eps) { return eps >= 0.0f && eps <= 3.0e38f; }
bool entries_ok(int n_tokens, int top_k) {
    return n_tokens >= 0 && top_k >= 1 && top_k <= 32 && (int64_t)n_tokens * top_k <= (1ll << 30);
}
int done(cudaError_t e) { return e == cudaSuccess ? QS_OK : cuda_fail(e); }
size_t norm_parts_bytes(int hidden) { return (size_t)kNormParts * ((hidden + 7) / 8 * 8) * 4; }

}  // namespace

extern "C" {

int qs_rmsnorm_residual(const void* x, int64_t x_stride, int x_dtype, const void* residual, int64_t residual_stride,
                        int residual_dtype, const float* weight, float eps, int n_rows, int hidden, void* sum_out,
                        int64_t sum_stride, int sum_dtype, void* y, int64_t y_stride, int y_dtype, void* q,
                        int64_t q_stride, float* q_scale, int64_t q_scale_stride, void* stream) {
    if (n_rows < 0 || hidden < 1 || hidden > kNormMaxHidden || !eps_ok(eps)) return QS_ERR_INVALID;
    if (!rows_ok(x, x_stride, x_dtype, n_rows, hidden) || !weight || ((uintptr_t)weight & 3u)) return QS_ERR_INVALID;
    if (residual && !rows_ok(residual, residual_stride, residual_dtype, n_rows, hidden)) return QS_ERR_INVALID;
    if (sum_out && !rows_ok(sum_out, sum_stride, sum_dtype, n_rows, hidden)) return QS_ERR_INVALID;
    if (y && !rows_ok(y, y_stride, y_dtype, n_rows, hidden)) return QS_ERR_INVALID;
    if ((q || q_scale) && !codes_ok(q, q_stride, q_scale, q_scale_stride, n_rows, hidden)) return QS_ERR_INVALID;
    if (n_rows > 0 && !sum_out && !y && !q) return QS_ERR_INVALID;
    NormArgs p = {};
    p.x = x;
    p.residual = residual;
    p.weight = weight;
    p.sum_out = sum_out;
    p.y = y;
    p.q = static_cast<uint8_t*>(q);
    p.q_scale = q_scale;
    p.x_stride = x_stride;
    p.residual_stride = residual_stride;
    p.sum_stride = sum_stride;
    p.y_stride = y_stride;
    p.q_stride = q_stride;
    p.q_scale_stride = q_scale_stride;
    p.x_dtype = x_dtype;
    p.residual_dtype = residual_dtype;
    p.sum_dtype = sum_dtype;
    p.y_dtype = y_dtype;
    p.n_rows = n_rows;
    p.hidden = hidden;
    p.eps = eps;
    return done(launch_rmsnorm(p, (cudaStream_t)stream));
}

size_t qs_rmsnorm_backward_workspace_bytes(int hidden) {
    return hidden < 1 || hidden > kNormMaxHidden ? 0 : norm_parts_bytes(hidden);
}

int qs_rmsnorm_residual_backward(const void* sum, int64_t sum_stride, int sum_dtype, const float* weight, float eps,
                                 const void* dy, int64_t dy_stride, int dy_dtype, const void* dsum,
                                 int64_t dsum_stride, int dsum_dtype, int n_rows, int hidden, void* dx,
                                 int64_t dx_stride, int dx_dtype, float* dweight, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    if (n_rows < 0 || hidden < 1 || hidden > kNormMaxHidden || !eps_ok(eps)) return QS_ERR_INVALID;
    if (!rows_ok(sum, sum_stride, sum_dtype, n_rows, hidden) || !weight || ((uintptr_t)weight & 3u)) return QS_ERR_INVALID;
    if (!rows_ok(dy, dy_stride, dy_dtype, n_rows, hidden)) return QS_ERR_INVALID;
    if (dsum && !rows_ok(dsum, dsum_stride, dsum_dtype, n_rows, hidden)) return QS_ERR_INVALID;
    if (!rows_ok(dx, dx_stride, dx_dtype, n_rows, hidden) || ((uintptr_t)dweight & 3u)) return QS_ERR_INVALID;
    if (dweight && (!workspace || ((uintptr_t)workspace & 255u) || workspace_bytes < norm_parts_bytes(hidden)))
        return QS_ERR_WORKSPACE;
    NormBwdArgs p = {};
    p.sum = sum;
    p.weight = weight;
    p.dy = dy;
    p.dsum = dsum;
    p.dx = dx;
    p.partial = dweight ? static_cast<float*>(workspace) : nullptr;
    p.sum_stride = sum_stride;
    p.dy_stride = dy_stride;
    p.dsum_stride = dsum_stride;
    p.dx_stride = dx_stride;
    p.sum_dtype = sum_dtype;
    p.dy_dtype = dy_dtype;
    p.dsum_dtype = dsum_dtype;
    p.dx_dtype = dx_dtype;
    p.n_rows = n_rows;
    p.hidden = hidden;
    p.part_stride = (hidden + 7) / 8 * 8;
    p.eps = eps;
    return done(launch_rmsnorm_backward(p, dweight, (cudaStream_t)stream));
}

int qs_silu_mul_quant(const void* gate_up, int64_t gate_up_stride, int gate_up_dtype, int n_rows,
                      const int32_t* n_rows_dev, int ffn, void* q, int64_t q_stride, float* q_scale,
                      int64_t q_scale_stride, void* stream) {
    if (n_rows < 0 || ffn < 1 || ffn > (1 << 24)) return QS_ERR_INVALID;
    if (!rows_ok(gate_up, gate_up_stride, gate_up_dtype, n_rows, 2 * ffn)) return QS_ERR_INVALID;
    if (!codes_ok(q, q_stride, q_scale, q_scale_stride, n_rows, ffn) || ((uintptr_t)n_rows_dev & 3u)) return QS_ERR_INVALID;
    SiluArgs p = {};
    p.gate_up = gate_up;
    p.n_rows_dev = n_rows_dev;
    p.q = static_cast<uint8_t*>(q);
    p.q_scale = q_scale;
    p.gate_up_stride = gate_up_stride;
    p.q_stride = q_stride;
    p.q_scale_stride = q_scale_stride;
    p.dtype = gate_up_dtype;
    p.n_rows = n_rows;
    p.ffn = ffn;
    return done(launch_silu_mul_quant(p, (cudaStream_t)stream));
}

static bool matmul_shape_ok(int n_rows, int n_cols, int n_inner, int n_experts) {
    return n_rows >= 0 && n_cols >= 1 && n_inner >= 1 && n_inner <= (1 << 30) && n_cols <= (1 << 30) &&
           n_experts >= 1 && n_experts <= 1024;
}

size_t qs_fp8_matmul_workspace_bytes(int n_rows, int n_cols, int n_inner, int n_experts) {
    return matmul_shape_ok(n_rows, n_cols, n_inner, n_experts) ? fp8_matmul_workspace(n_rows, n_cols, n_inner, n_experts) : 0;
}

int qs_fp8_matmul(const void* a, int64_t a_stride, const float* a_scale, int64_t a_scale_stride, const void* w,
                  int64_t w_stride, int64_t w_expert_stride, const float* w_scale, const int32_t* offsets,
                  int n_experts, int n_rows, int n_cols, int n_inner, void* out, int64_t out_stride, int out_dtype,
                  void* workspace, size_t workspace_bytes, void* stream) {
    if (!matmul_shape_ok(n_rows, n_cols, n_inner, n_experts) || (!offsets && n_experts != 1)) return QS_ERR_INVALID;
    // the strides are a tensor map's: multiples of 16 bytes below 2^40, also where there is one row
    const int64_t top = 1ll << 40;
    if (!codes_ok(a, a_stride, a_scale, a_scale_stride, n_rows, n_inner) || ((uintptr_t)a & 15u) || a_stride % 16 ||
        a_stride < n_inner || a_stride >= top)
        return QS_ERR_INVALID;
    if (!w || !w_scale || ((uintptr_t)w & 15u) || ((uintptr_t)w_scale & 3u) || w_stride % 16 || w_stride < n_inner ||
        w_stride >= top || w_expert_stride % 16 || w_expert_stride >= top ||
        w_expert_stride < (n_experts > 1 ? w_stride * (n_cols - 1) + n_inner : 0) || ((uintptr_t)offsets & 3u))
        return QS_ERR_INVALID;
    if (!rows_ok(out, out_stride, out_dtype, n_rows, n_cols)) return QS_ERR_INVALID;
    if (!workspace || ((uintptr_t)workspace & 255u) ||
        workspace_bytes < fp8_matmul_workspace(n_rows, n_cols, n_inner, n_experts))
        return QS_ERR_WORKSPACE;
    Fp8MmArgs p = {};
    p.a = a;
    p.a_scale = a_scale;
    p.w = w;
    p.w_scale = w_scale;
    p.offsets = offsets;
    p.out = out;
    p.status = static_cast<uint32_t*>(workspace);
    p.a_stride = a_stride;
    p.a_scale_stride = a_scale_stride;
    p.w_stride = w_stride;
    p.w_expert_stride = n_experts > 1 ? w_expert_stride : w_stride;
    p.out_stride = out_stride;
    p.n_experts = n_experts;
    p.n_rows = n_rows;
    p.n_cols = n_cols;
    p.n_inner = n_inner;
    p.out_dtype = out_dtype;
    return done(launch_fp8_matmul(p, workspace, (cudaStream_t)stream));
}

size_t qs_dispatch_workspace_bytes(int n_tokens, int top_k, int n_experts) {
    return entries_ok(n_tokens, top_k) && n_experts >= 1 && n_experts <= 1024
               ? dispatch_workspace(n_tokens, top_k, n_experts)
               : 0;
}

int qs_dispatch_tokens(const int32_t* topk_ids, int n_tokens, int top_k, int n_experts, int32_t* counts,
                       int32_t* offsets, int32_t* perm, int32_t* pos, const void* x, int64_t x_stride, int x_dtype,
                       const float* x_scale, int64_t x_scale_stride, int hidden, void* xs, int64_t xs_stride,
                       float* xs_scale, int64_t xs_scale_stride, void* workspace, size_t workspace_bytes,
                       void* stream) {
    if (!entries_ok(n_tokens, top_k) || n_experts < 1 || n_experts > 1024) return QS_ERR_INVALID;
    if (!counts || !offsets || (n_tokens > 0 && (!topk_ids || !perm || !pos))) return QS_ERR_INVALID;
    if (((uintptr_t)topk_ids | (uintptr_t)counts | (uintptr_t)offsets | (uintptr_t)perm | (uintptr_t)pos) & 3u)
        return QS_ERR_INVALID;
    DispatchArgs p = {};
    if (xs) {
        const int n = n_tokens * top_k;
        if (hidden < 1 || hidden > (1 << 24)) return QS_ERR_INVALID;
        if (x_dtype == QS_E4M3) {
            if (!codes_ok(x, x_stride, x_scale, x_scale_stride, n_tokens, hidden) ||
                !codes_ok(xs, xs_stride, xs_scale, xs_scale_stride, n, hidden))
                return QS_ERR_INVALID;
            p.n_scales = scale_blocks(hidden);
        } else if (!rows_ok(x, x_stride, x_dtype, n_tokens, hidden) || !rows_ok(xs, xs_stride, x_dtype, n, hidden)) {
            return QS_ERR_INVALID;
        }
        p.row_bytes = hidden * type_size(x_dtype);
        p.x_stride = x_stride * type_size(x_dtype);
        p.xs_stride = xs_stride * type_size(x_dtype);
    }
    if (!workspace || ((uintptr_t)workspace & 255u) || workspace_bytes < dispatch_workspace(n_tokens, top_k, n_experts))
        return QS_ERR_WORKSPACE;
    p.ids = topk_ids;
    p.counts = counts;
    p.offsets = offsets;
    p.perm = perm;
    p.pos = pos;
    p.x = x;
    p.xs = xs;
    p.x_scale = x_scale;
    p.xs_scale = xs_scale;
    p.hist = static_cast<int32_t*>(workspace);
    p.x_scale_stride = x_scale_stride;
    p.xs_scale_stride = xs_scale_stride;
    p.n_tokens = n_tokens;
    p.top_k = top_k;
    p.n_experts = n_experts;
    return done(launch_dispatch(p, (cudaStream_t)stream));
}

int qs_combine_tokens(const void* y, int64_t y_stride, int y_dtype, const int32_t* pos, const float* topk_w,
                      int n_tokens, int top_k, int hidden, void* out, int64_t out_stride, int out_dtype,
                      void* stream) {
    if (!entries_ok(n_tokens, top_k) || hidden < 1 || hidden > (1 << 24) || (!pos && n_tokens > 0)) return QS_ERR_INVALID;
    if (((uintptr_t)pos | (uintptr_t)topk_w) & 3u) return QS_ERR_INVALID;
    if (!rows_ok(y, y_stride, y_dtype, n_tokens * top_k, hidden) || !rows_ok(out, out_stride, out_dtype, n_tokens, hidden))
        return QS_ERR_INVALID;
    CombineArgs p = {};
    p.y = y;
    p.pos = pos;
    p.w = topk_w;
    p.out = out;
    p.y_stride = y_stride;
    p.out_stride = out_stride;
    p.y_dtype = y_dtype;
    p.out_dtype = out_dtype;
    p.n_tokens = n_tokens;
    p.top_k = top_k;
    p.hidden = hidden;
    return done(launch_combine(p, (cudaStream_t)stream));
}

int qs_combine_tokens_backward(const void* dout, int64_t dout_stride, int dout_dtype, const void* y, int64_t y_stride,
                               int y_dtype, const int32_t* pos, const float* topk_w, int n_tokens, int top_k,
                               int hidden, void* dy, int64_t dy_stride, int dy_dtype, float* dtopk_w, void* stream) {
    if (!entries_ok(n_tokens, top_k) || hidden < 1 || hidden > (1 << 24) || (!pos && n_tokens > 0)) return QS_ERR_INVALID;
    if (((uintptr_t)pos | (uintptr_t)topk_w | (uintptr_t)dtopk_w) & 3u) return QS_ERR_INVALID;
    const int n = n_tokens * top_k;
    if (!rows_ok(dout, dout_stride, dout_dtype, n_tokens, hidden) || !rows_ok(dy, dy_stride, dy_dtype, n, hidden))
        return QS_ERR_INVALID;
    if (dtopk_w && !rows_ok(y, y_stride, y_dtype, n, hidden)) return QS_ERR_INVALID;
    CombineBwdArgs p = {};
    p.dout = dout;
    p.y = y;
    p.pos = pos;
    p.w = topk_w;
    p.dy = dy;
    p.dw = dtopk_w;
    p.dout_stride = dout_stride;
    p.y_stride = y_stride;
    p.dy_stride = dy_stride;
    p.dout_dtype = dout_dtype;
    p.y_dtype = y_dtype;
    p.dy_dtype = dy_dtype;
    p.n_tokens = n_tokens;
    p.top_k = top_k;
    p.hidden = hidden;
    return done(launch_combine_backward(p, (cudaStream_t)stream));
}

}  // extern "C"
