// qs_rows_api.cu -- C ABI of the row operators: argument checks, then the kernels.
#include "qs_internal.h"
#include "qs_rows.cuh"

using namespace qs;

namespace {

bool wide_type(int dtype) { return dtype == QS_F32 || dtype == QS_BF16; }

// A matrix of fp32 or bf16 rows: there, aligned to its elements, rows not longer than their stride
// (one row may have any stride).  A matrix without rows may have no address.
bool rows_ok(const qs_rows& m, int n_rows, int cols) {
    return (m.data || n_rows == 0) && wide_type(m.dtype) && ((uintptr_t)m.data % type_size(m.dtype)) == 0 &&
           (m.stride >= cols || (n_rows <= 1 && m.stride >= 0));
}
bool codes_ok(const qs_codes& m, int n_rows, int cols) {
    const bool one = n_rows <= 1;
    return ((m.q && m.scale) || n_rows == 0) && ((uintptr_t)m.scale & 3u) == 0 &&
           (m.stride >= cols || (one && m.stride >= 0)) &&
           (m.scale_stride >= scale_blocks(cols) || (one && m.scale_stride >= 0));
}
bool eps_ok(float eps) { return eps >= 0.0f && eps <= 3.0e38f; }
bool entries_ok(int n_tokens, int top_k) {
    return n_tokens >= 0 && top_k >= 1 && top_k <= 32 && (int64_t)n_tokens * top_k <= (1ll << 30);
}
int done(cudaError_t e) { return e == cudaSuccess ? QS_OK : cuda_fail(e); }
size_t norm_parts_bytes(int hidden) { return (size_t)kNormParts * ((hidden + 7) / 8 * 8) * 4; }

}  // namespace

extern "C" {

int qs_rmsnorm_residual(const qs_rmsnorm_args* args, void* stream) {
    if (!args) return QS_ERR_INVALID;
    const qs_rmsnorm_args& a = *args;
    const int n = a.n_rows, h = a.hidden;
    if (n < 0 || h < 1 || h > kNormMaxHidden || !eps_ok(a.eps)) return QS_ERR_INVALID;
    if (!rows_ok(a.x, n, h) || !a.weight || ((uintptr_t)a.weight & 3u)) return QS_ERR_INVALID;
    if (a.residual.data && !rows_ok(a.residual, n, h)) return QS_ERR_INVALID;
    if (a.sum_out.data && !rows_ok(a.sum_out, n, h)) return QS_ERR_INVALID;
    if (a.y.data && !rows_ok(a.y, n, h)) return QS_ERR_INVALID;
    if ((a.q.q || a.q.scale) && !codes_ok(a.q, n, h)) return QS_ERR_INVALID;
    if (n > 0 && !a.sum_out.data && !a.y.data && !a.q.q) return QS_ERR_INVALID;
    NormArgs p = {};
    p.x = a.x.data;
    p.residual = a.residual.data;
    p.weight = a.weight;
    p.sum_out = a.sum_out.data;
    p.y = a.y.data;
    p.q = static_cast<uint8_t*>(a.q.q);
    p.q_scale = a.q.scale;
    p.x_stride = a.x.stride;
    p.residual_stride = a.residual.stride;
    p.sum_stride = a.sum_out.stride;
    p.y_stride = a.y.stride;
    p.q_stride = a.q.stride;
    p.q_scale_stride = a.q.scale_stride;
    p.x_dtype = a.x.dtype;
    p.residual_dtype = a.residual.dtype;
    p.sum_dtype = a.sum_out.dtype;
    p.y_dtype = a.y.dtype;
    p.n_rows = n;
    p.hidden = h;
    p.eps = a.eps;
    return done(launch_rmsnorm(p, (cudaStream_t)stream));
}

size_t qs_rmsnorm_backward_workspace_bytes(int hidden) {
    return hidden < 1 || hidden > kNormMaxHidden ? 0 : norm_parts_bytes(hidden);
}

int qs_rmsnorm_residual_backward(const qs_rmsnorm_backward_args* args, void* stream) {
    if (!args) return QS_ERR_INVALID;
    const qs_rmsnorm_backward_args& a = *args;
    const int n = a.n_rows, h = a.hidden;
    if (n < 0 || h < 1 || h > kNormMaxHidden || !eps_ok(a.eps)) return QS_ERR_INVALID;
    if (!rows_ok(a.sum, n, h) || !a.weight || ((uintptr_t)a.weight & 3u) || !rows_ok(a.dy, n, h)) return QS_ERR_INVALID;
    if (a.dsum.data && !rows_ok(a.dsum, n, h)) return QS_ERR_INVALID;
    if (!rows_ok(a.dx, n, h) || ((uintptr_t)a.dweight & 3u)) return QS_ERR_INVALID;
    if (a.dweight && (!a.workspace || ((uintptr_t)a.workspace & 255u) || a.workspace_bytes < norm_parts_bytes(h)))
        return QS_ERR_WORKSPACE;
    NormBwdArgs p = {};
    p.sum = a.sum.data;
    p.weight = a.weight;
    p.dy = a.dy.data;
    p.dsum = a.dsum.data;
    p.dx = a.dx.data;
    p.partial = a.dweight ? static_cast<float*>(a.workspace) : nullptr;
    p.sum_stride = a.sum.stride;
    p.dy_stride = a.dy.stride;
    p.dsum_stride = a.dsum.stride;
    p.dx_stride = a.dx.stride;
    p.sum_dtype = a.sum.dtype;
    p.dy_dtype = a.dy.dtype;
    p.dsum_dtype = a.dsum.dtype;
    p.dx_dtype = a.dx.dtype;
    p.n_rows = n;
    p.hidden = h;
    p.part_stride = (h + 7) / 8 * 8;
    p.eps = a.eps;
    return done(launch_rmsnorm_backward(p, a.dweight, (cudaStream_t)stream));
}

int qs_silu_mul_quant(const qs_silu_mul_args* args, void* stream) {
    if (!args) return QS_ERR_INVALID;
    const qs_silu_mul_args& a = *args;
    if (a.n_rows < 0 || a.ffn < 1 || a.ffn > (1 << 24)) return QS_ERR_INVALID;
    if (!rows_ok(a.gate_up, a.n_rows, 2 * a.ffn) || !codes_ok(a.q, a.n_rows, a.ffn)) return QS_ERR_INVALID;
    if ((uintptr_t)a.n_rows_dev & 3u) return QS_ERR_INVALID;
    SiluArgs p = {};
    p.gate_up = a.gate_up.data;
    p.n_rows_dev = a.n_rows_dev;
    p.q = static_cast<uint8_t*>(a.q.q);
    p.q_scale = a.q.scale;
    p.gate_up_stride = a.gate_up.stride;
    p.q_stride = a.q.stride;
    p.q_scale_stride = a.q.scale_stride;
    p.dtype = a.gate_up.dtype;
    p.n_rows = a.n_rows;
    p.ffn = a.ffn;
    return done(launch_silu_mul_quant(p, (cudaStream_t)stream));
}

static bool matmul_shape_ok(int n_rows, int n_cols, int n_inner, int n_experts) {
    return n_rows >= 0 && n_rows <= kMmMaxRows && n_cols >= 1 && n_inner >= 1 && n_inner <= (1 << 30) && n_cols <= (1 << 30) &&
           n_experts >= 1 && n_experts <= kMmMaxExperts;
}

size_t qs_fp8_matmul_workspace_bytes(int n_rows, int n_cols, int n_inner, int n_experts) {
    return matmul_shape_ok(n_rows, n_cols, n_inner, n_experts) ? fp8_matmul_workspace(n_rows, n_cols, n_inner, n_experts) : 0;
}

int qs_fp8_matmul(const qs_fp8_matmul_args* args, void* stream) {
    if (!args) return QS_ERR_INVALID;
    const qs_fp8_matmul_args& a = *args;
    const int m = a.n_rows, n = a.n_cols, k = a.n_inner, e = a.n_experts;
    if (!matmul_shape_ok(m, n, k, e) || (!a.offsets && e != 1)) return QS_ERR_INVALID;
    // the strides are a tensor map's: multiples of 16 bytes below 2^40, also where there is one row
    const int64_t top = 1ll << 40;
    if (!codes_ok(a.a, m, k) || ((uintptr_t)a.a.q & 15u) || a.a.stride % 16 || a.a.stride < k || a.a.stride >= top)
        return QS_ERR_INVALID;
    if (!a.w || !a.w_scale || ((uintptr_t)a.w & 15u) || ((uintptr_t)a.w_scale & 3u) || a.w_stride % 16 ||
        a.w_stride < k || a.w_stride >= top || a.w_expert_stride % 16 || a.w_expert_stride >= top ||
        ((uintptr_t)a.offsets & 3u))
        return QS_ERR_INVALID;
    // an expert's rows end before the next expert's begin; divided, since w_stride * (n - 1) may pass 64 bits
    if (a.w_expert_stride < 0 || (e > 1 && (a.w_expert_stride < k || (a.w_expert_stride - k) / a.w_stride < n - 1)))
        return QS_ERR_INVALID;
    if (!rows_ok(a.out, m, n)) return QS_ERR_INVALID;
    if (!a.workspace || ((uintptr_t)a.workspace & 255u) || a.workspace_bytes < fp8_matmul_workspace(m, n, k, e))
        return QS_ERR_WORKSPACE;
    Fp8MmArgs p = {};
    p.a = a.a.q;
    p.a_scale = a.a.scale;
    p.w = a.w;
    p.w_scale = a.w_scale;
    p.offsets = a.offsets;
    p.out = a.out.data;
    p.a_stride = a.a.stride;
    p.a_scale_stride = a.a.scale_stride;
    p.w_stride = a.w_stride;
    p.w_expert_stride = e > 1 ? a.w_expert_stride : a.w_stride;
    p.out_stride = a.out.stride;
    p.n_experts = e;
    p.n_rows = m;
    p.n_cols = n;
    p.n_inner = k;
    p.out_dtype = a.out.dtype;
    return done(launch_fp8_matmul(p, a.workspace, (cudaStream_t)stream));
}

size_t qs_dispatch_workspace_bytes(int n_tokens, int top_k, int n_experts) {
    return entries_ok(n_tokens, top_k) && n_experts >= 1 && n_experts <= 1024
               ? dispatch_workspace(n_tokens, top_k, n_experts)
               : 0;
}

int qs_dispatch_tokens(const qs_dispatch_args* args, void* stream) {
    if (!args) return QS_ERR_INVALID;
    const qs_dispatch_args& a = *args;
    if (!entries_ok(a.n_tokens, a.top_k) || a.n_experts < 1 || a.n_experts > 1024) return QS_ERR_INVALID;
    if (!a.counts || !a.offsets || (a.n_tokens > 0 && (!a.topk_ids || !a.perm || !a.pos))) return QS_ERR_INVALID;
    if (((uintptr_t)a.topk_ids | (uintptr_t)a.counts | (uintptr_t)a.offsets | (uintptr_t)a.perm | (uintptr_t)a.pos) & 3u)
        return QS_ERR_INVALID;
    DispatchArgs p = {};
    if (a.xs.data) {
        const int n = a.n_tokens * a.top_k;
        if (a.hidden < 1 || a.hidden > (1 << 24) || a.x.dtype != a.xs.dtype) return QS_ERR_INVALID;
        if (a.x.dtype == QS_E4M3) {
            const qs_codes x = {a.x.data, a.x.stride, const_cast<float*>(a.x_scale), a.x_scale_stride};
            const qs_codes xs = {a.xs.data, a.xs.stride, a.xs_scale, a.xs_scale_stride};
            if (!codes_ok(x, a.n_tokens, a.hidden) || !codes_ok(xs, n, a.hidden)) return QS_ERR_INVALID;
            p.n_scales = scale_blocks(a.hidden);
        } else if (!rows_ok(a.x, a.n_tokens, a.hidden) || !rows_ok(a.xs, n, a.hidden)) {
            return QS_ERR_INVALID;
        }
        p.row_bytes = a.hidden * type_size(a.x.dtype);
        p.x_stride = a.x.stride * type_size(a.x.dtype);
        p.xs_stride = a.xs.stride * type_size(a.x.dtype);
    }
    if (!a.workspace || ((uintptr_t)a.workspace & 255u) ||
        a.workspace_bytes < dispatch_workspace(a.n_tokens, a.top_k, a.n_experts))
        return QS_ERR_WORKSPACE;
    p.ids = a.topk_ids;
    p.counts = a.counts;
    p.offsets = a.offsets;
    p.perm = a.perm;
    p.pos = a.pos;
    p.x = a.x.data;
    p.xs = a.xs.data;
    p.x_scale = a.x_scale;
    p.xs_scale = a.xs_scale;
    p.hist = static_cast<int32_t*>(a.workspace);
    p.x_scale_stride = a.x_scale_stride;
    p.xs_scale_stride = a.xs_scale_stride;
    p.n_tokens = a.n_tokens;
    p.top_k = a.top_k;
    p.n_experts = a.n_experts;
    return done(launch_dispatch(p, (cudaStream_t)stream));
}

int qs_combine_tokens(const qs_combine_args* args, void* stream) {
    if (!args) return QS_ERR_INVALID;
    const qs_combine_args& a = *args;
    if (!entries_ok(a.n_tokens, a.top_k) || a.hidden < 1 || a.hidden > (1 << 24) || (!a.pos && a.n_tokens > 0))
        return QS_ERR_INVALID;
    if (((uintptr_t)a.pos | (uintptr_t)a.topk_w) & 3u) return QS_ERR_INVALID;
    if (!rows_ok(a.y, a.n_tokens * a.top_k, a.hidden) || !rows_ok(a.out, a.n_tokens, a.hidden)) return QS_ERR_INVALID;
    CombineArgs p = {};
    p.y = a.y.data;
    p.pos = a.pos;
    p.w = a.topk_w;
    p.out = a.out.data;
    p.y_stride = a.y.stride;
    p.out_stride = a.out.stride;
    p.y_dtype = a.y.dtype;
    p.out_dtype = a.out.dtype;
    p.n_tokens = a.n_tokens;
    p.top_k = a.top_k;
    p.hidden = a.hidden;
    return done(launch_combine(p, (cudaStream_t)stream));
}

int qs_combine_tokens_backward(const qs_combine_backward_args* args, void* stream) {
    if (!args) return QS_ERR_INVALID;
    const qs_combine_backward_args& a = *args;
    if (!entries_ok(a.n_tokens, a.top_k) || a.hidden < 1 || a.hidden > (1 << 24) || (!a.pos && a.n_tokens > 0))
        return QS_ERR_INVALID;
    if (((uintptr_t)a.pos | (uintptr_t)a.topk_w | (uintptr_t)a.dtopk_w) & 3u) return QS_ERR_INVALID;
    const int n = a.n_tokens * a.top_k;
    if (!rows_ok(a.dout, a.n_tokens, a.hidden) || !rows_ok(a.dy, n, a.hidden)) return QS_ERR_INVALID;
    if (a.dtopk_w && !rows_ok(a.y, n, a.hidden)) return QS_ERR_INVALID;
    CombineBwdArgs p = {};
    p.dout = a.dout.data;
    p.y = a.y.data;
    p.pos = a.pos;
    p.w = a.topk_w;
    p.dy = a.dy.data;
    p.dw = a.dtopk_w;
    p.dout_stride = a.dout.stride;
    p.y_stride = a.y.stride;
    p.dy_stride = a.dy.stride;
    p.dout_dtype = a.dout.dtype;
    p.y_dtype = a.y.dtype;
    p.dy_dtype = a.dy.dtype;
    p.n_tokens = a.n_tokens;
    p.top_k = a.top_k;
    p.hidden = a.hidden;
    return done(launch_combine_backward(p, (cudaStream_t)stream));
}

}  // extern "C"
