// qs_cache_api.cu -- C ABI of the paged cache's operators: argument checks, then the kernels.
#include <algorithm>

#include "qs_internal.h"
#include "qs_rows.cuh"

using namespace qs;

namespace {

constexpr int kMaxTokens = 1 << 24, kMaxSeqs = 1 << 16, kMaxHeads = 256, kMaxPositions = 1 << 30, kMaxNew = 256;

int done(cudaError_t e) { return e == cudaSuccess ? QS_OK : cuda_fail(e); }

bool head_dim_ok(int d) { return d >= 16 && d <= 256 && d % 16 == 0; }

// Dimensions of these strides and sizes under a contiguous inner one (of one element or more): whether no two places are the same.
struct Dim {
    int64_t stride, size;
};
bool distinct(Dim a, Dim b, Dim c, int64_t inner) {
    Dim d[3] = {a, b, c};
    std::sort(d, d + 3, [](const Dim& x, const Dim& y) { return x.stride < y.stride; });
    for (const Dim& x : d) {
        if (x.size <= 1) continue;
        if (x.stride < inner) return false;
        if (x.size - 1 > ((int64_t)1 << 60) / x.stride) return false;  // (three such extents are within 64 bits; their product may not be)
        inner += x.stride * (x.size - 1);
    }
    return true;
}

bool stride_ok(int64_t s) { return s >= 0 && s <= (int64_t)1 << 40; }

bool cache_ok(const qs_cache& c, bool written) {
    if ((c.dtype != QS_BF16 && c.dtype != QS_E4M3) || !head_dim_ok(c.head_dim)) return false;
    if (c.n_pages < 0 || c.page_size < 1 || c.page_size > kMaxPositions || c.n_kv_heads < 1 || c.n_kv_heads > kMaxHeads) return false;
    const int64_t step = c.dtype == QS_BF16 ? 8 : 16;
    // the stride of a dimension of one is never used
    for (const Dim& x : {Dim{c.page_stride, c.n_pages}, Dim{c.slot_stride, c.page_size}, Dim{c.head_stride, c.n_kv_heads}})
        if (x.size > 1 && (!stride_ok(x.stride) || x.stride % step)) return false;
    if ((!c.k || !c.v) && c.n_pages > 0) return false;
    if (((uintptr_t)c.k | (uintptr_t)c.v) & 15u) return false;
    if (written && !distinct({c.page_stride, c.n_pages}, {c.slot_stride, c.page_size}, {c.head_stride, c.n_kv_heads}, c.head_dim)) return false;
    if (c.dtype == QS_E4M3) {
        if ((!c.k_scale || !c.v_scale) && c.n_pages > 0) return false;
        if (((uintptr_t)c.k_scale | (uintptr_t)c.v_scale) & 3u) return false;
        for (const Dim& x : {Dim{c.scale_page_stride, c.n_pages}, Dim{c.scale_slot_stride, c.page_size}, Dim{c.scale_head_stride, c.n_kv_heads}})
            if (x.size > 1 && !stride_ok(x.stride)) return false;
        if (written && !distinct({c.scale_page_stride, c.n_pages}, {c.scale_slot_stride, c.page_size}, {c.scale_head_stride, c.n_kv_heads}, 1)) return false;
    }
    return true;
}

bool seqs_ok(const qs_seqs& s, const qs_cache& c, int n_tokens) {
    if (n_tokens < 0 || n_tokens > kMaxTokens || s.n_seqs < 0 || s.n_seqs > kMaxSeqs || s.n_seq_pages < 0) return false;
    if ((int64_t)s.n_seq_pages * c.page_size > kMaxPositions) return false;
    if (!s.table && s.n_seqs > 0 && s.n_seq_pages > 0) return false;
    if (s.n_seqs > 1 ? s.table_stride < s.n_seq_pages || s.table_stride > (int64_t)1 << 40 : !stride_ok(s.table_stride)) return false;
    if (!s.offsets && s.n_seqs != n_tokens) return false;
    return (((uintptr_t)s.table | (uintptr_t)s.starts | (uintptr_t)s.offsets) & 3u) == 0;
}

// Rows of heads: there, of fp32 or bf16, aligned to their elements; `written`: no two of them at the same place.
bool heads_ok(const qs_heads& x, int n_tokens, int n_heads, int head_dim, bool written) {
    if (x.dtype != QS_F32 && x.dtype != QS_BF16) return false;
    if ((!x.data && n_tokens > 0) || (uintptr_t)x.data % type_size(x.dtype)) return false;
    if (!stride_ok(x.token_stride) || !stride_ok(x.head_stride)) return false;
    return !written || distinct({x.token_stride, n_tokens}, {x.head_stride, n_heads}, {0, 1}, head_dim);
}

// Every row at 16-byte boundaries; the stride of a dimension of one is never used.
bool heads_aligned(const qs_heads& x, int n_tokens, int n_heads) {
    return al16(x.data, n_tokens > 1 ? x.token_stride : 0, x.dtype) && al16(x.data, n_heads > 1 ? x.head_stride : 0, x.dtype);
}

HeadsView view(const qs_heads& x) {
    const int64_t z = type_size(x.dtype);
    return {static_cast<uint8_t*>(x.data), x.token_stride * z, x.head_stride * z, x.dtype};
}

FastDiv fast_div_by(int d) {
    FastDiv f = {0, 0};
    while ((1ll << f.shift) < d) f.shift++;
    f.mul = (uint32_t)(((1ull << (31 + f.shift)) + d - 1) / d);
    return f;
}

CacheView view(const qs_cache& c) {
    const int64_t z = type_size(c.dtype);
    CacheView v = {};
    v.k = static_cast<uint8_t*>(c.k);
    v.v = static_cast<uint8_t*>(c.v);
    v.k_scale = c.k_scale;
    v.v_scale = c.v_scale;
    v.page_stride = c.page_stride * z;
    v.slot_stride = c.slot_stride * z;
    v.head_stride = c.head_stride * z;
    v.scale_page_stride = c.scale_page_stride;
    v.scale_slot_stride = c.scale_slot_stride;
    v.scale_head_stride = c.scale_head_stride;
    v.page_div = fast_div_by(c.page_size);
    v.dtype = c.dtype;
    v.n_pages = c.n_pages;
    v.page_size = c.page_size;
    v.n_kv = c.n_kv_heads;
    v.head_dim = c.head_dim;
    return v;
}

SeqsView view(const qs_seqs& s, const qs_cache& c) { return {s.table, s.starts, s.offsets, s.table_stride, s.n_seqs, s.n_seq_pages * c.page_size}; }

bool rows_args(const qs_cache_rows_args& a, bool write, CacheRowsArgs& p) {
    if (!cache_ok(a.cache, write) || !seqs_ok(a.seqs, a.cache, a.n_tokens)) return false;
    for (const qs_heads* x : {&a.k, &a.v})
        if (!heads_ok(*x, a.n_tokens, a.cache.n_kv_heads, a.cache.head_dim, !write)) return false;
    if (a.k.dtype != a.v.dtype) return false;
    p.cache = view(a.cache);
    p.seqs = view(a.seqs, a.cache);
    p.k = view(a.k);
    p.v = view(a.v);
    p.n_tokens = a.n_tokens;
    p.aligned = heads_aligned(a.k, a.n_tokens, a.cache.n_kv_heads) && heads_aligned(a.v, a.n_tokens, a.cache.n_kv_heads);
    return true;
}

bool attention_shape_ok(int n_heads, int n_kv, int head_dim, int max_new) {
    return n_kv >= 1 && n_kv <= kMaxHeads && n_heads >= n_kv && n_heads % n_kv == 0 && n_heads / n_kv <= kMaxHeads && head_dim_ok(head_dim) &&
           max_new >= 1 && max_new <= kMaxNew;
}

}  // namespace

extern "C" {

int qs_cache_write(const qs_cache_rows_args* args, void* stream) {
    if (!args) return QS_ERR_INVALID;
    CacheRowsArgs p = {};
    if (!rows_args(*args, true, p)) return QS_ERR_INVALID;
    return done(launch_cache_write(p, (cudaStream_t)stream));
}

int qs_cache_read(const qs_cache_rows_args* args, void* stream) {
    if (!args) return QS_ERR_INVALID;
    CacheRowsArgs p = {};
    if (!rows_args(*args, false, p)) return QS_ERR_INVALID;
    return done(launch_cache_read(p, (cudaStream_t)stream));
}

size_t qs_cache_attention_workspace_bytes(int n_heads, int n_kv_heads, int head_dim, int max_new) {
    return attention_shape_ok(n_heads, n_kv_heads, head_dim, max_new) ? attn_workspace(n_heads, n_kv_heads, head_dim, max_new) : 0;
}

int qs_cache_attention(const qs_cache_attention_args* args, void* stream) {
    if (!args) return QS_ERR_INVALID;
    const qs_cache_attention_args& a = *args;
    const int h = a.n_heads, kv = a.cache.n_kv_heads, d = a.cache.head_dim, n = a.n_tokens;
    if (!cache_ok(a.cache, false) || !seqs_ok(a.seqs, a.cache, n) || !attention_shape_ok(h, kv, d, a.max_new)) return QS_ERR_INVALID;
    if (!(a.scale >= -1.0e38f && a.scale <= 1.0e38f) || a.window < 0) return QS_ERR_INVALID;
    if (!heads_ok(a.q, n, h, d, false) || !heads_aligned(a.q, n, h)) return QS_ERR_INVALID;
    if (n > 0 && !a.out.data && !a.codes.q) return QS_ERR_INVALID;
    if (a.out.data && (!heads_ok(a.out, n, h, d, true) || !heads_aligned(a.out, n, h))) return QS_ERR_INVALID;
    if (a.codes.q || a.codes.scale) {
        if (d % kScaleCols || !a.codes.q || !a.codes.scale || ((uintptr_t)a.codes.q & 15u) || a.codes.stride % 16 || ((uintptr_t)a.codes.scale & 3u)) return QS_ERR_INVALID;
        if (!stride_ok(a.codes.stride) || !stride_ok(a.codes.scale_stride)) return QS_ERR_INVALID;
        if (n > 1 && (a.codes.stride < (int64_t)h * d || a.codes.scale_stride < h * d / kScaleCols)) return QS_ERR_INVALID;
    }
    if ((uintptr_t)a.lse & 3u) return QS_ERR_INVALID;
    // tiles of 16 positions and 8 rows, at most an eighth of the line's places: a CTA's share of these is counted in 32 bits
    if ((double)a.seqs.n_seqs * ((double)a.seqs.n_seq_pages * a.cache.page_size / 16 + 2) * kv * ((double)(h / kv) * a.max_new / 8 + 1) > 2.0e10) return QS_ERR_UNSUPPORTED;
    if (!a.workspace || ((uintptr_t)a.workspace & 255u) || a.workspace_bytes < attn_workspace(h, kv, d, a.max_new)) return QS_ERR_WORKSPACE;
    AttnArgs p = {};
    p.cache = view(a.cache);
    if (!p.places.set(p.cache)) return QS_ERR_UNSUPPORTED;
    p.seqs = view(a.seqs, a.cache);
    p.q = view(a.q);
    if (a.out.data) p.out = view(a.out);
    p.codes = static_cast<uint8_t*>(a.codes.q);
    p.codes_scale = a.codes.scale;
    p.codes_stride = a.codes.stride;
    p.codes_scale_stride = a.codes.scale_stride;
    p.lse = a.lse;
    p.scale = a.scale;
    p.n_tokens = n;
    p.n_heads = h;
    p.max_new = a.max_new;
    p.group = h / kv;
    p.group_div = fast_div_by(p.group);
    p.window = a.window;
    return done(launch_cache_attention(p, a.workspace, (cudaStream_t)stream));
}

}  // extern "C"
