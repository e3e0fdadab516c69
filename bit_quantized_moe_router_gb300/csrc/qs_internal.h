// qs_internal.h -- host-side declarations shared by the library's translation units.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "qs_moe.h"

namespace qs {

// Workspace regions (byte offsets from the workspace base; each 256-aligned).
struct WsLayout {
    size_t header = 0;
    size_t logits = 0;   // f32 [T x E]
    size_t ids = 0;      // i32 [T x k]
    size_t pw = 0;       // f32 [T x k]
    size_t counts = 0;   // i32 [E]
    size_t offsets = 0;  // i32 [E + 1]
    size_t perm = 0;     // i32 [T x k]
    size_t h = 0;        // f32 [T*k x F]
    size_t hs = 0;       // f32 [T x S]
    size_t gate = 0;     // f32 [T]
    size_t tickets = 0;  // u32 [ceil(T / kRouteTok)]
    // exchanged arrays of the persistent decode kernel (fp32; completion counters in the header)
    size_t xlog = 0;     // [Tf x E]
    size_t xhs = 0;      // [Tf x S]
    size_t xh = 0;       // [Tf*k x F]     (Tf = min(T, kFusedMaxT))
    // cluster decode kernel: its counters, per-entry routed down products, shared down products
    size_t cx = 0;       // kCxBytes of 64-bit counters, one per 32-byte sector
    size_t cpd = 0;      // f32 [Tc*k x H]  (Tc = min(T, kClusterMaxT))
    size_t csdp = 0;     // f32 [Tc x H]
    // tensor-core (prefill) path
    size_t wr3 = 0;      // bf16 [3 x E x H]  router weights as three bf16 planes
    size_t lpart = 0;    // f32 [kPrefillMaxKS x T x E] partial logits
    size_t xs = 0;       // fp16 [T*k x H] token rows in expert-sorted order
    size_t cursor = 0;   // i32 [E] fill pointers of the expert lists
    size_t h16 = 0;      // fp16 [T*k x F] (expert-sorted entries)
    size_t hs16 = 0;     // bf16 [T x S]
    size_t total = 0;
};

constexpr int kRouteTok = 8;    // tokens per router CTA chunk
constexpr int kFusedMaxT = 16;  // largest token count the persistent decode kernel takes
constexpr int kPrefillMaxKS = 4;  // largest split of H in the tensor-core router
constexpr int kClusterCtas = 8;   // CTAs per thread-block cluster of the cluster decode kernel
constexpr int kClusterMaxT = 8;   // largest token count the cluster decode kernel takes
constexpr int kCxBytes = 512;     // counter region of the cluster decode kernel

WsLayout ws_layout(const qs_moe_shape& s, int max_tokens);

// Record e as the calling thread's last CUDA failure (qs_last_cuda_error) and return QS_ERR_CUDA.
int cuda_fail(cudaError_t e);

// Decode-path launchers (qs_decode.cu).  All return the launch's cudaError_t.
cudaError_t launch_route(const qs_moe_shape& s, const void* x, const float* W, const float* bias, int T,
                         float* logits, int32_t* ids, float* pw, uint32_t* tickets, cudaStream_t st);
cudaError_t launch_group(int E, int k, int T, const int32_t* ids, int32_t* counts, int32_t* offsets, int32_t* perm,
                         cudaStream_t st);
cudaError_t launch_gateup(const qs_moe_shape& s, const void* x, const uint8_t* experts, int64_t stride,
                          const int32_t* offsets, const int32_t* perm, int T, float* h, cudaStream_t st);
cudaError_t launch_down(const qs_moe_shape& s, const uint8_t* experts, int64_t stride, const float* h,
                        const int32_t* ids, const float* pw, int n_slots, const uint16_t* sh_down,
                        const float* hs, const float* gate, int T, float* out, int accumulate, cudaStream_t st);
cudaError_t launch_shared_gateup(const qs_moe_shape& s, const void* x, const uint16_t* wg, const uint16_t* wu,
                                 const uint16_t* wsig, int T, float* hs, float* gate, cudaStream_t st);
cudaError_t launch_quantize(const float* w, int64_t n_blocks, uint8_t* out, cudaStream_t st);
cudaError_t launch_test_wait(void* ws, uint64_t limit_ns, cudaStream_t st);

// Q4_K routed experts (qs_q4k.cu): encoder, gate/up + SwiGLU into h, down + routing-weight
// combine into out (stored, not added).
cudaError_t launch_q4k_quantize(const float* w, int64_t n_blocks, uint8_t* out, cudaStream_t st);
cudaError_t launch_q4k_gateup(const qs_moe_shape& s, const void* x, const uint8_t* experts, int64_t stride,
                              const int32_t* offsets, const int32_t* perm, int T, float* h, cudaStream_t st);
cudaError_t launch_q4k_down(const qs_moe_shape& s, const uint8_t* experts, int64_t stride, const float* h,
                            const int32_t* ids, const float* pw, int T, float* out, cudaStream_t st);
size_t q4k_down_smem(int k, int F);

// Directional steering of output rows (qs_steer.cu): y <- y - scale * d * (d . y) per row.
cudaError_t launch_steer_rows(float* y, const float* d, float scale, int T, int H, cudaStream_t st);

// Persistent single-kernel decode path (qs_fused.cu).  cudaErrorNotSupported
// when the shape or token count is outside its plan; the caller then runs the
// per-step kernels.  sg == nullptr means no shared expert.  x_host_mapped: x and out are
// pinned host memory given by their device-mapped addresses (x read with plain loads).
cudaError_t launch_fused_decode(const qs_moe_shape& s, const void* x, const float* Wr, const float* bias,
                                const uint8_t* experts, int64_t stride, const uint16_t* sg, const uint16_t* su,
                                const uint16_t* sd, const uint16_t* ssig, int T, float* out, void* ws,
                                const WsLayout& W, cudaStream_t st, bool x_host_mapped = false,
                                int fmt = 0 /* 0: Q2_K, 1: Q4_K routed experts */);
bool fused_decode_supported(const qs_moe_shape& s, int T, cudaError_t* err);

// Decode path of thread-block clusters (qs_cluster.cu): one kernel; a cluster of
// kClusterCtas CTAs owns whole routed experts and shares h through distributed shared
// memory.  cudaErrorNotSupported when the shape or token count is outside its plan.
// x_host_mapped: x (and out) are pinned host memory given by their device-mapped
// addresses; the kernel reads x with plain loads instead of a bulk copy.
cudaError_t launch_cluster_decode(const qs_moe_shape& s, const void* x, const float* Wr, const float* bias,
                                  const uint8_t* experts, int64_t stride, const uint16_t* sg, const uint16_t* su,
                                  const uint16_t* sd, const uint16_t* ssig, int T, float* out, void* ws,
                                  const WsLayout& W, cudaStream_t st, bool x_host_mapped = false);
bool cluster_decode_supported(const qs_moe_shape& s, int T, cudaError_t* err);

// The one-kernel decode paths in qs_moe_ffn's order of preference for this token count
// (qs_api.cu): the first that takes the call is launched; cudaErrorNotSupported if neither.
cudaError_t launch_decode_kernel(const qs_moe_shape& s, const void* x, const float* Wr, const float* bias,
                                 const uint8_t* experts, int64_t stride, const uint16_t* sg, const uint16_t* su,
                                 const uint16_t* sd, const uint16_t* ssig, int T, float* out, void* ws,
                                 const WsLayout& W, cudaStream_t st, bool x_host_mapped);

// Tensor-core path for many tokens (qs_prefill.cu): prefill_launches() launches.  Needs bf16
// x and Q2_K row layouts it can stage (see prefill_shape_ok).
bool prefill_shape_ok(const qs_moe_shape& s);
int prefill_launches();
cudaError_t launch_prefill(const qs_moe_shape& s, const void* x, const float* Wr, const float* bias,
                           const uint8_t* experts, int64_t stride, const uint16_t* sg, const uint16_t* su,
                           const uint16_t* sd, const uint16_t* ssig, int T, float* out, void* ws, const WsLayout& W,
                           cudaStream_t st);

// Row operators (qs_norm.cu).  Strides in elements; a null pointer leaves its part out.
struct NormArgs {
    const void* x;
    const void* residual;
    const float* weight;
    void* sum_out;
    void* y;
    uint8_t* q;
    float* q_scale;
    int64_t x_stride, residual_stride, sum_stride, y_stride, q_stride, q_scale_stride;
    int x_dtype, residual_dtype, sum_dtype, y_dtype;
    int n_rows, hidden;
    float eps;
};
struct NormBwdArgs {
    const void* sum;
    const float* weight;
    const void* dy;
    const void* dsum;
    void* dx;
    float* partial;  // [a row a CTA x part_stride], or null without dweight
    int64_t sum_stride, dy_stride, dsum_stride, dx_stride;
    int sum_dtype, dy_dtype, dsum_dtype, dx_dtype;
    int n_rows, hidden, part_stride;
    float eps;
};
struct SiluArgs {
    const void* gate_up;
    const int32_t* n_rows_dev;
    uint8_t* q;
    float* q_scale;
    int64_t gate_up_stride, q_stride, q_scale_stride;
    int dtype, n_rows, ffn;
};
constexpr int kNormParts = 456;      // most CTAs of the gradient, a partial row of dweight each: three an SM
constexpr int kNormMaxHidden = 16384;
cudaError_t launch_rmsnorm(const NormArgs& p, cudaStream_t st);
cudaError_t launch_rmsnorm_backward(const NormBwdArgs& p, float* dweight, cudaStream_t st);
cudaError_t launch_silu_mul_quant(const SiluArgs& p, cudaStream_t st);

// Token rows to experts and back (qs_tokens.cu).
struct DispatchArgs {
    const int32_t* ids;
    int32_t *counts, *offsets, *perm, *pos;
    const void* x;
    void* xs;
    const float* x_scale;
    float* xs_scale;
    int32_t* hist;  // workspace: [chunks x n_experts]
    int64_t x_stride, xs_stride, x_scale_stride, xs_scale_stride;  // bytes of x and xs, floats of the scales
    int n_tokens, top_k, n_experts;
    int row_bytes, n_scales;
};
struct CombineArgs {
    const void* y;
    const int32_t* pos;
    const float* w;
    void* out;
    int64_t y_stride, out_stride;
    int y_dtype, out_dtype, n_tokens, top_k, hidden;
};
struct CombineBwdArgs {
    const void* dout;
    const void* y;
    const int32_t* pos;
    const float* w;
    void* dy;
    float* dw;
    int64_t dout_stride, y_stride, dy_stride;
    int dout_dtype, y_dtype, dy_dtype, n_tokens, top_k, hidden;
};
size_t dispatch_workspace(int n_tokens, int top_k, int n_experts);
cudaError_t launch_dispatch(const DispatchArgs& p, cudaStream_t st);
cudaError_t launch_combine(const CombineArgs& p, cudaStream_t st);
cudaError_t launch_combine_backward(const CombineBwdArgs& p, cudaStream_t st);

// e4m3 product with block scales (qs_fp8mm.cu).
struct Fp8MmArgs {
    const void* a;
    const float* a_scale;
    const void* w;
    const float* w_scale;
    const int32_t* offsets;
    void* out;
    int64_t a_stride, a_scale_stride, w_stride, w_expert_stride, out_stride;
    int n_experts, n_rows, n_cols, n_inner, out_dtype;
};
constexpr int kMmMaxRows = 1 << 30, kMmMaxExperts = 1024;
size_t fp8_matmul_workspace(int n_rows, int n_cols, int n_inner, int n_experts);
cudaError_t launch_fp8_matmul(const Fp8MmArgs& p, void* workspace, cudaStream_t st);

// The paged key-value cache and its operators (qs_cache.cu, qs_attn.cuh).  Strides of the cache and of rows of heads in
// bytes, of scales in floats.
struct FastDiv {
    uint32_t mul;
    int shift;
};
struct CacheView {
    uint8_t *k, *v;
    float *k_scale, *v_scale;
    int64_t page_stride, slot_stride, head_stride;
    int64_t scale_page_stride, scale_slot_stride, scale_head_stride;
    FastDiv page_div;  // by page_size
    int dtype, n_pages, page_size, n_kv, head_dim;
};
struct SeqsView {
    const int32_t *table, *starts, *offsets;
    int64_t table_stride;
    int n_seqs, positions;  // positions: what a row of the table covers
};
struct HeadsView {
    uint8_t* data;
    int64_t token_stride, head_stride;
    int dtype;
};
struct CacheRowsArgs {
    CacheView cache;
    SeqsView seqs;
    HeadsView k, v;
    int n_tokens;
    bool aligned;      // every row of k and v at 16-byte boundaries
    int lane_bits;     // set by the launch: 2^lane_bits lanes a head row
};
cudaError_t launch_cache_write(const CacheRowsArgs& p, cudaStream_t st);
cudaError_t launch_cache_read(const CacheRowsArgs& p, cudaStream_t st);

// Places of pages and slots as 32-bit numbers of `unit` bytes, the largest power of two that divides their strides.
struct Units {
    int page, slot, unit;
    bool set(const CacheView& c) {
        const int64_t page_stride = c.n_pages > 1 ? c.page_stride : 0, slot_stride = c.page_size > 1 ? c.slot_stride : 0;
        unit = 16;
        while (unit < (1 << 30) && (page_stride | slot_stride) % (2 * unit) == 0) unit *= 2;
        const int64_t most = 0x7fffffff;
        if (page_stride / unit > most || slot_stride / unit > most) return false;
        page = (int)(page_stride / unit);
        slot = (int)(slot_stride / unit);
        const double last = (double)page * (c.n_pages > 0 ? c.n_pages - 1 : 0) + (double)slot * (c.page_size - 1);
        return last <= (double)most;
    }
};
struct AttnArgs {
    CacheView cache;
    Units places;
    SeqsView seqs;
    HeadsView q, out;  // out.data null: left out
    uint8_t* codes;    // null: left out
    float* codes_scale;
    float* lse;        // null: left out
    int64_t codes_stride, codes_scale_stride;
    float scale;       // of the scores, times log2(e)
    int n_tokens, n_heads, max_new, window;
    FastDiv group_div;  // by group, the query heads of a key-value head
    int group;
    uint32_t* joined;  // workspace: three counters a CTA, and the parts of items that several teams or CTAs share
    float *parts, *merged, *heads;
};
constexpr int kAttnMaxCtas = 160;  // most CTAs of a call, one an SM
size_t attn_workspace(int n_heads, int n_kv, int head_dim, int max_new);
cudaError_t launch_cache_attention(const AttnArgs& p, void* workspace, cudaStream_t st);

}  // namespace qs
