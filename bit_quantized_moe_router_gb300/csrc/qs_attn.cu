// qs_attn.cu -- which attention kernel a call runs, and its workspace (sm_103a).
#include "qs_attn.cuh"

namespace qs {

// The header, three counters a CTA (zero between calls), and parts of items, each the sums of RT rows, their maxima and
// sums of weights: two a CTA (of the item that its run begins inside and of the one that it ends inside), two more where kFan
// CTAs' are joined first, and one a team (of the item that its run begins inside).
static constexpr size_t kPartsAt = kHeaderBytes + (3 * kAttnMaxCtas * 4 + 255) / 256 * 256;

static size_t part_floats(const int rows, int head_dim) { return (size_t)rows * (attn::padded_dim(head_dim) + 6); }

size_t attn_workspace(int n_heads, int n_kv, int head_dim, int max_new) {
    const int rows = attn::item_rows(n_heads / n_kv * max_new);
    return kPartsAt + kAttnMaxCtas * (4 + attn::most_teams(rows)) * part_floats(rows, head_dim) * 4;
}

cudaError_t launch_cache_attention(const AttnArgs& args, void* workspace, cudaStream_t st) {
    AttnArgs p = args;
    if (p.n_tokens == 0 || p.seqs.n_seqs == 0) return cudaSuccess;
    p.scale *= attn::kLog2e;
    if (p.cache.n_pages == 0) {  // copies of no bytes are still given an address
        p.cache.k = p.cache.v = static_cast<uint8_t*>(workspace);
        p.cache.k_scale = p.cache.v_scale = static_cast<float*>(workspace);
        p.cache.head_stride = p.cache.scale_head_stride = 0;
    }
    p.joined = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + kHeaderBytes);
    const size_t part = part_floats(attn::item_rows(p.n_heads / p.cache.n_kv * p.max_new), p.cache.head_dim);
    p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kPartsAt);
    p.merged = p.parts + 2 * kAttnMaxCtas * part;
    p.heads = p.merged + 2 * kAttnMaxCtas * part;
    // codes are made of unrounded rows: as near to the formula's as fp32 rows are, so that as few differ
    const bool wide = p.q.dtype == QS_F32 || (p.out.data && p.out.dtype == QS_F32) || p.codes;
    const int d = attn::padded_dim(p.cache.head_dim);
    if (p.cache.dtype == QS_E4M3)
        return d == 64 ? launch_attention<true, 64>(p, wide, st) : d == 128 ? launch_attention<true, 128>(p, wide, st) : launch_attention<true, 256>(p, wide, st);
    return d == 64 ? launch_attention<false, 64>(p, wide, st) : d == 128 ? launch_attention<false, 128>(p, wide, st) : launch_attention<false, 256>(p, wide, st);
}

}  // namespace qs
