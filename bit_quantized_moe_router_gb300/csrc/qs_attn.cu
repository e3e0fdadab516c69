// qs_attn.cu -- which attention kernel a call runs, and its workspace (sm_103a).
#include "qs_attn.cuh"

namespace qs {

// The header, a counter a CTA (zero between calls), and two parts of items a CTA: the one that its run begins inside
// and the one that it ends inside.  A part: sums of RT rows, and a maximum and a sum of weights each.
static constexpr size_t kPartsAt = kHeaderBytes + (kAttnMaxCtas * 4 + 255) / 256 * 256;

size_t attn_workspace(int n_heads, int n_kv, int head_dim, int max_new) {
    const size_t rows = attn::item_rows(n_heads / n_kv * max_new);
    return kPartsAt + (size_t)kAttnMaxCtas * 2 * rows * (attn::padded_dim(head_dim) + 2) * 4;
}

cudaError_t launch_cache_attention(const AttnArgs& args, void* workspace, cudaStream_t st) {
    AttnArgs p = args;
    if (p.n_tokens == 0 || p.seqs.n_seqs == 0) return cudaSuccess;
    p.scale *= attn::kLog2e;
    p.joined = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + kHeaderBytes);
    p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kPartsAt);
    // codes are made of unrounded rows: as near to the formula's as fp32 rows are, so that as few differ
    const bool wide = p.q.dtype == QS_F32 || (p.out.data && p.out.dtype == QS_F32) || p.codes;
    const int d = attn::padded_dim(p.cache.head_dim);
    if (p.cache.dtype == QS_E4M3)
        return d == 64 ? launch_attention<true, 64>(p, wide, st) : d == 128 ? launch_attention<true, 128>(p, wide, st) : launch_attention<true, 256>(p, wide, st);
    return d == 64 ? launch_attention<false, 64>(p, wide, st) : d == 128 ? launch_attention<false, 128>(p, wide, st) : launch_attention<false, 256>(p, wide, st);
}

}  // namespace qs
