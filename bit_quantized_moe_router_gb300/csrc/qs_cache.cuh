// qs_cache.cuh -- where a position of a sequence lies in the paged key-value cache, and which sequence a
// token belongs to.  Every index that comes from device memory (offsets, starts, page ids) is checked or
// clipped before an address is made of it; addresses are formed in 64 bits.
#pragma once

#include "qs_internal.h"
#include "qs_rows.cuh"

namespace qs {

// x / d for 0 <= x < 2^31 by a product: with 2^(31 + shift) >= 2^31 * d and mul = ceil(2^(31 + shift) / d), the product's
// error is below 1 / d for every such x.  mul < 2^32; the upper word of 2 x mul is x mul / 2^31.
__device__ __forceinline__ int fast_div(int x, const FastDiv& d) { return (int)(__umulhi(2u * (uint32_t)x, d.mul) >> d.shift); }

// The place of position pos of a sequence, in bytes of k and v (and floats of the scales, if asked for): -1 where the
// sequence has no such position or its page id names no page.  pos in 64 bits, as it was computed.
struct Place {
    int64_t at, scale_at;
};
__device__ __forceinline__ Place place_of(const CacheView& c, const SeqsView& s, int seq, int64_t pos) {
    Place r = {-1, -1};
    if (pos < 0 || pos >= s.positions) return r;
    const int page_of = fast_div((int)pos, c.page_div), slot = (int)pos - page_of * c.page_size;
    const int page = s.table[seq * s.table_stride + page_of];
    if ((unsigned)page >= (unsigned)c.n_pages) return r;
    r.at = page * c.page_stride + slot * c.slot_stride;
    r.scale_at = page * c.scale_page_stride + slot * c.scale_slot_stride;
    return r;
}

// The last sequence whose first token is not after token t, found by a whole warp, 32 offsets at a time: two steps for
// up to 1024 sequences where halving takes ten loads one after another.  Offsets that are not ascending give some
// sequence.
__device__ __forceinline__ int seq_of_token(const SeqsView& s, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = s.n_seqs;
    while (n > 1) {
        const int step = (n + 31) / 32, i = lo + lane * step;
        const unsigned before = __ballot_sync(0xffffffffu, lane * step < n && s.offsets[i] <= t);
        const int k = before ? 31 - __clz(before) : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

// Sequence and position of token t; false if it belongs to none.
__device__ __forceinline__ bool token_at(const SeqsView& s, int t, int& seq, int64_t& pos) {
    seq = s.offsets ? seq_of_token(s, t) : t;
    int first = t;
    if (s.offsets) {
        first = s.offsets[seq];
        if (t < first || t >= s.offsets[seq + 1]) return false;
    }
    pos = (s.starts ? (int64_t)s.starts[seq] : 0) + t - first;
    return true;
}

}  // namespace qs
