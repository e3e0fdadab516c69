// Attention over a cache of bf16, head sizes up to 128.
#include "qs_attn.cuh"

namespace qs {
template cudaError_t launch_attention<false, 128>(const AttnArgs&, bool, cudaStream_t);
}
