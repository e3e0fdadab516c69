// Attention over a cache of bf16, head sizes up to 64.
#include "qs_attn.cuh"

namespace qs {
template cudaError_t launch_attention<false, 64>(const AttnArgs&, bool, cudaStream_t);
}
