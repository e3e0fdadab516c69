// Attention over a cache of bf16, head sizes up to 256.
#include "qs_attn.cuh"

namespace qs {
template cudaError_t launch_attention<false, 256>(const AttnArgs&, bool, cudaStream_t);
}
