// Attention over a cache of e4m3, head sizes up to 256.
#include "qs_attn.cuh"

namespace qs {
template cudaError_t launch_attention<true, 256>(const AttnArgs&, bool, cudaStream_t);
}
