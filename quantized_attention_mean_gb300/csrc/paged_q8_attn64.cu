// 8-bit decode at head_dim 1 to 64.
#include "paged_q8_attn.cuh"

namespace sage {
cudaError_t launch_q8_decode_64(const Q8Args& p, const CUtensorMap* maps, cudaStream_t st) { return launch_q8<64>(p, maps, st); }
}  // namespace sage
