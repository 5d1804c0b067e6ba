// 8-bit decode at head_dim 65 to 128.
#include "paged_q8_attn.cuh"

namespace sage {
cudaError_t launch_q8_decode_128(const Q8Args& p, const CUtensorMap* maps, cudaStream_t st) { return launch_q8<128>(p, maps, st); }
}  // namespace sage
