// Attention over prompts and chunks (attn_tiles.cuh): causal and windowed calls.
#include "attn_tiles.cuh"

namespace cq {
cudaError_t launch_attn_tiles(const DeviceInfo& dev, const KvView& c, int dtype, const AttnArgs& a, const RowsPlan& pl,
                              cudaStream_t s) {
    return launch_tiles<false>(dev, c, dtype, a, pl, s);
}
}  // namespace cq
