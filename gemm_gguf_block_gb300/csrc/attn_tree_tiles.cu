// Attention over wide trees, and prompts beside them (attn_tiles.cuh), under a tree's masks.
#include "attn_tiles.cuh"

namespace cq {
cudaError_t launch_attn_tree_tiles(const DeviceInfo& dev, const KvView& c, int dtype, const AttnArgs& a, const RowsPlan& pl,
                                   cudaStream_t s) {
    return launch_tiles<true>(dev, c, dtype, a, pl, s);
}
}  // namespace cq
