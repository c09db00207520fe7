// Attention for few query rows (attn_rows.cuh) under a tree's masks.
#include "attn_rows.cuh"

namespace cq {
cudaError_t launch_attn_tree_rows(const DeviceInfo& dev, const KvView& c, int dtype, const AttnArgs& a, const RowsPlan& pl,
                                  cudaStream_t s) {
    return launch_rows<true>(dev, c, dtype, a, pl, s);
}
}  // namespace cq
