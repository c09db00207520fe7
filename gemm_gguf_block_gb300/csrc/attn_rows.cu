// Attention for few query rows (attn_rows.cuh): causal and windowed calls.
#include "attn_rows.cuh"

namespace cq {
cudaError_t launch_attn_rows(const DeviceInfo& dev, const KvView& c, int dtype, const AttnArgs& a, const RowsPlan& pl,
                             cudaStream_t s) {
    return launch_rows<false>(dev, c, dtype, a, pl, s);
}
}  // namespace cq
