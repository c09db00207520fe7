// Dispatch of the attention over the 8-bit paged cache (cq_attn_paged in
// include/cq_kv.h) and its workspace.
#include <climits>

#include "attn_common.cuh"

namespace cq {
namespace {

// Rows (token, head of a kv head) of a request from which its prompt goes to the
// 128-row tiles.
constexpr int TILE_ROWS = 128;

constexpr size_t COUNT_BYTES = ATTN_MAX_CTAS * sizeof(int);
size_t part_bytes(int64_t head_dim) { return size_t(ATTN_MAX_CTAS) * 2 * 16 * (head_dim + 4) * sizeof(float); }

}  // namespace

size_t attn_workspace_size(int64_t head_dim) { return COUNT_BYTES + part_bytes(head_dim); }

cudaError_t launch_attn(const DeviceInfo& dev, const KvView& c, int dtype, const AttnArgs& a, cudaStream_t s) {
    RowsPlan pl{};
    pl.count = static_cast<int*>(a.ws);
    pl.part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + COUNT_BYTES);
    const int64_t G = a.heads / c.heads;
    // Which kernel a request goes to is decided on the GPU by its own length: the host
    // only says whether there may be any for the tiles.
    const bool tiles = a.max_new * G >= TILE_ROWS;
    pl.tile_rows = tiles ? TILE_ROWS : INT_MAX;
    pl.after_tiles = tiles;
    if (tiles) {
        const cudaError_t e = launch_attn_tiles(dev, c, dtype, a, pl, s);
        if (e != cudaSuccess) return e;
    }
    return launch_attn_rows(dev, c, dtype, a, pl, s);
}

}  // namespace cq
