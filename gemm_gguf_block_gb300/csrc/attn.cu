// Dispatch of the attention over the 8-bit paged cache (cq_attn_paged in
// include/cq_kv.h, cq_attn_tree in
// include/cq_tree.h) and its workspace.
#include <climits>

#include "attn_common.cuh"

namespace cq {
namespace {

// Rows (token, head of a kv head) of a request from which it goes to the tiles.
// 32 query and 8 kv heads, time of the rows kernel at 16 / 32 / 48 rows and of the tiles: 16
// requests of 1500 keys, bf16 at 128: 33 / 48 / 62 against 39 us; fp32 at 128: 39 / 61 / 83
// against 52; 2 requests of 20000 keys, bf16 at 64: 32 / 42 / 54 against 53; 64 requests of 1500,
// bf16 at 128: 77 / 128 / 182 against 139.
constexpr int TILE_ROWS = 40;

// The workspace: the rows kernel's counters (the part that has to be zero) and parts, then the
// tiles kernel's. All but the counters is written by a call before it is read.
static_assert(ATTN_MAX_CTAS * sizeof(int) <= CQ_ATTN_WORKSPACE_ZERO, "the counters");
struct Layout {
    size_t count, part, share, tile_part, total;
};
Layout layout(int64_t head_dim) {
    const size_t row = static_cast<size_t>(head_dim + 4) * sizeof(float);
    Layout l{};
    l.part = CQ_ATTN_WORKSPACE_ZERO;
    l.share = l.part + size_t(ATTN_MAX_CTAS) * 2 * 16 * row;
    l.tile_part = l.share + ATTN_TILE_CTAS * sizeof(TileShare);
    l.total = l.tile_part + size_t(ATTN_TILE_CTAS) * 256 * row;
    return l;
}

}  // namespace

size_t attn_workspace_size(int64_t head_dim) { return layout(head_dim).total; }

cudaError_t launch_attn(const DeviceInfo& dev, const KvView& c, int dtype, const AttnArgs& a, cudaStream_t s) {
    const Layout l = layout(c.dim);
    char* ws = static_cast<char*>(a.ws);
    RowsPlan pl{};
    pl.count = reinterpret_cast<int*>(ws + l.count);
    pl.part = reinterpret_cast<float*>(ws + l.part);
    pl.share = reinterpret_cast<TileShare*>(ws + l.share);
    pl.tile_part = reinterpret_cast<float*>(ws + l.tile_part);
    pl.sms = dev.sm_count < ATTN_TILE_CTAS ? dev.sm_count : ATTN_TILE_CTAS;
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
