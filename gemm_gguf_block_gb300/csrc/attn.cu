// Dispatch of the attention over the 8-bit paged cache (cq_attn_paged in
// include/cq_kv.h, cq_attn_tree in
// include/cq_tree.h) and its workspace.
#include <algorithm>
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

// Trees: a call's requests go to one kernel, all of them, by the widest's rows -- a tree costs the tiles the same
// whatever its width, and tiles beside rows slow both (64 contexts of 200-8190, bf16, 12-36 rows: 276 us with the border
// at 33 rows, 113 all in the tiles, 162 all in the rows kernel). Few (request, kv head) pairs leave the rows kernel enough
// SMs for longer. Rows kernel / tiles, us, 32 query and 8 kv heads of 128, bf16 (binary16's tiles take 12% more, fp32 takes
// 1.2 to 1.75 times as long in both):
//   64 requests of 1500 keys    12 rows 75 / 101     16 rows 78 / 102    24 rows 129 / 103    64 rows 239 / 104
//   16 requests of 1500 keys    12 rows 31 / 28      16 rows 35 / 28     24 rows 45 / 29      64 rows 76 / 29
//   2 requests of 20000 keys    12 rows 46 / 52      24 rows 61 / 56     32 rows 67 / 57      64 rows 98 / 57
//   1 request of 1000 keys      16 rows 19 / 25      32 rows 19 / 25     64 rows 20 / 25      128 rows 22 / 26
// What decides is rows times keys for each SM, and the host is not told the keys: the borders suit many requests, and
// few with long contexts. One short context of 64 rows and more takes a quarter longer than it would in the rows kernel, 16
// requests of 16 rows a quarter longer than in the tiles.
constexpr int TREE_ROWS = 16, TREE_ROWS_FEW = 32, TREE_FEW = 32;

// 16-bit calls under masks take one row tile a CTA where the widest request fits it (bf16, 64 requests of 1500 keys, 48
// rows: 101 us, 135 with two tiles; 4 of 30k-60k keys and 96-192 rows: 222 in two items for 193). binary16 ones also up to this
// many new tokens: the probabilities' second part has columns there alone, and trees have it whatever stands beside them. For
// longer prompts two tiles are worth the trees' time in the rows kernel: a prompt of 2000 / 4000 tokens beside 31 trees of 16
// (1500 keys) takes 123 / 263 us in one tile and 196 / 288 the other way, beside 31 of 6 156 / 302 and 134 / 227.
constexpr int PAIRS_NEW = 2048;

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
    const bool trees = a.tree != nullptr && a.max_new <= CQ_TREE_MAX;
    const bool few = static_cast<int64_t>(a.R) * c.heads < TREE_FEW;
    const bool tiles = trees ? a.max_new * G > (few ? TREE_ROWS_FEW : TREE_ROWS) : a.max_new * G >= TILE_ROWS;
    pl.tile_rows = !tiles ? INT_MAX : trees ? 1 : TILE_ROWS;
    const bool pairs = a.tree != nullptr && dtype == CQ_F16;
    pl.one_tile = a.max_new * G <= 128 || (pairs && a.max_new <= PAIRS_NEW);
    // beyond that the two tiles' P, of 11 bits, is for prompts alone: the trees are the rows kernel's
    if (tiles && pairs && !pl.one_tile) pl.tile_rows = static_cast<int>(std::max<int64_t>(TILE_ROWS, CQ_TREE_MAX * G + 1));
    pl.after_tiles = tiles;
    if (tiles) {
        const cudaError_t e = launch_attn_tiles(dev, c, dtype, a, pl, s);
        if (e != cudaSuccess) return e;
    }
    return launch_attn_rows(dev, c, dtype, a, pl, s);
}

}  // namespace cq
