// Launchers of a tree decoding step's calls (include/cq_tree.h); arguments are validated by the
// caller (cq_api.cu).
#pragma once
#include <cstdint>

#include "cq_internal.h"
#include "cq_tree.h"
#include "kv.cuh"

namespace cq {

struct RopeArgs {
    const void* x[2];            // queries, keys
    void* y[2];
    const float* w[2];           // norms or NULL
    int64_t x_stride[2], y_stride[2];   // elements
    const int32_t* positions;
    const double* freqs;
    float eps;
    int T, heads[2], rot, adjacent;
};
cudaError_t launch_qk_rope(const DeviceInfo& dev, int in, int out, int64_t head_dim, const RopeArgs& a, cudaStream_t s);

cudaError_t launch_tree_plan(const DeviceInfo& dev, int R, int T, const int32_t* kv_len, const int32_t* q_start,
                             const int32_t* parent, uint64_t* mask, int32_t* positions, cudaStream_t s);

struct VerifyArgs {
    const float* logits;
    const float* draft;          // or NULL
    int64_t logits_stride, draft_stride;
    const int32_t* tokens;
    const int32_t* parent;
    const int32_t* q_start;
    const float* temperature;
    const float* u_accept;
    const float* u_sample;
    int32_t* count;
    int32_t* path;
    int32_t* next;
    int* status;
    int R, T, V, max_path;
};
cudaError_t launch_tree_verify(const DeviceInfo& dev, const VerifyArgs& a, cudaStream_t s);

struct MoveArgs {
    const int32_t* table;
    const int32_t* kv_len;
    const int32_t* q_start;
    const int32_t* count;
    const int32_t* path;
    int32_t* new_len;
    int* status;
    int64_t max_blocks;
    int R, max_path;
};
cudaError_t launch_kv_move(const DeviceInfo& dev, const KvView& c, const MoveArgs& a, cudaStream_t s);

cudaError_t launch_kv_release(const DeviceInfo& dev, int R, int page_shift, const int32_t* table, int64_t max_blocks,
                              int64_t num_pages, const int32_t* old_len, const int32_t* new_len, int32_t* freed,
                              int capacity, int32_t* used, cudaStream_t s);

}  // namespace cq
