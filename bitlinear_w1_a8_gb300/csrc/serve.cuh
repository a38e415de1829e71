// serve.cuh -- launchers of what a serving step needs beyond one independent token a
// sequence: probabilities and drafted tokens (sample.cu), chosen blocks of the cache
// (select.cu, attention_blocks.cu) and shared prefixes (attention_shared.cu).
#pragma once

#include "kv.cuh"

namespace bitlinear {

// sample.cu
cudaError_t launch_softmax(const float* y, float* p, const float* temperature, int64_t M, int64_t V, bool pdl,
                           const DeviceInfo& dev, cudaStream_t stream);
cudaError_t launch_verify(const float* p, const float* q, const int32_t* draft, const float* uniform, int64_t B, int K,
                          int64_t V, int32_t* tokens, int32_t* accepted, bool pdl, const DeviceInfo& dev,
                          cudaStream_t stream);

// select.cu.  A page's summary: int8 bounds of its keys [page][head][lower, upper][dim] and a step [page][head].
struct Summary {
  int8_t* bounds;
  float* step;
};
cudaError_t launch_summarise(const KvPages& cache, const Summary& summary, const int32_t* table, int64_t table_stride,
                             int64_t B, int64_t max_pages, const int32_t* first, const int32_t* lengths, bool pdl,
                             const DeviceInfo& dev, cudaStream_t stream);
constexpr int64_t kMostBlocks = 131072;  // of a sequence: their scores stay in shared memory
struct SelectArgs {
  const float* q;
  int64_t q_stride;
  int q_heads;
  const int32_t* table;
  int64_t table_stride, max_pages;
  const int32_t* lengths;
  int keep_first, keep_last, count;
  int32_t* blocks;
  int64_t B;
};
cudaError_t launch_select(const SelectArgs& a, const KvPages& cache, const Summary& summary, bool pdl,
                          const DeviceInfo& dev, cudaStream_t stream);

// attention_blocks.cu
cudaError_t launch_attention_blocks(const AttendArgs& a, const KvPages& cache, const int32_t* blocks, int count, bool pdl,
                                    const DeviceInfo& dev, cudaStream_t stream);

// attention_prefix.cu: the shared tokens of groups (a.B of them, a.lengths tokens each) for kPrefixWide q heads a CTA.
struct PrefixRows {
  int group, tiles;             // q heads of a group for a key head, in tiles of 128
  int group_rows, heads_a_key;  // its sequences, and their q heads a key head
  int slot_heads;               // places in a part
  const int32_t* lengths;       // of every sequence
  float* parts;                 // [CTA][slot_heads][dims, m, sum]
  int2* rows;                   // of each group, key head and tile: its first CTA and how many it has
};
cudaError_t launch_prefix_wide(const AttendArgs& a, const KvPages& c, const PrefixRows& p, bool pdl, const DeviceInfo& dev,
                               cudaStream_t stream);

// attention_shared.cu
size_t attention_shared_workspace_bytes(int64_t B, int q_heads, int kv_heads, int head_dim, int64_t groups);
cudaError_t launch_attention_shared(const AttendArgs& a, const KvPages& cache, const int32_t* shared, int64_t groups,
                                    void* workspace, bool pdl, const DeviceInfo& dev, cudaStream_t stream);

}  // namespace bitlinear
