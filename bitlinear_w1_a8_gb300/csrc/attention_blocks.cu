// attention_blocks.cu -- attention of one new token over chosen pages of its sequence (select.cu):
//   out[b, h] = sum_t p_t v_t / sum_t p_t over the tokens t of the pages that a list names for h's key head.
// The kernel is attend.cuh's; tokens are counted along the list, so a warp's step finds its
// page through two look-ups (list, page table), and the work of a row is known on the host.
//
// Bound as attention.cu's by the widening of the codes beside the bytes: 32 pages of 64 tokens each of 16 sequences, 32 heads of
// 80, int8: 38.1 us, 174 MB, 4.6 TB/s, one CTA a row and 512 of 608 places; 64 pages of 64 of one sequence, 8 key heads of 128,
// bf16: 9.8 us, four steps a warp; 8 of 32, 16 heads, fp8: 4.6 us, latency.
#include "attend.cuh"
#include "serve.cuh"

namespace bitlinear {
namespace {

template <int FORMAT, int DT>
cudaError_t launch_shape(AttendArgs a, const KvPages& c, const int32_t* blocks, int count, bool pdl, const DeviceInfo& dev,
                         cudaStream_t stream) {
  using S = Shape<FORMAT, DT>;
  set_factor(a);
  static thread_local int configured_device = -1, most_cluster;
  if (configured_device != dev.device) {
    const cudaError_t err = allow_clusters<S>(attend_kernel<FORMAT, DT, kBlocks>, &most_cluster);
    if (err != cudaSuccess) return err;
    configured_device = dev.device;
  }
  const int group = a.q_heads / c.heads, groups = (group + kRowHeads - 1) / kRowHeads;
  const int heads = group < kRowHeads ? group : kRowHeads;
  const int64_t rows = a.B * c.heads * groups;
  const int64_t steps = (((int64_t)count << c.page_shift) + S::kTokens - 1) / S::kTokens;
  const int smem = (int)S::kSmem + heads * S::kHeadBytes + kRowHeads * 4;
  const int ctas = resident_ctas<S>(dev, smem + received_bytes(heads, c.head_dim, kMaxCluster));
  Shares sh = {};
  sh.group = group;
  sh.groups = groups;
  sh.rows_a_seq = c.heads * groups;
  sh.splits = splits_for(rows, steps, ctas, most_cluster);
  while ((1 << sh.splits_log2) < sh.splits) ++sh.splits_log2;
  sh.blocks = blocks;
  sh.count = count;
  return launch_clusters<FORMAT, DT, kBlocks>(a, c, sh, smem + received_bytes(heads, c.head_dim, sh.splits), pdl, stream);
}

}  // namespace

cudaError_t launch_attention_blocks(const AttendArgs& a, const KvPages& cache, const int32_t* blocks, int count, bool pdl,
                                    const DeviceInfo& dev, cudaStream_t stream) {
  return of_shape(cache, [&](auto format, auto dims) {
    return launch_shape<decltype(format)::value, decltype(dims)::value>(a, cache, blocks, count, pdl, dev, stream);
  });
}

}  // namespace bitlinear
