// attention_shared.cu -- attention of a batch whose rows share their first tokens in groups.
//
// A group's sequences name the same pages for their first shared[g] tokens (a system prompt, a
// document, all of a sequence that several drafted tokens go on from).  Those tokens are
// attended to once for all of the group's q heads of a key head, eight to a CTA or 128 on the
// tensor cores; what a row has behind them is its own:
//   out = (P_shared + P_own) / (sum_shared + sum_own), each sum under its reference, joined as the
// parts of one sequence are (attend.cuh).  Two launches: the shared tokens, split over CTAs
// that leave their parts in the workspace, and each row's own tokens with the join.  The second begins while
// the first runs, as places on the SMs come free, and waits for it where it adds the parts.  shares.h has the rules by which a
// call goes one way or another, with what they were measured by.
//
// Measured (graph replays; the least is of bytes read once at 6684 GB/s): eight sequences of up to 2048 tokens with five
// drafted rows each, 32 heads of 80, int8, 20.6 us (10.1): the least time of a step a warp, two launches and the
// lookups; 64 rows behind 2039 tokens, up to 256 each of their own, 35.7 us (8.5): eight readings of the prefix out of L2
// (21 us, instructions: the schedulers issue in 53 cycles of 100), and own tokens whose warps begin and end with each
// row (2048 rows, 20 us alone, two thirds of it behind the first launch); 64 rows of 8 key heads of 128 behind 16384 tokens, bf16,
// 51.0 us (12.3; of fp8 53.5, of int8 55.1): ~42 of it the tensor cores' part (attention_prefix.cu), the rest the wait for SMs, lookups
// and the join.
#include "attend.cuh"
#include "serve.cuh"

namespace bitlinear {
namespace {

// The most CTAs that shared tokens are split over beside one a row.
constexpr int kPrefixCtas = 4 * kSms;

// How the shared tokens' q heads are cut into rows of work: eight a CTA (attend.cuh), or 128 on the tensor
// cores (attention_prefix.cu).
struct Sizes {
  int64_t group_rows, rows, slots;  // sequences a group; rows of all groups; parts that there may be
  int heads_a_key, tiles, tile, heads;  // q heads a key head; rows a key head of a group, of so many q heads; places in a part
};
Sizes sizes_of(int64_t B, int q_heads, int kv_heads, int64_t groups, bool wide) {
  Sizes s;
  s.group_rows = B / groups;
  s.heads_a_key = q_heads / kv_heads;
  const int64_t all = s.group_rows * s.heads_a_key;
  s.tile = wide ? kPrefixWide : kRowHeads;
  s.tiles = (int)((all + s.tile - 1) / s.tile);
  s.heads = (int)(all < s.tile ? all : s.tile);
  s.rows = groups * kv_heads * s.tiles;
  const int64_t ctas = wide ? kSms : kPrefixCtas;
  s.slots = s.rows > ctas ? s.rows : ctas;
  return s;
}
size_t workspace_of(const Sizes& s, int head_dim) {
  return (size_t)s.slots * s.heads * (head_dim + 4) * sizeof(float) + (size_t)s.rows * sizeof(int2);
}

constexpr int64_t kPackedRows = 300;  // a row a key head of a sequence: from so many on they fill the GPU without clusters

template <int FORMAT, int DT>
cudaError_t launch_shape(AttendArgs a, const KvPages& c, const int32_t* shared, int64_t groups, void* workspace, bool pdl,
                         const DeviceInfo& dev, cudaStream_t stream) {
  using S = Shape<FORMAT, DT>;
  set_factor(a);
  static thread_local int configured_device = -1, most_cluster;
  if (configured_device != dev.device) {
    cudaError_t err = allow_shared_memory<S>(attend_kernel<FORMAT, DT, kPrefix>);
    if (err == cudaSuccess)
      err = cudaFuncSetAttribute(attend_kernel<FORMAT, DT, kPacked>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem + kWarps * kRowHeads * (S::kHeadBytes + 4));
    if (err == cudaSuccess) err = allow_clusters<S>(attend_kernel<FORMAT, DT, kOwn>, &most_cluster);
    if (err != cudaSuccess) return err;
    configured_device = dev.device;
  }
  const bool wide = wide_wins(a.B / groups * (a.q_heads / c.heads), a.max_pages << c.page_shift, c.head_dim, S::kBytes);
  const Sizes sizes = sizes_of(a.B, a.q_heads, c.heads, groups, wide);
  const int64_t steps = ((a.max_pages << c.page_shift) + S::kTokens - 1) / S::kTokens;

  // The shared tokens: a group is a sequence, its rows' q heads those of one key head.
  AttendArgs g = a;
  g.B = groups;
  g.lengths = shared;
  g.table_stride = a.table_stride * sizes.group_rows;
  Shares sh = {};
  sh.group = (int)(sizes.group_rows * sizes.heads_a_key);
  sh.groups = sizes.tiles;
  sh.rows_a_seq = c.heads * sizes.tiles;
  sh.parts = static_cast<float*>(workspace);
  sh.rows = reinterpret_cast<int2*>(sh.parts + sizes.slots * sizes.heads * (c.head_dim + 4));
  sh.group_rows = (int)sizes.group_rows;
  sh.shared = shared;
  sh.lengths = a.lengths;
  sh.heads_a_key = sizes.heads_a_key;
  sh.prefix_tiles = sizes.tiles;
  sh.prefix_heads = sizes.tile;
  sh.slot_heads = sizes.heads;
  int smem = (int)S::kSmem + kRowHeads * (S::kHeadBytes + 4);
  cudaError_t err;
  if (wide) {
    const PrefixRows p = {sh.group, sizes.tiles, sh.group_rows, sizes.heads_a_key, sizes.heads, a.lengths, sh.parts, sh.rows};
    err = launch_prefix_wide(g, c, p, pdl, dev, stream);
  } else {
    const int ctas = resident_ctas<S>(dev, smem);
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    if (pdl) {
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.numAttrs = 1;
    }
    if (groups <= kShareSeqs && sizes.rows <= ctas / 3 && steps_fit(sizes.rows, steps)) {
      cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    } else {
      sh.splits = splits_for(sizes.rows, steps, ctas, kPortableCluster);
      while ((1 << sh.splits_log2) < sh.splits) ++sh.splits_log2;
      cfg.gridDim = dim3((unsigned)(sizes.rows * sh.splits), 1, 1);
    }
    err = cudaLaunchKernelEx(&cfg, attend_kernel<FORMAT, DT, kPrefix>, g, c, sh);
  }
  if (err != cudaSuccess) return err;

  // Each row's own tokens, and the join.
  sh.group = sizes.heads_a_key;
  sh.groups = (sh.group + kRowHeads - 1) / kRowHeads;
  sh.rows_a_seq = c.heads * sh.groups;
  const int heads = sh.group < kRowHeads ? sh.group : kRowHeads;
  const int64_t rows = a.B * sh.rows_a_seq;
  if (rows >= kPackedRows && a.B <= kShareSeqs) {
    smem = (int)S::kSmem + kWarps * (heads * S::kHeadBytes + kRowHeads * 4);
    // A warp finishes a head at a time, so rows of several have as many warps, while all are resident; where one a row
    // fills the GPU, rows are given more only if they are longer.
    const int64_t resident = resident_ctas<S>(dev, smem);
    sh.least_warps = heads >= 3 ? 4 : heads;
    while (sh.least_warps > 1 && rows * sh.least_warps > resident * kWarps) sh.least_warps /= 2;
    sh.warp_steps = rows > 2 * resident ? 8 : 4;
    return launch_grids(attend_kernel<FORMAT, DT, kPacked>, a, c, sh, sh.rows_a_seq, 1, smem, true, stream);
  }
  smem = (int)S::kSmem + heads * S::kHeadBytes + kRowHeads * 4;
  const int own_ctas = resident_ctas<S>(dev, smem + received_bytes(heads, c.head_dim, kMaxCluster));
  sh.splits = splits_for(rows, steps, own_ctas, most_cluster);
  sh.splits_log2 = 0;
  while ((1 << sh.splits_log2) < sh.splits) ++sh.splits_log2;
  return launch_clusters<FORMAT, DT, kOwn>(a, c, sh, smem + received_bytes(heads, c.head_dim, sh.splits), true, stream);
}

}  // namespace

size_t attention_shared_workspace_bytes(int64_t B, int q_heads, int kv_heads, int head_dim, int64_t groups) {
  const size_t alone = attention_workspace_bytes(B, q_heads, kv_heads, head_dim);
  if (groups == B) return alone;
  const size_t narrow = workspace_of(sizes_of(B, q_heads, kv_heads, groups, false), head_dim);
  const size_t wide = workspace_of(sizes_of(B, q_heads, kv_heads, groups, true), head_dim);
  const size_t need = narrow > wide ? narrow : wide;
  return need > alone ? need : alone;
}

cudaError_t launch_attention_shared(const AttendArgs& a, const KvPages& cache, const int32_t* shared, int64_t groups,
                                    void* workspace, bool pdl, const DeviceInfo& dev, cudaStream_t stream) {
  // Nothing is shared, or too little.
  if (groups == a.B || faster_alone(a.B, a.max_pages << cache.page_shift, cache.heads, cache.head_dim,
                                    cache.format == BITLINEAR_KV_BF16 ? 2 : 1, a.q_heads / cache.heads))
    return launch_attention(a, cache, workspace, pdl, dev, stream);
  return of_shape(cache, [&](auto format, auto dims) {
    return launch_shape<decltype(format)::value, decltype(dims)::value>(a, cache, shared, groups, workspace, pdl, dev, stream);
  });
}

}  // namespace bitlinear
