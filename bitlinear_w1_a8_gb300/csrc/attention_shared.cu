// attention_shared.cu -- attention of a batch whose rows share their first tokens in groups.
//
// A group's sequences name the same pages for their first shared[g] tokens (a system prompt, a
// document, all of a sequence that several drafted tokens go on from).  Those tokens are
// attended to once for all of the group's q heads of a key head, eight to a CTA or 128 on the
// tensor cores; what a row has behind them is its own:
//   out = (P_shared + P_own) / (sum_shared + sum_own), each sum under its reference, joined as the
// parts of one sequence are (attend.cuh).  Two launches: the shared tokens, split over CTAs
// that leave their parts in the workspace, and each row's own tokens with the join.  The second begins while
// the first runs, as places on the SMs come free, and waits for it where it adds the parts.
//
// Measured (graph replays; the least is of bytes read once at 6684 GB/s): eight sequences of up to 2048 tokens with five
// drafted rows each, 32 heads of 80, int8, 20.4 us (10.1): the least time of a step a warp, two launches and the
// lookups; 64 rows behind 2039 tokens, up to 256 each of their own, 35.7 us (8.5): eight readings of the prefix out of L2
// (21 us, instructions: the schedulers issue in 53 cycles of 100), and own tokens whose warps begin and end with each
// row (2048 rows, 20 us alone, two thirds of it behind the first launch); 64 rows of 8 key heads of 128 behind 16384 tokens, bf16,
// 51.0 us (12.3): ~42 of it the tensor cores' part (attention_prefix.cu), the rest the wait for SMs, lookups and the join.
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

// The tensor cores take 128 q heads of a key head in the time of 32, and ~8 us more to begin and to end.
// us, eight a CTA / 128 on the tensor cores, one group, up to 64 tokens of each row's own:
//   q heads a key head           24             32             48             64             96             128
//   int8, 32 heads of 80   512   11.8 / 16.9    12.3 / 16.9    16.7 / 24.1    17.3 / 24.8    23.6 / 28.5    29.2 / 33.1
//                         2048   18.1 / 27.8    20.0 / 28.2    23.7 / 29.2    27.2 / 29.5    41.0 / 35.3    49.9 / 39.8
//                         8192   30.2 / 50.4    38.4 / 50.7    52.2 / 53.3    69.5 / 54.1   108.7 / 59.2   136.4 / 66.4
//                        32768   89.1 / 142.2  125.5 / 142.5  166.4 / 153.1  241.9 / 154.1  377.5 / 159.6  479.9 / 173.2
//   bf16, 8 of 128         512   15.7 / 21.0    14.9 / 18.6    16.7 / 21.3    17.3 / 19.5    18.6 / 22.0    17.3 / 19.6
//                         2048   17.8 / 24.4    18.3 / 21.0    20.8 / 22.0    21.3 / 22.2    26.3 / 23.1    27.8 / 22.7
//                         8192   25.3 / 29.5    26.8 / 26.8    35.0 / 27.8    40.0 / 28.2    58.9 / 29.2    71.2 / 28.9
//                        32768   55.5 / 56.3    65.4 / 50.9    94.1 / 52.4   115.2 / 52.1   189.6 / 53.4   245.6 / 53.1
// Tokens are those that the table has room for.
bool wide_wins(const AttendArgs& a, const KvPages& c, int64_t groups) {
  const int64_t heads = a.B / groups * (a.q_heads / c.heads), tokens = a.max_pages << c.page_shift;
  return c.head_dim <= 128 && heads >= (c.format == BITLINEAR_KV_BF16 ? 28 : 40) + 65536 / tokens;
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
  const bool wide = wide_wins(a, c, groups);
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

// Whether attention that reads a group's tokens again for each of its rows is faster: it is one launch, and the
// second reading is of L2.  By the bytes that all rows read at most, the table's columns filled; us, shared / alone, one
// group, up to 64 tokens of each row's own:
//   32 heads of 80, int8, 24 rows x  512 tokens (63 MB) 11.8 / 20.0    16 heads of 128, int8, 24 x  512 (50 MB) 12.5 / 13.9
//   8 of 128 under 32 q heads, fp8, 16 x 2048 (67 MB) 20.2 / 16.3      24 x 2048 (100 MB) 21.7 / 21.7
//   the same, bf16, 8 x 2048 (67 MB) 18.3 / 14.5                       16 x 2048 (134 MB) 21.3 / 22.7
// and of 2 rows of 38 tokens, 16 heads of 128 dims: 8.7 / 3.1.
constexpr double kAloneBytes = 36e6;  // for each of the q heads of a key head, up to three
bool faster_alone(const AttendArgs& a, const KvPages& c) {
  const double code = c.format == BITLINEAR_KV_BF16 ? 2 : 1;
  const double bytes = (double)a.B * (double)a.max_pages * (double)(1 << c.page_shift) * c.heads * c.head_dim * 2 * code;
  const int group = a.q_heads / c.heads;
  return bytes <= kAloneBytes * (group < 3 ? group : 3);
}

cudaError_t launch_attention_shared(const AttendArgs& a, const KvPages& cache, const int32_t* shared, int64_t groups,
                                    void* workspace, bool pdl, const DeviceInfo& dev, cudaStream_t stream) {
  // Nothing is shared, or too little.
  if (groups == a.B || faster_alone(a, cache))
    return launch_attention(a, cache, workspace, pdl, dev, stream);
  return of_shape(cache, [&](auto format, auto dims) {
    return launch_shape<decltype(format)::value, decltype(dims)::value>(a, cache, shared, groups, workspace, pdl, dev, stream);
  });
}

}  // namespace bitlinear
