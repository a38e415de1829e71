// attention.cu -- attention of one new token over the paged key-value cache
// ("Hesper.Models.BitNet" page, section "KV cache": a token attends to the keys and
// values that earlier ones left).
//
//   out[b, h] = sum_t p_t v_t / sum_t p_t,  p_t = 2^(x_t - ref),  x_t = log2(e) scale q[b, h] . k_t
// over the tokens t of sequence b that its length and the window leave, in one
// pass over keys and values with a running reference, sum and weighted sum.
//
// One CTA takes a share of the tokens of one key head of one sequence, for up to 8
// of the q heads that share it; the shares of a sequence are the CTAs of one
// thread-block cluster.  A warp works alone: it streams its own steps of 16 or 32
// tokens (steps go round all warps of a sequence, so a warp's first page is known
// before the length is) through a ring of two shared-memory stages with asynchronous
// copies, and no barrier stands between copy and use.  At the end the warps' partials
// meet in shared memory, and each CTA sends each of its cluster its share of the dims
// to join: one cluster barrier, joins in a fixed order.
//
// Both products run on the warp-level MMA (m16n8k16, fp32 sums) whatever the
// number of q heads: a cache is bound by its bytes, and the MMA takes a token's
// key in fewer instructions than fp32 arithmetic on widened codes (one widening
// per code, no multiply-add; 8 q heads cost what one does).  Its 16 rows carry the
// 8 heads twice: rows 0-7 the leading parts of q (or p), rows 8-15 what they leave.
//   8-bit codes are exact in fp16; q and p are split into two fp16 parts (22 bits,
//   the second scaled by 2^11), q after scaling each head's row by a power of two.
//   bf16 values are used as they are; q and p are split into three bf16 parts (24
//   bits), the third in a second MMA, of rows 8-15 too: the adder cuts a sum toward zero
//   (-1.1 of 2^-24 of a logit of 80 dims; -3 with the third parts on the leading rows,
//   and twice the error of an output).
// So a logit and a weighted sum keep fp32 accuracy.  The key's step multiplies the
// logit, the value's step multiplies p.
//
// One lazy reference a head: p_t = 2^(x_t - ref), with ref moved only when some
// p_t times its value's step exceeds 2^8, to the largest x_t + log2(step).  So the
// weights that enter the second product stay in fp16's range and keep their bits
// whatever the steps are, and sum, weighted sum and ref need no other scale.
// The MMA sums of a step (16 or 32 tokens) start from zero and are added to fp32
// sums in registers: a chain of roundings no longer than the steps of a warp.
//
// With a workspace and long sequences, rows (a key head of a sequence, for up to 8 q
// heads) get CTAs in proportion to their steps instead, all of them resident at once,
// so lengths of any mix end together; a row of several CTAs leaves their partials in
// the workspace and a second small launch joins them in the order of the CTAs.
// Without one, rows that fill the GPU more than once (up to five times, of up to 128
// sequences) start with the longest.
//
// What bounds it (GB300, DRAM copy peak 6.78 TB/s; a graph's replay, so with launches):
// with the GPU full the cache's bytes and, for 8-bit codes, the instructions that widen
// them: 456 sequences of 1024 tokens, 8 key heads, are read at 100 % (bf16, 128 dims), 94 %
// (e4m3, 128, 4 q heads a key head) and 92 % (int8, 80) of the peak.  64 ragged sequences
// of up to 2048 tokens, 32 heads of 80, int8: 62.8 us, 81 %.  Few tokens are bound by
// latency: 2048 tokens of 32 heads take 5.9 us, 1.6 us of it bytes (a launch, the lookups,
// two steps of a warp one after the other, the joins).
// Tried and slower or no faster: five CTAs an SM at 96 registers (104 for 107 us with the
// GPU full, but 60 for 55 in one wave), three and four stages, two steps requested before the
// first is used, 8 warps a CTA, one logit a lane through shared memory where a key head has
// one q head, pieces of a single line through all rows (cut rows drain their pipelines
// twice), keys and values requested apart (a step and a half on their way, 75.5 for 67.8 us
// on the ragged batch), two CTAs a row where rows alone fill the GPU half to once (lengths
// are known on the GPU alone: 24.0 for 30.3 us on 48 ragged sequences of 8 key heads, 31.6
// for 26.6 on 12 equal ones of 32).
#include "attend.cuh"

namespace bitlinear {
namespace {

// Joins the parts of rows that several CTAs had: one CTA a (sequence, q head); teams of
// D threads, a thread a dim, take the parts in turn, each against a maximum of its own,
// and meet in order.  Two trips to memory: what the row has, and all of its parts.
constexpr int kJoinThreads = 512;
template <int T>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttendArgs a, KvPages c, Shares sh) {
  __shared__ float values[kJoinThreads];
  __shared__ float2 scales[kJoinThreads / 16];
  pdl_release_dependents();
  pdl_wait_primary();
  const int D = c.head_dim, team = threadIdx.x / D, teams = blockDim.x / D, d = threadIdx.x - team * D;
  const uint32_t b = blockIdx.x / (uint32_t)a.q_heads;
  const int h = blockIdx.x - b * a.q_heads, hk = h / sh.group, in_group = h - hk * sh.group;
  const int32_t length = a.lengths[b];
  const int2 row = sh.rows[(int64_t)b * sh.rows_a_seq + hk * sh.groups + in_group / kRowHeads];
  float* out = a.out + b * a.out_stride + (int64_t)h * D;
  const bool empty = Span<T>(length, a.max_pages << c.page_shift, a.window).steps() == 0;  // then no CTA had the row
  if (empty && threadIdx.x < D) out[d] = 0.0f;
  if (empty || row.y == 1) return;  // one CTA had all of it and has written it
  const int64_t apart = (int64_t)min(kRowHeads, sh.group) * (D + 4);
  const float* p = sh.parts + row.x * apart + in_group % kRowHeads * (D + 4);
  float m = kUnset, sum = 0.0f, value = 0.0f;
  if (team < teams) {
    constexpr int kTogether = 8;
    for (int i = team; i < row.y; i += kTogether * teams) {
      float2 s[kTogether];
      float v[kTogether], top = m;
#pragma unroll
      for (int n = 0; n < kTogether; ++n) {
        const float* q = p + (i + n * teams) * apart;
        const bool have = i + n * teams < row.y;
        s[n] = have ? *reinterpret_cast<const float2*>(q + D) : make_float2(kUnset, 0.0f);
        v[n] = have ? q[d] : 0.0f;
      }
#pragma unroll
      for (int n = 0; n < kTogether; ++n) top = fmaxf(top, s[n].x);
      const float down = exp2_of(m - top);
      m = top;
      sum *= down;
      value *= down;
#pragma unroll
      for (int n = 0; n < kTogether; ++n) {
        const float f = exp2_of(s[n].x - m);
        sum = fmaf(s[n].y, f, sum);
        value = fmaf(v[n], f, value);
      }
    }
    if (teams > 1) {
      values[threadIdx.x] = value;
      if (d == 0) scales[team] = make_float2(m, sum);
    }
  }
  if (teams > 1) {
    __syncthreads();
    if (threadIdx.x >= D) return;
    for (int t = 0; t < teams; ++t) m = fmaxf(m, scales[t].x);
    sum = value = 0.0f;
    for (int t = 0; t < teams; ++t) {
      const float f = exp2_of(scales[t].x - m);
      sum = fmaf(scales[t].y, f, sum);
      value = fmaf(values[t * D + d], f, value);
    }
  }
  if (team == 0) out[d] = output_of(value, m, sum);
}

int64_t rows_of(int64_t B, int q_heads, int kv_heads) {
  return B * kv_heads * ((q_heads / kv_heads + kRowHeads - 1) / kRowHeads);
}

// The most CTAs that rows are shared out over, of any format and padded head size,
// and whether so many rows are few enough for it (rows round up to whole CTAs).
constexpr int kShareCtas = 4 * kSms;
bool shares_fit(int64_t B, int64_t rows, int ctas) { return B <= kShareSeqs && rows <= ctas / 3; }

// Sharing out costs ~3 us more than clusters do (finding the row, the second launch)
// and fills what they leave idle.  Measured, clusters / shared out, us: one sequence of 8 key
// heads bf16, 8192 tokens 12.9 / 14.9, 16384 20.9 / 20.6, 32768 36.5 / 29.9; of one key head
// e4m3, 8192 9.2 / 10.4, 32768 21.8 / 16.0; of 32 heads of 80 int8, 16384 21.9 / 24.1; 4 ragged
// ones of 8 key heads e4m3, up to 16384 18.1 / 19.4, up to 32768 29.5 / 26.4; 8 equal ones of
// 8192 26.3 / 30.1.
bool share_out_wins(int64_t B, int64_t rows, int64_t tokens, int splits, int ctas) {
  const int64_t a_warp = tokens / (splits * kWarps);
  if (B > 1 && a_warp >= 512) return true;  // lengths may differ: the longest row would end alone
  return a_warp * (ctas - rows * splits) >= (int64_t)192 * ctas;
}

template <int FORMAT, int DT>
cudaError_t launch_shape(AttendArgs a, const KvPages& c, void* workspace, bool pdl, const DeviceInfo& dev,
                         cudaStream_t stream) {
  using S = Shape<FORMAT, DT>;
  set_factor(a);
  const auto clusters = attend_kernel<FORMAT, DT, kClusters>, shared_out = attend_kernel<FORMAT, DT, kSharedOut>;
  static thread_local int configured_device = -1, most_cluster;
  if (configured_device != dev.device) {
    cudaError_t err = allow_shared_memory<S>(shared_out);
    if (err == cudaSuccess) err = allow_clusters<S>(clusters, &most_cluster);
    if (err != cudaSuccess) return err;
    configured_device = dev.device;
  }
  const int64_t rows = rows_of(a.B, a.q_heads, c.heads);
  int64_t tokens = a.max_pages << c.page_shift;
  if (a.window > 0 && a.window < tokens) tokens = a.window + S::kTokens;  // a window may begin inside a step
  const int64_t steps = (tokens + S::kTokens - 1) / S::kTokens;
  const int group = a.q_heads / c.heads, groups = (group + kRowHeads - 1) / kRowHeads;
  const int heads = group < kRowHeads ? group : kRowHeads;
  const int smem = (int)S::kSmem + heads * S::kHeadBytes + kRowHeads * 4;  // the rings, q's parts and scales
  const int ctas = resident_ctas<S>(dev, smem), cluster_ctas = resident_ctas<S>(dev, smem + received_bytes(heads, c.head_dim, kMaxCluster));
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  auto programmatic = [&] {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  };
  Shares sh = {0, group, groups, c.heads * groups, splits_for(rows, steps, cluster_ctas, most_cluster), 0, false, nullptr, nullptr};
  while ((1 << sh.splits_log2) < sh.splits) ++sh.splits_log2;
  if (workspace && shares_fit(a.B, rows, ctas) && steps_fit(rows, steps) &&
      share_out_wins(a.B, rows, tokens, sh.splits, ctas)) {
    sh.parts = static_cast<float*>(workspace);
    sh.rows = reinterpret_cast<int2*>(sh.parts + (size_t)kShareCtas * heads * (c.head_dim + 4));
    cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    if (pdl) programmatic();
    const cudaError_t err = cudaLaunchKernelEx(&cfg, shared_out, a, c, sh);
    if (err != cudaSuccess) return err;
    cfg.gridDim = dim3((unsigned)(a.B * a.q_heads), 1, 1);
    // teams of D threads, 8 parts each at a time: as many as the parts of an average row want
    const int64_t parts = (ctas / rows + 7) / 8, most = kJoinThreads / c.head_dim;
    cfg.blockDim = dim3((unsigned)(c.head_dim * (parts < 1 ? 1 : parts < most ? parts : most)), 1, 1);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 0;
    programmatic();
    return cudaLaunchKernelEx(&cfg, join_kernel<S::kTokens>, a, c, sh);
  }
  // The longest sequences first, where rows come in more than one round and up to five: each
  // CTA then ranks all sequences.  Measured in their own order / sorted, us: 64 sequences of
  // up to 2048 tokens, 32 heads of 80, int8 (3.4 rounds) 69 / 63; 128 of 8 key heads e4m3 (1.7)
  // 60 / 48.5; 128 of up to 1024, 32 heads (6.7) 73 / 80.
  sh.sorted = a.B > 1 && a.B <= kSortSeqs && rows * sh.splits > ctas && rows <= 5 * (int64_t)ctas;
  return launch_clusters<FORMAT, DT, kClusters>(a, c, sh, smem + received_bytes(heads, c.head_dim, sh.splits), pdl, stream);
}

}  // namespace

size_t attention_workspace_bytes(int64_t B, int q_heads, int kv_heads, int head_dim) {
  const int64_t rows = rows_of(B, q_heads, kv_heads);
  if (!shares_fit(B, rows, kShareCtas)) return 0;
  const int group = q_heads / kv_heads, heads = group < kRowHeads ? group : kRowHeads;
  return (size_t)kShareCtas * heads * (head_dim + 4) * sizeof(float) + (size_t)rows * sizeof(int2);
}

cudaError_t launch_attention(const AttendArgs& a, const KvPages& cache, void* workspace, bool pdl,
                             const DeviceInfo& dev, cudaStream_t stream) {
  return of_shape(cache, [&](auto format, auto dims) {
    return launch_shape<decltype(format)::value, decltype(dims)::value>(a, cache, workspace, pdl, dev, stream);
  });
}

}  // namespace bitlinear
