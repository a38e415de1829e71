// attention.cu -- attention of one new token over the paged key-value cache.
//
//   out[b, h] = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale * q[b, h] . k_t - m)
// over the tokens t of sequence b that its length and the window leave, m the
// running maximum of the logits: one pass over keys and values.
//
// One CTA per (sequence, q head); its warps take every fourth token and a lane
// holds every 32nd dim; the warps' (m, sum, weighted sum) meet in shared memory.
#include <cuda_bf16.h>

#include "kv.cuh"

namespace bitlinear {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxHead = 256;
constexpr int kLaneDims = kMaxHead / 32;

template <int FORMAT>
__device__ __forceinline__ float value_at(const void* codes, int64_t i) {
  if constexpr (FORMAT == BITLINEAR_KV_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(codes)[i]);
  if constexpr (FORMAT == BITLINEAR_KV_INT8) return (float)static_cast<const int8_t*>(codes)[i];
  return __half2float(__ushort_as_half((unsigned short)half2_of_e4m3x2(static_cast<const uint8_t*>(codes)[i])));
}

template <int FORMAT>
__global__ void __launch_bounds__(kThreads) attend_kernel(AttendArgs a, KvPages c) {
  __shared__ float sm[kWarps], sl[kWarps], sacc[kWarps][kMaxHead];
  pdl_release_dependents();
  pdl_wait_primary();
  const int hq = blockIdx.x, hk = hq / (a.q_heads / c.heads), D = c.head_dim;
  const int64_t b = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
  if (b >= a.B) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t len = a.lengths[b];
  const int64_t most = a.max_pages << c.page_shift;
  len = len < most ? len : most;
  const int64_t first = a.window > 0 && len > a.window ? len - a.window : 0;
  float q[kLaneDims], acc[kLaneDims];
#pragma unroll
  for (int j = 0; j < kLaneDims; ++j) {
    const int d = lane + 32 * j;
    q[j] = d < D ? a.q[b * a.q_stride + (int64_t)hq * D + d] * a.scale : 0.0f;
    acc[j] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int64_t t = first + warp; t < len; t += kWarps) {
    const int32_t page = a.table[b * a.table_stride + (t >> c.page_shift)];
    if (page < 0 || page >= c.num_pages) continue;
    const int64_t row = (((int64_t)page * c.heads + hk) << c.page_shift) + (t & ((1 << c.page_shift) - 1));
    float x = 0.0f;
#pragma unroll
    for (int j = 0; j < kLaneDims; ++j)
      if (lane + 32 * j < D) x = fmaf(q[j], value_at<FORMAT>(c.k, row * D + lane + 32 * j), x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFullMask, x, o);
    if (FORMAT != BITLINEAR_KV_BF16) x *= c.k_step[row];
    const float up = fmaxf(m, x), f = expf(m - up), p = expf(x - up);
    const float w = FORMAT != BITLINEAR_KV_BF16 ? p * c.v_step[row] : p;
    m = up;
    l = fmaf(l, f, p);
#pragma unroll
    for (int j = 0; j < kLaneDims; ++j)
      if (lane + 32 * j < D) acc[j] = fmaf(acc[j], f, w * value_at<FORMAT>(c.v, row * D + lane + 32 * j));
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int j = 0; j < kLaneDims; ++j) sacc[warp][lane + 32 * j] = acc[j];
  __syncthreads();
  float top = -INFINITY, sum = 0.0f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
  for (int w = 0; w < kWarps; ++w)
    if (sm[w] > -INFINITY) sum += sl[w] * expf(sm[w] - top);
  for (int d = threadIdx.x; d < D; d += kThreads) {
    float o = 0.0f;
    for (int w = 0; w < kWarps; ++w)
      if (sm[w] > -INFINITY) o += sacc[w][d] * expf(sm[w] - top);
    a.out[b * a.out_stride + (int64_t)hq * D + d] = sum > 0.0f ? o / sum : 0.0f;  // no token: zeros
  }
}

}  // namespace

size_t attention_workspace_bytes(int64_t, int, int, int) { return 0; }

cudaError_t launch_attention(const AttendArgs& a, const KvPages& cache, void*, bool pdl, const DeviceInfo&,
                             cudaStream_t stream) {
  const auto kernel = cache.format == BITLINEAR_KV_INT8  ? attend_kernel<BITLINEAR_KV_INT8>
                      : cache.format == BITLINEAR_KV_FP8 ? attend_kernel<BITLINEAR_KV_FP8>
                                                         : attend_kernel<BITLINEAR_KV_BF16>;
  const int64_t rows = a.B < 65535 ? a.B : 65535;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.q_heads, (unsigned)rows, (unsigned)((a.B + rows - 1) / rows));
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a, cache);
}

}  // namespace bitlinear
