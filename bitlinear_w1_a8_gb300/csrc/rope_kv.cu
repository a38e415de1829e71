// rope_kv.cu -- rotary positions and the paged key-value cache: rows rotated,
// quantised and written where their page is, and read back.
//
// Rotation ("Hesper.Models.BitNet" page, section "Configuration": ropeBase):
// pair i of a head turns by the angle positions[t] * freq[i].  The angle is
// taken in turns in fp64, positions * (freq / 2 pi), and its whole turns are
// dropped before the sine and cosine, which are rounded once to fp32: a far
// position keeps its fraction of a turn to 2^-53 of the whole angle.  The
// rotation itself is two fp32 products and one sum, unfused.
//
// Quantisation follows activation_quant, a row being one (token, head):
//   int8: code = clamp(rne(x * s), -128, 127), s = 127 * (1 / a), a = max(max|x|, 1e-5)
//   e4m3: code = e4m3(x * s), s = 448 * (1 / a), round to nearest even, saturating
// with step = a / 127 or a / 448, the fp32 value of one unit; bf16 rounds.
#include <cuda_bf16.h>

#include "kv.cuh"

namespace bitlinear {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxHead = 256;             // head_dim limit
constexpr int kLaneDims = kMaxHead / 32;  // dims of a head that a lane holds

// cos and sin of every pair of one position, into shared memory.
__device__ __forceinline__ void fill_angles(const RopeArgs& r, int32_t pos, float2* cs) {
  for (int i = threadIdx.x; i < r.rot_dim / 2; i += blockDim.x) {
    const double turns = (double)pos * (r.freq[i] * 0.15915494309189533577);
    double s, c;
    sincospi(2.0 * (turns - rint(turns)), &s, &c);
    cs[i] = make_float2(__fmul_rn((float)c, r.amplitude), __fmul_rn((float)s, r.amplitude));
  }
}

// Dim d of the head at x, rotated.
__device__ __forceinline__ float rotated(const float* x, int d, const RopeArgs& r, const float2* cs) {
  const float own = x[d];
  if (!r.freq || d >= r.rot_dim) return own;
  const int n = r.rot_dim / 2;
  const bool second = r.layout == BITLINEAR_ROPE_HALF ? d >= n : (d & 1);
  const int i = r.layout == BITLINEAR_ROPE_HALF ? (second ? d - n : d) : d >> 1;
  const float other = x[r.layout == BITLINEAR_ROPE_HALF ? (second ? d - n : d + n) : d ^ 1];
  const float2 a = cs[i];
  return second ? __fadd_rn(__fmul_rn(own, a.x), __fmul_rn(other, a.y))
                : __fsub_rn(__fmul_rn(own, a.x), __fmul_rn(other, a.y));
}

// One warp per (token, head); blockIdx.x is the token, blockIdx.y shares its heads out.
__global__ void __launch_bounds__(kThreads) rope_kernel(const float* x, int64_t x_stride, int H, int D,
                                                        const int32_t* __restrict__ positions, RopeArgs r, float* y,
                                                        int64_t y_stride) {
  __shared__ float2 cs[kMaxHead / 2];
  pdl_release_dependents();
  pdl_wait_primary();
  const int64_t t = blockIdx.x;
  fill_angles(r, positions[t], cs);
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int h = blockIdx.y * kWarps + (threadIdx.x >> 5); h < H; h += gridDim.y * kWarps) {
    const float* in = x + t * x_stride + (int64_t)h * D;
    float* out = y + t * y_stride + (int64_t)h * D;
    float v[kLaneDims];
#pragma unroll
    for (int j = 0; j < kLaneDims; ++j)
      if (lane + 32 * j < D) v[j] = rotated(in, lane + 32 * j, r, cs);
    __syncwarp();  // y may be x: every lane has read its pairs
#pragma unroll
    for (int j = 0; j < kLaneDims; ++j)
      if (lane + 32 * j < D) out[lane + 32 * j] = v[j];
  }
}

// Quantises the D values of a row held by a warp and writes codes and step.
template <int FORMAT>
__device__ __forceinline__ void write_row(const float (&v)[kLaneDims], int D, int64_t row, void* codes, float* steps) {
  const int lane = threadIdx.x & 31;
  if constexpr (FORMAT == BITLINEAR_KV_BF16) {
#pragma unroll
    for (int j = 0; j < kLaneDims; ++j)
      if (lane + 32 * j < D) static_cast<__nv_bfloat16*>(codes)[row * D + lane + 32 * j] = __float2bfloat16_rn(v[j]);
    return;
  }
  constexpr float kTop = FORMAT == BITLINEAR_KV_INT8 ? 127.0f : 448.0f;
  float a = 0.0f;
#pragma unroll
  for (int j = 0; j < kLaneDims; ++j)
    if (lane + 32 * j < D) a = fmaxf(a, fabsf(v[j]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(kFullMask, a, o));
  a = fmaxf(a, 1e-5f);
  const float s = __fmul_rn(__frcp_rn(a), kTop);
#pragma unroll
  for (int j = 0; j < kLaneDims; ++j)
    if (lane + 32 * j < D) {
      const float x = __fmul_rn(v[j], s);
      static_cast<uint8_t*>(codes)[row * D + lane + 32 * j] =
          FORMAT == BITLINEAR_KV_INT8 ? (uint8_t)(int8_t)max(-128, min(127, __float2int_rn(x))) : (uint8_t)e4m3x2(0.0f, x);
    }
  if (lane == 0) steps[row] = __fdiv_rn(a, kTop);
}

// Units of a token: its q heads (rotated into q_out), its k heads (rotated and
// written) and its v heads (written); one warp a unit.
template <int FORMAT>
__global__ void __launch_bounds__(kThreads) append_kernel(const float* q, int64_t q_stride, int q_heads, float* q_out,
                                                          int64_t q_out_stride, const float* __restrict__ k,
                                                          int64_t k_stride, const float* __restrict__ v,
                                                          int64_t v_stride, KvRows rows, RopeArgs r, KvPages c) {
  __shared__ float2 cs[kMaxHead / 2];
  pdl_release_dependents();
  pdl_wait_primary();
  const int64_t t = blockIdx.x;
  const int64_t place = kv_place(rows, c, t);
  if (place < 0) return;
  if (r.freq) fill_angles(r, rows.positions[t], cs);
  __syncthreads();
  const int lane = threadIdx.x & 31, D = c.head_dim;
  const int units = q_heads + 2 * c.heads;
  RopeArgs none = {};
  for (int u = blockIdx.y * kWarps + (threadIdx.x >> 5); u < units; u += gridDim.y * kWarps) {
    const bool is_q = u < q_heads, is_v = u >= q_heads + c.heads;
    const int h = is_q ? u : u - q_heads - (is_v ? c.heads : 0);
    const float* in = (is_q ? q + t * q_stride : is_v ? v + t * v_stride : k + t * k_stride) + (int64_t)h * D;
    float val[kLaneDims];
#pragma unroll
    for (int j = 0; j < kLaneDims; ++j)
      if (lane + 32 * j < D) val[j] = rotated(in, lane + 32 * j, is_v ? none : r, cs);
    __syncwarp();  // q_out may be q: every lane has read its pairs
    if (is_q) {
#pragma unroll
      for (int j = 0; j < kLaneDims; ++j)
        if (lane + 32 * j < D) q_out[t * q_out_stride + (int64_t)h * D + lane + 32 * j] = val[j];
    } else {
      write_row<FORMAT>(val, D, place + ((int64_t)h << c.page_shift), is_v ? c.v : c.k, is_v ? c.v_step : c.k_step);
    }
  }
}

// One warp per (row, key or value head).
template <int FORMAT>
__global__ void __launch_bounds__(kThreads) read_kernel(KvPages c, KvRows rows, float* __restrict__ k_out,
                                                        int64_t k_stride, float* __restrict__ v_out, int64_t v_stride) {
  pdl_release_dependents();
  pdl_wait_primary();
  const int64_t t = blockIdx.x;
  const int64_t place = kv_place(rows, c, t);
  if (place < 0) return;
  const int lane = threadIdx.x & 31, D = c.head_dim;
  for (int u = blockIdx.y * kWarps + (threadIdx.x >> 5); u < 2 * c.heads; u += gridDim.y * kWarps) {
    const bool is_v = u >= c.heads;
    const int h = is_v ? u - c.heads : u;
    const int64_t row = place + ((int64_t)h << c.page_shift);
    const void* codes = is_v ? c.v : c.k;
    float* out = (is_v ? v_out + t * v_stride : k_out + t * k_stride) + (int64_t)h * D;
    const float step = FORMAT == BITLINEAR_KV_BF16 ? 1.0f : (is_v ? c.v_step : c.k_step)[row];
    for (int d = lane; d < D; d += 32) {
      if constexpr (FORMAT == BITLINEAR_KV_BF16) {
        out[d] = __bfloat162float(static_cast<const __nv_bfloat16*>(codes)[row * D + d]);
      } else if constexpr (FORMAT == BITLINEAR_KV_INT8) {
        out[d] = __fmul_rn((float)static_cast<const int8_t*>(codes)[row * D + d], step);
      } else {
        const uint32_t h2 = half2_of_e4m3x2(static_cast<const uint8_t*>(codes)[row * D + d]);
        out[d] = __fmul_rn(__half2float(__ushort_as_half((unsigned short)h2)), step);
      }
    }
  }
}

// One CTA per token and share of its units; shares only while the tokens
// alone leave SMs idle.
dim3 grid_for(int64_t T, int units, const DeviceInfo& dev) {
  const int64_t want = (2 * (int64_t)dev.num_sms + T - 1) / T;
  const int64_t most = (units + kWarps - 1) / kWarps;
  return dim3((unsigned)T, (unsigned)(want < most ? want : most), 1);
}

template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), dim3 grid, bool pdl, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

}  // namespace

cudaError_t launch_rope(const float* x, int64_t x_stride, int64_t T, int H, int D, const int32_t* positions,
                        const RopeArgs& rope, float* y, int64_t y_stride, bool pdl, const DeviceInfo& dev,
                        cudaStream_t stream) {
  return launch(rope_kernel, grid_for(T, H, dev), pdl, stream, x, x_stride, H, D, positions, rope, y, y_stride);
}

cudaError_t launch_kv_append(const float* q, int64_t q_stride, int q_heads, float* q_out, int64_t q_out_stride,
                             const float* k, int64_t k_stride, const float* v, int64_t v_stride, const KvRows& rows,
                             const RopeArgs& rope, const KvPages& cache, bool pdl, const DeviceInfo& dev,
                             cudaStream_t stream) {
  const auto kernel = cache.format == BITLINEAR_KV_INT8  ? append_kernel<BITLINEAR_KV_INT8>
                      : cache.format == BITLINEAR_KV_FP8 ? append_kernel<BITLINEAR_KV_FP8>
                                                         : append_kernel<BITLINEAR_KV_BF16>;
  return launch(kernel, grid_for(rows.T, q_heads + 2 * cache.heads, dev), pdl, stream, q, q_stride, q_heads, q_out,
                q_out_stride, k, k_stride, v, v_stride, rows, rope, cache);
}

cudaError_t launch_kv_read(const KvPages& cache, const KvRows& rows, float* k_out, int64_t k_stride, float* v_out,
                           int64_t v_stride, bool pdl, const DeviceInfo& dev, cudaStream_t stream) {
  const auto kernel = cache.format == BITLINEAR_KV_INT8  ? read_kernel<BITLINEAR_KV_INT8>
                      : cache.format == BITLINEAR_KV_FP8 ? read_kernel<BITLINEAR_KV_FP8>
                                                         : read_kernel<BITLINEAR_KV_BF16>;
  return launch(kernel, grid_for(rows.T, 2 * cache.heads, dev), pdl, stream, cache, rows, k_out, k_stride, v_out,
                v_stride);
}

}  // namespace bitlinear
