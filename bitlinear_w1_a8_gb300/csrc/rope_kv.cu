// rope_kv.cu -- rotary positions and the paged key-value cache: rows rotated,
// quantised and written where their page is, and read back.
//
// Rotation ("Hesper.Models.BitNet" page, section "Configuration": ropeBase):
// pair i of a head turns by the angle positions[t] * freq[i], taken in quarter
// turns in fp64, positions * (freq * 2 / pi), so its whole turns drop out without
// loss and a far position keeps its fraction of a turn to 2^-53 of the whole
// angle.  Sine and cosine of what is left (|a| <= pi / 4) are their Taylor series, the
// leading terms in fp64 and the tail, whose fp32 rounding is below 2^-38 of the
// result, in fp32 (the fp64 pipe is narrow: ~15 fp64 operations a pair), rounded
// once to fp32.  The rotation itself is two fp32 products and one sum, unfused, so
// it can be repeated bit for bit.
//
// Quantisation follows activation_quant, a row being one (token, head):
//   int8: code = clamp(rne(x * s), -128, 127), s = 127 * (1 / a), a = max(max|x|, 1e-5)
//   e4m3: code = e4m3(x * s), s = 448 * (1 / a), round to nearest even, saturating
// with step = a / 127 or a / 448, the fp32 value of one unit; bf16 rounds.
//
// Layout: four lanes hold a row, lane j its 16-byte chunks j, j + 4, ...: a warp
// takes 8 rows, every lane has a chunk in every load whatever the head size (80
// dims fill 20 of 32 lanes one row a warp), all of a row's loads are in flight
// together, and its maximum takes two shuffles.  A CTA takes one token (or, while
// the tokens alone leave SMs idle, a share of its heads), so a token's sines and
// cosines are made once, behind the loads of its first rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kv.cuh"

namespace bitlinear {
namespace {

constexpr int kMaxHead = 256;     // head_dim limit
constexpr int kMaxThreads = 512;
constexpr int kMinThreads = 64;
constexpr int kRowLanes = 4;      // lanes of a row
constexpr int kWarpRows = 32 / kRowLanes;

__device__ __forceinline__ void sin_cos_quarter(double q, float* sine, float* cosine) {
  const double whole = rint(q);
  const double a = (q - whole) * 1.57079632679489661923;  // |a| <= pi / 4
  const double a2 = a * a;
  const float u = (float)a2;
  // sin a = a - a^3/3! + a^5/5! - ..., cos a = 1 - a^2/2! + a^4/4! - ..., from a^7 and a^8 on in fp32
  const float ts = fmaf(u, fmaf(u, fmaf(u, 1.0f / 6227020800.0f, -1.0f / 39916800.0f), 1.0f / 362880.0f), -1.0f / 5040.0f);
  const float tc = fmaf(u, fmaf(u, 1.0f / 479001600.0f, -1.0f / 3628800.0f), 1.0f / 40320.0f);
  const double s = fma(a * a2, fma(a2, fma(a2, (double)ts, 1.0 / 120.0), -1.0 / 6.0), a);
  const double c = fma(a2, fma(a2, fma(a2, fma(a2, (double)tc, -1.0 / 720.0), 1.0 / 24.0), -0.5), 1.0);
  const int n = (int)(long long)whole & 3;  // quarter turns past whole turns
  const float fs = (float)s, fc = (float)c;
  const float x = n & 1 ? fs : fc, y = n & 1 ? fc : fs;
  *cosine = n == 1 || n == 2 ? -x : x;
  *sine = n >= 2 ? -y : y;
}

// cos and sin of every pair of one position, into shared memory.
__device__ __forceinline__ void fill_angles(const RopeArgs& r, int32_t pos, float2* cs) {
  for (int i = threadIdx.x; i < r.rot_dim / 2; i += blockDim.x) {
    float s, c;
    sin_cos_quarter((double)pos * (r.freq[i] * 0.63661977236758134308), &s, &c);
    cs[i] = make_float2(__fmul_rn(c, r.amplitude), __fmul_rn(s, r.amplitude));
  }
}

// The lane's chunks of a row of D floats.
template <int NC>
__device__ __forceinline__ void load_row(const float* row, int D, int j, float4 (&v)[NC]) {
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int d = 4 * (j + kRowLanes * i);
    if (d < D) v[i] = *reinterpret_cast<const float4*>(row + d);
  }
}

__device__ __forceinline__ float turn_first(float own, float other, float2 a) {
  return __fsub_rn(__fmul_rn(own, a.x), __fmul_rn(other, a.y));
}
__device__ __forceinline__ float turn_second(float own, float other, float2 a) {
  return __fadd_rn(__fmul_rn(own, a.x), __fmul_rn(other, a.y));
}

// Rotates the lane's chunks (v, of the row at `row`) in registers.
template <int NC>
__device__ __forceinline__ void rotate_row(const float* row, int D, int j, const RopeArgs& r, const float2* cs,
                                           float4 (&v)[NC]) {
  const int n = r.rot_dim / 2;
  if (r.layout == BITLINEAR_ROPE_INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int d = 4 * (j + kRowLanes * i);
      if (d < r.rot_dim) {
        const float2 a = cs[d / 2];
        const float x = turn_first(v[i].x, v[i].y, a), y = turn_second(v[i].y, v[i].x, a);
        v[i].x = x;
        v[i].y = y;
      }
      if (d + 2 < r.rot_dim) {
        const float2 a = cs[d / 2 + 1];
        const float z = turn_first(v[i].z, v[i].w, a), w = turn_second(v[i].w, v[i].z, a);
        v[i].z = z;
        v[i].w = w;
      }
    }
    return;
  }
  // Halves: the partners (loaded a moment ago by this row's lanes) come from the row again.
  if (n % 4 == 0) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int d = 4 * (j + kRowLanes * i);
      if (d >= r.rot_dim) continue;
      const bool second = d >= n;
      const float4 o = *reinterpret_cast<const float4*>(row + (second ? d - n : d + n));
      const float4* a4 = reinterpret_cast<const float4*>(cs + (second ? d - n : d));
      const float4 a = a4[0], b = a4[1];
      if (second) {
        v[i] = make_float4(turn_second(v[i].x, o.x, make_float2(a.x, a.y)), turn_second(v[i].y, o.y, make_float2(a.z, a.w)),
                           turn_second(v[i].z, o.z, make_float2(b.x, b.y)), turn_second(v[i].w, o.w, make_float2(b.z, b.w)));
      } else {
        v[i] = make_float4(turn_first(v[i].x, o.x, make_float2(a.x, a.y)), turn_first(v[i].y, o.y, make_float2(a.z, a.w)),
                           turn_first(v[i].z, o.z, make_float2(b.x, b.y)), turn_first(v[i].w, o.w, make_float2(b.z, b.w)));
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int d0 = 4 * (j + kRowLanes * i);
    float* e = reinterpret_cast<float*>(&v[i]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int d = d0 + k;
      if (d >= r.rot_dim) continue;
      e[k] = d < n ? turn_first(e[k], row[d + n], cs[d]) : turn_second(e[k], row[d - n], cs[d - n]);
    }
  }
}

template <int NC>
__device__ __forceinline__ void store_row(float* row, int D, int j, const float4 (&v)[NC]) {
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int d = 4 * (j + kRowLanes * i);
    if (d < D) *reinterpret_cast<float4*>(row + d) = v[i];
  }
}

// blockIdx.x is the token, blockIdx.y shares its heads out.
template <int NC>
__global__ void __launch_bounds__(kMaxThreads) rope_kernel(const float* x, int64_t x_stride, int H, int D,
                                                           const int32_t* __restrict__ positions, RopeArgs r, float* y,
                                                           int64_t y_stride) {
  __shared__ __align__(16) float2 cs[kMaxHead / 2];
  pdl_release_dependents();
  pdl_wait_primary();
  const int64_t t = blockIdx.x;
  const int j = threadIdx.x % kRowLanes, step = gridDim.y * (blockDim.x / kRowLanes);
  int h = blockIdx.y * (blockDim.x / kRowLanes) + threadIdx.x / kRowLanes;
  x += t * x_stride;
  y += t * y_stride;
  float4 v[NC];
  if (h < H) load_row(x + (int64_t)h * D, D, j, v);
  fill_angles(r, positions[t], cs);
  __syncthreads();
  // every lane of a warp makes every turn: y may be x, and a row's partners are read before it is written
  for (int at = h - (int)(threadIdx.x & 31) / kRowLanes; at < H; at += step, h += step) {
    if (h < H) rotate_row(x + (int64_t)h * D, D, j, r, cs, v);
    __syncwarp();
    if (h < H) store_row(y + (int64_t)h * D, D, j, v);
    if (h + step < H) load_row(x + (int64_t)(h + step) * D, D, j, v);
  }
}

// Quantises a row held by four lanes and writes codes and step.
template <int FORMAT, int NC>
__device__ __forceinline__ void write_row(const float4 (&v)[NC], int D, int j, int64_t row, void* codes, float* steps) {
  if constexpr (FORMAT == BITLINEAR_KV_BF16) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int d = 4 * (j + kRowLanes * i);
      if (d >= D) continue;
      const __nv_bfloat162 a = __floats2bfloat162_rn(v[i].x, v[i].y), b = __floats2bfloat162_rn(v[i].z, v[i].w);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(codes) + row * D + d) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
    return;
  }
  constexpr float kTop = FORMAT == BITLINEAR_KV_INT8 ? 127.0f : 448.0f;
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (4 * (j + kRowLanes * i) < D)
      a = fmaxf(fmaxf(a, fmaxf(fabsf(v[i].x), fabsf(v[i].y))), fmaxf(fabsf(v[i].z), fabsf(v[i].w)));
  a = fmaxf(a, __shfl_xor_sync(kFullMask, a, 1));
  a = fmaxf(a, __shfl_xor_sync(kFullMask, a, 2));
  a = fmaxf(a, 1e-5f);
  if (row < 0) return;  // a lane without a row: only its part in the shuffles
  const float s = __fmul_rn(__frcp_rn(a), kTop);
  uint8_t* out = static_cast<uint8_t*>(codes) + row * D;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int d = 4 * (j + kRowLanes * i);
    if (d >= D) continue;
    const float e[4] = {__fmul_rn(v[i].x, s), __fmul_rn(v[i].y, s), __fmul_rn(v[i].z, s), __fmul_rn(v[i].w, s)};
    uint32_t w;
    if constexpr (FORMAT == BITLINEAR_KV_INT8) {
      w = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) w |= (uint32_t)(uint8_t)(int8_t)max(-128, min(127, __float2int_rn(e[k]))) << (8 * k);
    } else {
      w = e4m3x2(e[1], e[0]) | e4m3x2(e[3], e[2]) << 16;
    }
    *reinterpret_cast<uint32_t*>(out + d) = w;
  }
  if (j == 0) steps[row] = __fdiv_rn(a, kTop);
}

// Units of a token: its q heads (rotated into q_out), its k heads (rotated and
// written) and its v heads (written).
struct Append {
  const float* q;
  const float* k;
  const float* v;
  float* q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  int q_heads;
};

template <int FORMAT, int NC>
__global__ void __launch_bounds__(kMaxThreads) append_kernel(Append a, KvRows rows, RopeArgs r, KvPages c) {
  __shared__ __align__(16) float2 cs[kMaxHead / 2];
  pdl_release_dependents();
  pdl_wait_primary();
  const int64_t t = blockIdx.x;
  const int D = c.head_dim, units = a.q_heads + 2 * c.heads;
  const int j = threadIdx.x % kRowLanes, step = gridDim.y * (blockDim.x / kRowLanes);
  int u = blockIdx.y * (blockDim.x / kRowLanes) + threadIdx.x / kRowLanes;
  auto input = [&](int unit) {
    if (unit < a.q_heads) return a.q + t * a.q_stride + (int64_t)unit * D;
    unit -= a.q_heads;
    if (unit < c.heads) return a.k + t * a.k_stride + (int64_t)unit * D;
    return a.v + t * a.v_stride + (int64_t)(unit - c.heads) * D;
  };
  float4 v[NC];
  if (u < units) load_row(input(u), D, j, v);
  const int64_t place = kv_place(rows, c, t);
  if (r.freq) fill_angles(r, rows.positions[t], cs);
  __syncthreads();
  if (place < 0) return;
  // every lane of a warp makes every turn: shuffles, and q_out may be q
  for (int at = u - (int)(threadIdx.x & 31) / kRowLanes; at < units; at += step, u += step) {
    const bool have = u < units, is_q = u < a.q_heads, is_v = u >= a.q_heads + c.heads;
    if (have && !is_v && r.freq) rotate_row(input(u), D, j, r, cs, v);
    __syncwarp();
    const int h = u - a.q_heads - (is_v ? c.heads : 0);
    const int64_t row = have && !is_q ? place + ((int64_t)h << c.page_shift) : -1;
    if (FORMAT != BITLINEAR_KV_BF16 || row >= 0)
      write_row<FORMAT>(v, D, j, row, is_v ? c.v : c.k, is_v ? c.v_step : c.k_step);
    if (have && is_q) store_row(a.q_out + t * a.q_out_stride + (int64_t)u * D, D, j, v);
    if (u + step < units) load_row(input(u + step), D, j, v);
  }
}

template <int FORMAT, int NC>
__global__ void __launch_bounds__(kMaxThreads) read_kernel(KvPages c, KvRows rows, float* __restrict__ k_out,
                                                           int64_t k_stride, float* __restrict__ v_out,
                                                           int64_t v_stride) {
  pdl_release_dependents();
  pdl_wait_primary();
  const int64_t t = blockIdx.x;
  const int64_t place = kv_place(rows, c, t);
  if (place < 0) return;
  const int D = c.head_dim, j = threadIdx.x % kRowLanes;
  for (int u = blockIdx.y * (blockDim.x / kRowLanes) + threadIdx.x / kRowLanes; u < 2 * c.heads;
       u += gridDim.y * (blockDim.x / kRowLanes)) {
    const bool is_v = u >= c.heads;
    const int h = is_v ? u - c.heads : u;
    const int64_t row = place + ((int64_t)h << c.page_shift);
    const void* codes = is_v ? c.v : c.k;
    float4 v[NC];
    if constexpr (FORMAT == BITLINEAR_KV_BF16) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int d = 4 * (j + kRowLanes * i);
        if (d >= D) continue;
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(codes) + row * D + d);
        v[i] = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                           __uint_as_float(w.y & 0xffff0000u));
      }
    } else {
      uint32_t w[NC];
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int d = 4 * (j + kRowLanes * i);
        if (d < D) w[i] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(codes) + row * D + d);
      }
      const float step = (is_v ? c.v_step : c.k_step)[row];
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float e[4];
        if constexpr (FORMAT == BITLINEAR_KV_INT8) {
#pragma unroll
          for (int k = 0; k < 4; ++k) e[k] = (float)(int8_t)(w[i] >> (8 * k));
        } else {
          const uint32_t lo = half2_of_e4m3x2((uint16_t)w[i]), hi = half2_of_e4m3x2((uint16_t)(w[i] >> 16));
          const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo)), b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
          e[0] = a.x; e[1] = a.y; e[2] = b.x; e[3] = b.y;
        }
        v[i] = make_float4(__fmul_rn(e[0], step), __fmul_rn(e[1], step), __fmul_rn(e[2], step), __fmul_rn(e[3], step));
      }
    }
    store_row((is_v ? v_out + t * v_stride : k_out + t * k_stride) + (int64_t)h * D, D, j, v);
  }
}

// One CTA per token while tokens fill the GPU (two CTAs an SM), else a token's
// units shared out; a CTA's threads take its units in one turn up to kMaxThreads.
struct Launch {
  dim3 grid;
  int threads;
};
Launch launch_for(int64_t T, int units, const DeviceInfo& dev) {
  int64_t shares = (2 * (int64_t)dev.num_sms + T - 1) / T;
  const int64_t most = ((int64_t)units * kRowLanes + kMinThreads - 1) / kMinThreads;
  if (shares > most) shares = most;
  const int64_t per = (units + shares - 1) / shares;
  int64_t threads = (per + kWarpRows - 1) / kWarpRows * 32;
  threads = threads < kMinThreads ? kMinThreads : threads > kMaxThreads ? kMaxThreads : threads;
  return Launch{dim3((unsigned)T, (unsigned)shares, 1), (int)threads};
}

template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), const Launch& l, bool pdl, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = l.grid;
  cfg.blockDim = dim3((unsigned)l.threads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// f(NC) with NC the smallest instantiated number of chunks a lane that holds D dims.
template <typename F>
cudaError_t with_chunks(int D, F f) {
  if (D <= 64) return f(std::integral_constant<int, 4>());
  if (D <= 80) return f(std::integral_constant<int, 5>());
  if (D <= 128) return f(std::integral_constant<int, 8>());
  return f(std::integral_constant<int, 16>());
}
template <typename F>
cudaError_t with_format(int format, F f) {
  if (format == BITLINEAR_KV_INT8) return f(std::integral_constant<int, BITLINEAR_KV_INT8>());
  if (format == BITLINEAR_KV_FP8) return f(std::integral_constant<int, BITLINEAR_KV_FP8>());
  return f(std::integral_constant<int, BITLINEAR_KV_BF16>());
}

}  // namespace

cudaError_t launch_rope(const float* x, int64_t x_stride, int64_t T, int H, int D, const int32_t* positions,
                        const RopeArgs& rope, float* y, int64_t y_stride, bool pdl, const DeviceInfo& dev,
                        cudaStream_t stream) {
  return with_chunks(D, [&](auto nc) {
    return launch(rope_kernel<decltype(nc)::value>, launch_for(T, H, dev), pdl, stream, x, x_stride, H, D, positions,
                  rope, y, y_stride);
  });
}

cudaError_t launch_kv_append(const float* q, int64_t q_stride, int q_heads, float* q_out, int64_t q_out_stride,
                             const float* k, int64_t k_stride, const float* v, int64_t v_stride, const KvRows& rows,
                             const RopeArgs& rope, const KvPages& cache, bool pdl, const DeviceInfo& dev,
                             cudaStream_t stream) {
  const Append a = {q, k, v, q_out, q_stride, k_stride, v_stride, q_out_stride, q_heads};
  return with_format(cache.format, [&](auto fmt) {
    return with_chunks(cache.head_dim, [&](auto nc) {
      return launch(append_kernel<decltype(fmt)::value, decltype(nc)::value>,
                    launch_for(rows.T, q_heads + 2 * cache.heads, dev), pdl, stream, a, rows, rope, cache);
    });
  });
}

cudaError_t launch_kv_read(const KvPages& cache, const KvRows& rows, float* k_out, int64_t k_stride, float* v_out,
                           int64_t v_stride, bool pdl, const DeviceInfo& dev, cudaStream_t stream) {
  return with_format(cache.format, [&](auto fmt) {
    return with_chunks(cache.head_dim, [&](auto nc) {
      return launch(read_kernel<decltype(fmt)::value, decltype(nc)::value>, launch_for(rows.T, 2 * cache.heads, dev),
                    pdl, stream, cache, rows, k_out, k_stride, v_out, v_stride);
    });
  });
}

}  // namespace bitlinear
