// sample.cu -- from the LM head's logits to tokens: probabilities, and the verification of
// drafted tokens against them ("Hesper.Models.BitNet" page, section "Performance (BitNet-3B
// on A100)": the LM head's logits end a token; several drafted ones can end in one pass).
//
// A row (of V logits, or a sequence's two rows of probabilities) is a thread-block cluster's,
// cut into runs of whole 16-byte chunks, one a CTA.
//
// softmax: p_v = 2^(c (y_v - m)) / sum, c = log2(e) / T, m the row's maximum.
//
// verify: with i the first draft that is refused, the next token is drawn from
// w = max(p_i - q_i, 0) (p_i where all drafts are taken, or where w is 0 everywhere).  Every
// weight counts as a whole number of 2^-s, s = 62 - ceil(log2 V), so that sums of V of them are exact
// in 64 bits whatever their order, and the token is the first whose running sum passes r * total.
#include "serve.cuh"

namespace bitlinear {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMostCtas = 8;  // of a cluster

__device__ __forceinline__ uint32_t smem_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void send64(uint32_t at, int rank, unsigned long long v) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(r), "l"(v) : "memory");
}
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A row's chunks: chunk i holds values 4 i - shift .. 4 i - shift + 3, so that whole chunks
// are 16-byte aligned whatever V is.
struct Row {
  int64_t V;
  int shift;       // values before the row in its first chunk
  int64_t chunks;
  __device__ __forceinline__ Row(const float* row, int64_t V_) : V(V_), shift((int)((reinterpret_cast<uintptr_t>(row) >> 2) & 3)), chunks((V_ + shift + 3) / 4) {}
};
__device__ __forceinline__ float4 load_chunk(const float* row, const Row& r, int64_t i, float none) {
  const int64_t v = 4 * i - r.shift;
  if (v >= 0 && v + 4 <= r.V) return __ldg(reinterpret_cast<const float4*>(row + v));
  float x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = v + j >= 0 && v + j < r.V ? __ldg(row + v + j) : none;
  return make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store_chunk(float* row, const Row& r, int64_t i, float4 x) {
  const int64_t v = 4 * i - r.shift;
  if (v >= 0 && v + 4 <= r.V) {
    *reinterpret_cast<float4*>(row + v) = x;
    return;
  }
  const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (v + j >= 0 && v + j < r.V) row[v + j] = y[j];
}

// A maximum and the sum of what is left under it, as one word to send.
__device__ __forceinline__ unsigned long long packed(float m, float s) {
  return (unsigned long long)__float_as_uint(m) << 32 | __float_as_uint(s);
}

// A key that orders logits as argmax does: larger first, of equal ones (-0 and +0 are) the earlier.
__device__ __forceinline__ unsigned long long order_key(float x, int64_t v) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (unsigned long long)(u & 0x80000000u ? ~u : u | 0x80000000u) << 32 | (uint32_t)~(uint32_t)v;
}

// A row's CTAs each keep their share of its values in registers: NV chunks a thread.  NV == 0: any
// number, read a second time.  Every warp sums under a maximum of its own and tells it to every CTA: one
// meeting of the cluster.
template <int NV>
__global__ void __launch_bounds__(kThreads) softmax_kernel(const float* __restrict__ y, float* __restrict__ p,
                                                           const float* __restrict__ temperature, int64_t V) {
  __shared__ unsigned long long told[kMostCtas * kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ctas = gridDim.x, rank = blockIdx.x;
  pdl_release_dependents();
  pdl_wait_primary();
  const int64_t m_row = blockIdx.y + (int64_t)gridDim.y * blockIdx.z;
  const float* in = y + m_row * V;
  float* out = p + m_row * V;
  const Row r(in, V);
  const int64_t share = (r.chunks + ctas - 1) / ctas, from = rank * share, to = min(r.chunks, from + share);
  const float T = temperature ? __ldg(temperature + m_row) : 1.0f;
  const bool greedy = !(T >= 1e-30f);
  const float c = 1.44269504f / fminf(T, 1e30f);

  constexpr int kHeld = NV ? NV : 1;
  float4 x[kHeld];
  float m = -INFINITY;
  if constexpr (NV > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t i = from + threadIdx.x + j * kThreads;
      x[j] = i < to ? load_chunk(in, r, i, -INFINITY) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      m = fmaxf(m, fmaxf(fmaxf(x[j].x, x[j].y), fmaxf(x[j].z, x[j].w)));
    }
  } else {
    for (int64_t i = from + threadIdx.x; i < to; i += kThreads) {
      const float4 v = load_chunk(in, r, i, -INFINITY);
      m = fmaxf(m, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
    }
  }
  auto each = [&](auto f) {  // f(chunk, its values)
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int64_t i = from + threadIdx.x + j * kThreads;
        if (i < to) f(i, x[j]);
      }
    } else {
      for (int64_t i = from + threadIdx.x; i < to; i += kThreads) {
        float4 v = load_chunk(in, r, i, -INFINITY);
        f(i, v);
      }
    }
  };
  unsigned long long mine;
  if (greedy) {
    mine = 0;
    each([&](int64_t i, float4& v) {
      const int64_t at = 4 * i - r.shift;
      const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (at + j >= 0 && at + j < V && e[j] > -INFINITY) mine = max(mine, order_key(e[j], at + j));
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine = max(mine, __shfl_xor_sync(kFullMask, mine, o));
  } else {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
    const float under = m == -INFINITY ? 0.0f : m;  // a row, or a warp's part, that is masked whole
    float s = 0.0f;
    each([&](int64_t, float4& v) {
      v.x = exp2_of((v.x - under) * c);
      v.y = exp2_of((v.y - under) * c);
      v.z = exp2_of((v.z - under) * c);
      v.w = exp2_of((v.w - under) * c);
      s += (v.x + v.y) + (v.z + v.w);
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFullMask, s, o);
    mine = packed(m, s);
  }
  if (ctas == 1) {
    if (lane == 0) told[warp] = mine;
    __syncthreads();
  } else {
    cluster_meet();  // all of the cluster's CTAs have begun
    if (lane < ctas) send64(smem_at(told + rank * kWarps + warp), lane, mine);
    cluster_meet();
  }
  if (greedy) {
    unsigned long long best = 0;
    for (int i = lane; i < ctas * kWarps; i += 32) best = max(best, told[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(kFullMask, best, o));
    const int64_t at = best ? (int64_t)(uint32_t)~(uint32_t)best : -1;
    each([&](int64_t i, float4& v) {
      const int64_t d = at - (4 * i - r.shift);
      v = make_float4(d == 0, d == 1, d == 2, d == 3);
      if (at < 0) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      store_chunk(out, r, i, v);
    });
    return;
  }
  float M = -INFINITY, S = 0.0f;
  for (int i = lane; i < ctas * kWarps; i += 32) M = fmaxf(M, __uint_as_float((uint32_t)(told[i] >> 32)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, o));
  const float top = M == -INFINITY ? 0.0f : M;
  for (int i = lane; i < ctas * kWarps; i += 32) {
    const float s = __uint_as_float((uint32_t)told[i]);
    S += s * exp2_of((__uint_as_float((uint32_t)(told[i] >> 32)) - top) * c);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(kFullMask, S, o);
  const float inverse = S == 0.0f ? 0.0f : 1.0f / S;
  const float f = NV > 0 ? exp2_of((m - top) * c) * inverse : inverse;
  each([&](int64_t i, float4& v) {
    if constexpr (NV == 0) {
      v.x = exp2_of((v.x - top) * c);
      v.y = exp2_of((v.y - top) * c);
      v.z = exp2_of((v.z - top) * c);
      v.w = exp2_of((v.w - top) * c);
    }
    store_chunk(out, r, i, make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
  });
}

// ---------------------------------------------------------------- verification

// A weight in units of 1 / `scale`, a power of two; what is not above 0 (NaN among it) is 0, what is above
// 2 counts as 2.
__device__ __forceinline__ unsigned long long units(float w, float scale) {
  return w > 0.0f ? __float2ull_rn(fminf(w, 2.0f) * scale) : 0ull;
}

struct VerifyArgs {
  const float *p, *q, *uniform;
  const int32_t* draft;
  int32_t *tokens, *accepted;
  int64_t V;
  int K;
  float scale;  // units of a weight of 1
};

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFullMask, x, o);
  return x;
}
__device__ __forceinline__ unsigned long long warp_upto(unsigned long long x, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long n = __shfl_up_sync(kFullMask, x, o);
    if (lane >= o) x += n;
  }
  return x;
}

__global__ void __launch_bounds__(kThreads) verify_kernel(VerifyArgs a) {
  __shared__ unsigned long long told[2][kMostCtas];
  __shared__ unsigned long long sums[2][kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ctas = gridDim.x, rank = blockIdx.x;
  pdl_release_dependents();
  pdl_wait_primary();
  const int64_t b = blockIdx.y + (int64_t)gridDim.y * blockIdx.z;
  const int K = a.K;
  const int64_t V = a.V;

  // The drafts taken: every warp asks for itself, 32 drafts at a time.
  int n = 0;
  bool refused = false;  // by the draw, and not because the drafts end
  for (int i0 = 0; i0 < K; i0 += 32) {
    const int i = i0 + lane;
    const int32_t x = i < K ? a.draft[b * K + i] : -1;
    const bool drafted = x >= 0 && x < V;
    bool take = false;
    if (drafted) {
      const float px = a.p[(b * (K + 1) + i) * V + x], qx = a.q[(b * K + i) * V + x], u = a.uniform[b * (K + 1) + i];
      take = (double)u * (double)qx < (double)px;
    }
    const uint32_t taken = __ballot_sync(kFullMask, take), drafts = __ballot_sync(kFullMask, drafted);
    const int run = taken == kFullMask ? 32 : __ffs(~taken) - 1;
    n += run;
    if (run < 32) {
      refused = (drafts >> run) & 1u;
      break;
    }
  }
  const float* p = a.p + (b * (K + 1) + n) * V;
  const float* q = refused ? a.q + (b * K + n) * V : nullptr;

  const int64_t share = (V + ctas - 1) / ctas, from = min(V, rank * share), to = min(V, from + share);
  unsigned long long total = 0, before = 0, mine = 0;
  for (int attempt = 0;; ++attempt) {
    auto weight = [&](int64_t v) {
      const float w = __ldg(p + v);
      return units(q ? __fsub_rn(w, __ldg(q + v)) : w, a.scale);
    };
    unsigned long long s = 0;
    for (int64_t v = from + threadIdx.x; v < to; v += kThreads) s += weight(v);
    s = warp_sum(s);
    if (lane == 0) sums[attempt][warp] = s;
    __syncthreads();
    mine = warp_sum(lane < kWarps ? sums[attempt][lane] : 0ull);
    if (ctas == 1) {
      total = mine;
    } else {
      if (attempt == 0) cluster_meet();  // all of the cluster's CTAs have begun
      if (threadIdx.x < ctas) send64(smem_at(told[attempt] + rank), threadIdx.x, mine);
      cluster_meet();
      const unsigned long long t = lane < ctas ? told[attempt][lane] : 0ull;
      total = warp_sum(t);
      before = warp_sum(lane < rank ? t : 0ull);
    }
    if (total != 0 || !q) break;
    q = nullptr;  // nothing is left of p - q: p itself
  }

  if (rank == 0) {
    for (int i = threadIdx.x; i <= K; i += kThreads)
      if (i != n) a.tokens[b * (K + 1) + i] = i < n ? a.draft[b * K + i] : -1;
    if (threadIdx.x == 0) {
      a.accepted[b] = n;
      if (total == 0) a.tokens[b * (K + 1) + n] = -1;
    }
  }
  // The first token whose running sum is above floor(r * total): r in [0, 1) as a 64-bit fraction.
  const float r = fminf(fmaxf(a.uniform[b * (K + 1) + K], 0.0f), 0.99999994f);
  const unsigned long long goal = __umul64hi((unsigned long long)((double)r * 18446744073709551616.0), total);
  if (total == 0 || goal < before || goal >= before + mine) return;
  // This CTA's run has it: walked through again.
  unsigned long long upto = before;
  for (int64_t v0 = from; v0 < to; v0 += kThreads) {
    const int64_t v = v0 + threadIdx.x;
    unsigned long long w = 0;
    if (v < to) {
      const float x = __ldg(p + v);
      w = units(q ? __fsub_rn(x, __ldg(q + v)) : x, a.scale);
    }
    const unsigned long long in_warp = warp_upto(w, lane);
    __syncthreads();
    if (lane == 31) sums[0][warp] = in_warp;
    __syncthreads();
    const unsigned long long of_warps = lane < kWarps ? sums[0][lane] : 0ull;
    const unsigned long long ahead = warp_sum(lane < warp ? of_warps : 0ull), all = warp_sum(of_warps);
    const unsigned long long end = upto + ahead + in_warp;
    if (w != 0 && end > goal && end - w <= goal) a.tokens[b * (K + 1) + n] = (int32_t)v;
    if (upto + all > goal) return;
    upto += all;
  }
}

template <typename... Kernel, typename... Args>
cudaError_t launch_rows(void (*kernel)(Kernel...), int64_t rows, int ctas, bool pdl, cudaStream_t stream, Args... args) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.blockDim = dim3(kThreads, 1, 1);
  if (ctas > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = (unsigned)ctas;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (pdl) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  cfg.gridDim = dim3((unsigned)ctas, (unsigned)rows, 1);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

constexpr int64_t kMostRows = 65535;  // of a launch

}  // namespace

cudaError_t launch_softmax(const float* y, float* p, const float* temperature, int64_t M, int64_t V, bool pdl,
                           const DeviceInfo&, cudaStream_t stream) {
  const int64_t chunks = (V + 6) / 4;
  int ctas = 1;
  while (ctas < kMostCtas && chunks > (int64_t)ctas * kThreads) ctas *= 2;
  const int64_t held = ((chunks + ctas - 1) / ctas + kThreads - 1) / kThreads;
  for (int64_t m = 0; m < M; m += kMostRows) {
    const int64_t rows = M - m < kMostRows ? M - m : kMostRows;
    const auto kernel = held <= 1 ? softmax_kernel<1> : held <= 2 ? softmax_kernel<2> : held <= 4 ? softmax_kernel<4> : held <= 8 ? softmax_kernel<8> : softmax_kernel<0>;
    const cudaError_t err = launch_rows(kernel, rows, ctas, pdl, stream, y + m * V, p + m * V, temperature ? temperature + m : nullptr, V);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

cudaError_t launch_verify(const float* p, const float* q, const int32_t* draft, const float* uniform, int64_t B, int K,
                          int64_t V, int32_t* tokens, int32_t* accepted, bool pdl, const DeviceInfo&, cudaStream_t stream) {
  int ctas = 1;
  while (ctas < kMostCtas && V > (int64_t)ctas * 2 * kThreads) ctas *= 2;
  int bits = 62;
  while (((int64_t)1 << (62 - bits)) < V) --bits;
  const float scale = (float)((int64_t)1 << bits);
  for (int64_t b = 0; b < B; b += kMostRows) {
    const int64_t rows = B - b < kMostRows ? B - b : kMostRows;
    const VerifyArgs a = {p + b * (K + 1) * V, q + b * K * V, uniform + b * (K + 1), draft + b * K, tokens + b * (K + 1), accepted + b, V, K, scale};
    const cudaError_t err = launch_rows(verify_kernel, rows, ctas, pdl, stream, a);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

}  // namespace bitlinear
