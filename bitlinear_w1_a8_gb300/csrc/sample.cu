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
//
// Measured.  softmax: 320 rows of 50000 25.7 us, 128 MB, 5.0 TB/s (a copy's 19.1 us): rows come in four rounds of clusters,
// each of which reads, meets once and writes (28.7 us while every warp told every CTA its sums: each then waits for what it
// published); one row 3.6 us, latency.  Rows streamed through rings in shared memory under
// resident CTAs took 43.3 where this took 33.9.  verify: 64 sequences of 4 drafts over 50000 tokens 11.2 us (3.8 us of bytes): the
// drafts' probabilities, then the two rows they point to, then the cluster's meeting, one after the other; one sequence 5.6.
#include <type_traits>

#include "serve.cuh"

namespace bitlinear {
namespace {

constexpr int kMostCtas = 8;  // of a cluster

__device__ __forceinline__ uint32_t smem_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void send64(uint32_t at, int rank, unsigned long long v) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(r), "l"(v) : "memory");
}
__device__ __forceinline__ void cluster_begun() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }  // publishes nothing
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A row's chunks: chunk i holds values 4 i - shift .. 4 i - shift + 3, so that whole chunks (lo .. hi - 1) are 16-byte
// aligned whatever V is.
struct Row {
  int64_t V;
  int shift;  // values before the row in its first chunk
  int chunks, lo, hi;
  __device__ __forceinline__ Row(const float* row, int64_t V_)
      : V(V_), shift((int)((reinterpret_cast<uintptr_t>(row) >> 2) & 3)), chunks((int)((V_ + shift + 3) / 4)), lo(shift > 0), hi((int)((V_ + shift) / 4)) {}
  __device__ __forceinline__ bool whole(int i) const { return i >= lo && i < hi; }
};
// The output may be the logits' own buffer, so logits are read by coherent loads.  ONCE: they are not read again, and come
// by relaxed loads (320 rows of 50000 out of DRAM 27.7 us, 28.4 by plain ones that leave L1 alone).
template <bool ONCE>
__device__ __forceinline__ float4 load4(const float4* p) {
  if constexpr (ONCE) {
    float4 x;
    asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "l"(p) : "memory");
    return x;
  } else {
    return *p;
  }
}
template <bool ONCE>
__device__ __forceinline__ float4 load_chunk(const float* row, const Row& r, int i, float none) {
  if (r.whole(i)) return load4<ONCE>(reinterpret_cast<const float4*>(row - r.shift) + i);
  const int64_t v = 4 * (int64_t)i - r.shift;
  float x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = v + j >= 0 && v + j < r.V ? row[v + j] : none;
  return make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store_chunk(float* row, const Row& r, int i, float4 x) {
  if (r.whole(i)) {
    reinterpret_cast<float4*>(row - r.shift)[i] = x;
    return;
  }
  const int64_t v = 4 * (int64_t)i - r.shift;
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

constexpr int kRowThreads = 256;  // of a CTA

// The cluster's exchange: a CTA's words, one a warp, are joined to one, which it tells every CTA: one warp publishes,
// the others have nothing to.  `told` has room for WARPS + kMostCtas words; the CTAs' begin at WARPS.
template <int WARPS, typename Join>
__device__ __forceinline__ void tell(unsigned long long* told, unsigned long long mine, int ctas, int rank, int lane, int warp, Join join) {
  if (lane == 0) told[warp] = mine;
  __syncthreads();
  if (warp == 0) {
    const unsigned long long all = join(told, WARPS);
    if (ctas == 1) {
      if (lane == 0) told[WARPS] = all;
    } else if (lane < ctas) {
      send64(smem_at(told + WARPS + rank), lane, all);
    }
  }
  if (ctas == 1) {
    __syncthreads();
    return;
  }
  __syncwarp();
  if (warp == 0)
    cluster_arrive();
  else
    cluster_begun();
  cluster_wait();
}

// A row's probabilities from what its threads hold: `each` calls its argument with (chunk, its values) for
// every chunk of the thread's.  m: the thread's largest logit.  AGAIN: `each` reads the logits anew.
template <int WARPS, bool AGAIN, bool ALIGNED, typename Each>
__device__ __forceinline__ void finish_row(const Row& r, float* out, float T, float m, unsigned long long* told, int ctas, int rank,
                                           int lane, int warp, Each each) {
  const bool greedy = !(T >= 1e-30f);
  const float c = 1.44269504f / fminf(T, 1e30f);
  if (greedy) {
    unsigned long long mine = 0;
    each([&](int i, float4& v) {
      const int64_t at = 4 * (int64_t)i - r.shift;
      const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (at + j >= 0 && at + j < r.V && e[j] > -INFINITY) mine = max(mine, order_key(e[j], at + j));
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine = max(mine, __shfl_xor_sync(kFullMask, mine, o));
    const auto largest = [&](const unsigned long long* t, int n) {
      unsigned long long best = lane < n ? t[lane] : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(kFullMask, best, o));
      return best;
    };
    tell<WARPS>(told, mine, ctas, rank, lane, warp, largest);
    const unsigned long long best = largest(told + WARPS, ctas);
    const int64_t at = best ? (int64_t)(uint32_t)~(uint32_t)best : -1;
    each([&](int i, float4&) {
      const int64_t d = at < 0 ? -1 : at - (4 * (int64_t)i - r.shift);
      store_chunk(out, r, i, make_float4(d == 0, d == 1, d == 2, d == 3));
    });
    return;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
  const float under = m == -INFINITY ? 0.0f : m;  // a row, or a warp's part, that is masked whole
  float s = 0.0f;
  each([&](int, float4& v) {
    v.x = exp2_of((v.x - under) * c);
    v.y = exp2_of((v.y - under) * c);
    v.z = exp2_of((v.z - under) * c);
    v.w = exp2_of((v.w - under) * c);
    s += (v.x + v.y) + (v.z + v.w);
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFullMask, s, o);
  const auto joined = [&](const unsigned long long* t, int n) {
    const unsigned long long word = lane < n ? t[lane] : packed(-INFINITY, 0.0f);
    const float of = __uint_as_float((uint32_t)(word >> 32));
    float most = of;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(kFullMask, most, o));
    float sum = __uint_as_float((uint32_t)word) * exp2_of((of - (most == -INFINITY ? 0.0f : most)) * c);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
    return packed(most, sum);
  };
  tell<WARPS>(told, packed(m, s), ctas, rank, lane, warp, joined);
  const unsigned long long row = joined(told + WARPS, ctas);
  const float M = __uint_as_float((uint32_t)(row >> 32)), S = __uint_as_float((uint32_t)row), top = M == -INFINITY ? 0.0f : M;
  const float inverse = S == 0.0f ? 0.0f : 1.0f / S;
  const float f = AGAIN ? inverse : exp2_of((m - top) * c) * inverse;
  each([&](int i, float4& v) {
    if constexpr (AGAIN) {
      v.x = exp2_of((v.x - top) * c);
      v.y = exp2_of((v.y - top) * c);
      v.z = exp2_of((v.z - top) * c);
      v.w = exp2_of((v.w - top) * c);
    }
    const float4 w = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
    if constexpr (ALIGNED)
      reinterpret_cast<float4*>(out)[i] = w;
    else
      store_chunk(out, r, i, w);
  });
}

__device__ __forceinline__ float largest_of(float m, const float4& v) { return fmaxf(m, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w))); }

// CTAs an SM, as many as the registers of NV chunks allow; said, because the compiler stops short of it (seven chunks: 54
// registers where 48 do, in place 21.7 us for 19.6 on 320 rows of 50000).
__host__ __device__ constexpr int softmax_ctas(int nv, bool aligned) { return nv == 7 ? (aligned ? 5 : 4) : nv == 4 ? 6 : 8; }

// p may be y: a thread has read a chunk for the last time when it writes it.
// A row a cluster.  A CTA keeps its share of the row in registers, NV chunks a thread; NV == 0: any number of
// them, read a second and a third time.  ALIGNED: V is a multiple of four, so that every chunk is whole (320 rows of
// 50000 25.7 us; of 50001 26.8).  Every warp sums under a maximum of its own, so
// the cluster meets once.
template <int THREADS, int NV, bool ALIGNED>
__global__ void __launch_bounds__(THREADS, softmax_ctas(NV, ALIGNED)) softmax_kernel(const float* y, float* p, const float* __restrict__ temperature, int64_t V) {
  constexpr int kWarps = THREADS / 32;
  __shared__ unsigned long long told[kWarps + kMostCtas];
  const int ctas = gridDim.x, rank = blockIdx.x;
  pdl_release_dependents();
  if (ctas > 1) cluster_begun();  // waited for before the first word goes to another CTA
  pdl_wait_primary();
  const int64_t m_row = blockIdx.y;
  const float* in = y + m_row * V;
  const Row r(in, V);
  const int share = (int)((uint32_t)(r.chunks + ctas - 1) / (uint32_t)ctas), from = min(r.chunks, rank * share), to = min(r.chunks, from + share);
  float4 x[NV ? NV : 1];
  float m = -INFINITY;
  if constexpr (NV > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = from + (int)threadIdx.x + j * THREADS;
      x[j] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if constexpr (ALIGNED) {
        if (i < to) x[j] = load4<true>(reinterpret_cast<const float4*>(in) + i);
      } else {
        if (i < to) x[j] = load_chunk<true>(in, r, i, -INFINITY);
      }
    }
  }
  const float T = temperature ? __ldg(temperature + m_row) : 1.0f;
  if constexpr (NV > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) m = largest_of(m, x[j]);
  } else {
    for (int i = from + (int)threadIdx.x; i < to; i += THREADS) m = largest_of(m, load_chunk<false>(in, r, i, -INFINITY));
  }
  if (ctas > 1) cluster_wait();
  finish_row<kWarps, NV == 0, ALIGNED>(r, p + m_row * V, T, m, told, ctas, rank, threadIdx.x & 31, threadIdx.x >> 5, [&](auto f) {
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i = from + (int)threadIdx.x + j * THREADS;
        if (i < to) f(i, x[j]);
      }
    } else {
      for (int i = from + (int)threadIdx.x; i < to; i += THREADS) {
        float4 v = load_chunk<false>(in, r, i, -INFINITY);
        f(i, v);
      }
    }
  });
}

// ---------------------------------------------------------------- verification

// A weight in units of 2^-places (31 to 62), to the nearest, ties to even; what is not above 0 (NaN among it) is 0, what is
// above 2 counts as 2.  By shifts: the conversion to 64 bits runs on the fp64 pipe, which it kept busy for half of the
// kernel's time (64 sequences of 50000 tokens 14.6 us with it, 11.6 without; 11.2 by now).
__device__ __forceinline__ unsigned long long units(float w, int places) {
  const uint32_t u = __float_as_uint(fminf(w, 2.0f)), m = (u & 0x7fffffu) | 0x800000u;
  const int shift = (int)(u >> 23) - 150 + places;  // the weight is m 2^(its exponent's field - 150), below 2^-126 nothing is left
  const int down = min(31, max(1, -shift));
  const uint32_t rounded = (m + (1u << (down - 1)) - 1u + ((m >> down) & 1u)) >> down;
  const unsigned long long units = shift >= 0 ? (unsigned long long)m << shift : rounded;
  return w > 0.0f ? units : 0ull;
}

struct VerifyArgs {
  const float *p, *q, *uniform;
  const int32_t* draft;
  int32_t *tokens, *accepted;
  int64_t V;
  int K;
  int places;  // a weight counts in units of 2^-places
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

// Four values from v on, of a row of V; those past its end are 0.
template <bool ALIGNED>
__device__ __forceinline__ float4 load_four(const float* row, int64_t v, int64_t V) {
  if constexpr (ALIGNED) {
    return __ldg(reinterpret_cast<const float4*>(row + v));
  } else {
    float x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = v + j < V ? __ldg(row + v + j) : 0.0f;
    return make_float4(x[0], x[1], x[2], x[3]);
  }
}

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;

// A warp takes a run of the row in turns of four values a lane; the weights of NV turns stay in registers, and where
// there are more of them (NV == 0) the run that has the token is walked through again.  Sums are told warp by
// warp: the cluster meets once, and every warp then knows whether the token is in its run.  ALIGNED: rows start on
// 16 bytes.  CTAS: as many fit an SM.
template <int NV, bool ALIGNED, int CTAS>
__global__ void __launch_bounds__(kVerifyThreads, CTAS) verify_kernel(VerifyArgs a) {
  __shared__ unsigned long long told[2][kMostCtas * kVerifyWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ctas = gridDim.x, rank = blockIdx.x;
  pdl_release_dependents();
  if (ctas > 1) cluster_begun();  // waited for before the first word goes to another CTA
  pdl_wait_primary();
  const int64_t b = blockIdx.y;
  const int K = a.K;
  const int64_t V = a.V;

  // The drafts taken: every warp asks for itself, 32 drafts at a time.
  int n = 0;
  bool refused = false;  // by the draw, and not because the drafts end
  const float last = __ldg(a.uniform + b * (K + 1) + K);
  for (int i0 = 0; i0 < K; i0 += 32) {
    const int i = i0 + lane;
    const float u = i < K ? __ldg(a.uniform + b * (K + 1) + i) : 0.0f;
    const int32_t x = i < K ? __ldg(a.draft + b * K + i) : -1;
    const bool drafted = x >= 0 && x < V;
    bool take = false;
    if (drafted) {
      const float px = __ldg(a.p + (b * (K + 1) + i) * V + x), qx = __ldg(a.q + (b * K + i) * V + x);
      // exactly: the rounded product, and what the rounding left where that decides; in fp64 (a slow pipe) where it may not be whole
      const float h = __fmul_rn(u, qx);
      take = fabsf(h) >= 7.8886091e-31f && fabsf(h) < INFINITY ? h < px || (h == px && __fmaf_rn(u, qx, -h) < 0.0f) : (double)u * (double)qx < (double)px;
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

  const int fours = (int)((V + 3) / 4), share = (fours + ctas * kVerifyWarps - 1) / (ctas * kVerifyWarps);
  const int from = min(fours, (rank * kVerifyWarps + warp) * share), to = min(fours, from + share);
  auto weights = [&](int i) {
    float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i < to) {
      w = load_four<ALIGNED>(p, 4 * (int64_t)i, V);
      if (q) {
        const float4 d = load_four<ALIGNED>(q, 4 * (int64_t)i, V);
        w = make_float4(__fsub_rn(w.x, d.x), __fsub_rn(w.y, d.y), __fsub_rn(w.z, d.z), __fsub_rn(w.w, d.w));
      }
    }
    return w;
  };
  auto sum_of = [&](const float4& w) { return units(w.x, a.places) + units(w.y, a.places) + units(w.z, a.places) + units(w.w, a.places); };
  constexpr int kHeld = NV ? NV : 1;
  float4 held[kHeld];
  unsigned long long total = 0, before = 0, mine = 0;
  for (int attempt = 0;; ++attempt) {
    mine = 0;
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) held[j] = weights(from + lane + 32 * j);
#pragma unroll
      for (int j = 0; j < NV; ++j) mine += sum_of(held[j]);
    } else {
      for (int i = from + lane; i < to; i += 32) mine += sum_of(weights(i));
    }
    mine = warp_sum(mine);
    const int here = rank * kVerifyWarps + warp;
    if (ctas == 1) {
      if (lane == 0) told[attempt][warp] = mine;
      __syncthreads();
    } else {
      if (attempt == 0) cluster_wait();  // all of the cluster's CTAs have begun
      if (lane < ctas) send64(smem_at(told[attempt] + here), lane, mine);
      cluster_arrive();
      cluster_wait();
    }
    unsigned long long all = 0, ahead = 0;
    for (int i = lane; i < ctas * kVerifyWarps; i += 32) {
      const unsigned long long t = told[attempt][i];
      all += t;
      ahead += i < here ? t : 0ull;
    }
    total = warp_sum(all);
    before = warp_sum(ahead);
    if (total != 0 || !q) break;
    q = nullptr;  // nothing is left of p - q: p itself
  }

  if (rank == 0) {
    for (int i = threadIdx.x; i <= K; i += kVerifyThreads)
      if (i != n) a.tokens[b * (K + 1) + i] = i < n ? a.draft[b * K + i] : -1;
    if (threadIdx.x == 0) {
      a.accepted[b] = n;
      if (total == 0) a.tokens[b * (K + 1) + n] = -1;
    }
  }
  // The first token whose running sum is above floor(r * total): r in [0, 1) as a 64-bit fraction.
  const float r = fminf(fmaxf(last, 0.0f), 0.99999994f);
  const uint32_t r_bits = __float_as_uint(r), r_m = (r_bits & 0x7fffffu) | 0x800000u;
  const int r_shift = (int)(r_bits >> 23) - 150 + 64;  // below 40; from -23 on nothing is left
  const unsigned long long fraction = r_shift >= 0 ? (unsigned long long)r_m << r_shift : r_m >> min(31, -r_shift);
  const unsigned long long goal = __umul64hi(fraction, total);
  if (total == 0 || goal < before || goal >= before + mine) return;
  // This warp's run has it.
  auto look_at = [&](const float4& w, int i) {  // the i-th four of the row, a lane each
    unsigned long long s = sum_of(w), upto = before + warp_upto(s, lane);
    before = __shfl_sync(kFullMask, upto, 31);
    upto -= s;
    const float x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned long long u = units(x[j], a.places);
      if (upto <= goal && upto + u > goal) a.tokens[b * (K + 1) + n] = (int32_t)(4 * i + j);
      upto += u;
    }
  };
  if constexpr (NV > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (before <= goal) look_at(held[j], from + lane + 32 * j);
  } else {
    for (int i = from; i < to && before <= goal; i += 32) look_at(weights(i + lane), i + lane);
  }
}

template <typename... Kernel, typename... Args>
cudaError_t launch_grid(void (*kernel)(Kernel...), int threads, dim3 grid, int ctas, int smem, bool pdl, cudaStream_t stream, Args... args) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
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
  cfg.gridDim = grid;
  cfg.dynamicSmemBytes = (size_t)smem;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

constexpr int64_t kMostRows = 65535;  // of a launch

}  // namespace

cudaError_t launch_softmax(const float* y, float* p, const float* temperature, int64_t M, int64_t V, bool pdl,
                           const DeviceInfo& dev, cudaStream_t stream) {
  const int64_t chunks = (V + 6) / 4;
  // As few CTAs as hold a row, and more while they do not fill the GPU
  int ctas = 1;
  while (ctas < kMostCtas && (chunks > (int64_t)ctas * kRowThreads * 7 || (chunks > (int64_t)ctas * kRowThreads && M * ctas < 4 * (int64_t)dev.num_sms)))
    ctas *= 2;
  const int64_t held = ((chunks + ctas - 1) / ctas + kRowThreads - 1) / kRowThreads;
  const auto of = [&](auto aligned) {
    constexpr bool A = decltype(aligned)::value;
    return held <= 1   ? softmax_kernel<kRowThreads, 1, A>
           : held <= 2 ? softmax_kernel<kRowThreads, 2, A>
           : held <= 4 ? softmax_kernel<kRowThreads, 4, A>
           : held <= 7 ? softmax_kernel<kRowThreads, 7, A>
                       : softmax_kernel<kRowThreads, 0, false>;
  };
  const auto kernel = V % 4 == 0 ? of(std::true_type()) : of(std::false_type());
  for (int64_t m = 0; m < M; m += kMostRows) {
    const int64_t rows = M - m < kMostRows ? M - m : kMostRows;
    const cudaError_t err = launch_grid(kernel, kRowThreads, dim3((unsigned)ctas, (unsigned)rows, 1), ctas, 0, pdl, stream, y + m * V, p + m * V,
                                        temperature ? temperature + m : nullptr, V);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

cudaError_t launch_verify(const float* p, const float* q, const int32_t* draft, const float* uniform, int64_t B, int K,
                          int64_t V, int32_t* tokens, int32_t* accepted, bool pdl, const DeviceInfo& dev, cudaStream_t stream) {
  const int64_t fours = (V + 3) / 4;
  int ctas = 1;
  while (ctas < kMostCtas && (fours > (int64_t)ctas * kVerifyThreads * 7 || (fours > (int64_t)ctas * kVerifyThreads && B * ctas < 4 * (int64_t)dev.num_sms)))
    ctas *= 2;
  const int64_t held = ((fours + ctas * kVerifyWarps - 1) / (ctas * kVerifyWarps) + 31) / 32;
  const bool aligned = V % 4 == 0;
  // Seven turns take more registers than four CTAs an SM have: 5.6 us for one sequence of 50000 tokens with two and
  // 6.8 with four, 13.5 and 11.0 for 64.
  const bool few = B * ctas <= 2 * (int64_t)dev.num_sms;
  const auto of_turns = [&](auto turns) {
    constexpr int NV = decltype(turns)::value;
    if (few) return aligned ? verify_kernel<NV, true, 2> : verify_kernel<NV, false, 2>;
    return aligned ? verify_kernel<NV, true, 4> : verify_kernel<NV, false, 4>;
  };
  const auto kernel = held <= 1   ? of_turns(std::integral_constant<int, 1>())
                      : held <= 4 ? of_turns(std::integral_constant<int, 4>())
                      : held <= 7 ? of_turns(std::integral_constant<int, 7>())
                                  : of_turns(std::integral_constant<int, 0>());
  int bits = 62;
  while (((int64_t)1 << (62 - bits)) < V) --bits;
  for (int64_t b = 0; b < B; b += kMostRows) {
    const int64_t rows = B - b < kMostRows ? B - b : kMostRows;
    const VerifyArgs a = {p + b * (K + 1) * V, q + b * K * V, uniform + b * (K + 1), draft + b * K, tokens + b * (K + 1), accepted + b, V, K, bits};
    const cudaError_t err = launch_grid(kernel, kVerifyThreads, dim3((unsigned)ctas, (unsigned)rows, 1), ctas, 0, pdl, stream, a);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

}  // namespace bitlinear
