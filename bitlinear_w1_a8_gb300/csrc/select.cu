// select.cu -- a cheap score for every page of a long sequence, and the pages that it chooses
// ("Hesper.Models.BitNet" page, section "KV cache": attention reads all of it for each token;
// over chosen pages it reads a fixed part).
//
// Summary of a page's keys for a head: per dim the least and the largest value, lo and hi, of
// code * step (one fp32 product) over the tokens that are there, kept as int8 codes under one step,
//   a = max(max_d |lo_d|, max_d |hi_d|, 1e-5), s = 127 / a, step = a / 127,
//   lower_d = max(floor(lo_d s), -127), upper_d = min(ceil(hi_d s), 127),
// rounded outwards (the fp32 products and quotients before that, to the nearest).  Least and largest do not depend on an order, so neither does a summary.
//
// Score of a page for a q head: with q's codes c_d = rne(q_d (127 / max(max|q|, 1e-5))) as
// activation_quant has them,
//   acc = sum_d max(c_d lower_d, c_d upper_d) = sum_d max(c_d, 0) upper_d + min(c_d, 0) lower_d,
// an exact whole number (dp4a), and score = (acc * step) * (max|q| / 127), two fp32 products: no key of the
// page has a larger product with those codes by more than the roundings, six of 2^-24 of step max|q| sum |c_d| at most.  A
// key head's score is the largest of its q heads'.
//
// Measured.  Summaries of three prompts of up to 2039 tokens, 32 heads of 80, int8: 9.7 us for 15 MB (2.2 us of copying): two
// rounds and a half of CTAs whose loads, join in shared memory and lookups follow one another (a warp waits for memory half
// of its time); of the page that a token was just written to, 16 sequences of 32 heads: 3.9 us, latency.  A warp a page,
// whose lanes join by shuffles, took 10.6 and 8.7.  The choice of 32 of 256 pages for 16 sequences of 32 heads: 8.9 us, of 64 of 2048
// for one of 8 key heads 8.4: latency, a dozen meetings of a CTA's threads among it (a byte at a time over all CTAs'
// keys, the way of more than 8192 pages, and bounds that waited for q's codes took 16 and 22).
#include <cuda_fp16.h>

#include <type_traits>

#include "serve.cuh"
#include "shares.h"

namespace bitlinear {
namespace {

constexpr float kLeastTop = 1e-5f;

// ---------------------------------------------------------------- summaries

constexpr int kSumThreads = 128;
constexpr int kSumWarps = kSumThreads / 32;
constexpr int kSumCtas = 8;  // of an SM
constexpr int kDims = 8;    // of a thread
constexpr int kTurns = 4;   // rows that a thread has on their way together

// Two fp32 sums, or products, an instruction, each rounded as alone.
__device__ __forceinline__ float2 plus2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; add.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z;}" : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 times2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z;}" : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// Eight codes as fp32 values times their row's step: 8 bytes of int8 or e4m3, 16 of bf16 (no step).
template <int FORMAT>
using Codes = std::conditional_t<FORMAT == BITLINEAR_KV_BF16, uint4, uint2>;
template <int FORMAT>
__device__ __forceinline__ void widen(Codes<FORMAT> w, float step, float (&x)[kDims]) {
  if constexpr (FORMAT == BITLINEAR_KV_BF16) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else if constexpr (FORMAT == BITLINEAR_KV_INT8) {
    // code + 128 in the mantissa of 2^23: exact, and not on the unit that converts (a quarter of the rate)
    const uint32_t u[2] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u};
#pragma unroll
    for (int i = 0; i < kDims; i += 2) {
      const float2 b = make_float2(__uint_as_float(__byte_perm(u[i / 4], 0x4b000000u, 0x7650 | i % 4)),
                                   __uint_as_float(__byte_perm(u[i / 4], 0x4b000000u, 0x7650 | (i + 1) % 4)));
      const float2 f = times2(plus2(b, make_float2(-8388736.0f, -8388736.0f)), make_float2(step, step));
      x[i] = f.x;
      x[i + 1] = f.y;
    }
  } else {
    const uint32_t u[2] = {w.x, w.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t h = half2_of_e4m3x2((uint16_t)(u[i / 2] >> (16 * (i % 2))));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      x[2 * i] = __fmul_rn(f.x, step);
      x[2 * i + 1] = __fmul_rn(f.y, step);
    }
  }
}

__device__ __forceinline__ float least_of(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float most_of(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

struct SummariseArgs {
  KvPages c;
  Summary summary;
  const int32_t *table, *first, *lengths;
  int64_t table_stride, max_pages;
  int shares;  // CTAs a key head of a sequence, each every shares-th of its pages
};

// A CTA takes a page of a head, a thread eight dims of every few rows, eight rows on their way at once.
template <int FORMAT>
__global__ void __launch_bounds__(kSumThreads, kSumCtas) summarise_kernel(SummariseArgs a) {
  constexpr int kBytes = FORMAT == BITLINEAR_KV_BF16 ? 2 : 1;
  __shared__ __align__(16) float least[kSumThreads * kDims], most[kSumThreads * kDims];
  __shared__ uint32_t tops[kSumWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_release_dependents();
  pdl_wait_primary();
  const KvPages& c = a.c;
  const int hk = blockIdx.y;
  const int64_t b = blockIdx.z;
  const int D = c.head_dim, chunks = D / kDims, rows = kSumThreads / chunks;  // rows a turn, 4 at least
  const int row = threadIdx.x / chunks, chunk = threadIdx.x - row * chunks;
  const int page_size = 1 << c.page_shift;
  const int64_t length = max((int64_t)0, min((int64_t)a.lengths[b], a.max_pages << c.page_shift));
  const int first = max(0, a.first[b]);
  // no page of a range of no token, not the one that both ends lie in either
  const int begin = (first >> c.page_shift) + blockIdx.x, end = first < length ? (int)((length + page_size - 1) >> c.page_shift) : 0;
  const int32_t* table = a.table + b * a.table_stride;
  int32_t next = begin < end ? table[begin] : -1;
  for (int column = begin; column < end; column += a.shares) {
    const int32_t page = next;
    if (column + a.shares < end) next = table[column + a.shares];
    if (page < 0 || page >= c.num_pages) continue;
    const int here = (int)min((int64_t)page_size, length - ((int64_t)column << c.page_shift));
    const int64_t head = (int64_t)page * c.heads + hk, first_row = head << c.page_shift;
    const uint8_t* k = static_cast<const uint8_t*>(c.k) + (first_row * D + kDims * chunk) * kBytes;
    const float* steps = FORMAT == BITLINEAR_KV_BF16 ? nullptr : c.k_step + first_row;
    float lo[kDims], hi[kDims];
#pragma unroll
    for (int i = 0; i < kDims; ++i) {
      lo[i] = INFINITY;
      hi[i] = -INFINITY;
    }
    for (int t0 = row; t0 < here; t0 += kTurns * rows) {
      Codes<FORMAT> w[kTurns];
      float step[kTurns];
#pragma unroll
      for (int n = 0; n < kTurns; ++n) {  // past the last token: that token again
        const int t = min(t0 + n * rows, here - 1);
        w[n] = __ldg(reinterpret_cast<const Codes<FORMAT>*>(k + t * D * kBytes));
        step[n] = FORMAT == BITLINEAR_KV_BF16 ? 1.0f : __ldg(steps + t);
      }
#pragma unroll
      for (int n = 0; n < kTurns; n += 2) {
        if (t0 - row + n * rows >= here) break;  // for all threads alike
        float x[kDims], y[kDims];
        widen<FORMAT>(w[n], step[n], x);
        widen<FORMAT>(w[n + 1], step[n + 1], y);
#pragma unroll
        for (int i = 0; i < kDims; ++i) {
          lo[i] = least_of(lo[i], x[i], y[i]);
          hi[i] = most_of(hi[i], x[i], y[i]);
        }
      }
    }
    __syncthreads();  // the last page's are read
    if (row < rows) {
#pragma unroll
      for (int i = 0; i < kDims; i += 4) {
        *reinterpret_cast<float4*>(&least[row * D + kDims * chunk + i]) = make_float4(lo[i], lo[i + 1], lo[i + 2], lo[i + 3]);
        *reinterpret_cast<float4*>(&most[row * D + kDims * chunk + i]) = make_float4(hi[i], hi[i + 1], hi[i + 2], hi[i + 3]);
      }
    }
    __syncthreads();
    // a dim or two a thread
    const int taken = min(rows, here);
    float dim_lo[2], dim_hi[2], top = kLeastTop;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int d = threadIdx.x + i * kSumThreads;
      if (d >= D) break;
      dim_lo[i] = least[d];
      dim_hi[i] = most[d];
#pragma unroll 4
      for (int r = 1; r < taken; ++r) {
        dim_lo[i] = fminf(dim_lo[i], least[r * D + d]);
        dim_hi[i] = fmaxf(dim_hi[i], most[r * D + d]);
      }
      top = fmaxf(top, fmaxf(fabsf(dim_lo[i]), fabsf(dim_hi[i])));
    }
    const uint32_t warp_top = __reduce_max_sync(kFullMask, __float_as_uint(top));  // above 0: ordered as their bits
    if (lane == 0) tops[warp] = warp_top;
    __syncthreads();
    top = __uint_as_float(__reduce_max_sync(kFullMask, tops[lane & (kSumWarps - 1)]));
    const float s = __fdiv_rn(127.0f, top);
    int8_t* to = a.summary.bounds + head * 2 * D;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int d = threadIdx.x + i * kSumThreads;
      if (d >= D) break;
      to[d] = (int8_t)(int)fmaxf(floorf(__fmul_rn(dim_lo[i], s)), -127.0f);
      to[D + d] = (int8_t)(int)fminf(ceilf(__fmul_rn(dim_hi[i], s)), 127.0f);
    }
    if (threadIdx.x == 0) a.summary.step[head] = __fdiv_rn(top, 127.0f);
  }
}

// ---------------------------------------------------------------- the choice

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHeadsAtOnce = 16;  // q heads whose codes are in shared memory together
constexpr int kMostCtas = 8;      // of a cluster
constexpr int kDigits = 256;
constexpr uint32_t kKept = 0xffffffffu, kAbsent = 0u;  // keys of pages that are chosen whatever their score, and that are none

__device__ __forceinline__ uint32_t smem_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void send32(uint32_t at, int rank, uint32_t v) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(r), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_begun() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }  // publishes nothing
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_meet() {
  cluster_arrive();
  cluster_wait();
}

// Larger scores have larger keys, between kAbsent and kKept; NaN has the least.
__device__ __forceinline__ uint32_t key_of(float score) {
  const uint32_t u = __float_as_uint(score + 0.0f);
  if (score != score) return 1u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kGathered = 8192;  // pages whose keys one CTA chooses from
constexpr int kRanked = 64;      // and those that one warp ranks
constexpr int kBins = 2048, kBinBits = 11, kListed = 128;

struct Scratch {
  union {
    uint32_t bins[kBins];
    uint32_t histogram[kMostCtas][kDigits];
  };
  uint32_t listed[kListed];
  uint32_t of_warps[kWarps][4];
  uint32_t counted[kMostCtas][2];
  uint32_t found[4];
};

// Over the CTA's threads: sums of x and y, smallest z, largest w.
struct Totals {
  uint32_t x, y, z, w;
};
__device__ __forceinline__ Totals totals(Scratch& t, uint32_t x, uint32_t y, uint32_t z, uint32_t w, int lane, int warp) {
  x = __reduce_add_sync(kFullMask, x);
  y = __reduce_add_sync(kFullMask, y);
  z = __reduce_min_sync(kFullMask, z);
  w = __reduce_max_sync(kFullMask, w);
  __syncthreads();
  if (lane == 0) {
    t.of_warps[warp][0] = x;
    t.of_warps[warp][1] = y;
    t.of_warps[warp][2] = z;
    t.of_warps[warp][3] = w;
  }
  __syncthreads();
  const int i = lane & (kWarps - 1);
  return {__reduce_add_sync(kFullMask, lane < kWarps ? t.of_warps[i][0] : 0u), __reduce_add_sync(kFullMask, lane < kWarps ? t.of_warps[i][1] : 0u),
          __reduce_min_sync(kFullMask, t.of_warps[i][2]), __reduce_max_sync(kFullMask, t.of_warps[i][3])};
}

// The count-th largest of the CTA's keys (`known`), and how many that equal it are among the count largest
// (`wanted`); known kAbsent and wanted 0 where there are fewer.  Keys of scores are put into 2048 bins of the range that
// they cover, so that neighbours in score are neighbours in place: one round leaves a few, which are ranked.
__device__ __forceinline__ void find_here(const uint32_t* keys, int here, uint32_t count, Scratch& t, uint32_t& known, uint32_t& wanted,
                                          int lane, int warp) {
  uint32_t kept = 0, scored = 0, lo = 0xffffffffu, hi = 0;
  for (int i = threadIdx.x; i < here; i += kThreads) {
    const uint32_t k = keys[i];
    kept += k == kKept;
    if (k != kKept && k != kAbsent) {
      ++scored;
      lo = min(lo, k);
      hi = max(hi, k);
    }
  }
  const Totals all = totals(t, kept, scored, lo, hi, lane, warp);
  known = kAbsent;
  wanted = 0;
  if (all.x + all.y <= count) return;
  if (all.x >= count) {
    known = kKept;
    wanted = count;
    return;
  }
  wanted = count - all.x;  // of keys lo .. hi
  lo = all.z;
  hi = all.w;
  for (;;) {
    const int shift = max(0, 32 - __clz(hi - lo) - kBinBits);
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kThreads) t.bins[i] = 0;
    if (threadIdx.x == 0) t.found[2] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < here; i += kThreads) {
      const uint32_t k = keys[i];
      if (k >= lo && k <= hi && k != kAbsent) atomicAdd(&t.bins[(k - lo) >> shift], 1u);
    }
    __syncthreads();
    // a thread has 8 bins, the highest in thread 0
    uint32_t n[kBins / kThreads], mine = 0;
#pragma unroll
    for (int i = 0; i < kBins / kThreads; ++i) mine += n[i] = t.bins[kBins - 1 - (kBins / kThreads * threadIdx.x + i)];
    uint32_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(kFullMask, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane == 31) t.of_warps[warp][0] = upto;
    __syncthreads();
    upto += __reduce_add_sync(kFullMask, lane < warp ? t.of_warps[lane & (kWarps - 1)][0] : 0u);
    uint32_t above = upto - mine;
    if (wanted > above && wanted <= upto) {
#pragma unroll
      for (int i = 0; i < kBins / kThreads; ++i) {
        if (wanted > above && wanted <= above + n[i]) {
          t.found[0] = kBins - 1 - (kBins / kThreads * threadIdx.x + i);
          t.found[1] = above;
          t.found[3] = n[i];
        }
        above += n[i];
      }
    }
    __syncthreads();
    const uint32_t bin = t.found[0], inside = t.found[3];
    wanted -= t.found[1];
    lo += bin << shift;
    hi = min(hi, lo + ((1u << shift) - 1));
    if (shift == 0) {
      known = lo;
      return;
    }
    if (inside <= kListed) break;
  }
  for (int i = threadIdx.x; i < here; i += kThreads) {
    const uint32_t k = keys[i];
    if (k >= lo && k <= hi && k != kAbsent) t.listed[atomicAdd(&t.found[2], 1u)] = k;
  }
  __syncthreads();
  const uint32_t n = t.found[2];
  if (threadIdx.x < n) {
    const uint32_t k = t.listed[threadIdx.x];
    uint32_t greater = 0, equal = 0;
    for (uint32_t i = 0; i < n; ++i) {
      greater += t.listed[i] > k;
      equal += t.listed[i] == k;
    }
    if (greater < wanted && wanted <= greater + equal) {  // the same from every equal key
      t.found[0] = k;
      t.found[1] = greater;
    }
  }
  __syncthreads();
  known = t.found[0];
  wanted -= t.found[1];
}

// The same of all CTAs' keys together, a byte at a time from histograms that all CTAs add up.
__device__ __forceinline__ void find_in_cluster(const uint32_t* keys, int here, uint32_t count, Scratch& t, uint32_t& known, uint32_t& wanted,
                                                int ctas, int rank, int lane) {
  known = 0;
  wanted = count;
  uint32_t mask = 0;  // where the bytes found are
  for (int shift = 24; shift >= 0; shift -= 8) {
    uint32_t* mine = t.histogram[rank];
    for (int i = threadIdx.x; i < kDigits; i += kThreads) mine[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < here; i += kThreads) {
      const uint32_t k = keys[i];
      if (k != kAbsent && (k & mask) == known) atomicAdd(&mine[(k >> shift) & 0xff], 1u);
    }
    __syncthreads();
    for (int r = 0; r < ctas; ++r)
      if (r != rank)
        for (int i = threadIdx.x; i < kDigits; i += kThreads) send32(smem_at(&t.histogram[rank][i]), r, mine[i]);
    cluster_meet();
    // every warp finds the byte for itself: a lane has 8 digits, the highest digits in lane 0
    uint32_t n[8], all = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      n[i] = 0;
      for (int r = 0; r < ctas; ++r) n[i] += t.histogram[r][kDigits - 1 - (8 * lane + i)];
      all += n[i];
    }
    uint32_t upto = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(kFullMask, upto, o);
      if (lane >= o) upto += x;
    }
    uint32_t above = upto - all, digit = 0;
    const uint32_t has = __ballot_sync(kFullMask, wanted > above && wanted <= upto);
    if (has == 0) {  // fewer keys than are wanted: all of them
      known = kAbsent;
      wanted = 0;
      cluster_meet();
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (wanted > above && wanted <= above + n[i]) {
        digit = kDigits - 1 - (8 * lane + i);
        break;
      }
      above += n[i];
    }
    const int owner = __ffs(has) - 1;
    digit = __shfl_sync(kFullMask, digit, owner);
    wanted -= __shfl_sync(kFullMask, above, owner);
    known |= digit << shift;
    mask |= 0xffu << shift;
    cluster_meet();  // the histograms are read
  }
}

// A lane's 16 of a page's bounds at a time: LANES of them (a power of two) have a row, of lower or of upper bounds, a
// warp 16 / LANES pages an instruction and kLoads of these on their way.  (Two lanes a page, each reading a row from end to
// end, took 3.9 us for 256 pages of 128 dims where this takes 2.1: every load touched 32 lines.)
constexpr int kLoads = 8;

// A cluster chooses for one key head of one sequence.  Every CTA scores a run of the pages; up to kGathered of them
// (`gather`) all keys go to the first CTA, which chooses, and beyond each keeps its own and writes its chosen
// pages where those of the CTAs before it end.
template <int LANES, bool FEW>  // dims / 16 at most; kRanked pages and kThreads chosen ones at most, one CTA
__global__ void __launch_bounds__(kThreads) select_kernel(SelectArgs a, KvPages c, Summary summary, int share, bool gather) {
  extern __shared__ __align__(16) uint8_t smem[];
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem);
  __shared__ __align__(16) int8_t codes[kHeadsAtOnce][2][LANES * 16];  // parts below and above 0
  __shared__ float steps[kHeadsAtOnce];
  __shared__ Scratch scratch;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int ctas = gridDim.x, rank = blockIdx.x;
  pdl_release_dependents();
  if (!FEW && ctas > 1) cluster_begun();  // waited for before the first word goes to another CTA
  pdl_wait_primary();
  const int64_t b = (int64_t)blockIdx.z, hk = blockIdx.y;
  const int D = c.head_dim, chunks = D / 16, group = a.q_heads / c.heads;
  const int64_t length = max((int64_t)0, min((int64_t)a.lengths[b], a.max_pages << c.page_shift));
  const int pages = (int)((length + (1 << c.page_shift) - 1) >> c.page_shift);
  // runs as short as the sequence allows
  const int run = min(share, (pages + ctas - 1) / ctas);
  int from = min(pages, rank * run), here = min(pages, from + run) - from;
  const int32_t* table = a.table + b * a.table_stride;
  int32_t* out = a.blocks + (b * c.heads + hk) * a.count;

  constexpr int kTogether = 16 / LANES, kPages = kLoads * kTogether;  // pages of an instruction, and of a warp
  static_assert(kLoads == 8 && LANES >= 4, "three halvings leave a page a lane");
  const int chunk = lane & (LANES - 1), side = (lane / LANES) & 1;
  const int mine = ((lane & 1) << 2 | (lane & 2) | ((lane >> 2) & 1)) * kTogether + lane / (2 * LANES);  // the page that this lane ends with
  const bool writes = (lane & (2 * LANES - 1)) < 8;  // one of those that end with it
  uint4 w[kLoads];
  float step;
  int32_t page_here;
  auto look_up = [&](int i0) { return lane < kPages && i0 + warp * kPages + lane < here ? table[from + i0 + warp * kPages + lane] : -1; };
  int32_t listed = look_up(0);
  auto bring = [&](int i0) {
    if (listed >= c.num_pages) listed = -1;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int32_t page = __shfl_sync(kFullMask, listed, j * kTogether + lane / (2 * LANES));
      w[j] = page >= 0 && chunk < chunks ? __ldg(reinterpret_cast<const uint4*>(summary.bounds + (((int64_t)page * c.heads + hk) * 2 + side) * D) + chunk)
                                         : make_uint4(0, 0, 0, 0);
    }
    page_here = __shfl_sync(kFullMask, listed, mine);
    step = page_here >= 0 ? __ldg(summary.step + (int64_t)page_here * c.heads + hk) : 0.0f;
    listed = look_up(i0 + kWarps * kPages);
  };
  bring(0);  // on their way while q is turned into codes
  for (int h0 = 0; h0 < group; h0 += kHeadsAtOnce) {
    const int heads = min(kHeadsAtOnce, group - h0);
    if (h0 > 0) __syncthreads();
    for (int h = warp; h < heads; h += kWarps) {  // a warp quantises a head
      const float* q = a.q + b * a.q_stride + (hk * group + h0 + h) * D;
      float x[(LANES * 16 + 31) / 32], top = kLeastTop;
#pragma unroll
      for (int i = 0; i < (LANES * 16 + 31) / 32; ++i) {
        x[i] = lane + 32 * i < D ? q[lane + 32 * i] : 0.0f;
        top = fmaxf(top, fabsf(x[i]));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
      const float s = __fdiv_rn(127.0f, top);
#pragma unroll
      for (int i = 0; i < (LANES * 16 + 31) / 32; ++i) {
        if (lane + 32 * i < D) {
          const int code = max(-127, min(127, __float2int_rn(__fmul_rn(x[i], s))));
          codes[h][0][lane + 32 * i] = (int8_t)min(code, 0);
          codes[h][1][lane + 32 * i] = (int8_t)max(code, 0);
        }
      }
      if (lane == 0) steps[h] = __fdiv_rn(top, 127.0f);
    }
    __syncthreads();
    if (h0 > 0) listed = look_up(0);
    for (int i0 = 0; i0 < here; i0 += kWarps * kPages) {
      const int i = i0 + warp * kPages + mine, column = from + i;
      if (i0 > 0 || h0 > 0) bring(i0);
      float best = -INFINITY;
      bool nan = false;
      for (int h = 0; h < heads; ++h) {
        const uint4 x = *reinterpret_cast<const uint4*>(&codes[h][side][16 * chunk]);
        int acc[kLoads];
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
          acc[j] = __dp4a((int)w[j].w, (int)x.w, __dp4a((int)w[j].z, (int)x.z, __dp4a((int)w[j].y, (int)x.y, __dp4a((int)w[j].x, (int)x.x, 0))));
        // three halvings: a lane keeps half of its loads and gives the others away
#pragma unroll
        for (int n = kLoads / 2, o = 1; n > 0; n /= 2, o *= 2) {
#pragma unroll
          for (int j = 0; j < n; ++j) {
            const bool upper = lane & o;
            acc[j] = (upper ? acc[j + n] : acc[j]) + __shfl_xor_sync(kFullMask, upper ? acc[j] : acc[j + n], o);
          }
        }
#pragma unroll
        for (int o = 8; o < 2 * LANES; o *= 2) acc[0] += __shfl_xor_sync(kFullMask, acc[0], o);
        const float score = __fmul_rn(__fmul_rn((float)acc[0], step), steps[h]);
        nan |= score != score;
        best = fmaxf(best, score);
      }
      if (i < here && writes) {
        uint32_t key = nan ? 1u : key_of(best);
        if (h0 > 0) key = keys[i] == 1u || key == 1u ? 1u : max(key, keys[i]);
        if (h0 + heads >= group && (column < a.keep_first || column >= pages - a.keep_last)) key = kKept;
        keys[i] = page_here >= 0 ? key : kAbsent;
      }
    }
  }
  __syncthreads();
  if (!FEW && ctas > 1) {
    cluster_wait();  // all of the cluster's CTAs have begun
    if (gather) {
      if (rank > 0)
        for (int i = threadIdx.x; i < here; i += kThreads) send32(smem_at(keys + from + i), 0, keys[i]);
      cluster_meet();
      if (rank > 0) return;
      ctas = 1;
      from = 0;
      here = pages;
    }
  }

  // Few pages: a warp ranks them (a step of three calls over 8 of 22 pages, 16 heads of 128: 9.6 us, 11.4 by the way below).
  if constexpr (FEW) {
    if (warp > 0) return;
    const uint32_t k0 = lane < here ? keys[lane] : kAbsent, k1 = lane + 32 < here ? keys[lane + 32] : kAbsent;
    int before0 = 0, before1 = 0;
    for (int i = 0; i < here; ++i) {
      const uint32_t k = keys[i];
      before0 += k > k0 || (k == k0 && i < lane);
      before1 += k > k1 || (k == k1 && i < lane + 32);
    }
    const uint32_t c0 = __ballot_sync(kFullMask, k0 != kAbsent && before0 < a.count), c1 = __ballot_sync(kFullMask, k1 != kAbsent && before1 < a.count);
    const uint32_t below = (1u << lane) - 1;
    if ((c0 >> lane) & 1u) out[__popc(c0 & below)] = lane;
    if ((c1 >> lane) & 1u) out[__popc(c0) + __popc(c1 & below)] = lane + 32;
    for (int i = __popc(c0) + __popc(c1) + lane; i < a.count; i += 32) out[i] = -1;
    return;
  }
  // Chosen: keys above `known`, and the first `wanted` that equal it.
  uint32_t known, wanted;
  if (ctas == 1)
    find_here(keys, here, a.count, scratch, known, wanted, lane, warp);
  else
    find_in_cluster(keys, here, a.count, scratch, known, wanted, ctas, rank, lane);
  uint32_t more_before = 0, equal_before = 0;
  if (ctas > 1) {
    uint32_t more = 0, equal = 0;
    for (int i = threadIdx.x; i < here; i += kThreads) {
      more += keys[i] > known;
      equal += keys[i] == known;
    }
    const Totals all = totals(scratch, more, equal, 0, 0, lane, warp);
    if (threadIdx.x < ctas) {
      send32(smem_at(&scratch.counted[rank][0]), threadIdx.x, all.x);
      send32(smem_at(&scratch.counted[rank][1]), threadIdx.x, all.y);
    }
    cluster_meet();
    for (int r = 0; r < rank; ++r) {
      more_before += scratch.counted[r][0];
      equal_before += scratch.counted[r][1];
    }
  }
  // Written in order: a thread has a run of the keys, and counts what is before it.
  const int each = (here + kThreads - 1) / kThreads, first = min(here, (int)threadIdx.x * each), last = min(here, first + each);
  uint32_t counts = 0;  // more above, equal below
  for (int i = first; i < last; ++i) counts += (uint32_t)(keys[i] > known) << 16 | (uint32_t)(keys[i] == known);
  uint32_t upto = counts;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(kFullMask, upto, o);
    if (lane >= o) upto += x;
  }
  __syncthreads();
  if (lane == 31) scratch.of_warps[warp][0] = upto;
  __syncthreads();
  const uint32_t of_warp = lane < kWarps ? scratch.of_warps[lane][0] : 0u;
  const uint32_t before = upto - counts + __reduce_add_sync(kFullMask, lane < warp ? of_warp : 0u), whole = __reduce_add_sync(kFullMask, of_warp);
  uint32_t m_at = more_before + (before >> 16), e_at = equal_before + (before & 0xffffu);
  for (int i = first; i < last; ++i) {
    const uint32_t k = keys[i];
    if (k > known || (k == known && e_at < wanted)) out[m_at + min(e_at, wanted)] = from + i;
    m_at += k > known;
    e_at += k == known;
  }
  more_before += whole >> 16;
  equal_before += whole & 0xffffu;
  if (rank == ctas - 1)  // whose counts are of all
    for (uint32_t i = more_before + min(equal_before, wanted) + threadIdx.x; i < (uint32_t)a.count; i += kThreads) out[i] = -1;
}

}  // namespace

cudaError_t launch_summarise(const KvPages& cache, const Summary& summary, const int32_t* table, int64_t table_stride,
                             int64_t B, int64_t max_pages, const int32_t* first, const int32_t* lengths, bool pdl,
                             const DeviceInfo& dev, cudaStream_t stream) {
  const int64_t shares = page_shares(max_pages, B * cache.heads, (int64_t)dev.num_sms * kSumCtas);
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.blockDim = dim3(kSumThreads, 1, 1);
  if (pdl) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
  }
  const auto kernel = cache.format == BITLINEAR_KV_INT8  ? summarise_kernel<BITLINEAR_KV_INT8>
                      : cache.format == BITLINEAR_KV_FP8 ? summarise_kernel<BITLINEAR_KV_FP8>
                                                         : summarise_kernel<BITLINEAR_KV_BF16>;
  constexpr int64_t kMostSeqs = 65535;
  for (int64_t b = 0; b < B; b += kMostSeqs) {
    const SummariseArgs a = {cache, summary, table + b * table_stride, first + b, lengths + b, table_stride, max_pages, (int)shares};
    cfg.gridDim = dim3((unsigned)shares, (unsigned)cache.heads, (unsigned)(B - b < kMostSeqs ? B - b : kMostSeqs));
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, a);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

template <int LANES>
static cudaError_t launch_select_lanes(SelectArgs a, const KvPages& cache, const Summary& summary, bool pdl,
                                        const DeviceInfo& dev, cudaStream_t stream) {
  constexpr int kMostShare = 24576;  // pages a CTA: 96 KB of keys, counted in 16 bits
  const int64_t heads = a.B * cache.heads;
  int ctas = 1;
  while (ctas < kMostCtas && (a.max_pages > (int64_t)ctas * kMostShare ||
                              (a.max_pages > (int64_t)ctas * 128 && heads * ctas * 2 <= 4 * dev.num_sms)))
    ctas *= 2;
  const int share = (int)((a.max_pages + ctas - 1) / ctas);
  const bool few = a.max_pages <= kRanked && a.count <= kThreads;
  const auto kernel = few ? select_kernel<LANES, true> : select_kernel<LANES, false>;
  static thread_local int configured_device = -1;
  if (configured_device != dev.device) {
    const cudaError_t err = cudaFuncSetAttribute(select_kernel<LANES, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShare * 4);
    if (err != cudaSuccess) return err;
    configured_device = dev.device;
  }
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.blockDim = dim3(kThreads, 1, 1);
  const bool gather = a.max_pages <= kGathered;
  cfg.dynamicSmemBytes = (size_t)(gather ? a.max_pages : share) * 4;
  if (ctas > 1) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.numAttrs = 1;
  }
  if (pdl) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  constexpr int64_t kMostSeqs = 65535;
  const int64_t B = a.B;
  for (int64_t b = 0; b < B; b += kMostSeqs) {
    SelectArgs part = a;
    part.q += b * a.q_stride;
    part.table += b * a.table_stride;
    part.lengths += b;
    part.blocks += b * cache.heads * a.count;
    cfg.gridDim = dim3((unsigned)ctas, (unsigned)cache.heads, (unsigned)(B - b < kMostSeqs ? B - b : kMostSeqs));
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, part, cache, summary, share, gather);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

cudaError_t launch_select(const SelectArgs& a, const KvPages& cache, const Summary& summary, bool pdl,
                          const DeviceInfo& dev, cudaStream_t stream) {
  if (cache.head_dim <= 64) return launch_select_lanes<4>(a, cache, summary, pdl, dev, stream);
  if (cache.head_dim <= 128) return launch_select_lanes<8>(a, cache, summary, pdl, dev, stream);
  return launch_select_lanes<16>(a, cache, summary, pdl, dev, stream);
}

}  // namespace bitlinear
