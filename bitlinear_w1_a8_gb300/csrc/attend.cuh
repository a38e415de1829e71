// attend.cuh -- the kernel that attends to the paged key-value cache, and what it is made of.
// attention.cu says how it works and what bounds it; MODE says what a CTA's rows and tokens are:
// the tokens of one sequence (kClusters, kSharedOut: attention.cu), the pages that a list names
// (kBlocks: attention_blocks.cu), the tokens that a group of rows shares, and a row's own tokens
// joined with those (kPrefix, kOwn, kPacked: attention_shared.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kv.cuh"
#include "shares.h"

namespace bitlinear {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kRowHeads = 8;   // q heads of one CTA
constexpr int kStages = 2;     // the step in hand and the next
constexpr int kMaxCluster = 16;  // where the device schedules one; else kPortableCluster
constexpr int kPortableCluster = 8;
constexpr int kSms = 152;
constexpr int kOtherSmem = 1024 + 640;  // of a CTA, beside the dynamic: the system's and the static arrays
constexpr int kLeastSteps = 2;    // steps a warp at least: short rows take fewer CTAs
constexpr int kSortSeqs = kThreads;  // sequences that a CTA ranks by length
constexpr float kLimit = 256.0f;  // the largest weight before the reference moves
constexpr float kUnset = -1e30f;  // a reference below every logit
constexpr float kLeastStep = 8.2718061e-25f;  // 2^-80: a value's step counts as that at least (a cache of zeros holds 0)

// Sizes of one instantiation: DT dims a head (a smaller head_dim is padded with
// zeros), codes of kBytes, steps of kTokens tokens.
template <int FORMAT, int DT>
struct Shape {
  static constexpr int kBytes = FORMAT == BITLINEAR_KV_BF16 ? 2 : 1;
  static constexpr int kRow = DT * kBytes;
  // Where chunk c (16 bytes) of row n is, so that the fragments' loads (8 rows x 4 words for
  // keys, 4 even or 4 odd rows x 8 words for values) touch every bank once.  Rows of an odd
  // number of chunks do so as they are.  Else the last kTurn bits of the chunk are xor-ed
  // with the first of the row's place among eight, and each eight rows are kept in the order
  // 0 2 4 6 1 3 5 7 (one bit), 0 2 1 3 4 6 5 7 (two) or as they come (three).  Both chunks of
  // a 32-byte sector stay in one such block, so that a copied sector is one write; a pad of
  // 16 bytes a row splits every other row's (95.3 for 85.3 us on one sequence of 131072
  // tokens bf16, 32.7 for 29.2 on 64 x 2048 of 8 key heads of 64, int8).
  static constexpr int kTurn = (kRow / 16) % 2 ? 0 : (kRow / 16) % 4 ? 1 : (kRow / 16) % 8 ? 2 : 3;
  static constexpr int kNext = kTurn == 1 ? 4 : kTurn == 2 ? 2 : 1;  // from an even row to the one after
  static __device__ __forceinline__ uint32_t place(int n, int chunk) {
    const int slot = kTurn == 1 ? (n & ~7) | (n & 1) << 2 | (n & 6) >> 1 : kTurn == 2 ? (n & ~3) | (n & 1) << 1 | (n & 2) >> 1 : n;
    return slot * kRow + (kTurn ? chunk ^ ((slot & 7) >> (3 - kTurn)) : chunk) * 16;
  }
  static constexpr int kTokens = kRow <= 96 ? 32 : 16;
  static constexpr int kTiles = kTokens / 8;       // n-tiles of the logits
  static constexpr int kSteps = DT / 16;           // k-steps of the logits
  static constexpr int kChunks = kRow / 16;
  static constexpr int kOutTiles = DT / 8;         // n-tiles of the weighted sums
  static constexpr int kStage = 2 * kTokens * kRow + 2 * kTokens * 4;
  static constexpr int kWarpBytes = kStages * kStage;
  static constexpr int kPartial = (DT + 4) * 4;    // a head's weighted sum, m and sum, padded to 16 bytes
  static constexpr size_t kSmem = (size_t)kWarps * kWarpBytes;
  static constexpr int kCtas = kRow <= 192 ? 4 : kRow <= 256 && kBytes == 2 ? 3 : 2;  // CTAs an SM that the registers allow
  // q's parts of a head: 4 lanes' 16 bytes a k-step (leading part and rest, two words each), and 8
  // bytes of third parts for bf16
  static constexpr int kHeadBytes = 4 * kSteps * (kBytes == 1 ? 16 : 24);
  // of any call: the rings, q's parts and scales, and what a CTA of the largest cluster receives
  static constexpr int kMostShared = (int)kSmem + kRowHeads * (kHeadBytes + 4) +
                                     kMaxCluster * ((kRowHeads * DT + kMaxCluster - 1) / kMaxCluster + 1 + 2 * kRowHeads) * 4;
  static_assert(kRowHeads * kPartial <= kWarpBytes, "a warp's partials reuse its ring");
  static_assert(kTokens * kRow % 128 == 0 && kStage % 128 == 0, "chunks are turned within 128 bytes");
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ float4 lds_float4(uint32_t a) {
  const uint4 w = lds128(a);
  return make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
}
__device__ __forceinline__ float2 lds_float2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
  return v;
}
// Stores a float in CTA `rank` of the cluster, at the address that `a` has in this CTA.
__device__ __forceinline__ void sts_cluster(uint32_t a, int rank, float v) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(r), "f"(v) : "memory");
}
__device__ __forceinline__ float lds_float(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ float exp2_of(float x) {  // relative error 2^-22, 0 below -126
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float at_least(float x, float least) {  // NaN stays NaN
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(least));
  return y;
}
__device__ __forceinline__ float log2_of(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^e for |e| <= 126, and the exponent of a positive normal x.
__device__ __forceinline__ float power2(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ int exponent_of(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }
__device__ __forceinline__ int clamp_exponent(int e) { return max(-100, min(100, e)); }

// Two at a time: one instruction for both, each rounded as alone.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// c = a b (FIRST) or c += a b.
template <int FORMAT, bool FIRST>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  const float c0 = FIRST ? 0.0f : c[0], c1 = FIRST ? 0.0f : c[1], c2 = FIRST ? 0.0f : c[2], c3 = FIRST ? 0.0f : c[3];
  if constexpr (FORMAT == BITLINEAR_KV_BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// The bytes `pair` selects of two code words, widened to two halves.  int8 codes
// come with their sign bit flipped (excess 128): 0x6400 | u is the half 1024 + u.
__device__ __forceinline__ uint32_t halves_of_int8(uint32_t w, uint32_t selector) {
  const uint32_t u = __byte_perm(w, 0x64646464u, selector);
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <int FORMAT>
__device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) {  // bytes 0, 1 and 2, 3
  if constexpr (FORMAT == BITLINEAR_KV_INT8) {
    w ^= 0x80808080u;
    lo = halves_of_int8(w, 0x4140);
    hi = halves_of_int8(w, 0x4342);
  } else {
    lo = half2_of_e4m3x2((uint16_t)w);
    hi = half2_of_e4m3x2((uint16_t)(w >> 16));
  }
}

// x, y as leading parts and what they leave, the latter times 2^11 (fp16).  MORE: of x and y
// (1 + more 2^-11) each.
template <bool MORE = false>
__device__ __forceinline__ void split2(float x, float y, uint32_t& lead, uint32_t& rest, float more = 0.0f) {
  const __half2 h = __floats2half2_rn(x, y);
  // exact, as (x - h) 2^11 is: h is x's leading part
  float2 d = fma2(__half22float2(h), both(-2048.0f), mul2(make_float2(x, y), both(2048.0f)));
  if constexpr (MORE) d = fma2(make_float2(x, y), both(more), d);
  const __half2 r = __floats2half2_rn(d.x, d.y);
  lead = *reinterpret_cast<const uint32_t*>(&h);
  rest = *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t next_part(float& x, float& y) {  // bf16 parts, taken off x and y
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  x -= __low2float(h);
  y -= __high2float(h);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A key head's part of the cache and the tokens of the sequence that count.
struct Source {
  const uint8_t *k, *v;    // the head's rows of page 0
  const float *ks, *vs;
  uint32_t first, len;     // first <= t < len
};

// Requests a step whose every token counts and has a page, head_dim == DT: a
// half's 16 rows are one run of bytes, 512 of them an instruction.
template <int FORMAT, int DT>
__device__ __forceinline__ void request_whole(const Source& r, const int64_t (&row)[2], uint32_t stage, int lane) {
  using S = Shape<FORMAT, DT>;
  constexpr int kTurns = 16 * S::kChunks / 32;  // whole turns of the warp over a half's chunks
  auto place = [](int i) { return S::place(i / S::kChunks, i % S::kChunks); };
#pragma unroll
  for (int s = 0; s < S::kTokens / 16; ++s) {
    const uint8_t* k = r.k + row[s] * S::kRow;
    const uint8_t* v = r.v + row[s] * S::kRow;
    const uint32_t kd = stage + 16 * s * S::kRow, vd = kd + S::kTokens * S::kRow;
#pragma unroll
    for (int j = 0; j < kTurns; ++j) {
      copy16(kd + place(lane + 32 * j), k + 16 * (lane + 32 * j));
      copy16(vd + place(lane + 32 * j), v + 16 * (lane + 32 * j));
    }
    if constexpr (S::kChunks % 2) {  // half a turn of each is left
      const int i = (lane & 15) + 32 * kTurns;
      copy16((lane < 16 ? kd : vd) + place(i), (lane < 16 ? k : v) + 16 * i);
    }
  }
  if constexpr (FORMAT != BITLINEAR_KV_BF16) {
    if (lane < S::kTokens / 2) {  // 16 bytes: key steps of the halves, then value steps
      const int in_kind = lane % (S::kTokens / 4), half = in_kind / 4;
      copy16(stage + 2 * S::kTokens * S::kRow + 16 * lane,
             (lane < S::kTokens / 4 ? r.ks : r.vs) + (half ? row[1] : row[0]) + 4 * (in_kind % 4));
    }
  }
}

// Requests any step; `ok` says which halves have a page.  Rows that do not count
// are zeroed, so that whatever they hold (NaN among it) meets no weight of 0.
// COUNTED: the first left[s] rows of a half count, else those of the source's tokens.
template <int FORMAT, int DT, bool COUNTED>
__device__ __forceinline__ void request_part(const Source& r, const KvPages& c, uint32_t t0, const int64_t (&row)[2],
                                             uint32_t ok, uint32_t stage, int lane, const int (&left)[2]) {
  using S = Shape<FORMAT, DT>;
  const int row_bytes = c.head_dim * S::kBytes, chunks = row_bytes / 16;
#pragma unroll
  for (int s = 0; s < S::kTokens / 16; ++s) {
    const uint32_t t = t0 + 16 * s;
    const bool have = (ok >> s) & 1u;
    const uint8_t* k = r.k + row[s] * row_bytes;
    const uint8_t* v = r.v + row[s] * row_bytes;
    const uint32_t kd = stage + 16 * s * S::kRow, vd = kd + S::kTokens * S::kRow;
#pragma unroll 1
    for (int i = lane; i < 16 * S::kChunks; i += 32) {
      const int n = i / S::kChunks, ch = i % S::kChunks;
      if (ch >= chunks) continue;
      const bool there = have && (COUNTED ? n < left[s] : t + n >= r.first && t + n < r.len);
      const int off = there ? n * row_bytes + 16 * ch : 0;
      copy16(kd + S::place(n, ch), k + off, there);
      copy16(vd + S::place(n, ch), v + off, there);
    }
    if constexpr (FORMAT != BITLINEAR_KV_BF16) {
      const int n = lane & 15;
      const bool there = have && (COUNTED ? n < left[s] : t + n >= r.first && t + n < r.len);
      copy4(stage + 2 * S::kTokens * S::kRow + (lane >> 4) * S::kTokens * 4 + (16 * s + n) * 4,
            (lane < 16 ? r.ks : r.vs) + row[s] + (there ? n : 0), there);
    }
  }
}

// A row's output: zeros where no token counted (no reference, no sum).  Whatever else the
// sum is, a NaN on the way here is one of the output too.
__device__ __forceinline__ float output_of(float value, float m, float sum) {
  return value / (m == kUnset && sum == 0.0f ? 1.0f : sum);
}

// Joins `parts` partials, at most MOST: the values are at `value` and every `apart`
// bytes on, the references and sums (side by side) at `scale` and every `scales_apart`.
// Unrolled, so that all of them are on their way together.
struct Joined {
  float value, m, sum;
};
template <int MOST>
__device__ __forceinline__ Joined join(uint32_t value, uint32_t apart, uint32_t scale, uint32_t scales_apart, int parts) {
  Joined j = {0.0f, kUnset, 0.0f};
  float2 s[MOST];
  float v[MOST];
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    s[i] = i < parts ? lds_float2(scale + i * scales_apart) : make_float2(kUnset, 0.0f);
    v[i] = i < parts ? lds_float(value + i * apart) : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < MOST; ++i) j.m = fmaxf(j.m, s[i].x);
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    const float f = exp2_of(s[i].x - j.m);
    j.sum = fmaf(s[i].y, f, j.sum);
    j.value = fmaf(v[i], f, j.value);
  }
  return j;
}

// Where a CTA receives what its cluster's CTAs have for its share of a row's dims (dim
// i of the row is CTA i % splits's): [CTA][share's dims] and [CTA][head][m, sum], behind
// the rings.
__host__ __device__ __forceinline__ int share_of(int heads, int D, int splits) { return (heads * D + splits - 1) / splits; }
__host__ __device__ __forceinline__ int received_bytes(int heads, int D, int splits) {
  return splits > 1 ? splits * (share_of(heads, D, splits) + 1 + 2 * heads) * 4 : 0;
}

// What the rows of a launch are, and which tokens each attends to.
enum Mode {
  kClusters,   // a key head of a sequence, its tokens split over a cluster
  kSharedOut,  // the same, its tokens split in proportion over CTAs that leave parts behind
  kBlocks,     // a key head of a sequence and the pages that its list names, over a cluster
  kPrefix,     // a key head of a group of sequences and the tokens that they share; leaves parts behind
  kOwn,        // a key head of a sequence and its tokens behind the shared ones, joined with kPrefix's parts
  kPacked      // the same, up to four rows of a sequence a CTA: one, two or four warps a row, by its tokens
};

// How rows are shared out.
struct Shares {
  int64_t b0;      // the launch's first sequence
  int group, groups, rows_a_seq;  // q heads a key head, groups of them, rows of a sequence
  int splits;      // CTAs a row where each has as many: a power of two
  int splits_log2;
  bool sorted;     // sequences in order of length, the longest first
  float* parts;    // rows shared out by their steps: [CTA][q heads of a row, at most 8][dims, m, sum]
  int2* rows;      // and a row's first CTA and how many it has
  // kBlocks: the pages' columns, `count` a key head of a sequence
  const int32_t* blocks;
  int count;
  // kPrefix, kOwn, kPacked: sequences a group, the tokens that each group shares, every sequence's length, and
  // q heads a key head (kPrefix's `group` holds those of all the group's sequences)
  int group_rows;
  const int32_t* shared;
  const int32_t* lengths;
  int heads_a_key;
  int prefix_tiles;  // rows a key head of a group, of
  int prefix_heads;  // so many q heads, and
  int slot_heads;    // their places in a part
  // kPacked: warps a row at least, and steps a warp at most while the row has fewer than four
  int least_warps, warp_steps;
};

// Tokens first <= t < len of a sequence that count, in steps of T from first / T on.
// A length is at most 2^31 - 1, so tokens and the steps past them fit in 32 bits.
template <int T>
struct Span {
  uint32_t first, len;
  __device__ __forceinline__ Span(int32_t length, int64_t most, int64_t window) {
    len = length <= 0 ? 0u : length < most ? (uint32_t)length : (uint32_t)most;
    first = window > 0 && len > window ? len - (uint32_t)window : 0u;
  }
  __device__ __forceinline__ uint32_t begin() const { return first / T * T; }
  __device__ __forceinline__ int steps() const { return len > first ? (int)((len + T - 1) / T - first / T) : 0; }
};

// This CTA's row and which part of it.  Every row with any step has ceil(steps /
// share) CTAs, in the order of the rows; share is the least for which the grid has
// enough of them (each row rounds up by less than one).
// Every warp finds it for itself, a lane for one sequence in 32: no barrier.
struct Part {
  int64_t b;
  int row, part, parts;  // parts == 0: the CTA has nothing
};
template <int T>
__device__ __forceinline__ Part find_part(const AttendArgs& a, int64_t most, int rows_a_seq, int least = kLeastSteps * kWarps) {
  const int lane = threadIdx.x & 31, here = blockIdx.x;
  const int each = ((int)a.B + 31) / 32, from = min((int)a.B, lane * each), to = min((int)a.B, from + each);
  auto steps_of = [&](int b) { return Span<T>(a.lengths[b], most, a.window).steps(); };
  int steps = 0, some = 0;
  for (int b = from; b < to; ++b) {
    const int n = steps_of(b);
    steps += n;
    some += n > 0;
  }
  const int total = __reduce_add_sync(kFullMask, steps) * rows_a_seq, rows = __reduce_add_sync(kFullMask, some) * rows_a_seq;
  const int spare = (int)gridDim.x - rows;  // > 0: the host takes this path for rows well below the grid
  const int share = share_of_steps(total, spare, least);
  auto parts_of = [&](int b) { return (steps_of(b) + share - 1) / share; };
  int ctas = 0;
  for (int b = from; b < to; ++b) ctas += parts_of(b) * rows_a_seq;
  int upto = ctas;  // CTAs of this lane's sequences and all before
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(kFullMask, upto, o);
    if (lane >= o) upto += n;
  }
  const uint32_t mine = __ballot_sync(kFullMask, here >= upto - ctas && here < upto);
  if (mine == 0) return {0, 0, 0, 0};
  int b = from, at = upto - ctas, n = 0;
  if ((mine >> lane) & 1u)
    for (; n = parts_of(b), here >= at + n * rows_a_seq; ++b) at += n * rows_a_seq;
  const int owner = __ffs(mine) - 1;
  n = __shfl_sync(kFullMask, n, owner);
  const int i = here - __shfl_sync(kFullMask, at, owner), row = i / n;
  return {__shfl_sync(kFullMask, b, owner), row, i - row * n, n};
}

// kPacked: this CTA's sequence, its first row there and how many warps a row has.
struct Pack {
  int64_t b;
  int row, warps;  // warps == 0: the CTA has nothing
};
template <int T>
__device__ __forceinline__ Pack find_pack(const AttendArgs& a, const Shares& sh, int64_t most) {
  const int lane = threadIdx.x & 31, here = blockIdx.x;
  const int each = ((int)a.B + 31) / 32, from = min((int)a.B, lane * each), to = min((int)a.B, from + each);
  auto warps_of = [&](int b) {
    Span<T> span(a.lengths[b], most, 0);
    span.first = min(span.len, (uint32_t)max(0, sh.shared[b / sh.group_rows]));
    const int steps = span.steps();
    return max(sh.least_warps, steps <= sh.warp_steps ? 1 : steps <= 2 * sh.warp_steps ? 2 : 4);
  };
  auto ctas_of = [&](int b) { return (sh.rows_a_seq * warps_of(b) + kWarps - 1) / kWarps; };
  int ctas = 0;
  for (int b = from; b < to; ++b) ctas += ctas_of(b);
  int upto = ctas;  // CTAs of this lane's sequences and all before
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(kFullMask, upto, o);
    if (lane >= o) upto += n;
  }
  const uint32_t mine = __ballot_sync(kFullMask, here >= upto - ctas && here < upto);
  if (mine == 0) return {0, 0, 0};
  int b = from, at = upto - ctas;
  if ((mine >> lane) & 1u)
    for (int n; n = ctas_of(b), here >= at + n; ++b) at += n;
  const int owner = __ffs(mine) - 1;
  b = __shfl_sync(kFullMask, b, owner);
  const int warps = warps_of(b);
  return {b, (here - __shfl_sync(kFullMask, at, owner)) * (kWarps / warps), warps};
}

// The sequence that comes at place `at` when the longest is first (of equal ones, and
// beyond 2^24 tokens, the one with the lowest number).  A key holds length and number:
// one compare a pair of sequences.
__device__ __forceinline__ int64_t by_length(const AttendArgs& a, int at) {
  __shared__ __align__(16) int keys[kSortSeqs];
  __shared__ int found;
  const int B = (int)a.B, b = threadIdx.x;
  const int mine = b < B ? min(max(a.lengths[b], 0), 0xffffff) * kSortSeqs + (kSortSeqs - 1 - b) : -1;
  keys[b] = mine;
  __syncthreads();
  if (b < B) {
    int rank = 0;
    for (int i = 0; i < B; i += 4) {
      const int4 k = *reinterpret_cast<const int4*>(keys + i);
      rank += (k.x > mine) + (k.y > mine) + (k.z > mine) + (k.w > mine);
    }
    if (rank == at) found = b;
  }
  __syncthreads();
  return found;
}

// A head's sums of a lane's dims 4 lane .. 4 lane + 3 (and 128 more), under reference m.
template <int DT>
struct HeadSums {
  static constexpr int kTurns = (DT + 127) / 128;
  float4 v[kTurns];
  float m, sum;
};
// Adds the parts `first`, `first` + `every`, ... below `end` of a head, the first of which lies at p and the next ones
// `apart` floats on.  Parts on their way together: 8, or 4 of 256 dims.
template <int DT>
__device__ __forceinline__ void add_parts(HeadSums<DT>& t, const float* p, int64_t apart, int first, int every, int end, int D, int lane) {
  constexpr int kTurns = HeadSums<DT>::kTurns, kTogether = 8 / kTurns;
  for (int i = first; i < end; i += kTogether * every) {
    float2 s[kTogether];
    float4 x[kTogether][kTurns];
    float top = t.m;
#pragma unroll
    for (int n = 0; n < kTogether; ++n) {
      const bool have = i + n * every < end;
      const float* q = p + (i + n * every) * apart;
      s[n] = have ? *reinterpret_cast<const float2*>(q + D) : make_float2(kUnset, 0.0f);
#pragma unroll
      for (int k = 0; k < kTurns; ++k) {
        const int d = 4 * lane + 128 * k;
        x[n][k] = have && d < D ? *reinterpret_cast<const float4*>(q + d) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
      top = fmaxf(top, s[n].x);
    }
    const float down = exp2_of(t.m - top);
    t.m = top;
    t.sum *= down;
#pragma unroll
    for (int k = 0; k < kTurns; ++k) t.v[k] = make_float4(t.v[k].x * down, t.v[k].y * down, t.v[k].z * down, t.v[k].w * down);
#pragma unroll
    for (int n = 0; n < kTogether; ++n) {
      const float f = exp2_of(s[n].x - top);
      t.sum = fmaf(s[n].y, f, t.sum);
#pragma unroll
      for (int k = 0; k < kTurns; ++k) {
        t.v[k].x = fmaf(x[n][k].x, f, t.v[k].x);
        t.v[k].y = fmaf(x[n][k].y, f, t.v[k].y);
        t.v[k].z = fmaf(x[n][k].z, f, t.v[k].z);
        t.v[k].w = fmaf(x[n][k].w, f, t.v[k].w);
      }
    }
  }
}

// kOwn, kPacked: where the parts of what the sequence's group shares lie, of q head `lane` of the row's: the first
// part's floats and how many there are.
struct HeadParts {
  int64_t at;
  int n;
};
__device__ __forceinline__ HeadParts parts_of(const KvPages& c, const Shares& sh, int64_t b, int hk, int first_head, int heads, int lane) {
  const int64_t g = b / sh.group_rows;
  if (lane >= heads || sh.shared[g] <= 0) return {0, 0};  // nothing shared: no CTA had the group's rows
  const int of_group = (int)(b - g * sh.group_rows) * sh.heads_a_key + first_head + lane, tile = of_group / sh.prefix_heads;
  const int2 row = sh.rows[(g * c.heads + hk) * sh.prefix_tiles + tile];
  return {((int64_t)row.x * sh.slot_heads + of_group - tile * sh.prefix_heads) * (c.head_dim + 4), row.y};
}

// kOwn: adds the parts `first`, `first` + `every`, ... to a warp's own partials at `at`.
template <int PARTIAL, int DT>
__device__ __forceinline__ void add_prefix(const KvPages& c, const Shares& sh, const HeadParts& of, int heads, int first, int every,
                                           uint32_t at, int lane) {
  const int D = c.head_dim;
  for (int h = 0; h < heads; ++h) {
    const int64_t p = __shfl_sync(kFullMask, of.at, h);
    const int n = __shfl_sync(kFullMask, of.n, h);
    const uint32_t mine = at + h * PARTIAL;
    HeadSums<DT> t;
    const float2 own = lds_float2(mine + 4 * DT);
    t.m = own.x;
    t.sum = own.y;
#pragma unroll
    for (int k = 0; k < t.kTurns; ++k) {
      const int d = 4 * lane + 128 * k;
      t.v[k] = d < D ? lds_float4(mine + 4 * d) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    add_parts<DT>(t, sh.parts + p, (int64_t)sh.slot_heads * (D + 4), first, every, n, D, lane);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < t.kTurns; ++k) {
      const int d = 4 * lane + 128 * k;
      if (d < D)
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(mine + 4 * d), "f"(t.v[k].x), "f"(t.v[k].y), "f"(t.v[k].z), "f"(t.v[k].w) : "memory");
    }
    if (lane == 0) {
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(mine + 4 * DT), "f"(t.m) : "memory");
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(mine + 4 * DT + 4), "f"(t.sum) : "memory");
    }
  }
}

// kPacked: a row's output.  A head is a warp's: its parts, then the own partials of the row's warps, at `at` and
// `apart` bytes on.
template <int PARTIAL, int DT>
__device__ __forceinline__ void finish_packed(const KvPages& c, const Shares& sh, const HeadParts& of, int heads, int me, int warps,
                                              uint32_t at, int apart, float* out, int lane) {
  const int D = c.head_dim;
  for (int h = me; h < heads; h += warps) {
    HeadSums<DT> t;
    t.m = kUnset;
    t.sum = 0.0f;
#pragma unroll
    for (int k = 0; k < t.kTurns; ++k) t.v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    add_parts<DT>(t, sh.parts + __shfl_sync(kFullMask, of.at, h), (int64_t)sh.slot_heads * (D + 4), 0, 1, __shfl_sync(kFullMask, of.n, h), D, lane);
    for (int w = 0; w < warps; ++w) {
      const uint32_t own = at + w * apart + h * PARTIAL;
      const float2 s = lds_float2(own + 4 * DT);
      const float top = fmaxf(t.m, s.x), down = exp2_of(t.m - top), f = exp2_of(s.x - top);
      t.m = top;
      t.sum = fmaf(s.y, f, t.sum * down);
#pragma unroll
      for (int k = 0; k < t.kTurns; ++k) {
        const int d = 4 * lane + 128 * k;
        const float4 x = d < D ? lds_float4(own + 4 * d) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        t.v[k] = make_float4(fmaf(x.x, f, t.v[k].x * down), fmaf(x.y, f, t.v[k].y * down), fmaf(x.z, f, t.v[k].z * down), fmaf(x.w, f, t.v[k].w * down));
      }
    }
#pragma unroll
    for (int k = 0; k < t.kTurns; ++k) {
      const int d = 4 * lane + 128 * k;
      if (d < D) {
        float* to = out + h * D + d;
        to[0] = output_of(t.v[k].x, t.m, t.sum);
        to[1] = output_of(t.v[k].y, t.m, t.sum);
        to[2] = output_of(t.v[k].z, t.m, t.sum);
        to[3] = output_of(t.v[k].w, t.m, t.sum);
      }
    }
  }
}

// Rows of `splits` CTAs each, a cluster but in kPrefix, or (sh.rows given) of CTAs in proportion to their steps.
template <int FORMAT, int DT, Mode MODE>
__global__ void __launch_bounds__(kThreads, Shape<FORMAT, DT>::kCtas)
attend_kernel(AttendArgs a, KvPages c, Shares sh) {
  using S = Shape<FORMAT, DT>;
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr bool kCluster = MODE == kClusters || MODE == kBlocks || MODE == kOwn;
  if constexpr (MODE != kPrefix) pdl_release_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, qd = lane & 3;
  const int group = sh.group, rows_a_seq = sh.rows_a_seq;
  const int D = c.head_dim;
  const int64_t most = MODE == kBlocks ? (int64_t)sh.count << c.page_shift : a.max_pages << c.page_shift;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * S::kWarpBytes;
  if (D < DT) {  // the padding of every row, once: copies never write it
    for (int i = lane; i < S::kWarpBytes / 16; i += 32)
      reinterpret_cast<uint4*>(smem + warp * S::kWarpBytes)[i] = make_uint4(0, 0, 0, 0);
    __syncwarp();
  }
  if (kCluster && sh.splits > 1) cluster_arrive();  // waited for before the first word goes to another CTA
  // kOwn, kPacked: begun when every CTA of the shared tokens' kernel has waited for what was before; its parts are
  // waited for where they are added.
  if constexpr (MODE != kOwn && MODE != kPacked) pdl_wait_primary();
  if constexpr (MODE == kPrefix) pdl_release_dependents();

  // The CTA's row (sequence b, head `row` of its key heads and groups of q heads)
  // and its place among the row's CTAs.
  int64_t b;
  int row, split, splits, row_warps = kWarps;
  if (MODE == kSharedOut || (MODE == kPrefix && sh.splits == 0)) {
    const Part p = find_part<S::kTokens>(a, most, rows_a_seq);
    if (p.parts == 0) return;
    b = p.b;
    row = p.row;
    split = p.part;
    splits = p.parts;
    if (split == 0 && threadIdx.x == 0) sh.rows[b * rows_a_seq + row] = make_int2(blockIdx.x, splits);
  } else if constexpr (MODE == kPacked) {
    const Pack p = find_pack<S::kTokens>(a, sh, most);
    row_warps = p.warps;
    if (row_warps == 0) return;
    b = p.b;
    row = p.row + warp / row_warps;
    if (row >= rows_a_seq) return;  // whole rows' warps: nobody waits for them
    split = 0;
    splits = 1;
  } else {
    splits = sh.splits;
    split = blockIdx.x & (splits - 1);
    const uint32_t rest = blockIdx.x >> sh.splits_log2, place = rest / (uint32_t)rows_a_seq;
    row = (int)(rest - place * rows_a_seq);
    b = MODE == kClusters && sh.sorted ? by_length(a, (int)place) : sh.b0 + place;
    if (MODE == kPrefix && split == 0 && threadIdx.x == 0) sh.rows[b * rows_a_seq + row] = make_int2(blockIdx.x, splits);
  }

  constexpr bool kBehind = MODE == kOwn || MODE == kPacked;  // tokens behind the shared ones
  const int workers = splits * row_warps, first_warp = MODE == kPacked ? warp & ~(row_warps - 1) : 0, me = split * row_warps + warp - first_warp;
  // the warps of a row meet
  auto meet = [&]() {
    if (MODE != kPacked || row_warps == kWarps)
      __syncthreads();
    else if (row_warps == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, 64;" ::"r"(1 + warp / 2) : "memory");
  };
  const int hk = sh.groups == 1 ? row : row / sh.groups, first_of_group = (row - hk * sh.groups) * kRowHeads;
  const int heads = min(kRowHeads, group - first_of_group), hq = hk * group + first_of_group;
  // q of the row's heads, on its way while the pages are looked up: 0.2 us of the smallest
  // calls, 1 to 3 % of full ones.  One warp splits it for all.
  constexpr bool kBf16 = FORMAT == BITLINEAR_KV_BF16;
  // kPrefix: row g is q head `in_key` of the key head's, of the group's sequence `member`
  const uint32_t of_group = MODE == kPrefix ? first_of_group + min(g, heads - 1) : 0;
  const uint32_t member = MODE == kPrefix ? of_group / (uint32_t)sh.heads_a_key : 0, in_key = of_group - member * sh.heads_a_key;
  float2 qx[S::kSteps], qy[S::kSteps];
  if (MODE == kPacked || warp == 0) {
    const float* q = MODE == kPrefix ? a.q + (b * sh.group_rows + member) * a.q_stride + (int64_t)(hk * sh.heads_a_key + in_key) * D
                                     : a.q + b * a.q_stride + (int64_t)(hq + min(g, heads - 1)) * D;
#pragma unroll
    for (int s = 0; s < S::kSteps; ++s) {
      // 8-bit: dims 4 qd .. 4 qd + 3 of the k-step (one word); bf16: dims 2 qd, 2 qd + 1 and 8 more
      const int d0 = 16 * s + (kBf16 ? 2 : 4) * qd, d1 = kBf16 ? d0 + 8 : d0 + 2;
      qx[s] = d0 < D ? *reinterpret_cast<const float2*>(q + d0) : make_float2(0.0f, 0.0f);
      qy[s] = d1 < D ? *reinterpret_cast<const float2*>(q + d1) : make_float2(0.0f, 0.0f);
    }
  }

  // The warp's steps are every (splits * kWarps)-th one of the row's.
  const int32_t* table = a.table + b * a.table_stride;
  const uint32_t columns = (uint32_t)(most < 0x7fffffff ? most : 0x7fffffff);  // tokens that the table has room for
  int32_t page[2] = {-1, -1};
  // kBlocks: tokens are counted along the list; a list's page may end a sequence, so each half of
  // a step has a number of rows that count
  const int32_t* list = MODE == kBlocks ? sh.blocks + (b * c.heads + hk) * sh.count : nullptr;
  const int64_t there = MODE == kBlocks ? max((int64_t)0, min((int64_t)a.lengths[b], a.max_pages << c.page_shift)) : 0;
  int left[2] = {0, 0};
  auto look_up_listed = [&](uint32_t t, int s) {
    page[s] = -1;
    left[s] = 0;
    if (t >= columns) return;
    const int64_t column = list[t >> c.page_shift];
    if (column < 0 || column >= a.max_pages) return;
    left[s] = (int)max((int64_t)0, min((int64_t)16, there - (column << c.page_shift) - (t & ((1u << c.page_shift) - 1))));
    if (left[s] > 0) page[s] = table[column];
  };
  auto look_up = [&](uint32_t t) {  // the pages of the step at t (columns of the table, whatever the length)
    if constexpr (MODE == kBlocks) {
      look_up_listed(t, 0);
      if constexpr (S::kTokens == 32) look_up_listed(t + 16, 1);
      return;
    }
    page[0] = t < columns ? table[t >> c.page_shift] : -1;
    if constexpr (S::kTokens == 32) {
      page[1] = page[0];
      if (c.page_shift == 4) page[1] = t + 16 < columns ? table[(t + 16) >> 4] : -1;
    }
  };
  const uint32_t lap = (uint32_t)workers * S::kTokens;
  uint32_t t_ask = (uint32_t)me * S::kTokens;
  if (!kBehind && a.window <= 0) look_up(t_ask);  // the first page is known before the length
  Span<S::kTokens> span(MODE == kBlocks ? 0 : a.lengths[b], most, a.window);
  if constexpr (MODE == kBlocks) span.len = (uint32_t)most;
  if constexpr (kBehind) span.first = min(span.len, (uint32_t)max(0, sh.shared[b / sh.group_rows]));
  if (kBehind || a.window > 0) {
    t_ask += span.begin();
    look_up(t_ask);
  }
  Source r;
  const int64_t head_row = (int64_t)hk << c.page_shift;
  r.k = static_cast<const uint8_t*>(c.k) + head_row * D * S::kBytes;
  r.v = static_cast<const uint8_t*>(c.v) + head_row * D * S::kBytes;
  r.ks = c.k_step + head_row;
  r.vs = c.v_step + head_row;
  r.first = span.first;
  r.len = span.len;
  uint32_t t0 = t_ask;  // the step in hand
  // kPrefix: tokens end with the group's longest sequence, and a row's with its own
  uint32_t row_end = r.len, rows_end = r.len;
  if constexpr (MODE == kPrefix) {
    int longest = 0;
    for (int i = lane; i < sh.group_rows; i += 32) longest = max(longest, sh.lengths[b * sh.group_rows + i]);
    r.len = min(r.len, (uint32_t)__reduce_max_sync(kFullMask, longest));
    row_end = min(r.len, (uint32_t)max(0, sh.lengths[b * sh.group_rows + member]));
    rows_end = __reduce_min_sync(kFullMask, row_end);
  }

  uint32_t lefts = 0;  // kBlocks: a byte a half of a requested step, the newest lowest
  uint32_t oks = 0;  // two bits a requested step (its halves have pages), the newest lowest
  uint32_t ask_at = ring;
  auto ask = [&]() {  // requests the step at t_ask into the next stage and looks the one after up
    oks <<= 2;
    if constexpr (MODE == kBlocks) lefts = lefts << 16 | (uint32_t)left[0] | (uint32_t)left[1] << 8;
    if (t_ask < r.len) {
      int64_t place[2] = {0, 0};
      uint32_t ok = 0;
#pragma unroll
      for (int s = 0; s < S::kTokens / 16; ++s) {
        if (t_ask + 16 * s < r.len && (uint32_t)page[s] < (uint32_t)c.num_pages) {
          ok |= 1u << s;
          place[s] = (((int64_t)page[s] * c.heads) << c.page_shift) + ((t_ask + 16 * s) & ((1u << c.page_shift) - 1));
        }
      }
      oks |= ok;
      const bool all = MODE == kBlocks ? (left[0] == 16 && (S::kTokens == 16 || left[1] == 16))
                                       : (t_ask >= r.first && t_ask + S::kTokens <= r.len);
      if (D == DT && ok == (S::kTokens == 32 ? 3u : 1u) && all)
        request_whole<FORMAT, DT>(r, place, ask_at, lane);
      else
        request_part<FORMAT, DT, MODE == kBlocks>(r, c, t_ask, place, ok, ask_at, lane, left);
    }
    copies_commit();
    t_ask += lap;
    look_up(t_ask);
    ask_at = ask_at == ring + (kStages - 1) * S::kStage ? ring : ask_at + S::kStage;
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) ask();

  // q as the MMA's A operand: rows g the leading parts of head g, rows g + 8 the
  // next, the dims of a k-step in the order the key words give them.  Kept in shared
  // memory behind the rings and read again in every step: in registers it was 20 to 64
  // of them a thread, a CTA less an SM, and spills.
  // kPacked: each warp has parts of its own.
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem);
  const uint32_t q_area = base + (uint32_t)S::kSmem + (MODE == kPacked ? warp * (min(kRowHeads, group) * S::kHeadBytes + kRowHeads * 4) : 0);
  const uint32_t thirds = q_area + S::kSteps * heads * 64, q_scales = q_area + heads * S::kHeadBytes;
  if (MODE == kPacked || warp == 0) {
    // scale log2(e) is a pair: its second part goes into q's last, so a row's logits have no
    // rounding of it in common
    const float factor = a.factor, more = a.factor_rest;
    float v[S::kSteps][4], top = 0.0f;
#pragma unroll
    for (int s = 0; s < S::kSteps; ++s) {
      v[s][0] = qx[s].x * factor; v[s][1] = qx[s].y * factor; v[s][2] = qy[s].x * factor; v[s][3] = qy[s].y * factor;
#pragma unroll
      for (int j = 0; j < 4; ++j) top = fmaxf(top, fabsf(v[s][j]));
    }
    float down = 1.0f, up = 1.0f;
    if constexpr (!kBf16) {
      top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 2));
      const int e = clamp_exponent(exponent_of(top));
      up = power2(e);
      down = power2(-e);
    }
    if (g < heads) {
      const uint32_t to = q_area + (g * 4 + qd) * 16, to_third = thirds + (g * 4 + qd) * 8;
#pragma unroll
      for (int s = 0; s < S::kSteps; ++s) {
        uint4 w;
        if constexpr (!kBf16) {
          split2<true>(v[s][0] * down, v[s][1] * down, w.x, w.y, more * 2048.0f);
          split2<true>(v[s][2] * down, v[s][3] * down, w.z, w.w, more * 2048.0f);
        } else {
          uint2 third;
          const float2 x = mul2(make_float2(v[s][0], v[s][1]), both(more)), y = mul2(make_float2(v[s][2], v[s][3]), both(more));
          w.x = next_part(v[s][0], v[s][1]); w.y = next_part(v[s][0], v[s][1]);
          w.z = next_part(v[s][2], v[s][3]); w.w = next_part(v[s][2], v[s][3]);
          v[s][0] += x.x; v[s][1] += x.y; v[s][2] += y.x; v[s][3] += y.y;
          third.x = next_part(v[s][0], v[s][1]); third.y = next_part(v[s][2], v[s][3]);
          asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(to_third + s * (heads * 32)), "r"(third.x), "r"(third.y) : "memory");
        }
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + s * (heads * 64)), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
      }
      if (qd == 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(q_scales + 4 * g), "f"(up) : "memory");
    }
  }
  if constexpr (MODE == kPacked)
    __syncwarp();
  else
    __syncthreads();
  const uint32_t q_lane = min(g, heads - 1) * 4 + qd, q_stride = heads * 64;  // [k-step][head][lane]: no bank twice
  const float row_scale = lds_float(q_scales + 4 * min(g, heads - 1));

  float ref = kUnset;                                  // of row g
  float2 sums = both(0.0f);                            // over this lane's tokens, the even and the odd ones
  float2 out[S::kOutTiles];                            // row g: dims 2 qd, 2 qd + 1 of every n-tile (in the tiles' order)
#pragma unroll
  for (int n = 0; n < S::kOutTiles; ++n) out[n] = both(0.0f);
  constexpr float kRest = kBf16 ? 1.0f : 1.0f / 2048.0f;

  for (uint32_t st = ring; t0 < r.len; t0 += lap, st = st == ring + (kStages - 1) * S::kStage ? ring : st + S::kStage) {
    // The next step is asked for once this one has come, into the stage that the last one
    // has left: one meeting of the warp a step.  Asked for before the wait (a second
    // meeting): 51.2 for 47.4 us on 64 x 2048 tokens of 8 key heads e4m3, 47.6 for 45.8 on
    // 32 x 2048 bf16; with the GPU full several times 159.0 for 161.0 (456 x 1024, e4m3).
    copies_wait<0>();
    __syncwarp();
    ask();
    if (MODE == kBlocks && ((oks >> (2 * (kStages - 1))) & 3u) == 0) continue;  // a list's unused place
    const uint32_t vst = st + S::kTokens * S::kRow, kst = vst + S::kTokens * S::kRow;

    // where this lane's words are: keys of row g, chunk 0; values of row 2 qd, chunk g / 4
    const uint32_t key_at = st + S::place(g, 0) + 4 * qd, value_at = vst + S::place(2 * qd, g >> 2) + 4 * (g & 3);
    auto in_row = [](uint32_t at, int chunk) {  // the same place of a row, `chunk` (a constant) chunks on
      constexpr int kMask = (1 << S::kTurn) - 1;
      return (at ^ ((chunk & kMask) * 16)) + (chunk & ~kMask) * 16;
    };
    float x[S::kTiles][4];
#pragma unroll
    for (int s = 0; s < S::kSteps; ++s) {
      const uint4 w = lds128(q_area + q_lane * 16 + s * q_stride);
      const uint32_t qa[4] = {w.x, w.y, w.z, w.w};
      uint32_t third[4] = {0u, 0u, 0u, 0u};
      if constexpr (kBf16) {
        third[1] = lds32(thirds + q_lane * 8 + s * (q_stride / 2));
        third[3] = lds32(thirds + q_lane * 8 + s * (q_stride / 2) + 4);
      }
#pragma unroll
      for (int j = 0; j < S::kTiles; ++j) {
        uint32_t k0, k1;
        const uint32_t rows = 8 * j * S::kRow;
        if constexpr (kBf16) {
          k0 = lds32(in_row(key_at, 2 * s) + rows);
          k1 = lds32(in_row(key_at, 2 * s + 1) + rows);
        } else {
          widen<FORMAT>(lds32(in_row(key_at, s) + rows), k0, k1);
        }
        if (s == 0)
          mma<FORMAT, true>(x[j], qa, k0, k1);
        else
          mma<FORMAT, false>(x[j], qa, k0, k1);
        if constexpr (kBf16) mma<FORMAT, false>(x[j], third, k0, k1);
      }
    }

    // logits of row g (times 1 / row_scale), tokens 8 j + 2 qd and the next
    float2 lg[S::kTiles], p[S::kTiles], w[S::kTiles];
#pragma unroll
    for (int j = 0; j < S::kTiles; ++j) {
      lg[j] = fma2(make_float2(x[j][2], x[j][3]), both(kRest), make_float2(x[j][0], x[j][1]));
      if constexpr (!kBf16) {
        lg[j] = mul2(lg[j], lds_float2(kst + (8 * j + 2 * qd) * 4));
      }
    }
    const uint32_t ok = (oks >> (2 * (kStages - 1))) & 3u;
    if constexpr (MODE == kBlocks) {
      const uint32_t counts = lefts >> (16 * (kStages - 1));
      if (ok != (S::kTokens == 32 ? 3u : 1u) || (counts & 0xffffu) != (S::kTokens == 32 ? 0x1010u : 0x10u)) {
#pragma unroll
        for (int j = 0; j < S::kTiles; ++j) {
          const int n = 8 * (j & 1) + 2 * qd, have = (ok >> (j / 2)) & 1u ? (int)((counts >> (8 * (j / 2))) & 0xffu) : 0;
          if (n >= have) lg[j].x = -INFINITY;
          if (n + 1 >= have) lg[j].y = -INFINITY;
        }
      }
    } else if (ok != (S::kTokens == 32 ? 3u : 1u) || t0 < r.first || t0 + S::kTokens > (MODE == kPrefix ? rows_end : r.len)) {
      const uint32_t end = MODE == kPrefix ? row_end : r.len;
#pragma unroll
      for (int j = 0; j < S::kTiles; ++j) {
        const uint32_t t = t0 + 8 * j + 2 * qd;
        const bool have = (ok >> (j / 2)) & 1u;
        if (!have || t < r.first || t >= end) lg[j].x = -INFINITY;
        if (!have || t + 1 < r.first || t + 1 >= end) lg[j].y = -INFINITY;
      }
    }
    // p and its weights (p times the value's step); `high` the largest
    auto weights = [&](float& high) {
#pragma unroll
      for (int j = 0; j < S::kTiles; ++j) {
        const float2 z = fma2(lg[j], both(row_scale), both(-ref));
        p[j] = make_float2(exp2_of(z.x), exp2_of(z.y));
        w[j] = p[j];
        if constexpr (!kBf16) {
          const float2 step = lds_float2(kst + (S::kTokens + 8 * j + 2 * qd) * 4);
          w[j] = mul2(w[j], make_float2(at_least(step.x, kLeastStep), at_least(step.y, kLeastStep)));
        }
        high = fmaxf(high, fmaxf(w[j].x, w[j].y));
      }
    };
    float high = 0.0f;
    weights(high);
    if (__any_sync(kFullMask, high > kLimit)) {
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < S::kTiles; ++j) {
        float2 z = make_float2(lg[j].x * row_scale, lg[j].y * row_scale);
        if constexpr (!kBf16) {
          const float2 step = lds_float2(kst + (S::kTokens + 8 * j + 2 * qd) * 4);
          z.x += log2_of(fmaxf(step.x, kLeastStep));
          z.y += log2_of(fmaxf(step.y, kLeastStep));
        }
        top = fmaxf(top, fmaxf(z.x, z.y));
      }
      top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 2));
      if (top > ref) {
        const float f = exp2_of(ref - top);  // 0 from the first reference
        ref = top;
        sums = mul2(sums, both(f));
#pragma unroll
        for (int n = 0; n < S::kOutTiles; ++n) {
          out[n] = mul2(out[n], both(f));
        }
      }
      weights(high);
    }
#pragma unroll
    for (int j = 0; j < S::kTiles; ++j) sums = add2(sums, p[j]);

    // the weights as the A operand: token pairs of tiles 2 kk, 2 kk + 1
    uint32_t pa[S::kTokens / 16][4], pb[kBf16 ? S::kTokens / 16 : 1][2];
#pragma unroll
    for (int kk = 0; kk < S::kTokens / 16; ++kk) {
      if constexpr (kBf16) {
        pa[kk][0] = next_part(w[2 * kk].x, w[2 * kk].y);
        pa[kk][1] = next_part(w[2 * kk].x, w[2 * kk].y);
        pb[kk][0] = next_part(w[2 * kk].x, w[2 * kk].y);
        pa[kk][2] = next_part(w[2 * kk + 1].x, w[2 * kk + 1].y);
        pa[kk][3] = next_part(w[2 * kk + 1].x, w[2 * kk + 1].y);
        pb[kk][1] = next_part(w[2 * kk + 1].x, w[2 * kk + 1].y);
      } else {
        split2(w[2 * kk].x, w[2 * kk].y, pa[kk][0], pa[kk][1]);
        split2(w[2 * kk + 1].x, w[2 * kk + 1].y, pa[kk][2], pa[kk][3]);
      }
    }

    // weighted sums: a word of 4 tokens gives the B operands of as many n-tiles as it
    // holds dims; n-tile i of a group takes dim (dims a word) * g + i
    constexpr int kWide = kBf16 ? 2 : 4;             // dims a word
    constexpr int kGroups = DT / (8 * kWide);
    auto add = [&](int n, const float (&t)[4]) {
      out[n] = add2(out[n], fma2(make_float2(t[2], t[3]), both(kRest), make_float2(t[0], t[1])));
    };
#pragma unroll
    for (int dg = 0; dg < kGroups; ++dg) {
      float t[kWide][4];
#pragma unroll
      for (int kk = 0; kk < S::kTokens / 16; ++kk) {
        const uint32_t even = in_row(value_at, 2 * dg) + 16 * kk * S::kRow;  // row 2 qd; the next one's last bit is turned
        const uint32_t odd = in_row(S::kTurn ? value_at ^ 16 : value_at, 2 * dg) + (16 * kk + S::kNext) * S::kRow;
        uint32_t w[4] = {lds32(even), lds32(odd), lds32(even + 8 * S::kRow), lds32(odd + 8 * S::kRow)};
        if constexpr (kBf16) {
          const uint32_t third[4] = {0u, pb[kk][0], 0u, pb[kk][1]};
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const uint32_t sel = n ? 0x7632 : 0x5410;
            const uint32_t v0 = __byte_perm(w[0], w[1], sel), v1 = __byte_perm(w[2], w[3], sel);
            if (kk == 0)
              mma<FORMAT, true>(t[n], pa[kk], v0, v1);
            else
              mma<FORMAT, false>(t[n], pa[kk], v0, v1);
            mma<FORMAT, false>(t[n], third, v0, v1);
          }
        } else {
#pragma unroll
          for (int n = 0; n < 4; n += 2) {
            uint32_t v0[2], v1[2];  // bytes n, n + 1 of both tokens of a pair, side by side
            widen<FORMAT>(__byte_perm(w[0], w[1], n ? 0x7362 : 0x5140), v0[0], v0[1]);
            widen<FORMAT>(__byte_perm(w[2], w[3], n ? 0x7362 : 0x5140), v1[0], v1[1]);
            if (kk == 0) {
              mma<FORMAT, true>(t[n], pa[kk], v0[0], v1[0]);
              mma<FORMAT, true>(t[n + 1], pa[kk], v0[1], v1[1]);
            } else {
              mma<FORMAT, false>(t[n], pa[kk], v0[0], v1[0]);
              mma<FORMAT, false>(t[n + 1], pa[kk], v0[1], v1[1]);
            }
          }
        }
      }
#pragma unroll
      for (int n = 0; n < kWide; ++n) add(kWide * dg + n, t[n]);
    }
    if constexpr (!kBf16 && DT % 32 == 16) {  // the last 16 dims: two a token, n-tile i takes dim 2 g + i
      constexpr int n0 = S::kOutTiles - 2;
      float t[2][4];
#pragma unroll
      for (int kk = 0; kk < S::kTokens / 16; ++kk) {
        const uint32_t row = vst + (16 * kk + 2 * qd) * S::kRow + (DT - 16) + 2 * g;
        const uint32_t w0 = lds16(row), w1 = lds16(row + S::kRow), w2 = lds16(row + 8 * S::kRow), w3 = lds16(row + 9 * S::kRow);
        uint32_t v0[2], v1[2];
        widen<FORMAT>(__byte_perm(w0, w1, 0x5140), v0[0], v0[1]);
        widen<FORMAT>(__byte_perm(w2, w3, 0x5140), v1[0], v1[1]);
        if (kk == 0) {
          mma<FORMAT, true>(t[0], pa[kk], v0[0], v1[0]);
          mma<FORMAT, true>(t[1], pa[kk], v0[1], v1[1]);
        } else {
          mma<FORMAT, false>(t[0], pa[kk], v0[0], v1[0]);
          mma<FORMAT, false>(t[1], pa[kk], v0[1], v1[1]);
        }
      }
      add(n0, t[0]);
      add(n0 + 1, t[1]);
    }
  }
  copies_wait<0>();
  __syncwarp();

  // The warp's partials over its ring: [head][dims, m, sum].
  float sum = sums.x + sums.y;
  sum += __shfl_xor_sync(kFullMask, sum, 1);
  sum += __shfl_xor_sync(kFullMask, sum, 2);
  float* part = reinterpret_cast<float*>(smem + warp * S::kWarpBytes + g * S::kPartial);
  constexpr int kWideOut = kBf16 ? 2 : 4;
#pragma unroll
  for (int n = 0; n < S::kOutTiles; ++n) {
    const bool tail = !kBf16 && DT % 32 == 16 && n >= S::kOutTiles - 2;
    const int wide = tail ? 2 : kWideOut, first = tail ? DT - 16 : n / kWideOut * 8 * kWideOut;
    const int of = tail ? n - (S::kOutTiles - 2) : n % kWideOut;
    part[first + wide * (2 * qd) + of] = out[n].x;
    part[first + wide * (2 * qd + 1) + of] = out[n].y;
  }
  if (qd == 0) {
    part[DT] = ref;
    part[DT + 1] = sum;
  }
  if constexpr (MODE == kPacked) {
    meet();
    pdl_wait_primary();
    finish_packed<S::kPartial, DT>(c, sh, parts_of(c, sh, b, hk, first_of_group, heads, lane), heads, me, row_warps, base + first_warp * S::kWarpBytes,
                                   S::kWarpBytes, a.out + b * a.out_stride + (int64_t)hq * D, lane);
    return;
  }
  if constexpr (MODE == kOwn) {
    __syncwarp();
    pdl_wait_primary();
    add_prefix<S::kPartial, DT>(c, sh, parts_of(c, sh, b, hk, first_of_group, heads, lane), heads, me, workers, base + warp * S::kWarpBytes, lane);
  }
  __syncthreads();

  auto of_warps = [&](int h, int d) {
    const uint32_t p = base + h * S::kPartial;
    return join<kWarps>(p + 4 * d, S::kWarpBytes, p + 4 * DT, S::kWarpBytes, kWarps);
  };
  auto head_of = [&](int i) { return heads == 1 ? 0 : (int)((uint32_t)i / (uint32_t)D); };
  auto finish = [&](int h, int d, const Joined& j) {
    a.out[b * a.out_stride + (int64_t)(hq + h) * D + d] = output_of(j.value, j.m, j.sum);
  };
  if (MODE == kSharedOut || MODE == kPrefix || splits == 1) {
    const bool whole = MODE != kPrefix && splits == 1;
    float* part = whole ? nullptr : sh.parts + (int64_t)blockIdx.x * min(kRowHeads, group) * (D + 4);
    for (int i = threadIdx.x; i < heads * D; i += kThreads) {
      const int h = head_of(i), d = i - h * D;
      const Joined j = of_warps(h, d);
      if (whole) {
        finish(h, d, j);
      } else {
        part[h * (D + 4) + d] = j.value;
        if (d == 0) *reinterpret_cast<float2*>(part + h * (D + 4) + D) = make_float2(j.m, j.sum);
      }
    }
    return;
  }
  // Every CTA sends each of the cluster its share of the dims, then joins its own.
  const int share = (heads * D + splits - 1) >> sh.splits_log2;
  const uint32_t values = q_scales + kRowHeads * 4, scales = values + (splits * share + 1) / 2 * 8;
  cluster_wait();  // all of the cluster's CTAs have begun
  for (int i = threadIdx.x; i < heads * D; i += kThreads) {
    const int h = head_of(i), d = i - h * D;
    const Joined j = of_warps(h, d);
    sts_cluster(values + (split * share + (i >> sh.splits_log2)) * 4, i & (splits - 1), j.value);
    if (d < splits) {  // dim r's thread tells CTA r (16 dims at least, 16 CTAs at most)
      sts_cluster(scales + (split * heads + h) * 8, d, j.m);
      sts_cluster(scales + (split * heads + h) * 8 + 4, d, j.sum);
    }
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  for (int n = threadIdx.x; n < share; n += kThreads) {
    const int i = n * splits + split;
    if (i >= heads * D) break;
    const int h = head_of(i);
    const uint32_t value = values + 4 * n, scale = scales + 8 * h;
    finish(h, i - h * D, splits > 8 ? join<16>(value, 4 * share, scale, 8 * heads, splits)
                                    : join<8>(value, 4 * share, scale, 8 * heads, splits));
  }
}

// CTAs of a cluster: a power of two up to `most`, while all CTAs are resident at once and
// every warp may have a step, or two from 16 CTAs on.  (One sequence, 8 / 16 CTAs at most, us:
// 8192 tokens of 32 heads of 80, int8 15.5 / 14.3; 4096 of 8 key heads bf16 10.1 / 8.9, of one
// e4m3 8.9 / 7.1; a step a warp: 2048 of 32 heads 5.8 / 6.0, 1024 of one key head 5.7 / 5.5.)
int splits_for(int64_t rows, int64_t steps, int ctas, int most) {
  int s = 1;
  while (s < most && rows * s * 2 <= ctas && steps >= (s >= 8 ? 4 : 2) * s * kWarps) s *= 2;
  return s;
}

// ---------------------------------------------------------------- host side

// Allows a kernel the most shared memory that any of its calls takes.
template <typename S, typename Kernel>
cudaError_t allow_shared_memory(Kernel kernel) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kMostShared);
}
// The same for a kernel of clusters, and how large they may be: kMaxCluster where the device schedules one.
template <typename S, typename Kernel>
cudaError_t allow_clusters(Kernel kernel, int* most_cluster) {
  const cudaError_t err = allow_shared_memory<S>(kernel);
  if (err != cudaSuccess) return err;
  *most_cluster = kPortableCluster;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {kMaxCluster, 1, 1};
  cfg.gridDim = dim3(kMaxCluster, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = S::kMostShared;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int fit = 0;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
      cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg) == cudaSuccess && fit > 0)
    *most_cluster = kMaxCluster;
  else
    cudaGetLastError();  // not this call's: the smaller size always runs
  return cudaSuccess;
}

// CTAs resident at once, of so much dynamic shared memory each.
template <typename S>
int resident_ctas(const DeviceInfo& dev, int smem) {
  const int fit = (int)(dev.smem_per_sm / (smem + kOtherSmem));
  return (dev.num_sms < kSms ? dev.num_sms : kSms) * (fit < S::kCtas ? fit : S::kCtas);
}

inline void set_factor(AttendArgs& a) {  // scale log2(e), to the base of the weights
  const double factor = (double)a.scale * 1.4426950408889634;
  a.factor = (float)factor;
  a.factor_rest = (float)(a.factor != 0.0f ? factor / a.factor - 1.0 : 0.0);
}

// `a_seq` CTAs a sequence, in clusters of `cluster`, in launches of as many sequences as a grid holds.
template <typename Kernel>
cudaError_t launch_grids(Kernel kernel, const AttendArgs& a, const KvPages& c, Shares sh, int64_t a_seq, int cluster, int smem, bool pdl,
                         cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  const int64_t per_launch = (int64_t)0x7fffffff / a_seq;  // sequences a grid holds
  for (sh.b0 = 0; sh.b0 < a.B; sh.b0 += per_launch) {
    const int64_t n = a.B - sh.b0 < per_launch ? a.B - sh.b0 : per_launch;
    cfg.gridDim = dim3((unsigned)(n * a_seq), 1, 1);
    cfg.numAttrs = 0;
    if (cluster > 1) {
      attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
      attr[cfg.numAttrs].val.clusterDim.x = (unsigned)cluster;
      attr[cfg.numAttrs].val.clusterDim.y = 1;
      attr[cfg.numAttrs].val.clusterDim.z = 1;
      ++cfg.numAttrs;
    }
    if (pdl) {
      attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
      ++cfg.numAttrs;
    }
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, a, c, sh);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

// sh.splits CTAs a row, a cluster.
template <int FORMAT, int DT, Mode MODE>
cudaError_t launch_clusters(const AttendArgs& a, const KvPages& c, const Shares& sh, int smem, bool pdl, cudaStream_t stream) {
  return launch_grids(attend_kernel<FORMAT, DT, MODE>, a, c, sh, (int64_t)sh.rows_a_seq * sh.splits, sh.splits, smem, pdl, stream);
}

// f(format, padded head size) of a cache, as constants.
template <typename F>
cudaError_t of_shape(const KvPages& c, F f) {
  auto of_dims = [&](auto format) {
    if (c.head_dim <= 64) return f(format, std::integral_constant<int, 64>());
    if (c.head_dim <= 80) return f(format, std::integral_constant<int, 80>());
    if (c.head_dim <= 96) return f(format, std::integral_constant<int, 96>());
    if (c.head_dim <= 112) return f(format, std::integral_constant<int, 112>());
    if (c.head_dim <= 128) return f(format, std::integral_constant<int, 128>());
    return f(format, std::integral_constant<int, 256>());
  };
  if (c.format == BITLINEAR_KV_INT8) return of_dims(std::integral_constant<int, BITLINEAR_KV_INT8>());
  if (c.format == BITLINEAR_KV_FP8) return of_dims(std::integral_constant<int, BITLINEAR_KV_FP8>());
  return of_dims(std::integral_constant<int, BITLINEAR_KV_BF16>());
}

}  // namespace
}  // namespace bitlinear
