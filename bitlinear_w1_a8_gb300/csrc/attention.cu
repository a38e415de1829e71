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
#include <cuda_bf16.h>
#include <cuda_fp16.h>

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
constexpr int kShareSeqs = 1024;  // sequences that a CTA adds up to find its row
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
template <int FORMAT, int DT>
__device__ __forceinline__ void request_part(const Source& r, const KvPages& c, uint32_t t0, const int64_t (&row)[2],
                                             uint32_t ok, uint32_t stage, int lane) {
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
      const bool there = have && t + n >= r.first && t + n < r.len;
      const int off = there ? n * row_bytes + 16 * ch : 0;
      copy16(kd + S::place(n, ch), k + off, there);
      copy16(vd + S::place(n, ch), v + off, there);
    }
    if constexpr (FORMAT != BITLINEAR_KV_BF16) {
      const int n = lane & 15;
      const bool there = have && t + n >= r.first && t + n < r.len;
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

// How rows are shared out.
struct Shares {
  int64_t b0;      // the launch's first sequence
  int group, groups, rows_a_seq;  // q heads a key head, groups of them, rows of a sequence
  int splits;      // CTAs a row where each has as many: a power of two
  int splits_log2;
  bool sorted;     // sequences in order of length, the longest first
  float* parts;    // rows shared out by their steps: [CTA][q heads of a row, at most 8][dims, m, sum]
  int2* rows;      // and a row's first CTA and how many it has
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
__device__ __forceinline__ Part find_part(const AttendArgs& a, int64_t most, int rows_a_seq) {
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
  const int share = share_of_steps(total, spare, kLeastSteps * kWarps);
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

// Rows of `splits` CTAs each, a cluster, or (SHARED_OUT) of CTAs in proportion to their steps.
template <int FORMAT, int DT, bool SHARED_OUT>
__global__ void __launch_bounds__(kThreads, Shape<FORMAT, DT>::kCtas)
attend_kernel(AttendArgs a, KvPages c, Shares sh) {
  using S = Shape<FORMAT, DT>;
  extern __shared__ __align__(128) uint8_t smem[];
  pdl_release_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, qd = lane & 3;
  const int group = sh.group, rows_a_seq = sh.rows_a_seq;
  const int D = c.head_dim;
  const int64_t most = a.max_pages << c.page_shift;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * S::kWarpBytes;
  if (D < DT) {  // the padding of every row, once: copies never write it
    for (int i = lane; i < S::kWarpBytes / 16; i += 32)
      reinterpret_cast<uint4*>(smem + warp * S::kWarpBytes)[i] = make_uint4(0, 0, 0, 0);
    __syncwarp();
  }
  if (!SHARED_OUT && sh.splits > 1) cluster_arrive();  // waited for before the first word goes to another CTA
  pdl_wait_primary();

  // The CTA's row (sequence b, head `row` of its key heads and groups of q heads)
  // and its place among the row's CTAs.
  int64_t b;
  int row, split, splits;
  if constexpr (SHARED_OUT) {
    const Part p = find_part<S::kTokens>(a, most, rows_a_seq);
    if (p.parts == 0) return;
    b = p.b;
    row = p.row;
    split = p.part;
    splits = p.parts;
    if (split == 0 && threadIdx.x == 0) sh.rows[b * rows_a_seq + row] = make_int2(blockIdx.x, splits);
  } else {
    splits = sh.splits;
    split = blockIdx.x & (splits - 1);
    const uint32_t rest = blockIdx.x >> sh.splits_log2, place = rest / (uint32_t)rows_a_seq;
    row = (int)(rest - place * rows_a_seq);
    b = sh.sorted ? by_length(a, (int)place) : sh.b0 + place;
  }

  const int hk = sh.groups == 1 ? row : row / sh.groups, first_of_group = (row - hk * sh.groups) * kRowHeads;
  const int heads = min(kRowHeads, group - first_of_group), hq = hk * group + first_of_group;
  // q of the row's heads, on its way while the pages are looked up: 0.2 us of the smallest
  // calls, 1 to 3 % of full ones.  One warp splits it for all.
  constexpr bool kBf16 = FORMAT == BITLINEAR_KV_BF16;
  float2 qx[S::kSteps], qy[S::kSteps];
  if (warp == 0) {
    const float* q = a.q + b * a.q_stride + (int64_t)(hq + min(g, heads - 1)) * D;
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
  auto look_up = [&](uint32_t t) {  // the pages of the step at t (columns of the table, whatever the length)
    page[0] = t < columns ? table[t >> c.page_shift] : -1;
    if constexpr (S::kTokens == 32) {
      page[1] = page[0];
      if (c.page_shift == 4) page[1] = t + 16 < columns ? table[(t + 16) >> 4] : -1;
    }
  };
  const uint32_t lap = (uint32_t)splits * (kWarps * S::kTokens);
  uint32_t t_ask = (uint32_t)(split * kWarps + warp) * S::kTokens;
  if (a.window <= 0) look_up(t_ask);  // the first page is known before the length
  const Span<S::kTokens> span(a.lengths[b], most, a.window);
  if (a.window > 0) {
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

  uint32_t oks = 0;  // two bits a requested step (its halves have pages), the newest lowest
  uint32_t ask_at = ring;
  auto ask = [&]() {  // requests the step at t_ask into the next stage and looks the one after up
    oks <<= 2;
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
      if (D == DT && ok == (S::kTokens == 32 ? 3u : 1u) && t_ask >= r.first && t_ask + S::kTokens <= r.len)
        request_whole<FORMAT, DT>(r, place, ask_at, lane);
      else
        request_part<FORMAT, DT>(r, c, t_ask, place, ok, ask_at, lane);
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
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem), q_area = base + (uint32_t)S::kSmem;
  const uint32_t thirds = q_area + S::kSteps * heads * 64, q_scales = q_area + heads * S::kHeadBytes;
  if (warp == 0) {
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
    if (ok != (S::kTokens == 32 ? 3u : 1u) || t0 < r.first || t0 + S::kTokens > r.len) {
#pragma unroll
      for (int j = 0; j < S::kTiles; ++j) {
        const uint32_t t = t0 + 8 * j + 2 * qd;
        const bool have = (ok >> (j / 2)) & 1u;
        if (!have || t < r.first || t >= r.len) lg[j].x = -INFINITY;
        if (!have || t + 1 < r.first || t + 1 >= r.len) lg[j].y = -INFINITY;
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
  __syncthreads();

  auto of_warps = [&](int h, int d) {
    const uint32_t p = base + h * S::kPartial;
    return join<kWarps>(p + 4 * d, S::kWarpBytes, p + 4 * DT, S::kWarpBytes, kWarps);
  };
  auto head_of = [&](int i) { return heads == 1 ? 0 : (int)((uint32_t)i / (uint32_t)D); };
  auto finish = [&](int h, int d, const Joined& j) {
    a.out[b * a.out_stride + (int64_t)(hq + h) * D + d] = output_of(j.value, j.m, j.sum);
  };
  if (SHARED_OUT || splits == 1) {
    float* part = splits == 1 ? nullptr : sh.parts + (int64_t)blockIdx.x * min(kRowHeads, group) * (D + 4);
    for (int i = threadIdx.x; i < heads * D; i += kThreads) {
      const int h = head_of(i), d = i - h * D;
      const Joined j = of_warps(h, d);
      if (splits == 1) {
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

// CTAs of a cluster: a power of two up to `most`, while all CTAs are resident at once and
// every warp may have a step, or two from 16 CTAs on.  (One sequence, 8 / 16 CTAs at most, us:
// 8192 tokens of 32 heads of 80, int8 15.5 / 14.3; 4096 of 8 key heads bf16 10.1 / 8.9, of one
// e4m3 8.9 / 7.1; a step a warp: 2048 of 32 heads 5.8 / 6.0, 1024 of one key head 5.7 / 5.5.)
int splits_for(int64_t rows, int64_t steps, int ctas, int most) {
  int s = 1;
  while (s < most && rows * s * 2 <= ctas && steps >= (s >= 8 ? 4 : 2) * s * kWarps) s *= 2;
  return s;
}

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
  const double factor = (double)a.scale * 1.4426950408889634;  // to the base of the weights
  a.factor = (float)factor;
  a.factor_rest = (float)(a.factor != 0.0f ? factor / a.factor - 1.0 : 0.0);
  const auto clusters = attend_kernel<FORMAT, DT, false>, shared_out = attend_kernel<FORMAT, DT, true>;
  static thread_local int configured_device = -1, most_cluster;
  if (configured_device != dev.device) {
    const int most = (int)S::kSmem + kRowHeads * (S::kHeadBytes + 4) + received_bytes(kRowHeads, DT, kMaxCluster);
    for (const auto kernel : {clusters, shared_out}) {
      const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
      if (err != cudaSuccess) return err;
    }
    most_cluster = kPortableCluster;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {kMaxCluster, 1, 1};
    cfg.gridDim = dim3(kMaxCluster, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = most;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int fit = 0;
    if (cudaFuncSetAttribute(clusters, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&fit, clusters, &cfg) == cudaSuccess && fit > 0)
      most_cluster = kMaxCluster;
    else
      cudaGetLastError();  // not this call's: the smaller size always runs
    configured_device = dev.device;
  }
  const int64_t rows = rows_of(a.B, a.q_heads, c.heads), per_seq = rows / a.B;
  int64_t tokens = a.max_pages << c.page_shift;
  if (a.window > 0 && a.window < tokens) tokens = a.window + S::kTokens;  // a window may begin inside a step
  const int64_t steps = (tokens + S::kTokens - 1) / S::kTokens;
  const int group = a.q_heads / c.heads, groups = (group + kRowHeads - 1) / kRowHeads;
  const int heads = group < kRowHeads ? group : kRowHeads;
  const int smem = (int)S::kSmem + heads * S::kHeadBytes + kRowHeads * 4;  // the rings, q's parts and scales
  // CTAs resident at once, with so much shared memory more each
  auto resident = [&](int more) {
    const int fit = (int)(dev.smem_per_sm / (smem + more + kOtherSmem));
    return (dev.num_sms < kSms ? dev.num_sms : kSms) * (fit < S::kCtas ? fit : S::kCtas);
  };
  const int ctas = resident(0), cluster_ctas = resident(received_bytes(heads, c.head_dim, kMaxCluster));
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
  cfg.dynamicSmemBytes = smem + received_bytes(heads, c.head_dim, sh.splits);
  const int64_t per_launch = (int64_t)0x7fffffff / (per_seq * sh.splits);  // sequences a grid holds
  for (; sh.b0 < a.B; sh.b0 += per_launch) {
    const int64_t n = a.B - sh.b0 < per_launch ? a.B - sh.b0 : per_launch;
    cfg.gridDim = dim3((unsigned)(n * per_seq * sh.splits), 1, 1);
    cfg.numAttrs = 0;
    if (sh.splits > 1) {
      attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
      attr[cfg.numAttrs].val.clusterDim.x = (unsigned)sh.splits;
      attr[cfg.numAttrs].val.clusterDim.y = 1;
      attr[cfg.numAttrs].val.clusterDim.z = 1;
      ++cfg.numAttrs;
    }
    if (pdl) programmatic();
    const cudaError_t err = cudaLaunchKernelEx(&cfg, clusters, a, c, sh);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

template <int FORMAT>
cudaError_t launch_format(const AttendArgs& a, const KvPages& c, void* workspace, bool pdl, const DeviceInfo& dev,
                          cudaStream_t s) {
  if (c.head_dim <= 64) return launch_shape<FORMAT, 64>(a, c, workspace, pdl, dev, s);
  if (c.head_dim <= 80) return launch_shape<FORMAT, 80>(a, c, workspace, pdl, dev, s);
  if (c.head_dim <= 96) return launch_shape<FORMAT, 96>(a, c, workspace, pdl, dev, s);
  if (c.head_dim <= 112) return launch_shape<FORMAT, 112>(a, c, workspace, pdl, dev, s);
  if (c.head_dim <= 128) return launch_shape<FORMAT, 128>(a, c, workspace, pdl, dev, s);
  return launch_shape<FORMAT, 256>(a, c, workspace, pdl, dev, s);
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
  if (cache.format == BITLINEAR_KV_INT8) return launch_format<BITLINEAR_KV_INT8>(a, cache, workspace, pdl, dev, stream);
  if (cache.format == BITLINEAR_KV_FP8) return launch_format<BITLINEAR_KV_FP8>(a, cache, workspace, pdl, dev, stream);
  return launch_format<BITLINEAR_KV_BF16>(a, cache, workspace, pdl, dev, stream);
}

}  // namespace bitlinear
