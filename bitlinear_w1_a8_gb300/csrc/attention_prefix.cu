// attention_prefix.cu -- the tokens that many rows share, on the fifth-generation tensor cores.
//
// A row of work is 128 q heads (all of a group's rows' for one key head, or 128 of them) and a run
// of the group's shared tokens, in tiles of 128:
//   S = Q K^T (TMEM), P = 2^(S - ref) in registers, back to TMEM as the next product's A operand, O = P V (TMEM).
// fp32 accuracy takes two MMAs for one, or three.  Codes are exact in fp16, and q and the weights are split into two fp16
// parts (22 bits): q's row is scaled to 2^13 .. 2^14 and the weights to at most 2^15, so that what a leading part
// leaves is still a whole fp16 (its last place 2^-38 of the row's largest q, 2^-36 of the largest weight), and
// both parts add up in one accumulator, the small ones first.  bf16 keys are used as they are, with q in three
// bf16 parts (24 bits).  bf16 values become fp16 under a power of two that a tile of 128 tokens has in common
// (below): those above 2^-32 of the tile's largest are exact.
// Each tile's O starts from zero and is added to fp32 sums in registers: the tensor cores' adder cuts toward
// zero, and a chain of tiles in it would show.
//
// 28 warps: two groups of eight that turn logits into weights and add up O, each for every other tile with a
// reference and sums of its own (two threads a row, half of a tile's tokens and half of the dims each: they tell each
// other their largest logits); eight that widen codes (bf16: values) and lay them out for the MMA (128-byte swizzle,
// the same image for both: K is the B operand along its rows, V across them); one that looks pages up, four
// tiles ahead, and asks for them to come into L2; one that copies rows as they are needed (bulk copies, TMA for
// bf16); one thread that issues the products of S and one that issues those of O.  Two S and two O are in
// flight, K and V tiles take turns in one ring, and a weight overwrites its logit's place.
//
// Measured: 256 q heads over 16384 tokens, 8 key heads of 128, bf16: ~42 us, 15 tiles a CTA at ~4000 cycles each beside ~17,000 to
// the first weights' product and ~7,000 to hand over.  What bounds it: a tile's logits, weights, their product and the place
// for the next but one's logits follow one another (1600 + 4200 + 1500 cycles), for two tiles at a time; five MMAs a tile need
// 2700, and with what TMA, the turning of values and both operands of the MMAs read and write of shared memory it is busy
// for ~3300.  The tensor pipe is busy 53 cycles of 100 on an SM that has work.
// Slower: a thread a row in the adding groups (its loops are fetched, not issued); unrolled loops (three times as long: the
// code is fetched as it runs); values turned in one pass that holds them in registers (spills).
#include "attend.cuh"
#include "serve.cuh"
#include "tc_util.cuh"
#include "tensor_map.cuh"

namespace bitlinear {
namespace {

constexpr int kRows = kPrefixWide;      // q heads of a CTA: the MMA's rows
constexpr int kTile = kPrefixTile;      // tokens
constexpr int kWideThreads = 896;
constexpr int kBring = 16, kIssue = 24;  // the first warps that bring keys and values, and that issue
constexpr int kBringThreads = 256;
constexpr int kEntries = 4;             // tiles whose pages and steps are known
constexpr int kPanel = 128 * 128;       // bytes of 128 rows of 64 fp16 values
constexpr float kTarget = 12.0f, kMost = 15.0f;  // log2 of the largest weight: where the reference puts it, what moves it
// Registers a thread: at the launch, and as the groups of warps then share them out.
constexpr int kLaunchRegisters = 72, kAddRegisters = 104, kBringRegisters = 32, kIssueRegisters = 24;
static_assert(512 * kAddRegisters + kBringThreads * kBringRegisters + 128 * kIssueRegisters <= kWideThreads * kLaunchRegisters,
              "more registers than were launched with would be waited for");

struct Maps {  // of a bf16 cache: [page][head and token][dim], boxes of 64 dims of a page's tokens, 128 at most
  CUtensorMap keys, values;
};
struct Entry {
  // of each 16 tokens: ((page * heads) + head) * page_size + offset (bf16: the page above 32 bits of the rest), or -1
  int64_t row[kTile / 16];
};

// What the roles tell each other.
template <bool BF16>
struct State {
  float k_steps[kEntries][BF16 ? 4 : kTile], v_steps[kEntries][BF16 ? 4 : kTile];
  float v_most[kEntries][4];  // the largest of the latter, by warp; bf16: a tile's power of two, first
  Entry entries[kEntries];
  float row_tops[2][2][kRows];  // by tile's parity and half of its tokens; before the first tile q's scales, in the first
  uint32_t tops[2][8];
  unsigned long long meta_full[kEntries], meta_empty[kEntries], raw_full[4], raw_empty[4], stage_full[4], stage_empty[4], s_full[2], p_full[2],
      o_full[2], q_full, drained[2];
  uint32_t entry_ok[kEntries], tmem_at;
  int abort_flag;
};

template <int FORMAT, int DT>
struct Wide {
  static constexpr bool kBf16 = FORMAT == BITLINEAR_KV_BF16;
  static constexpr int kBytes = kBf16 ? 2 : 1;
  static constexpr int kPanels = (DT + 63) / 64;
  static constexpr int kOperand = kPanels * kPanel;
  static constexpr int kPieces = DT / 16;              // 16-byte pieces of a token's 8-bit codes
  static constexpr int kTurn = kBringThreads / 8;      // tokens whose codes are widened at once
  static constexpr int kStages = kBf16 ? 4 : 3;        // K and V tiles as operands
  static constexpr int kRaw = kTile * DT;              // and 8-bit codes as they come, rows of the cache's size side by side
  static constexpr int kRaws = kBf16 ? 0 : 3;          // (bf16 comes as operands)
  static constexpr int kParts = kBf16 ? 3 : 2;         // of q
  static constexpr int kOperands = kParts * kOperand + kStages * kOperand + kRaws * kRaw;  // Q's parts first
  static constexpr int kNeed = kOperands + (int)sizeof(State<kBf16>);
  // the base is rounded up to 1024, where it is not there already (a kernel without static arrays has it there)
  static constexpr int kSmem = kNeed + 1024 < 232448 ? kNeed + 1024 : 232448;
  static_assert(kNeed <= 232448, "what a CTA may have");
};

__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
// The B operand across its rows (N along the row): panels of 64 columns a panel apart, 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t across_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3fffu) | (uint64_t)(kPanel >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
__device__ __forceinline__ void tmem_load16(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}
__device__ __forceinline__ void tmem_load8(uint32_t at, uint32_t (&r)[16]) {  // the first 8
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(at));
#pragma unroll
  for (int i = 8; i < 16; ++i) r[i] = 0;
}
// After the wait: the registers of earlier loads are used behind it.
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ float largest_of(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two values as the leading fp16 parts and what they leave, both whole.
__device__ __forceinline__ void parts_of(float2 w, uint32_t& lead, uint32_t& rest) {
  const __half2 h = __floats2half2_rn(w.x, w.y);
  const float2 d = fma2(__half22float2(h), both(-1.0f), w);  // exact
  const __half2 r = __floats2half2_rn(d.x, d.y);
  lead = *reinterpret_cast<const uint32_t*>(&h);
  rest = *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t of_panel(int row, int dim) {  // where a 16-byte piece (8 dims) of an operand is
  return (uint32_t)((dim >> 6) * kPanel + row * 128 + ((((dim >> 3) & 7) ^ (row & 7)) << 4));
}

// The bounded wait of tc_util.cuh, inlined whole: a call has no place where warps' registers differ.
__device__ __forceinline__ bool wait_bounded(unsigned long long* bar, uint32_t parity, int* abort_flag, int* status) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = tc::global_timer();
#pragma unroll 1
  for (uint32_t i = 1;; ++i) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 0u) {
      if (*reinterpret_cast<volatile int*>(abort_flag)) return false;
      if (tc::global_timer() - t0 > tc::kTimeoutNs) {
        atomicExch(abort_flag, 1);
        atomicExch(status, (int)BITLINEAR_ERR_TIMEOUT);
        return false;
      }
    }
  }
}

// Waits, with the same limit, for what this thread has issued, also after others have given up.
__device__ __forceinline__ void drain(unsigned long long* bar, uint32_t parity, int* status) {
  const unsigned long long t0 = tc::global_timer();
#pragma unroll 1
  for (uint32_t i = 0; !tc::mbar_try_wait(bar, parity); ++i) {
    if ((i & 63u) == 63u && tc::global_timer() - t0 > tc::kTimeoutNs) {
      atomicExch(status, (int)BITLINEAR_ERR_TIMEOUT);
      return;
    }
  }
}

template <int FORMAT, int DT>
__global__ void __launch_bounds__(kWideThreads, 1) prefix_wide_kernel(AttendArgs a, KvPages c, Shares sh, const __grid_constant__ Maps maps,
                                                                      int* status) {
  using W = Wide<FORMAT, DT>;
  extern __shared__ __align__(1024) uint8_t raw[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = c.head_dim;
  const uint32_t base = ((uint32_t)__cvta_generic_to_shared(raw) + 1023u) & ~1023u;
  const uint32_t q_at = base, stage_at = base + W::kParts * W::kOperand, raw_at = stage_at + W::kStages * W::kOperand;
  uint32_t given;
  asm volatile("mov.u32 %0, %%dynamic_smem_size;" : "=r"(given));
  if (base + W::kNeed > (uint32_t)__cvta_generic_to_shared(raw) + given) {  // not where it was expected
    if (threadIdx.x == 0) atomicExch(status, (int)BITLINEAR_ERR_UNSUPPORTED);
    return;
  }
  State<W::kBf16>& st = *reinterpret_cast<State<W::kBf16>*>(raw + (base - (uint32_t)__cvta_generic_to_shared(raw)) + W::kOperands);

  if (warp == kIssue + 3 && lane == 0) {
    st.abort_flag = 0;
#pragma unroll 1
    for (int i = 0; i < kEntries; ++i) {
      tc::mbar_init(&st.meta_full[i], 1);
      tc::mbar_init(&st.meta_empty[i], 8);
    }
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(&st.raw_full[i], 1);
      tc::mbar_init(&st.raw_empty[i], kBringThreads / 32);
      tc::mbar_init(&st.stage_full[i], kBringThreads / 32);
      tc::mbar_init(&st.stage_empty[i], 1);
    }
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&st.p_full[i], 8);
      tc::mbar_init(&st.s_full[i], 1);
      tc::mbar_init(&st.o_full[i], 1);
      tc::mbar_init(&st.drained[i], 1);
    }
    tc::mbar_init(&st.q_full, kBring);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait_primary();
  pdl_release_dependents();
  // The CTA's row of work: group b, key head and tile of q heads `row`, and its run of tiles.
  const int64_t most = a.max_pages << c.page_shift;
  int64_t b;
  int row, part, parts;
  if (sh.splits == 0) {
    const Part p = find_part<kTile>(a, most, sh.rows_a_seq, 1);
    if (p.parts == 0) return;
    b = p.b;
    row = p.row;
    part = p.part;
    parts = p.parts;
  } else {
    const uint32_t at = blockIdx.x / (uint32_t)sh.splits;
    b = at / (uint32_t)sh.rows_a_seq;
    row = at - (uint32_t)b * sh.rows_a_seq;
    part = blockIdx.x - at * sh.splits;
    // as few parts as leave the longest as short
    const int steps = max(1, Span<kTile>(a.lengths[b], most, 0).steps()), each = (steps + sh.splits - 1) / sh.splits;
    parts = (steps + each - 1) / each;
    if (part >= parts) return;
  }
  if (warp == kIssue) tc::tmem_alloc(&st.tmem_at, 512);
  if (part == 0 && threadIdx.x == 0) sh.rows[b * sh.rows_a_seq + row] = make_int2(blockIdx.x, parts);
  const int hk = row / sh.groups, first_head = (row - hk * sh.groups) * kRows, heads = min(kRows, sh.group - first_head);
  uint32_t len;
  {
    int longest = 0;
#pragma unroll 1
    for (int i = lane; i < sh.group_rows; i += 32) longest = max(longest, sh.lengths[b * sh.group_rows + i]);
    const Span<kTile> span(a.lengths[b], most, 0);
    len = min(span.len, (uint32_t)__reduce_max_sync(kFullMask, longest));
    const int steps = span.steps();  // shared out by what the group may share, whatever its rows have of it
    const int each = (steps + parts - 1) / parts;
    part *= each;
    parts = min(steps, part + each);
  }
  const uint32_t begin = (uint32_t)part * kTile;
  // the first tile's pages are on their way while the CTA meets
  const int32_t* table = a.table + b * a.table_stride;
  int32_t page = -1;
  if (warp == kIssue + 2 && begin + 16 * (lane & 7) < len) page = table[(begin + 16 * (lane & 7)) >> c.page_shift];
  if constexpr (W::kBf16) {
    if (warp == kIssue + 3 && lane < 2) asm volatile("prefetch.tensormap [%0];" ::"l"(lane ? &maps.values : &maps.keys) : "memory");
  }
  const int tiles = max(0, min(parts, (int)((len + kTile - 1) / kTile)) - part);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = st.tmem_at;
  auto s_of = [&](int par) { return tmem + par * 128; };
  auto o_of = [&](int par) { return tmem + 256 + par * 128; };

  // K and V tiles take turns in one ring, in the order in which they are used: K0 K1 V0 K2 V1 ... and the last V.
  auto place_of_k = [&](int n) { return n == 0 ? 0 : 2 * n - 1; };
  auto place_of_v = [&](int n) { return n + 1 < tiles ? 2 * n + 2 : 2 * n + 1; };
  auto at_place = [&](int i, int& operand, int& n) {
    operand = i > 0 && ((i & 1) == 0 || i == 2 * tiles - 1);
    n = operand ? (i == 2 * tiles - 1 ? tiles - 1 : i / 2 - 1) : (i + 1) / 2;
  };

  // Every role runs through all of its tiles, also after a wait has run out (`alive` false): it then
  // waits and reads no more, and still arrives wherever others count it.
  bool alive = true;
  auto wait = [&](unsigned long long* bar, int phase) { alive = alive && wait_bounded(bar, phase & 1, &st.abort_flag, status); };

  if (warp < kBring) {
    // ------------------------------------------------------- logits to weights, sums
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAddRegisters));
    const int par = warp >> 3, side = (warp >> 2) & 1, r = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's lanes of TMEM
    const bool there = r < heads;
    const uint32_t of_group = first_head + (there ? r : 0), member = of_group / (uint32_t)sh.heads_a_key;
    const int64_t seq = b * sh.group_rows + member;
    // q's rows, a warp a row, four at a time: a lane has 4 dims
    {
      const float factor = a.factor, more = a.factor_rest;
      const bool have = 4 * lane < D;
#pragma unroll 1
      for (int i0 = warp; i0 < kRows; i0 += 4 * kBring) {
        float4 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = i0 + kBring * j;
          const uint32_t head = first_head + min(i, heads - 1), who = head / (uint32_t)sh.heads_a_key;
          const float* q = a.q + (b * sh.group_rows + who) * a.q_stride + (int64_t)(hk * sh.heads_a_key + (head - who * sh.heads_a_key)) * D;
          w[j] = have && i < heads ? *reinterpret_cast<const float4*>(q + 4 * lane) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = i0 + kBring * j;
          const float2 x = mul2(make_float2(w[j].x, w[j].y), both(factor)), y = mul2(make_float2(w[j].z, w[j].w), both(factor));
          uint32_t words[W::kParts][2];
          if constexpr (W::kBf16) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float u = k ? y.x : x.x, v = k ? y.y : x.y;
              const float2 rest = mul2(make_float2(u, v), both(more));
              words[0][k] = next_part(u, v);
              words[1][k] = next_part(u, v);
              u += rest.x;
              v += rest.y;
              words[2][k] = next_part(u, v);
            }
          } else {
            const float top = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y)));
            const int e = clamp_exponent(exponent_of(__uint_as_float(__reduce_max_sync(kFullMask, __float_as_uint(top)))));
            const float2 up = both(power2(13 - e)), rest_up = both(power2(13 - e) * more);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float2 z = k ? y : x, v = mul2(z, up);
              const __half2 h = __floats2half2_rn(v.x, v.y);
              const float2 d = fma2(z, rest_up, fma2(__half22float2(h), both(-1.0f), v));
              const __half2 g = __floats2half2_rn(d.x, d.y);
              words[0][k] = *reinterpret_cast<const uint32_t*>(&h);
              words[1][k] = *reinterpret_cast<const uint32_t*>(&g);
            }
            if (lane == 0) st.row_tops[0][0][i] = power2(e - 13);
          }
          if (4 * lane < DT) {
            const uint32_t at = q_at + of_panel(i, 4 * lane) + (lane & 1) * 8;
#pragma unroll
            for (int k = 0; k < W::kParts; ++k)
              asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at + k * W::kOperand), "r"(words[k][0]), "r"(words[k][1]) : "memory");
          }
        }
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&st.q_full);
    }
    tc::named_bar_sync(3, 32 * kBring);
    const float unit = W::kBf16 ? 1.0f : st.row_tops[0][0][r];  // of a logit in S
    tc::named_bar_sync(3, 32 * kBring);
    const bool none = (warp & 3) * 32 >= heads;  // rows of no q head: whatever comes of them is theirs
    const uint32_t row_end = there ? min(len, (uint32_t)max(0, sh.lengths[seq])) : len;  // beside none: masked as the others are

    constexpr int kSide = kTile / 2, kGranules = kSide / 16;  // tokens of this thread, and 16s of them
    constexpr int kDims = DT / 2;                             // and dims
    float ref = kUnset;
    float2 sums = both(0.0f);
    float2 out[kDims / 2];
#pragma unroll
    for (int i = 0; i < kDims / 2; ++i) out[i] = both(0.0f);
    const uint32_t s_at = s_of(par) + lanes + side * kSide, o_at = o_of(par) + lanes + side * kDims;

#pragma unroll 1
    for (int n = par; n < tiles; n += 2) {
      const int entry = n % kEntries;
      const uint32_t t0 = begin + n * kTile + side * kSide;
      wait(&st.s_full[par], n >> 1);
      if (none) {
        if (lane == 0) tc::mbar_arrive(&st.p_full[par]);
        tc::named_bar_sync(1 + par, 256);
        wait(&st.o_full[par], n >> 1);
        if (lane == 0) tc::mbar_arrive(&st.meta_empty[entry]);
        continue;
      }
      tc::tc_fence_after();
      // the columns that count: all of them, or the first `count` of those 16 whose page is there
      const uint32_t ok = alive ? st.entry_ok[entry] >> (kGranules * side) & 0xfu : 0u;
      const int count = row_end > t0 ? (int)min((uint32_t)kSide, row_end - t0) : 0;
      const bool whole = __all_sync(kFullMask, ok == 0xfu && count == kSide);
      const uint32_t ks = (uint32_t)__cvta_generic_to_shared(st.k_steps[entry]) + (W::kBf16 ? 0 : 4 * kSide * side);
      const uint32_t vs = (uint32_t)__cvta_generic_to_shared(st.v_steps[entry]) + (W::kBf16 ? 0 : 4 * kSide * side);
      // The 16 logits over `unit` of granule g.  Loops over granules stay rolled up: code is fetched as it runs, and
      // unrolled they took three times as long.
      auto logits = [&](int g, uint32_t (&s)[16], float2 (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
        if constexpr (!W::kBf16) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 k = lds_float4(ks + (16 * g + 4 * i) * 4);
            x[2 * i] = mul2(x[2 * i], make_float2(k.x, k.y));
            x[2 * i + 1] = mul2(x[2 * i + 1], make_float2(k.z, k.w));
          }
        }
        if (!whole) {
          const int here = (ok >> g) & 1u ? count - 16 * g : 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (2 * i >= here) x[i].x = -INFINITY;
            if (2 * i + 1 >= here) x[i].y = -INFINITY;
          }
        }
      };
      // the row's largest
      float top = -INFINITY;
      constexpr int kTogether = DT <= 96 ? 2 : 1;  // granules, as the registers allow
#pragma unroll 1
      for (int g = 0; g < kGranules; g += kTogether) {
        uint32_t s[kTogether][16];
        float2 x[8];
#pragma unroll
        for (int k = 0; k < kTogether; ++k) tmem_load16(s_at + 16 * (g + k), s[k]);
#pragma unroll
        for (int k = 0; k < kTogether; ++k) tmem_loaded(s[k]);
#pragma unroll
        for (int k = 0; k < kTogether; ++k) {
          logits(g + k, s[k], x);
#pragma unroll
          for (int i = 0; i < 8; ++i) top = largest_of(top, x[i].x, x[i].y);
        }
      }
      st.row_tops[par][side][r] = top;
      tc::named_bar_sync(1 + par, 256);
      top = fmaxf(top, st.row_tops[par][1 - side][r]) * unit;
      if constexpr (!W::kBf16) {  // of a weight: a power times the value's step
        const float4 vm = lds_float4((uint32_t)__cvta_generic_to_shared(st.v_most[entry]));
        top += log2_of(at_least(fmaxf(fmaxf(vm.x, vm.y), fmaxf(vm.z, vm.w)), kLeastStep));
      }
      if (top > ref + kMost) {
        const float next = top - kTarget, down = exp2_of(ref - next);  // 0 from the first reference
        ref = next;
        sums = mul2(sums, both(down));
#pragma unroll
        for (int i = 0; i < kDims / 2; ++i) out[i] = mul2(out[i], both(down));
      }
      float2 more = both(0.0f);
#pragma unroll 1
      for (int g = 0; g < kGranules; ++g) {
        uint32_t s[16], w[16];
        float2 x[8];
        tmem_load16(s_at + 16 * g, s);
        tmem_loaded(s);
        logits(g, s, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = W::kBf16 ? add2(x[i], both(-ref)) : fma2(x[i], both(unit), both(-ref));
          x[i] = make_float2(exp2_of(x[i].x), exp2_of(x[i].y));
          more = add2(more, x[i]);
        }
        if constexpr (!W::kBf16) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 v = lds_float4(vs + (16 * g + 4 * i) * 4);
            x[2 * i] = mul2(x[2 * i], make_float2(v.x, v.y));
            x[2 * i + 1] = mul2(x[2 * i + 1], make_float2(v.z, v.w));
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) parts_of(x[i], w[i], w[8 + i]);
        tc::tmem_st16(s_at + 16 * g, w);
      }
      tc::tmem_st_wait();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&st.p_full[par]);
      sums = add2(sums, more);
      wait(&st.o_full[par], n >> 1);
      float2 v_unit = both(1.0f);
      if constexpr (W::kBf16) {  // the values' power of two
        v_unit = both(st.v_most[entry][0]);
        __syncwarp();
      }
      // Not before O: the weights wait for keys alone, and the copies and the laying out of the tile's values read its entry
      // too.  O shows that they have.
      if (lane == 0) tc::mbar_arrive(&st.meta_empty[entry]);
      tc::tc_fence_after();
#pragma unroll
      for (int d = 0; d < kDims; d += 16) {  // 8 or 16 dims
        uint32_t o[16];
        if (d + 16 <= kDims)
          tmem_load16(o_at + d, o);
        else
          tmem_load8(o_at + d, o);
        tmem_loaded(o);
#pragma unroll
        for (int i = 0; i < (d + 16 <= kDims ? 8 : 4); ++i)
          out[d / 2 + i] = W::kBf16 ? fma2(make_float2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), v_unit, out[d / 2 + i])
                                    : add2(out[d / 2 + i], make_float2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])));
      }
    }
    // The two groups meet in what was K's and V's place, [dim][row], 129 apart, then references and sums: each
    // thread gives half of its dims and joins the other half of the other's.
    constexpr int kApart = kRows + 1, kGiven = kDims / 4;  // in pairs of dims
    const uint32_t meet = stage_at + (side * kDims * kApart + r) * 4, scales = stage_at + DT * kApart * 4;
    static_assert((DT * kApart + 8 * kRows) * 4 <= W::kStages * W::kOperand + W::kRaws * W::kRaw, "what is joined fits where K and V were");
    auto store = [](uint32_t at, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory"); };
    auto give = [&](auto half) {
      constexpr int h = decltype(half)::value;
#pragma unroll
      for (int i = h * kGiven; i < (h + 1) * kGiven; ++i) {
        store(meet + 2 * i * kApart * 4, out[i].x);
        store(meet + (2 * i + 1) * kApart * 4, out[i].y);
      }
    };
    auto take = [&](auto half, float mine, float theirs) {
      constexpr int h = decltype(half)::value;
#pragma unroll
      for (int i = h * kGiven; i < (h + 1) * kGiven; ++i) {
        const uint32_t at = meet + 2 * i * kApart * 4;
        store(at, out[i].x * mine + lds_float(at) * theirs);
        store(at + kApart * 4, out[i].y * mine + lds_float(at + kApart * 4) * theirs);
      }
    };
    static_assert(kDims % 8 == 0, "whole pairs to give and to take");
    tc::named_bar_sync(3, 32 * kBring);
    if (par == 0)
      give(std::integral_constant<int, 1>());
    else
      give(std::integral_constant<int, 0>());
    // a row's: [group][reference, sum of one half, sum of the other]
    if (side == 0) store(scales + 32 * r + 16 * par, ref);
    store(scales + 32 * r + 16 * par + 4 + 4 * side, sums.x + sums.y);
    tc::named_bar_sync(3, 32 * kBring);
    const float4 first = lds_float4(scales + 32 * r), second = lds_float4(scales + 32 * r + 16);
    const float m = fmaxf(first.x, second.x), f0 = exp2_of(first.x - m), f1 = exp2_of(second.x - m);
    if (par == 0)
      take(std::integral_constant<int, 0>(), f0, f1);
    else
      take(std::integral_constant<int, 1>(), f1, f0);
    tc::named_bar_sync(3, 32 * kBring);  // all references and sums are read
    if (par == 0 && side == 0) {
      store(scales + 32 * r, m);
      store(scales + 32 * r + 4, (first.y + first.z) * f0 + (second.y + second.z) * f1);
    }
    tc::named_bar_sync(3, 32 * kBring);
    float* slot = sh.parts + (int64_t)blockIdx.x * sh.slot_heads * (D + 4);
    for (int i = warp; i < heads; i += kBring) {
      for (int d = lane; d < D; d += 32) slot[i * (D + 4) + d] = lds_float(stage_at + (d * kApart + i) * 4);
      if (lane == 0) *reinterpret_cast<float2*>(slot + i * (D + 4) + D) = lds_float2(scales + 32 * i);
    }
  } else if (warp < kIssue) {
    // ------------------------------------------------------- keys and values, widened
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kBringRegisters));
    const int tid = threadIdx.x - 32 * kBring;
    auto done = [&](int stage) {
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&st.stage_full[stage]);
    };
    if constexpr (!W::kBf16) {
      // A thread takes the same 16 bytes of every kTurn-th token's row.
      const int of_turn = tid / 8, chunk = tid % 8;
      const bool loads = 16 * chunk < D, stores = chunk < W::kPieces, turned = chunk & 4;
      // and 128 kTurn bytes on for each turn; the second panel's pieces go in the other order, so that each
      // eighth of a store meets every bank once
      const uint32_t place = of_panel(of_turn, 16 * chunk) ^ (turned ? 16 : 0);
#pragma unroll 1
      for (int i = 0; i < 2 * tiles; ++i) {
        int operand, n;
        at_place(i, operand, n);
        const int entry = n % kEntries, stage = i % W::kStages, slot = i % W::kRaws;
        const uint32_t to = stage_at + stage * W::kOperand + place, from = raw_at + slot * W::kRaw + of_turn * D + 16 * chunk;
        wait(&st.raw_full[slot], i / W::kRaws);
        // the tokens that are there: of each 16 those whose page is, and the first `count`
        const uint32_t ok = alive ? st.entry_ok[entry] : 0u;
        const int count = (int)(len - begin) - n * kTile;
        const bool whole = ok == 0xffu && count >= kTile;
        if (!operand) {  // the steps of both come with the keys, so that weights need not wait for values
          const int token = tid % kTile;
          float* steps = tid < kTile ? st.k_steps[entry] : st.v_steps[entry];
          float step = token < count && ((ok >> (token >> 4)) & 1u) ? steps[token] : 0.0f;
          if (tid >= kTile) {
            const uint32_t m = __reduce_max_sync(kFullMask, __float_as_uint(step));
            if (lane == 0) st.v_most[entry][warp - kBring - kTile / 32] = __uint_as_float(m);
            step = at_least(step, kLeastStep);
          }
          steps[token] = step;
        }
        if (i >= W::kStages) wait(&st.stage_empty[stage], i / W::kStages - 1);
        if (stores) {
#pragma unroll
          for (int t = 0; t < kTile / W::kTurn; ++t) {
            const int token = t * W::kTurn + of_turn;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (loads && (whole || (token < count && ((ok >> (token >> 4)) & 1u)))) w = lds128(from + t * W::kTurn * D);
            uint32_t h[8];
            widen<FORMAT>(turned ? w.z : w.x, h[0], h[1]);
            widen<FORMAT>(turned ? w.w : w.y, h[2], h[3]);
            widen<FORMAT>(turned ? w.x : w.z, h[4], h[5]);
            widen<FORMAT>(turned ? w.y : w.w, h[6], h[7]);
            tc::st_shared_v4(to + t * W::kTurn * 128, h[0], h[1], h[2], h[3]);
            tc::st_shared_v4((to + t * W::kTurn * 128) ^ 16, h[4], h[5], h[6], h[7]);
          }
        }
        done(stage);
        if (lane == 0) tc::mbar_arrive(&st.raw_empty[slot]);
      }
    } else {
      // bf16 values become fp16 where they are, under the power of two that puts the tile's largest to 2^14 .. 2^15
      // (what is below 2^-32 of that is rounded to a multiple of 2^-38); those of tokens that are not there become 0.
      constexpr int kTurns = W::kOperand / (kBringThreads * 16);
#pragma unroll 1
      for (int n = 0; n < tiles; ++n) {
        const int i = place_of_v(n), entry = n % kEntries, stage = i % W::kStages;
        // how often the place has had values before: the even ones every other tile's, the last one's odd place none
        wait(&st.raw_full[stage], i & 1 ? 0 : n >> 1);
        const uint32_t ok = alive ? st.entry_ok[entry] : 0u;
        const int count = (int)(len - begin) - n * kTile;
        const bool whole = ok == 0xffu && count >= kTile;
        const uint32_t at = stage_at + stage * W::kOperand + 16 * tid;
        auto counts = [&](int t) {  // whether turn t's piece of this thread is of a token that is there
          const int token = (tid >> 3) + (t * (kBringThreads / 8)) % kTile;
          return whole || (token < count && ((ok >> (token >> 4)) & 1u));
        };
        uint32_t top = 0;
#pragma unroll
        for (int t = 0; t < kTurns; ++t) {
          if (!counts(t)) continue;
          const uint4 w = lds128(at + t * kBringThreads * 16);
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
        }
        top = __reduce_max_sync(kFullMask, max(top & 0xffffu, top >> 16));
        if (lane == 0) st.tops[n & 1][warp - kBring] = top;
        tc::named_bar_sync(4, kBringThreads);
        top = __reduce_max_sync(kFullMask, st.tops[n & 1][lane & 7]);
        const int e = max(30, min(254, (int)(top >> 7)));
        const float2 scale = both(power2(141 - e));
#pragma unroll
        for (int t = 0; t < kTurns; ++t) {
          uint4 w = make_uint4(0, 0, 0, 0);
          if (counts(t)) w = lds128(at + t * kBringThreads * 16);
          uint32_t* u[4] = {&w.x, &w.y, &w.z, &w.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = mul2(make_float2(__uint_as_float(*u[k] << 16), __uint_as_float(*u[k] & 0xffff0000u)), scale);
            const __half2 x = __floats2half2_rn(f.x, f.y);
            *u[k] = *reinterpret_cast<const uint32_t*>(&x);
          }
          tc::st_shared_v4(at + t * kBringThreads * 16, w.x, w.y, w.z, w.w);
        }
        // beside an infinity or a NaN the others are lost: whoever meets the tile has NaN
        if (tid == 0) st.v_most[entry][0] = top >= 0x7f80u ? NAN : power2(e - 141);
        done(stage);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegisters));
    if (warp == kIssue) {
      // ----------------------------------------------------- S = Q K^T
      if (lane == 0) {
        // bf16 is format 1 of both operands, fp16 0
        const uint32_t idesc = tc::make_idesc(kRows, kTile) | (W::kBf16 ? 1u << 7 | 1u << 10 : 0u);
        wait(&st.q_full, 0);
#pragma unroll 1
        for (int n = 0; n < tiles; ++n) {
          const int at = place_of_k(n), stage = at % W::kStages;
          wait(&st.stage_full[stage], at / W::kStages);
          if (n >= 2) wait(&st.o_full[n & 1], (n >> 1) - 1);  // the weights that lie over the last S of this place are used
          if (alive) {
            tc::tc_fence_after();
            uint32_t add = 0;
#pragma unroll 1
            for (int part = W::kParts - 1; part >= 0; --part) {
#pragma unroll
              for (int k = 0; k < DT / 16; ++k) {
                const uint32_t off = (k / 4) * kPanel + (k % 4) * 32;
                mma_f16_ss(s_of(n & 1), tc::smem_desc_sw128(q_at + part * W::kOperand + off), tc::smem_desc_sw128(stage_at + stage * W::kOperand + off), idesc, add);
                add = 1;
              }
            }
            tc::mma_commit(&st.s_full[n & 1]);
            tc::mma_commit(&st.stage_empty[stage]);
          }
        }
        tc::mma_commit(&st.drained[0]);
        drain(&st.drained[0], 0, status);
      }
    } else if (warp == kIssue + 1) {
      // ----------------------------------------------------- O = P V
      if (lane == 0) {
        constexpr uint32_t kAcross = 1u << 16;
        const uint32_t idesc = tc::make_idesc(kRows, DT) | kAcross;
#pragma unroll 1
        for (int n = 0; n < tiles; ++n) {
          const int at = place_of_v(n), stage = at % W::kStages;
          wait(&st.stage_full[stage], at / W::kStages);
          wait(&st.p_full[n & 1], n >> 1);
          if (alive) {
            tc::tc_fence_after();
            uint32_t add = 0;
#pragma unroll 1
            for (int part = 1; part >= 0; --part) {
#pragma unroll
              for (int k = 0; k < kTile / 16; ++k) {
                tc::mma_f16_ta(o_of(n & 1), s_of(n & 1) + 16 * k + 8 * part, across_desc(stage_at + stage * W::kOperand + k * 2048), idesc, add);
                add = 1;
              }
            }
            tc::mma_commit(&st.o_full[n & 1]);
            tc::mma_commit(&st.stage_empty[stage]);
          }
        }
        tc::mma_commit(&st.drained[1]);
        drain(&st.drained[1], 0, status);
      }
    } else if (warp == kIssue + 2) {
      // ----------------------------------------------------- pages
      const int64_t head_row = (int64_t)hk << c.page_shift;
      const int half = lane & 7;
#pragma unroll 1
      for (int n = 0; n < tiles; ++n) {
        const int entry = n % kEntries;
        const uint32_t t = begin + n * kTile + 16 * half;
        int64_t at = -1, row = 0;
        if (t < len) {
          if (n > 0) page = table[t >> c.page_shift];
          if (page >= 0 && page < c.num_pages) {
            const int64_t in_page = head_row + (t & ((1u << c.page_shift) - 1)), page_row = ((int64_t)page * c.heads) << c.page_shift;
            row = page_row + in_page;
            at = W::kBf16 ? (int64_t)page << 32 | in_page : row;
          }
        }
        if (n >= kEntries) wait(&st.meta_empty[entry], n / kEntries - 1);
        if (lane < 8) st.entries[entry].row[half] = at;
        const uint32_t ok = __ballot_sync(kFullMask, at >= 0) & 0xffu;
        if (lane == 0) st.entry_ok[entry] = ok;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&st.meta_full[entry]);
        if (n > 0 && lane < 16 && at >= 0) {  // 16 tokens of a head are one run of bytes
          const uint8_t* from = static_cast<const uint8_t*>(lane < 8 ? c.k : c.v) + row * D * W::kBytes;
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(16 * D * W::kBytes) : "memory");
        }
      }
    } else {
      // ----------------------------------------------------- copies of the cache's rows, or of their steps: a lane a page's
      // part of the tile by TMA (16 tokens a lane: 51.9 us for 51.0 of 64 rows over 16384 tokens of 8 key heads of 128, ~110 cycles a
      // copy, one after the other), 16 tokens by bulk copies (a page's part: 55.4 for 52.0, fp8).
      const int half = lane & 7, run = W::kBf16 ? min(kTile, 1 << c.page_shift) : 16;
      const bool leads = (16 * half & (run - 1)) == 0;
#pragma unroll 1
      for (int i = 0; i < 2 * tiles; ++i) {
        int operand, n;
        at_place(i, operand, n);
        const int entry = n % kEntries, stage = i % W::kStages;
        if (!operand) wait(&st.meta_full[entry], n / kEntries);
        const int64_t first = st.entries[entry].row[half];
        const int rows = min(run, (int)(len - begin) - n * kTile - 16 * half);
        if constexpr (W::kBf16) {
          // by TMA into their place as an operand, a lane a panel of the page's; whole boxes, of which the tokens that are
          // not there do not count
          if (i >= W::kStages) wait(&st.stage_empty[stage], i / W::kStages - 1);
          unsigned long long* bar = operand ? &st.raw_full[stage] : &st.stage_full[stage];
          const bool copies = alive && first >= 0 && rows > 0 && leads && lane < 8 * W::kPanels;
          const uint32_t all = __popc(__ballot_sync(kFullMask, copies)) * 128u * run;
          if (!operand && lane < kBringThreads / 32 - 1) tc::mbar_arrive(bar);  // as many arrive as where warps widen
          if (lane == 31) tc::mbar_arrive_expect_tx(bar, all);
          __syncwarp();
          if (copies)
            asm volatile(
                "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                    stage_at + stage * W::kOperand + (lane >> 3) * kPanel + half * 2048),
                "l"(reinterpret_cast<uint64_t>(operand ? &maps.values : &maps.keys)), "r"((lane >> 3) * 64), "r"((int)first), "r"((int)(first >> 32)),
                "r"(tc::smem_u32(bar))
                : "memory");
        } else {
          const int slot = i % W::kRaws;
          if (i >= W::kRaws) wait(&st.raw_empty[slot], i / W::kRaws - 1);
          const bool copies = alive && first >= 0 && rows > 0 && leads && lane < (operand ? 8 : 24);  // rows; k's steps, v's steps
          const uint32_t bytes = lane < 8 ? rows * D : (rows + 15) / 16 * 64;
          const uint32_t all = __reduce_add_sync(kFullMask, copies ? bytes : 0u);
          if (lane == 0) tc::mbar_arrive_expect_tx(&st.raw_full[slot], all);
          __syncwarp();
          if (copies) {
            if (lane < 8)
              tc::bulk_copy_g2s(raw_at + slot * W::kRaw + 16 * half * D, static_cast<const uint8_t*>(operand ? c.v : c.k) + first * D, bytes, &st.raw_full[slot]);
            else
              tc::bulk_copy_g2s((uint32_t)__cvta_generic_to_shared(&(lane < 16 ? st.k_steps : st.v_steps)[entry][16 * half]), (lane < 16 ? c.k_step : c.v_step) + first, bytes, &st.raw_full[slot]);
          }
        }
        __syncwarp();
      }
    }
    __syncwarp();
  }
  tc::tc_fence_before();
  __syncthreads();
  // No copy is on its way when the CTA ends.  Each was waited for by the role that used it, but after a wait that has
  // run out, in whatever role: then for a millisecond, long after the last one.
  if (warp == kIssue + 3 && lane == 0 && *reinterpret_cast<volatile int*>(&st.abort_flag)) {
    const unsigned long long t0 = tc::global_timer();
#pragma unroll 1
    while (tc::global_timer() - t0 < 1000000ull) {
    }
  }
  if (warp == kIssue) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <int FORMAT, int DT>
cudaError_t launch_shape(const AttendArgs& a, const KvPages& c, Shares sh, int64_t rows, bool pdl, const DeviceInfo& dev,
                         cudaStream_t stream) {
  using W = Wide<FORMAT, DT>;
  const auto kernel = prefix_wide_kernel<FORMAT, DT>;
  static thread_local int configured_device = -1;
  if (configured_device != dev.device) {
    cudaFuncAttributes built;
    cudaError_t err = cudaFuncGetAttributes(&built, kernel);
    if (err == cudaSuccess && built.numRegs != kLaunchRegisters) err = cudaErrorInvalidKernelImage;  // what its groups share out
    if (err == cudaSuccess) err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, W::kSmem);
    if (err != cudaSuccess) return err;
    configured_device = dev.device;
  }
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.blockDim = dim3(kWideThreads, 1, 1);
  cfg.dynamicSmemBytes = W::kSmem;
  if (pdl) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
  }
  const int sms = dev.num_sms < kSms ? dev.num_sms : kSms;
  const int64_t steps = ((a.max_pages << c.page_shift) + kTile - 1) / kTile;
  sh.splits = wide_splits(a.B, rows, steps, sms);
  cfg.gridDim = dim3((unsigned)(sh.splits ? rows * sh.splits : sms), 1, 1);
  Maps maps = {};
  if constexpr (W::kBf16) {
    const cuuint64_t sizes[3] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.heads << c.page_shift, (cuuint64_t)c.num_pages};
    const cuuint64_t strides[2] = {sizes[0] * 2, sizes[0] * sizes[1] * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)(1 << c.page_shift < kTile ? 1 << c.page_shift : kTile), 1}, each[3] = {1, 1, 1};
    const EncodeTiledFn encode = encode_fn();
    for (int i = 0; i < 2; ++i)
      if (!encode || encode(i ? &maps.values : &maps.keys, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, i ? c.v : c.k, sizes, strides, box, each,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorUnknown;
  }
  return cudaLaunchKernelEx(&cfg, kernel, a, c, sh, maps, dev.status);
}

}  // namespace

cudaError_t launch_prefix_wide(const AttendArgs& a, const KvPages& c, const PrefixRows& p, bool pdl, const DeviceInfo& dev,
                               cudaStream_t stream) {
  Shares sh = {};
  sh.group = p.group;
  sh.groups = p.tiles;
  sh.rows_a_seq = c.heads * p.tiles;
  sh.parts = p.parts;
  sh.rows = p.rows;
  sh.group_rows = p.group_rows;
  sh.lengths = p.lengths;
  sh.heads_a_key = p.heads_a_key;
  sh.slot_heads = p.slot_heads;
  const int64_t rows = a.B * sh.rows_a_seq;
  return of_shape(c, [&](auto format, auto dims) {
    constexpr int kDims = decltype(dims)::value;
    if constexpr (kDims <= 128)
      return launch_shape<decltype(format)::value, kDims>(a, c, sh, rows, pdl, dev, stream);
    else
      return cudaErrorInvalidValue;  // not asked for
  });
}

}  // namespace bitlinear
