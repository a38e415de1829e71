// rope_kv.cu -- rotary positions and the paged key-value cache: rows rotated,
// quantised and written where their page is, and read back.
//
// Rotation ("Hesper.Models.BitNet" page, section "Configuration": ropeBase):
// pair i of a head turns by the angle positions[t] * freq[i].  The angle is kept in
// turns as a 64-bit fraction, positions times the frequency's fraction modulo 2^64, so
// whole turns drop out exactly.  It is off by what rounds the frequency's fraction (1.5 *
// 2^-53 of it for 1 / (2 pi) and the product, and 2^-65 turns for the last place), times the
// position, and by what the series drop of it (below 2^-48 turns).
// What is left of the nearest quarter turn, |a| <= pi / 4, becomes a pair of fp32
// (leading part and rest), its sine and cosine the Taylor series with the first three
// terms in such pairs, rounded once to fp32: the nearest fp32 value to those of that angle
// but for one in ~10^4.  (In fp64 the same took ~20 instructions a pair of a pipe that takes one in
// ~14 cycles: 3 us of 11 for 2048 tokens of 32 heads.)  The
// rotation itself is two fp32 products and one sum, unfused, so that it can be
// repeated bit for bit.
//
// Quantisation follows activation_quant, a row being one (token, head):
//   int8: code = clamp(rne(x * s), -128, 127), s = 127 * (1 / a), a = max(max|x|, 1e-5)
//   e4m3: code = e4m3(x * s), s = 448 * (1 / a), round to nearest even, saturating
// with step = a / 127 or a / 448, the fp32 value of one unit; bf16 rounds.
//
// Layout: four or eight lanes hold a row, each 16-byte chunks in pairs; the chunks of
// a pair are the two halves of the same rotated dims, so both of a rotation's operands
// and its angle are one lane's (loading the partners a second time took 5 us of 27 for
// 2039 tokens), and nearly every lane has a chunk in every load whatever the head size
// (80 dims fill 20 of 24; 20 of 32 with a row a warp).  A warp works alone: one token,
// or a share of its heads while tokens alone do not fill the GPU, with the next turn's
// rows loaded before this one's are used and the token's sines and cosines in its own
// shared memory, so no barrier holds it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kv.cuh"

namespace bitlinear {
namespace {

constexpr int kMaxHead = 256;     // head_dim limit
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

// The fraction of a turn that a position adds, in units of 2^-64 turns.
__device__ __forceinline__ uint64_t turn_fraction(double freq) {
  const uint64_t bits = (uint64_t)__double_as_longlong(freq * 0.15915494309189533577);
  const int shift = (int)((bits >> 52) & 0x7ff) - 1011;  // mantissa * 2^(exponent - 1075) turns
  const uint64_t m = (bits & 0xfffffffffffffull) | 0x10000000000000ull;
  uint64_t f;
  if (shift >= 0)
    f = shift < 64 ? m << shift : 0;
  else
    f = shift > -54 ? ((m >> (-shift - 1)) + 1) >> 1 : 0;
  return (bits >> 63) ? 0 - f : f;
}

// Sine and cosine of `phase` / 2^64 turns.  h and l name a value's leading part and
// rest; a product's rest is an exact fma, and a sum's follows from larger + smaller.
__device__ __forceinline__ void sin_cos_turns(uint64_t phase, float* sine, float* cosine) {
  const uint64_t from_eighth = phase + (1ull << 61);
  const int quarter = (int)(from_eighth >> 62);
  const int64_t r = (int64_t)(from_eighth & ((1ull << 62) - 1)) - (1ll << 61);
  const float top = (float)(int)(r >> 40), low = (float)((uint32_t)(r >> 16) & 0xffffffu) * 5.9604644775390625e-8f;
  // a = 2 pi / 2^24 (top + low)
  constexpr float kH = 3.7450704e-07f, kL = -1.0421607e-14f;
  float h = top * kH, l = fmaf(low, kH, fmaf(top, kL, fmaf(top, kH, -h)));
  const float ah = h + l, al = l - (ah - h);
  const float uh = ah * ah, ul = fmaf(ah + ah, al, fmaf(ah, ah, -uh));  // a^2
  const float zh = uh * uh, zl = fmaf(uh + uh, ul, fmaf(uh, uh, -zh));  // a^4
  // sin a = a + a q, q = -a^2 / 3! + a^4 / 5! + a^4 (-a^2 / 7! + a^4 / 9! - a^6 / 11!)
  constexpr float k6H = 0.16666667f, k6L = -4.967054e-09f, k120H = 0.008333334f, k120L = -4.346172e-10f;
  h = zh * k120H;
  l = fmaf(zl, k120H, fmaf(zh, k120L, fmaf(zh, k120H, -h)));
  l = fmaf(zh, uh * fmaf(uh, fmaf(uh, -1.0f / 39916800.0f, 1.0f / 362880.0f), -1.0f / 5040.0f), l);
  const float th = uh * k6H, tl = fmaf(ul, k6H, fmaf(uh, k6L, fmaf(uh, k6H, -th)));
  const float qh = h - th, ql = ((-th - qh) + h) + (l - tl);
  const float ch = ah * qh, cl = fmaf(al, qh, fmaf(ah, ql, fmaf(ah, qh, -ch))) + al;
  const float sh = ah + ch, s = sh + ((ch - (sh - ah)) + cl);
  // cos a = 1 - a^2 / 2! + a^4 / 4! + a^4 (-a^2 / 6! + a^4 / 8! - a^6 / 10! + a^8 / 12!)
  constexpr float k24H = 0.041666668f, k24L = -1.2417635e-09f;
  const float yh = zh * k24H;
  float yl = fmaf(zl, k24H, fmaf(zh, k24L, fmaf(zh, k24H, -yh)));
  yl = fmaf(zh, uh * fmaf(uh, fmaf(uh, fmaf(uh, 1.0f / 479001600.0f, -1.0f / 3628800.0f), 1.0f / 40320.0f), -1.0f / 720.0f), yl);
  const float dh = -0.5f * uh, dl = -0.5f * ul;
  const float c1 = 1.0f + dh, e1 = dh - (c1 - 1.0f), c2 = c1 + yh, e2 = yh - (c2 - c1);
  const float c = c2 + ((e1 + e2) + (dl + yl));
  const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;
  *cosine = quarter == 1 || quarter == 2 ? -x : x;
  *sine = quarter >= 2 ? -y : y;
}

// cos and sin of every pair of one position, into the warp's shared memory; two pairs
// a lane side by side, their chains of operations overlapping.
__device__ __forceinline__ void fill_angles(const RopeArgs& r, int32_t pos, float2* cs) {
  const int n = r.rot_dim / 2;
  const uint64_t p = (uint64_t)(int64_t)pos;
  for (int i = threadIdx.x & 31; i < n; i += 64) {
    const double f0 = r.freq[i], f1 = r.freq[min(i + 32, n - 1)];
    float s0, c0, s1, c1;
    sin_cos_turns(turn_fraction(f0) * p, &s0, &c0);
    sin_cos_turns(turn_fraction(f1) * p, &s1, &c1);
    cs[i] = make_float2(__fmul_rn(c0, r.amplitude), __fmul_rn(s0, r.amplitude));
    if (i + 32 < n) cs[i + 32] = make_float2(__fmul_rn(c1, r.amplitude), __fmul_rn(s1, r.amplitude));
  }
  __syncwarp();
}

// Asks for `rows` rows of D floats to come into L2, by one lane.
__device__ __forceinline__ void rows_to_l2(const float* row, int rows, int D) {
  if (rows > 0) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(row), "r"(rows * D * 4) : "memory");
}

// A warp's work: units first <= u < end of one token, ROWS a turn.
struct Task {
  int64_t token;
  int first, end;
};
template <int ROWS>
__device__ __forceinline__ Task task_of_warp(int64_t T, int units, int shares) {
  const uint32_t w = blockIdx.x * kWarps + (threadIdx.x >> 5);  // T <= 2^30, and more than one share only of few
  const uint32_t token = shares == 1 ? w : w / (uint32_t)shares, share = w - token * shares;
  const uint32_t turns = (units + ROWS - 1) / ROWS;
  Task t = {token, (int)(turns * share / shares * ROWS), (int)(turns * (share + 1) / shares * ROWS)};
  t.end = t.token < T ? min(t.end, units) : t.first;
  return t;
}

// A head size and where a lane's chunks are: DX dims known at compile time, or, DX == 0,
// any up to 8 * L * NP.  Pair p = j + L i of lane j of a row is chunks p and p + together
// for p < together (the pairs of a rotation by halves), else the next two in order.
template <int NP_, int L_, int DX>
struct Head {
  static constexpr int NP = NP_, L = L_, kRows = 32 / L;
  static constexpr int kCtas = NP == 1 ? 8 : NP == 2 ? 5 : 4;        // CTAs an SM, without spilled registers up to 128 dims (4 bytes of 96)
  static constexpr int kReadCtas = NP == 1 ? 12 : NP <= 3 ? 8 : 6;  // the same of the reading kernel
  int D, j, a[NP], b[NP];  // first dims of the two chunks of each pair
  __device__ __forceinline__ Head(int dims, int together) : D(DX ? DX : dims), j((threadIdx.x & 31) % L) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int p = j + L * i;
      a[i] = 4 * (p < together ? p : 2 * p);
      b[i] = 4 * (p < together ? p + together : 2 * p + 1);
    }
  }
  __device__ __forceinline__ bool has_a(int i) const { return 8 * L * (i + 1) <= DX || 8 * (j + L * i) < D; }
  __device__ __forceinline__ bool has_b(int i) const { return has_a(i) && (DX || b[i] < D); }
};
// How many pairs of chunks a rotation keeps together in heads of D dims.
__host__ __device__ __forceinline__ int pairs_together(int D, const RopeArgs& r) {
  return r.freq && r.layout == BITLINEAR_ROPE_HALF && r.rot_dim % 8 == 0 ? r.rot_dim / 8 : D / 8;
}

// The lane's chunks of a row.
template <typename H>
struct Row {
  float4 a[H::NP], b[H::NP];
};
template <typename H>
__device__ __forceinline__ void load_row(const H& head, const float* row, Row<H>& v) {
  const float4 none = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < H::NP; ++i) {
    v.a[i] = head.has_a(i) ? *reinterpret_cast<const float4*>(row + head.a[i]) : none;
    v.b[i] = head.has_b(i) ? *reinterpret_cast<const float4*>(row + head.b[i]) : none;
  }
}
template <typename H>
__device__ __forceinline__ void store_row(const H& head, float* row, const Row<H>& v) {
#pragma unroll
  for (int i = 0; i < H::NP; ++i) {
    if (head.has_a(i)) *reinterpret_cast<float4*>(row + head.a[i]) = v.a[i];
    if (head.has_b(i)) *reinterpret_cast<float4*>(row + head.b[i]) = v.b[i];
  }
}

// own * c + other * s, each step rounded; the first of a pair takes -s.
__device__ __forceinline__ float turn(float own, float other, float c, float s) {
  return __fadd_rn(__fmul_rn(own, c), __fmul_rn(other, s));
}
__device__ __forceinline__ void turn_halves(float4& v, float4& o, const float2* cs) {
  const float4 p = reinterpret_cast<const float4*>(cs)[0], q = reinterpret_cast<const float4*>(cs)[1];
  const float4 x = make_float4(turn(v.x, o.x, p.x, -p.y), turn(v.y, o.y, p.z, -p.w), turn(v.z, o.z, q.x, -q.y), turn(v.w, o.w, q.z, -q.w));
  o = make_float4(turn(o.x, v.x, p.x, p.y), turn(o.y, v.y, p.z, p.w), turn(o.z, v.z, q.x, q.y), turn(o.w, v.w, q.z, q.w));
  v = x;
}
// Interleaved pairs of the chunk at dim d, of which those below rot turn.
__device__ __forceinline__ void turn_pairs(float4& v, const float2* cs, int d, int rot) {
  const float4 p = *reinterpret_cast<const float4*>(cs + d / 2);
  if (d < rot) {
    const float x = turn(v.x, v.y, p.x, -p.y);
    v.y = turn(v.y, v.x, p.x, p.y);
    v.x = x;
  }
  if (d + 2 < rot) {
    const float z = turn(v.z, v.w, p.z, -p.w);
    v.w = turn(v.w, v.z, p.z, p.w);
    v.z = z;
  }
}
// Halves whose length is no multiple of a chunk: the partners come from the row again.
__device__ __forceinline__ void turn_scattered(float4& v, const float* row, const float2* cs, int d0, int rot) {
  float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int d = d0 + k, n = rot / 2, other = d < n ? d + n : d - n;
    if (d >= rot) continue;
    const float2 p = cs[min(d, other)];
    e[k] = turn(e[k], row[other], p.x, d < n ? -p.y : p.y);
  }
  v = make_float4(e[0], e[1], e[2], e[3]);
}

// Rotates the lane's chunks (of the row at `row`) in registers.
template <typename H>
__device__ __forceinline__ void rotate_row(const H& head, const float* row, const RopeArgs& r, const float2* cs,
                                           Row<H>& v) {
  if (r.layout == BITLINEAR_ROPE_INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < H::NP; ++i) {
      if (head.has_a(i)) turn_pairs(v.a[i], cs, head.a[i], r.rot_dim);
      if (head.has_b(i)) turn_pairs(v.b[i], cs, head.b[i], r.rot_dim);
    }
  } else if (r.rot_dim % 8 == 0) {
#pragma unroll
    for (int i = 0; i < H::NP; ++i)
      if (head.has_a(i) && 2 * head.a[i] < r.rot_dim) turn_halves(v.a[i], v.b[i], cs + head.a[i]);
  } else {
#pragma unroll
    for (int i = 0; i < H::NP; ++i) {
      if (head.has_a(i)) turn_scattered(v.a[i], row, cs, head.a[i], r.rot_dim);
      if (head.has_b(i)) turn_scattered(v.b[i], row, cs, head.b[i], r.rot_dim);
    }
  }
}

// Lanes past the last head of a turn repeat it: no turn asks whether a lane has a row.
template <typename H>
__global__ void __launch_bounds__(kThreads, H::kCtas)
rope_kernel(const float* x, int64_t x_stride, int64_t T, int heads, int D, int shares, bool early,
            const int32_t* __restrict__ positions, RopeArgs r, float* y, int64_t y_stride) {
  __shared__ __align__(16) float2 angles[kWarps][kMaxHead / 2];
  pdl_release_dependents();
  pdl_wait_primary();
  const H head(D, pairs_together(D, r));
  const Task task = task_of_warp<H::kRows>(T, heads, shares);
  if (task.first >= task.end) return;
  float2* cs = angles[threadIdx.x >> 5];
  const int sub = (threadIdx.x & 31) / H::L;
  x += task.token * x_stride;
  y += task.token * y_stride;
  int at = task.first, h = min(at + sub, task.end - 1);
  if (early && (threadIdx.x & 31) == 0) rows_to_l2(x + (at + H::kRows) * head.D, task.end - at - H::kRows, head.D);
  Row<H> v;
  load_row(head, x + h * head.D, v);
  fill_angles(r, positions[task.token], cs);
  while (true) {
    at += H::kRows;
    const int h_next = min(at + sub, task.end - 1);
    Row<H> next;
    if (at < task.end) load_row(head, x + h_next * head.D, next);
    rotate_row(head, x + h * head.D, r, cs, v);
    __syncwarp();  // y may be x: a row is read before it is written
    store_row(head, y + h * head.D, v);
    if (at >= task.end) return;
    h = h_next;
    v = next;
  }
}

// Four floats as codes of 8 bits, x * s each.
template <int FORMAT>
__device__ __forceinline__ uint32_t codes_of(const float4& v, float s) {
  float e[4] = {__fmul_rn(v.x, s), __fmul_rn(v.y, s), __fmul_rn(v.z, s), __fmul_rn(v.w, s)};
  if constexpr (FORMAT == BITLINEAR_KV_INT8) {
    // |x * s| <= 127 (1 + 2^-22): plus 1.5 * 2^23 the sum's last bits are the code, rounded half to even
#pragma unroll
    for (int k = 0; k < 4; ++k) e[k] = __fadd_rn(e[k], 12582912.0f);
    return __byte_perm(__byte_perm(__float_as_uint(e[0]), __float_as_uint(e[1]), 0x0040),
                       __byte_perm(__float_as_uint(e[2]), __float_as_uint(e[3]), 0x0040), 0x5410);
  } else {
    return e4m3x2(e[1], e[0]) | e4m3x2(e[3], e[2]) << 16;
  }
}
__device__ __forceinline__ uint2 bf16_of(const float4& v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ float largest(float a, const float4& v) {
  return fmaxf(fmaxf(a, fmaxf(fabsf(v.x), fabsf(v.y))), fmaxf(fabsf(v.z), fabsf(v.w)));
}

// Quantises a row held by its lanes and writes codes and step.  Only the row's
// lanes need to be here (a warp may hold q rows beside it).
template <int FORMAT, typename H>
__device__ __forceinline__ void write_row(const H& head, const Row<H>& v, int64_t row, void* codes, float* steps) {
  if constexpr (FORMAT == BITLINEAR_KV_BF16) {
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(codes) + row * head.D;
#pragma unroll
    for (int i = 0; i < H::NP; ++i) {
      if (head.has_a(i)) *reinterpret_cast<uint2*>(out + head.a[i]) = bf16_of(v.a[i]);
      if (head.has_b(i)) *reinterpret_cast<uint2*>(out + head.b[i]) = bf16_of(v.b[i]);
    }
  } else {
    constexpr float kTop = FORMAT == BITLINEAR_KV_INT8 ? 127.0f : 448.0f;
    const unsigned lanes = ((1u << H::L) - 1) << ((threadIdx.x & 31) / H::L * H::L);
    float a = 1e-5f;
#pragma unroll
    for (int i = 0; i < H::NP; ++i) a = largest(largest(a, v.a[i]), v.b[i]);
#pragma unroll
    for (int o = 1; o < H::L; o <<= 1) a = fmaxf(a, __shfl_xor_sync(lanes, a, o));
    const float s = __fmul_rn(__frcp_rn(a), kTop);
    uint8_t* out = static_cast<uint8_t*>(codes) + row * head.D;
#pragma unroll
    for (int i = 0; i < H::NP; ++i) {
      if (head.has_a(i)) *reinterpret_cast<uint32_t*>(out + head.a[i]) = codes_of<FORMAT>(v.a[i], s);
      if (head.has_b(i)) *reinterpret_cast<uint32_t*>(out + head.b[i]) = codes_of<FORMAT>(v.b[i], s);
    }
    if (head.j == 0) steps[row] = __fdiv_rn(a, kTop);
  }
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

template <int FORMAT, typename H>
__global__ void __launch_bounds__(kThreads, H::kCtas)
append_kernel(Append a, KvRows rows, RopeArgs r, KvPages c, int shares) {
  __shared__ __align__(16) float2 angles[kWarps][kMaxHead / 2];
  pdl_release_dependents();
  pdl_wait_primary();
  const H head(c.head_dim, pairs_together(c.head_dim, r));
  const int units = a.q_heads + 2 * c.heads;
  const Task task = task_of_warp<H::kRows>(rows.T, units, shares);
  if (task.first >= task.end) return;
  float2* cs = angles[threadIdx.x >> 5];
  const int64_t t = task.token;
  const int sub = (threadIdx.x & 31) / H::L;
  const float* qt = a.q + t * a.q_stride;
  const float* kt = a.k + t * a.k_stride;
  const float* vt = a.v + t * a.v_stride;
  float* qo = a.q_out + t * a.q_out_stride;
  auto input = [&](int u) {
    const int kv = u - a.q_heads;
    return kv < 0 ? qt + u * head.D : kv < c.heads ? kt + kv * head.D : vt + (kv - c.heads) * head.D;
  };
  int at = task.first, u = min(at + sub, task.end - 1);
  const float* in = input(u);
  Row<H> v;
  load_row(head, in, v);
  const int64_t place = kv_place(rows, c, t);
  if (r.freq && at < a.q_heads + c.heads) fill_angles(r, rows.positions[t], cs);
  if (place < 0) return;
  while (true) {
    at += H::kRows;
    const int u_next = min(at + sub, task.end - 1);
    const float* in_next = input(u_next);
    Row<H> next;
    if (at < task.end) load_row(head, in_next, next);
    const int kv = u - a.q_heads;
    const bool is_v = kv >= c.heads;
    if (!is_v && r.freq) rotate_row(head, in, r, cs, v);
    __syncwarp();  // q_out may be q: a row is read before it is written
    if (kv < 0) {
      store_row(head, qo + u * head.D, v);
    } else {
      const int64_t row = place + ((int64_t)(is_v ? kv - c.heads : kv) << c.page_shift);
      write_row<FORMAT>(head, v, row, is_v ? c.v : c.k, is_v ? c.v_step : c.k_step);
    }
    if (at >= task.end) return;
    u = u_next;
    in = in_next;
    v = next;
  }
}

// The codes of a chunk (8-bit: one word) as floats.
template <int FORMAT>
__device__ __forceinline__ float4 widened(uint32_t w) {
  if constexpr (FORMAT == BITLINEAR_KV_INT8) {
    return make_float4((float)(int8_t)w, (float)(int8_t)(w >> 8), (float)(int8_t)(w >> 16), (float)(int8_t)(w >> 24));
  } else {
    const uint32_t lo = half2_of_e4m3x2((uint16_t)w), hi = half2_of_e4m3x2((uint16_t)(w >> 16));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo)), b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return make_float4(a.x, a.y, b.x, b.y);
  }
}

// The lane's chunks of a row of codes: a word each of 8-bit codes, two of bf16.
template <int FORMAT, typename H>
struct CodeRow {
  uint2 a[H::NP], b[H::NP];
  float step;
};
template <int FORMAT>
__device__ __forceinline__ uint2 load_codes(const uint8_t* row, int d) {
  if constexpr (FORMAT == BITLINEAR_KV_BF16) return *reinterpret_cast<const uint2*>(row + 2 * d);
  return make_uint2(*reinterpret_cast<const uint32_t*>(row + d), 0u);
}
template <int FORMAT>
__device__ __forceinline__ float4 values_of(const uint2& w, float step) {
  if constexpr (FORMAT == BITLINEAR_KV_BF16)
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
  const float4 e = widened<FORMAT>(w.x);
  return make_float4(__fmul_rn(e.x, step), __fmul_rn(e.y, step), __fmul_rn(e.z, step), __fmul_rn(e.w, step));
}

template <int FORMAT, typename H>
__global__ void __launch_bounds__(kThreads, H::kReadCtas)
read_kernel(KvPages c, KvRows rows, int shares, float* __restrict__ k_out, int64_t k_stride,
            float* __restrict__ v_out, int64_t v_stride) {
  pdl_release_dependents();
  pdl_wait_primary();
  const H head(c.head_dim, c.head_dim / 8);
  const Task task = task_of_warp<H::kRows>(rows.T, 2 * c.heads, shares);
  if (task.first >= task.end) return;
  const int64_t t = task.token, place = kv_place(rows, c, t);
  if (place < 0) return;
  const int sub = (threadIdx.x & 31) / H::L;
  float* kt = k_out + t * k_stride;
  float* vt = v_out + t * v_stride;
  auto fetch = [&](int u, CodeRow<FORMAT, H>& w) {
    const bool is_v = u >= c.heads;
    const int64_t row = place + ((int64_t)(is_v ? u - c.heads : u) << c.page_shift);
    const uint8_t* codes = static_cast<const uint8_t*>(is_v ? c.v : c.k) + row * head.D * (FORMAT == BITLINEAR_KV_BF16 ? 2 : 1);
#pragma unroll
    for (int i = 0; i < H::NP; ++i) {
      w.a[i] = head.has_a(i) ? load_codes<FORMAT>(codes, head.a[i]) : make_uint2(0u, 0u);
      w.b[i] = head.has_b(i) ? load_codes<FORMAT>(codes, head.b[i]) : make_uint2(0u, 0u);
    }
    w.step = FORMAT == BITLINEAR_KV_BF16 ? 1.0f : (is_v ? c.v_step : c.k_step)[row];
  };
  int at = task.first, u = min(at + sub, task.end - 1);
  CodeRow<FORMAT, H> w;
  fetch(u, w);
  while (true) {
    at += H::kRows;
    const int u_next = min(at + sub, task.end - 1);
    CodeRow<FORMAT, H> next;
    if (at < task.end) fetch(u_next, next);
    Row<H> v;
#pragma unroll
    for (int i = 0; i < H::NP; ++i) {
      v.a[i] = values_of<FORMAT>(w.a[i], w.step);
      v.b[i] = values_of<FORMAT>(w.b[i], w.step);
    }
    store_row(head, u >= c.heads ? vt + (u - c.heads) * head.D : kt + u * head.D, v);
    if (at >= task.end) return;
    u = u_next;
    w = next;
  }
}

// Warps that share a token's units.  A warp's time is its turns and about two more
// (the lookups, the angles, the first rows' way), and warps beyond those resident wait
// for a whole round: the number that makes rounds * time least.  (2039 tokens of 96
// heads of 80: one warp a token 20.4 us, two 25.9.)
int shares_for(int64_t T, int units, int rows, int ctas, const DeviceInfo& dev) {
  const int64_t resident = (int64_t)dev.num_sms * ctas * kWarps;
  const int turns = (units + rows - 1) / rows;
  int best = 1;
  double least = 0.0;
  for (int s = 1; s <= turns; ++s) {
    const double time = (double)((T * s + resident - 1) / resident) * ((turns + s - 1) / s + 2);
    if (s == 1 || time < least) {
      least = time;
      best = s;
    }
    if (T * s >= 8 * resident) break;
  }
  return best;
}

// Whether a token's rows are all asked for (into L2) before the first one's turn: when
// warps come in three rounds or more.  Measured without / with: 16384 tokens of 32 heads of
// 80 55.9 / 50.7 us, 8192 30.7 / 28.7, 2048 9.6 / 10.7.  (Appending has three times the
// rows: all at once displace one another, 128 / 142 us for 16384 tokens; a turn more ahead
// 128 / 123, but 0.1 to 0.3 us more for few tokens, where the kernel carries it unused.)
bool early_for(int64_t warps, int ctas, const DeviceInfo& dev) { return warps >= 3 * (int64_t)dev.num_sms * ctas * kWarps; }

template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), int64_t warps, bool pdl, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((warps + kWarps - 1) / kWarps), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// f(type) with the Head of D dims: of its own up to 128 in steps that models use, else of any.
template <typename T>
struct Tag {
  using type = T;
};
template <typename F>
cudaError_t with_head(int D, F f) {
  switch (D) {
    case 64: return f(Tag<Head<1, 8, 64>>());
    case 80: return f(Tag<Head<3, 4, 80>>());
    case 96: return f(Tag<Head<3, 4, 96>>());
    case 128: return f(Tag<Head<2, 8, 128>>());
    default: return D <= 128 ? f(Tag<Head<2, 8, 0>>()) : f(Tag<Head<4, 8, 0>>());
  }
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
  return with_head(D, [&](auto head) {
    const int shares = shares_for(T, H, decltype(head)::type::kRows, decltype(head)::type::kCtas, dev);
    return launch(rope_kernel<typename decltype(head)::type>, T * shares, pdl, stream, x, x_stride, T, H, D, shares,
                  early_for(T * shares, decltype(head)::type::kCtas, dev), positions, rope, y, y_stride);
  });
}

cudaError_t launch_kv_append(const float* q, int64_t q_stride, int q_heads, float* q_out, int64_t q_out_stride,
                             const float* k, int64_t k_stride, const float* v, int64_t v_stride, const KvRows& rows,
                             const RopeArgs& rope, const KvPages& cache, bool pdl, const DeviceInfo& dev,
                             cudaStream_t stream) {
  const Append a = {q, k, v, q_out, q_stride, k_stride, v_stride, q_out_stride, q_heads};
  return with_format(cache.format, [&](auto fmt) {
    return with_head(cache.head_dim, [&](auto head) {
      const int shares = shares_for(rows.T, q_heads + 2 * cache.heads, decltype(head)::type::kRows, decltype(head)::type::kCtas, dev);
      return launch(append_kernel<decltype(fmt)::value, typename decltype(head)::type>, rows.T * shares, pdl, stream,
                    a, rows, rope, cache, shares);
    });
  });
}

cudaError_t launch_kv_read(const KvPages& cache, const KvRows& rows, float* k_out, int64_t k_stride, float* v_out,
                           int64_t v_stride, bool pdl, const DeviceInfo& dev, cudaStream_t stream) {
  return with_format(cache.format, [&](auto fmt) {
    return with_head(cache.head_dim, [&](auto head) {
      const int shares = shares_for(rows.T, 2 * cache.heads, decltype(head)::type::kRows, decltype(head)::type::kReadCtas, dev);
      return launch(read_kernel<decltype(fmt)::value, typename decltype(head)::type>, rows.T * shares, pdl, stream,
                    cache, rows, shares, k_out, k_stride, v_out, v_stride);
    });
  });
}

}  // namespace bitlinear
