// shares.h -- the arithmetic by which attention.cu shares rows out over CTAs in proportion
// to their steps, and by which attention_shared.cu, attention_prefix.cu and select.cu choose their way and
// their CTAs.  Plain functions of numbers, for the host, the device and tests.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define BITLINEAR_BOTH __host__ __device__ __forceinline__
#else
#define BITLINEAR_BOTH inline
#endif

namespace bitlinear {

// Whether the steps of `rows` rows, `steps` each at most, are counted in 31 bits.
BITLINEAR_BOTH bool steps_fit(int64_t rows, int64_t steps) { return steps <= 0x7fffffff / rows; }

// Steps that a CTA has at most, so that rows of ceil(steps / share) CTAs each, `total` steps
// in all, fit `spare` CTAs beside one a row.  total may be 2^31 - 1, and total + spare more.
BITLINEAR_BOTH int share_of_steps(int total, int spare, int least) {
  const int share = (int)(((uint32_t)total + (uint32_t)spare - 1u) / (uint32_t)spare);
  return share > least ? share : least;
}

constexpr int kShareSeqs = 1024;   // sequences that a CTA adds up to find its row
constexpr int kPrefixWide = 128;   // q heads of a CTA on the tensor cores: the MMA's rows
constexpr int kPrefixTile = 128;   // tokens of one of its tiles

// Whether attention that reads a group's tokens again for each of its rows is faster: it is one launch, and the
// second reading is of L2.  By the bytes that all rows read at most, the table's columns filled; us, shared / alone, one
// group, up to 64 tokens of each row's own:
//   32 heads of 80, int8, 24 rows x  512 tokens (63 MB) 11.8 / 20.0    16 heads of 128, int8, 24 x  512 (50 MB) 12.5 / 13.9
//   8 of 128 under 32 q heads, fp8, 16 x 2048 (67 MB) 20.2 / 16.3      24 x 2048 (100 MB) 21.7 / 21.7
//   the same, bf16, 8 x 2048 (67 MB) 18.3 / 14.5                       16 x 2048 (134 MB) 21.3 / 22.7
// and of 2 rows of 38 tokens, 16 heads of 128 dims: 8.7 / 3.1.  Lengths are on the device: rows that fill little of a wide
// table take the way of those that fill it, here the 8.7 us.
constexpr double kAloneBytes = 36e6;  // for each of the q heads of a key head, up to three
inline bool faster_alone(int64_t B, int64_t tokens, int kv_heads, int head_dim, int code_bytes, int heads_a_key) {
  const double bytes = (double)B * (double)tokens * kv_heads * head_dim * 2 * code_bytes;
  return bytes <= kAloneBytes * (heads_a_key < 3 ? heads_a_key : 3);
}

// Whether a group's shared tokens go to the tensor cores, `heads` q heads of the group a key head and `tokens` that the
// table has room for.  The tensor cores take 128 q heads of a key head in the time of 32, and ~8 us more to begin and to end.
// us, eight a CTA / 128 on the tensor cores, one group, up to 64 tokens of each row's own:
//   q heads a key head           24             32             48             64             96             128
//   int8, 32 heads of 80   512   11.8 / 16.9    12.3 / 16.9    16.7 / 24.1    17.3 / 24.8    23.6 / 28.5    29.2 / 33.1
//                         2048   18.1 / 27.8    20.0 / 28.2    23.7 / 29.2    27.2 / 29.5    41.0 / 35.3    49.9 / 39.8
//                         8192   30.2 / 50.4    38.4 / 50.7    52.2 / 53.3    69.5 / 54.1   108.7 / 59.2   136.4 / 66.4
//                        32768   89.1 / 142.2  125.5 / 142.5  166.4 / 153.1  241.9 / 154.1  377.5 / 159.6  479.9 / 173.2
//   bf16, 8 of 128         512   15.7 / 21.0    14.9 / 18.6    16.7 / 21.3    17.3 / 19.5    18.6 / 22.0    17.3 / 19.6
//                         2048   17.8 / 24.4    18.3 / 21.0    20.8 / 22.0    21.3 / 22.2    26.3 / 23.1    27.8 / 22.7
//                         8192   25.3 / 29.5    26.8 / 26.8    35.0 / 27.8    40.0 / 28.2    58.9 / 29.2    71.2 / 28.9
//                        32768   55.5 / 56.3    65.4 / 50.9    94.1 / 52.4   115.2 / 52.1   189.6 / 53.4   245.6 / 53.1
// All of tables as wide as their longest row.  512 tokens of a table with room for 16384 take the tensor cores from 44 heads
// on, which 64 heads would do without in 17.3 us for 24.8.
inline bool wide_wins(int64_t heads, int64_t tokens, int head_dim, int code_bytes) {
  return head_dim <= 128 && heads >= (code_bytes == 2 ? 28 : 40) + 65536 / tokens;
}

// CTAs that each of `rows` rows of work has on the tensor cores, of `groups` groups and at most `steps` tiles: 0 for CTAs in
// proportion to the tokens, where groups differ and rows round up to whole CTAs well below the GPU, else as many a row as
// there is room for.
inline int wide_splits(int64_t groups, int64_t rows, int64_t steps, int sms) {
  if (groups > 1 && groups <= kShareSeqs && rows <= sms / 3 && steps_fit(rows, steps)) return 0;
  return rows < sms ? (int)(sms / rows) : 1;
}

// CTAs that share the pages of each of `heads` key heads (of all sequences): as many as are resident together, in equal
// rounds of pages.  max_pages <= 2^30 and heads <= 2^42, whose product does not fit.
inline int64_t page_shares(int64_t max_pages, int64_t heads, int64_t resident) {
  if (heads >= resident) return 1;
  const int64_t rounds = (max_pages * heads + resident - 1) / resident;
  return (max_pages + rounds - 1) / rounds;
}

}  // namespace bitlinear
