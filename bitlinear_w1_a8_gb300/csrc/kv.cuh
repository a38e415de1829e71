// kv.cuh -- what the attention-side kernels share: the rotary positions, the
// paged key-value cache's layout and its three formats, and their launchers.
#pragma once

#include "common.cuh"

namespace bitlinear {

// The rows of one call: row i belongs to sequence seq[i] (i when seq is NULL)
// and sits at positions[i]; page positions[i] / page_size of that sequence is
// table[seq * table_stride + page].
struct KvRows {
  const int32_t* positions;
  const int32_t* seq;
  const int32_t* table;
  int64_t table_stride;
  int64_t num_seqs;
  int64_t max_pages;
  int64_t T;
};

// The cache with its page size as a shift.
struct KvPages {
  void* k;
  void* v;
  float* k_step;
  float* v_step;
  int64_t num_pages;
  int heads, page_shift, head_dim, format;
};

struct RopeArgs {
  const double* freq;  // NULL: no rotation
  int rot_dim, layout;
  float amplitude;
};

// The row index ((page * heads) + head) * page_size + offset of (row i, head 0)
// and the distance between heads, or -1 when the row has no place in the
// cache: a negative position, a sequence, page column or page number out of
// range.  64-bit throughout: a cache may hold more than 2^31 rows.
__device__ __forceinline__ int64_t kv_place(const KvRows& r, const KvPages& c, int64_t i) {
  const int32_t pos = r.positions[i];
  const int64_t s = r.seq ? (int64_t)r.seq[i] : i;
  const int64_t col = (int64_t)pos >> c.page_shift;
  if (pos < 0 || s < 0 || s >= r.num_seqs || col >= r.max_pages) return -1;
  const int32_t page = r.table[s * r.table_stride + col];
  if (page < 0 || page >= c.num_pages) return -1;
  return (((int64_t)page * c.heads) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

// fp32 -> e4m3, round to nearest even, saturating at +-448.
__device__ __forceinline__ uint32_t e4m3x2(float hi, float lo) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// The two e4m3 values of the low 16 bits, as two halves (exact).
__device__ __forceinline__ uint32_t half2_of_e4m3x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}

// rope_kv.cu
cudaError_t launch_rope(const float* x, int64_t x_stride, int64_t T, int H, int D, const int32_t* positions,
                        const RopeArgs& rope, float* y, int64_t y_stride, bool pdl, const DeviceInfo& dev,
                        cudaStream_t stream);
cudaError_t launch_kv_append(const float* q, int64_t q_stride, int q_heads, float* q_out, int64_t q_out_stride,
                             const float* k, int64_t k_stride, const float* v, int64_t v_stride, const KvRows& rows,
                             const RopeArgs& rope, const KvPages& cache, bool pdl, const DeviceInfo& dev,
                             cudaStream_t stream);
cudaError_t launch_kv_read(const KvPages& cache, const KvRows& rows, float* k_out, int64_t k_stride, float* v_out,
                           int64_t v_stride, bool pdl, const DeviceInfo& dev, cudaStream_t stream);

// attention.cu
struct AttendArgs {
  const float* q;
  float* out;
  int64_t q_stride, out_stride;
  const int32_t* table;
  int64_t table_stride, max_pages;
  const int32_t* lengths;
  int64_t window;  // 0: none
  float scale;
  int64_t B;
  int q_heads;
  float factor, factor_rest;  // launch_attention's: scale log2(e) = factor (1 + factor_rest)
};
size_t attention_workspace_bytes(int64_t B, int q_heads, int kv_heads, int head_dim);
cudaError_t launch_attention(const AttendArgs& a, const KvPages& cache, void* workspace, bool pdl,
                             const DeviceInfo& dev, cudaStream_t stream);

}  // namespace bitlinear
