// Host/device interface of the cache operators: rotation with the page write, the 4-bit and
// 8-bit writes and reads, attention over pages.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "specdec.h"

namespace specdec {

constexpr int kGroup4 = 16;  // values that share a scale in a 4-bit cache

// The pages as the kernels see them.  Strides are in bytes.
struct Pages {
  char *k, *v;
  char *k_scales, *v_scales;
  int64_t page_stride, slot_stride, head_stride;
  int64_t scale_page_stride, scale_slot_stride, scale_head_stride;
  const int32_t* table;  // [B, max_pages]
  int num_pages, page_size, max_pages;
  int kv_heads, head_dim;
  float k_scale, v_scale;
  uint64_t page_magic;   // 2^64 / page_size, rounded up (0 for pages of one slot)
  int scale_block;       // 8-bit pages: slots that share a scale
  uint64_t block_magic;  // 2^64 / scale_block, rounded up
};

struct RotateParams {
  const void *q, *k, *v;           // [B, n, heads, D]; strides in elements, the last is 1
  int64_t q_sb, q_st, q_sh, k_sb, k_st, k_sh, v_sb, v_st, v_sh;
  const void *q_weight, *k_weight;  // [D] or nullptr: no norm
  const uint64_t* turns;            // [rot / 2], in 2^-64 turns for a position
  const int32_t *context_len, *query_len, *depth;
  int B, n, Hq, Hkv, D, rot, interleaved;
  float eps;
  void* q_out;                      // [B, n, Hq, D]
  void* k_out;                      // [B, n, Hkv, D] or nullptr: pages
  int32_t* out_status;
  Pages pages;
};
cudaError_t launch_rotate_qk(const RotateParams& P, specdec_dtype dt, cudaStream_t stream);

// The write and read of pages held in few bits.
struct KvParams {
  const void *k, *v;  // append: [B, n, Hkv, D] inputs, strides in elements
  int64_t k_sb, k_st, k_sh, v_sb, v_st, v_sh;
  float k_inv, v_inv;   // append: 1 / the tensor-wide scales, rounded to fp32
  void *k_out, *v_out;  // read: [B, n, Hkv, D] outputs
  const int32_t *context_len, *query_len;
  int B, n;
  int32_t* out_status;
  Pages pages;
};
cudaError_t launch_append_kv4(const KvParams& P, specdec_dtype dt, cudaStream_t stream);
cudaError_t launch_read_kv4(const KvParams& P, specdec_dtype dt, cudaStream_t stream);
cudaError_t launch_append_kv8(const KvParams& P, specdec_dtype dt, cudaStream_t stream);
cudaError_t launch_read_kv8(const KvParams& P, specdec_dtype dt, cudaStream_t stream);

struct AttendParams {
  const void* q;  // [B, n, Hq, D]; strides in elements, the last is 1
  int64_t q_sb, q_st, q_sh;
  const int32_t *context_len, *query_len, *depth;
  const uint8_t* tree_mask;  // [n, n] or nullptr: the chain
  int B, n, Hq, G;
  int window, sinks;
  float scale_log2;  // softmax scale * log2(e) * the keys' tensor-wide scale
  void* out;         // [B, n, Hq, D]
  float* lse;        // [B, n, Hq] or nullptr
  int32_t* out_status;
  uint64_t g_magic;  // 2^40 / G, rounded up: n * G < 2^24 rows
  int row_tiles;     // tiles of the n * G query rows that share a key head
  int tracks;        // rows of CTAs: 1, or a key head each
  int ctas;
  int4* split;       // workspace [ctas]: the item whose first part a CTA left, and its parts
  int* gave_up;      // workspace [ctas]: a bounded wait of the CTA ran out
  float2* part_ml;   // workspace [ctas, 2, rows]: (running maximum, sum) of a part
  float* part_o;     // workspace [ctas, 2, rows, D]: its unnormalised output
  Pages pages;
};
// The tensor-memory kernel: the rows of its tile, and its launches for 16-bit, 4-bit and 8-bit pages.
int attend_tc_rows(int64_t rows);
cudaError_t launch_attend_tc(const AttendParams& P, specdec_dtype dt, int mr, cudaStream_t stream);
cudaError_t launch_attend_tc4(const AttendParams& P, specdec_dtype dt, int mr, cudaStream_t stream);
cudaError_t launch_attend_tc8(const AttendParams& P, specdec_dtype dt, int mr, cudaStream_t stream);
// The warp-level kernel over 8-bit pages: the rows of its tile, and its launch.
int attend8_rows(int64_t rows);
cudaError_t launch_attend8(const AttendParams& P, specdec_dtype dt, int mr, cudaStream_t stream);
size_t attend_workspace_bytes(int n, int G, int D);
cudaError_t launch_attend(AttendParams P, specdec_dtype dt, specdec_dtype format, void* workspace,
                          cudaStream_t stream);

}  // namespace specdec
