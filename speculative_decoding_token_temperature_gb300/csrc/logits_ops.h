// Host/device interface of the logits' processing and of the table of token counts.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "specdec.h"

namespace specdec {

constexpr int kMaxProcessRows = 8192;

struct ProcessParams {
  const void* logits;  // [B, rows, V]
  const int32_t *tokens, *parents, *gammas;
  const int32_t* counts;  // [B, V] or nullptr
  const float *repetition, *presence, *frequency;
  const int32_t* bias_tokens;  // [B, num_bias]
  const float* bias_values;
  const uint32_t* mask;  // [B, rows, words] or nullptr
  int num_bias, words, B, rows, V;
  int alike;  // logits and out lie alike on 16 bytes
  int group;  // rows of a CTA
  void* out;
  int32_t* out_status;
};
cudaError_t launch_process_logits(const ProcessParams& P, specdec_dtype dt, cudaStream_t stream);

struct CountParams {
  int32_t* counts;  // [B, V]
  const int32_t* tokens;
  int64_t token_stride;
  const int32_t* num_tokens;
  int B, n, V, prompt;
  int32_t* out_status;
};
cudaError_t launch_count_tokens(const CountParams& P, bool reset, cudaStream_t stream);

}  // namespace specdec
