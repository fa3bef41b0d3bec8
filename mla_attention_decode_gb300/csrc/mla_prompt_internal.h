// mla_prompt_internal.h -- parameters of the prompt attention (include/mla_prompt.h),
// shared by its entry points and its kernels.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "mla_prompt.h"

namespace mla {

constexpr int kPromptQ = 256;   // query tokens of a CTA: two tiles of 128
constexpr int kPromptTile = 128;
constexpr int kPromptMaxSplits = 16;
constexpr int kPromptSplitCtas = 304;  // no split beyond two CTAs for each of the 152 SMs

struct PromptParams {
  // (columns, heads, tokens) of 64 columns x 1 head x 128 tokens a box, 128-byte
  // swizzle; k_pe (columns, tokens)
  CUtensorMap q_nope, q_pe, k_nope, k_pe, v;
  const int32_t* qo_indptr;
  const int32_t* kv_indptr;
  const int32_t* prefix;
  uint16_t* out;
  float* lse;
  int64_t out_token_stride, out_head_stride;
  int32_t num_q, num_kv, batch, heads, causal;
  int32_t slots;        // upper bound of the batch's 256-token tiles
  int32_t splits;       // CTAs that share a tile's keys; > 1: partial results in
  float* part_o;        //   fp32 [splits][num_q][heads][128], each over its own sum
  float* part_lse;      //   fp32 [splits][num_q][heads]
  float scale_log2;     // sm_scale * log2(e)
  int32_t* ws_err;
};

cudaError_t launch_prompt(const PromptParams& p, cudaStream_t s);

}  // namespace mla
