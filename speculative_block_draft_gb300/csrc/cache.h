// Internal declarations of the paged 8-bit context cache (pool.cu, cache_append.cu, cache_attn.cu,
// cache_abi.cu). Not part of the public ABI (include/dflash.h).
#pragma once

#include "internal.h"

namespace dfl {

inline bool block_tokens_ok(int t) { return t == 16 || t == 32 || t == 64 || t == 128; }

// Smallest scale: 2^kMinScaleExp. A block of zeros has it, and sums of weight / scale stay in fp32's range.
constexpr int kMinScaleExp = -64;

constexpr unsigned kErrTimeoutCache = 4u;

struct CacheAppendArgs {
  uint8_t* codes[2];        // K, V
  float* scales[2];
  const void* rows[2];
  int64_t row_layer[2], row_row[2], row_head[2];   // strides of the rows, elements
  int64_t c_layer, c_block, c_head, c_token;       // strides of the codes, bytes
  int layer0, n_layers, n_rows, n_blocks, n_kv, hd, log_t;
  int rows_per_cta;
  const int32_t* slots;
  unsigned* err;
};

cudaError_t launch_cache_append(int dtype, const CacheAppendArgs& a, cudaStream_t s);

struct CacheAttnArgs {
  const uint8_t *k, *v;
  const float *k_scale, *v_scale;                  // of the call's layer
  int64_t c_block, c_head, c_token;
  int n_blocks, n_kv, hd, log_t, grp;
  int n_req, n_rows, max_q, table_rows, table_blocks, causal, window;
  const int32_t *requests, *lens, *table, *row_start;
  const void *q, *k_own, *v_own;
  void* out;
  int64_t q_row, q_head, o_row, o_head, ko_row, ko_head, vo_row, vo_head;   // elements
  float scale_log2;                                // scale * log2(e)
  unsigned* err;
};

cudaError_t launch_cache_attn(int dtype, const CacheAttnArgs& a, cudaStream_t s);

}  // namespace dfl
