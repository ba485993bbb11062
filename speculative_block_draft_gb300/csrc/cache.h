// Internal declarations of the paged 8-bit context cache (pool.cu, cache_append.cu, cache_attn.cu,
// cache_abi.cu). Not part of the public ABI (include/dflash.h).
#pragma once

#include "internal.h"

namespace dfl {

inline bool block_tokens_ok(int t) { return t == 16 || t == 32 || t == 64 || t == 128; }

// Smallest scale: 2^kMinScaleExp. A block of zeros has it, and sums of weight / scale stay in fp32's range.
constexpr int kMinScaleExp = -64;

constexpr unsigned kErrTimeoutCache = 4u;
constexpr unsigned kWaitNs = 1000000000u;   // default limit of the attention's waits

struct CacheAppendArgs {
  uint8_t* codes[2];        // K, V
  float* scales[2];
  const void* rows[2];
  int64_t row_layer[2], row_row[2], row_head[2];   // strides of the rows, elements
  int64_t c_layer, c_block, c_head, c_token;       // strides of the codes, bytes
  int layer0, n_layers, n_rows, n_blocks, n_kv, hd, log_t;
  int heads, rows_per_cta;  // set by the launcher
  const int32_t* slots;
  unsigned* err;
};

cudaError_t launch_cache_append(int dtype, const CacheAppendArgs& a, cudaStream_t s);

// How a call's query rows are laid out over CTAs (plan_cache_attn): the grp * n rows of one request and
// KV head are cut into chunks of rc rows, each padded to rp columns.
struct CacheAttnPlan {
  int chunks, rc, rp;
  int ctas_per_sm, stages, tmem_cols;
  int setup;               // tiles that the start and end of a chunk count for when the work is shared out
  size_t smem;
};
CacheAttnPlan plan_cache_attn(int dtype, int hd, int grp, int max_q, int n_req);

struct CacheAttnArgs {
  const float *k_scale, *v_scale;                  // of the call's layer
  int layer, n_blocks, n_kv, hd, log_t, grp;
  unsigned grp_mul;                                // 2^32 / grp, rounded up
  int n_req, n_rows, max_q, table_rows, table_blocks, causal, window;
  int held;                                        // tokens that a table row can name
  const int32_t *requests, *lens, *table, *row_start;
  const void *q, *k_own, *v_own;
  void* out;
  int64_t q_row, q_head, o_row, o_head, ko_row, ko_head, vo_row, vo_head;   // elements
  float scale_log2;                                // scale * log2(e)
  unsigned* err;
  unsigned wait_ns;                                // limit of the waits
  int stall;                                       // test hook: CTA stall - 1 gets no keys (0: none)
  CacheAttnPlan p;
  int grid;                                        // CTAs of the first kernel
  int4* words;                                     // [n_req] what the call says about each request (read_request)
  int2* held_by;                                   // [n_req * n_kv * chunks] first and last CTA with tiles
  float* part_o;                                   // [grid + n_req * n_kv * chunks][rp][hd]
  float2* part_ml;                                 // [..][rp] (reference, sum)
};

cudaError_t launch_cache_attn(int dtype, const CacheAttnArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                              cudaStream_t s);

// Host numbers into device arrays (a launch of their own, so they may be captured): d_req[i] = req[i], d_n[i] = n[i].
struct PoolNumbers {
  int n_req;
  int32_t req[DFLASH_MAX_BATCH], n[DFLASH_MAX_BATCH];
};
cudaError_t launch_pool_numbers(const PoolNumbers& v, int32_t* d_req, int32_t* d_n, cudaStream_t s);
// All blocks free: free_list = n_blocks - 1 .. 0 (taken from block 0 on), free_count = n_blocks.
cudaError_t launch_pool_init(int n_blocks, int32_t* free_list, int32_t* free_count, cudaStream_t s);

}  // namespace dfl
