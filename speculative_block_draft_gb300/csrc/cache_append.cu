// Quantising append of the paged context cache (include/dflash.h, dflash_cache_append).
//
//   amax  = largest finite |x| of a block's new rows (per layer, head, side)
//   s     = 2^k, k = the smallest integer >= -64 with amax <= 448 * 2^k   (448: the largest e4m3)
//   scale = s if the block starts anew in this call, else max(old, s)
//   code  = e4m3(x / scale), codes that stay in the block = e4m3(code * old / scale)
// e4m3 keeps 4 significant bits at any magnitude, so a scale only has to keep the block in range: a
// power of two loses nothing against amax / 448, and when it grows, the codes that stay move by
// whole exponents (only those that become subnormal are rounded again).
//
// A run is the rows of one block. A CTA takes the runs that start among some rows, for some heads of one side and
// layer, each in one of two ways by its length:
//  * long (prompts: whole blocks): its 256 threads together, HBM-bound; the rows stay in registers between the
//    amax and the rounding, so they are read once, and the next head's are on their way meanwhile;
//  * at most kShortRun rows (rounds): a warp per run and head, latency-bound.
// Measured, 5 layers x 8 heads x 128 columns of bf16: 128 rows in 2 runs 4.4 us together, 16.5 us by warps; 512
// rows in 64 runs 33.9 us together, 7.0 us by warps. 16384 rows: 94 us, 5.4 TB/s read and written (the floor at the
// measured copy bandwidth is 74 us).
#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>

#include "cache.h"
#include "common.cuh"

namespace dfl {

namespace {

constexpr int kAppendThreads = 256;
constexpr int kShortRun = 16;

// 8 consecutive elements of a row: fetched as they are, read as fp32.
template <typename T>
struct Row8 {
  uint4 v[sizeof(T) / 2];
  __device__ void fetch(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; i++) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ void get(float (&x)[8]) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if constexpr (sizeof(T) == 4) {
        x[2 * i] = __uint_as_float(u[2 * i]);
        x[2 * i + 1] = __uint_as_float(u[2 * i + 1]);
      } else if constexpr (__is_same(T, __nv_bfloat16)) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
      }
    }
  }
  // The largest magnitude as bits of T (they order as the magnitudes do, NaN above infinity above all else).
  __device__ uint32_t top(uint32_t m) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
    for (int i = 0; i < 2 * (int)sizeof(T); i++)
      m = sizeof(T) == 4 ? max(m, u[i] & 0x7fffffffu) : __vmaxu2(m, u[i] & 0x7fff7fffu);
    return m;
  }
  // The largest finite magnitude.
  __device__ float finite_amax(float amax) const {
    float x[8];
    get(x);
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const float m = fabsf(x[j]);
      if (m <= 3.402823466e38f) amax = fmaxf(amax, m);   // false for infinities and NaN
    }
    return amax;
  }
  // Magnitude bits over a warp's lanes; `finite`: no infinity and no NaN among them, `value` is the magnitude.
  __device__ static uint32_t warp_top(uint32_t m) {
    if constexpr (sizeof(T) == 2) m = max(m & 0xffffu, m >> 16);
    return __reduce_max_sync(0xffffffffu, m);
  }
  __device__ static bool finite(uint32_t m) {
    return m < (sizeof(T) == 4 ? 0x7f800000u : __is_same(T, __nv_bfloat16) ? 0x7f80u : 0x7c00u);
  }
  __device__ static float value(uint32_t m) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(m);
    if constexpr (__is_same(T, __nv_bfloat16)) return __uint_as_float(m << 16);
    return __half2float(__ushort_as_half((unsigned short)m));
  }
};

// 2^k for -126 <= k <= 127.
__device__ __forceinline__ float pow2i(int k) { return __int_as_float((k + 127) << 23); }

// The smallest power of two >= 2^kMinScaleExp with amax <= 448 * scale; amax finite and >= 0.
// amax = m * 2^e with 1 <= m < 2 and 448 = 1.75 * 2^8, so the exponent is e - 8, one more if m > 1.75.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int k = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return pow2i(max(k, kMinScaleExp));
}

__device__ __forceinline__ uint2 to_codes(const float (&x)[8]) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; i++) h[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i], x[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// Codes of x / scale: a multiplication where scale is a power of two, as it is unless the caller wrote another
// one into the cache.
struct Divide {
  float s, inv;
  bool exact;
  __device__ explicit Divide(float scale) : s(scale) {
    const uint32_t u = __float_as_uint(scale);
    exact = (u & 0x807fffffu) == 0 && (u >> 23) > 0 && (u >> 23) < 254;
    inv = __uint_as_float((254u << 23) - u);           // exact reciprocal of a power of two
  }
  __device__ uint2 codes(float (&x)[8]) const {
    if (exact) {
#pragma unroll
      for (int j = 0; j < 8; j++) x[j] *= inv;
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) x[j] = __fdiv_rn(x[j], s);
    }
    return to_codes(x);
  }
};

__device__ __forceinline__ void from_codes(uint2 c, float (&x)[8]) {
  const uint32_t u[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u[i / 2] >> (16 * (i & 1))), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
}

// The block of a row, -1 for a row to skip.
__device__ __forceinline__ int block_at(const CacheAppendArgs& a, int row) {
  const int s = a.slots[row];
  if (s < 0) return -1;
  const int b = s >> a.log_t;
  return in_bounds(b < a.n_blocks, a.err) ? b : -1;
}

// Whether a run starts at `row`, whose block is `block`: the last row before it that has a block has another.
__device__ __forceinline__ bool starts_run(const CacheAppendArgs& a, int row, int block) {
  int before = row - 1;
  while (before >= 0) {
    const int b = block_at(a, before);
    if (b >= 0) return b != block;
    before--;
  }
  return true;
}

struct Target {                    // codes and scale of one (layer, block, head, side)
  uint8_t* codes;
  float* scale;
  float old, now;
  bool regrade;
  __device__ Target(const CacheAppendArgs& a, int layer, int block, int head, int side)
      : codes(a.codes[side] + layer * a.c_layer + block * a.c_block + head * a.c_head),
        scale(a.scales[side] + ((int64_t)layer * a.n_blocks + block) * a.n_kv + head), old(*scale) {}
  __device__ void settle(float amax, bool fresh) {
    const float fit = scale_for(amax);
    now = fresh ? fit : fmaxf(old, fit);
    regrade = !fresh && now > old;
  }
};

// Codes that stay in a block whose scale grew.
__device__ __forceinline__ void regrade8(uint2* at, float ratio) {
  float x[8];
  from_codes(*at, x);
#pragma unroll
  for (int j = 0; j < 8; j++) x[j] *= ratio;
  *at = to_codes(x);
}

constexpr int kHeld = 4;           // eighths of a row that a lane holds at once

// The run that starts at `row`, by one warp; owner: block_tokens words of shared memory of its own.
template <typename T>
__device__ __forceinline__ void append_by_warp(const CacheAppendArgs& a, int row, int layer, int head, int side, int* owner) {
  const int lane = threadIdx.x & 31, n_tok = 1 << a.log_t, block = block_at(a, row);
  Target to(a, layer, block, head, side);
  for (int t = lane; t < n_tok; t += 32) owner[t] = -1;
  __syncwarp();
  // its rows: up to the first one of another block
  int end = row;
  for (int r0 = row;; r0 += 32) {
    const int b = r0 + lane < a.n_rows ? block_at(a, r0 + lane) : -1;
    const unsigned other = __ballot_sync(0xffffffffu, b >= 0 && b != block);
    const int stop = other ? __ffs(other) - 1 : 32;
    if (lane < stop && b == block) atomicMax(&owner[a.slots[r0 + lane] & (n_tok - 1)], r0 + lane);
    end = r0 + stop;
    if (other || end >= a.n_rows) break;
  }
  end = min(end, a.n_rows);
  __syncwarp();
  const T* src = static_cast<const T*>(a.rows[side]) + (layer - a.layer0) * a.row_layer[side] + head * a.row_head[side];
  const int per_row = a.hd / 8, at_once = 32 / per_row, c8 = (lane % per_row) * 8;
  // kHeld rows of this lane's group of lanes at a time, all their loads in flight; a short run is read once
  Row8<T> x[kHeld];
  int tok[kHeld];
  auto fetch = [&](int r0) {
#pragma unroll
    for (int i = 0; i < kHeld; i++) {
      const int r = r0 + i * at_once, s = r < end ? a.slots[r] : -1;
      tok[i] = s >= 0 && owner[s & (n_tok - 1)] == r ? s & (n_tok - 1) : -1;
      if (tok[i] >= 0) x[i].fetch(src + r * a.row_row[side] + c8);
    }
  };
  float v[8];
  uint32_t top = 0;
  const int step = kHeld * at_once;
  for (int r0 = row; r0 < end; r0 += step) {
    fetch(r0 + lane / per_row);
#pragma unroll
    for (int i = 0; i < kHeld; i++)
      if (tok[i] >= 0) top = x[i].top(top);
  }
  top = Row8<T>::warp_top(top);
  float amax = Row8<T>::value(top);
  if (!Row8<T>::finite(top)) {
    amax = 0.f;
    for (int r0 = row; r0 < end; r0 += step) {
      fetch(r0 + lane / per_row);
#pragma unroll
      for (int i = 0; i < kHeld; i++)
        if (tok[i] >= 0) amax = x[i].finite_amax(amax);
    }
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  }
  to.settle(amax, owner[0] >= 0);
  const Divide div(to.now);
  for (int r0 = row; r0 < end; r0 += step) {
    if (end - row > step) fetch(r0 + lane / per_row);
#pragma unroll
    for (int i = 0; i < kHeld; i++)
      if (tok[i] >= 0) {
        x[i].get(v);
        *reinterpret_cast<uint2*>(to.codes + tok[i] * a.c_token + c8) = div.codes(v);
      }
  }
  if (to.regrade) {
    const float ratio = __fdiv_rn(to.old, to.now);
    for (int t = lane / per_row; t < n_tok; t += at_once)
      if (owner[t] < 0) regrade8(reinterpret_cast<uint2*>(to.codes + t * a.c_token + c8), ratio);
  }
  if (lane == 0) *to.scale = to.now;
  __syncwarp();   // owner belongs to the next run
}

// PER: eighths of a row per thread, block_tokens * head_dim / 8 / 256 (at least 1). CTAS per SM: five for prompts, for
// the loads in flight (16384 rows: 93.8 us, 98.0 with four, 118.6 with six, which spills); four for rounds, which the
// fewer registers slow (32 requests x 1-8 rows: 5.9 us, 6.8 with five). Measured on bf16 blocks of 64 x 128. In fp32 blocks of
// up to 4096 elements spill at five (444 bytes: 16384 rows in blocks of 16 x 128 291.6 us for a floor of 123.8); above PER *
// sizeof(T) = 8 a thread holds so much that one CTA fits an SM (8192 rows in blocks of 64 x 256 158.4 us for 74.2).
template <typename T, int PER, int CTAS>
__global__ void __launch_bounds__(kAppendThreads, PER * sizeof(T) <= 8 ? CTAS : 1)
    cache_append_kernel(const __grid_constant__ CacheAppendArgs a) {
  __shared__ int owners[kAppendThreads / 32][128];   // last row of the call for each token of the block, -1: none
  int* owner = owners[0];
  __shared__ uint32_t wtop[2][kAppendThreads / 32];
  __shared__ int starts[2][128], n_starts[2], run_end;   // first rows of the short and of the long runs
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int side = blockIdx.y & 1, head0 = (blockIdx.y >> 1) * a.heads, head1 = min(a.n_kv, head0 + a.heads);
  const int layer = a.layer0 + blockIdx.z, n_tok = 1 << a.log_t, per_row = a.hd / 8;
  if (tid < 2) n_starts[tid] = 0;
  pdl_launch_dependents();
  pdl_wait();
  __syncthreads();
  {
    const int row = blockIdx.x * a.rows_per_cta + tid;
    if (tid < a.rows_per_cta && row < a.n_rows) {
      const int b = block_at(a, row);
      if (b >= 0 && starts_run(a, row, b)) {
        const int is_long = row + kShortRun < a.n_rows && block_at(a, row + kShortRun) == b;
        starts[is_long][atomicAdd(&n_starts[is_long], 1)] = row;
      }
    }
  }
  __syncthreads();
  {
    const int runs = n_starts[0], tasks = runs * (head1 - head0);
    for (int u = warp; u < tasks; u += kAppendThreads / 32)
      append_by_warp<T>(a, starts[0][u % runs], layer, head0 + u / runs, side, owners[warp]);
  }
  if (n_starts[1] == 0) return;
  __syncthreads();                 // owners
  const int runs = n_starts[1];
  const T* src = static_cast<const T*>(a.rows[side]) + blockIdx.z * a.row_layer[side];
  for (int u = 0; u < runs; u++) {
    const int row = starts[1][u], block = block_at(a, row);
    for (int t = tid; t < n_tok; t += kAppendThreads) owner[t] = -1;
    if (tid == 0) run_end = a.n_rows;
    __syncthreads();
    // its end: the first later row of another block
    for (int r0 = row; r0 < a.n_rows; r0 += kAppendThreads) {
      const int r = r0 + tid, b = r < a.n_rows ? block_at(a, r) : -1;
      if (b >= 0 && b != block) atomicMin(&run_end, r);
      if (__syncthreads_or(b >= 0 && b != block)) break;
    }
    const int end = run_end;
    for (int r = row + tid; r < end; r += kAppendThreads)
      if (block_at(a, r) == block) atomicMax(&owner[a.slots[r] & (n_tok - 1)], r);
    __syncthreads();
    const bool fresh = owner[0] >= 0;
    int from[PER];                 // the row of the call that each of this thread's pieces comes from
    Row8<T> x[PER];
#pragma unroll
    for (int i = 0; i < PER; i++) {
      const int t = (tid + i * kAppendThreads) / per_row;
      from[i] = t < n_tok ? owner[t] : -1;
    }
    auto fetch = [&](int head) {
#pragma unroll
      for (int i = 0; i < PER; i++)
        if (from[i] >= 0)
          x[i].fetch(src + head * a.row_head[side] + from[i] * a.row_row[side] + ((tid + i * kAppendThreads) & (per_row - 1)) * 8);
    };
    fetch(head0);
    for (int head = head0; head < head1; head++) {
      Target to(a, layer, block, head, side);
      Row8<T> y[PER];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < PER; i++) {
        y[i] = x[i];
        if (from[i] >= 0) top = y[i].top(top);
      }
      if (head + 1 < head1) fetch(head + 1);
      top = Row8<T>::warp_top(top);
      if (lane == 0) wtop[head & 1][warp] = top;
      __syncthreads();
      top = wtop[head & 1][0];
#pragma unroll
      for (int w = 1; w < kAppendThreads / 32; w++) top = max(top, wtop[head & 1][w]);
      float amax = Row8<T>::value(top);
      if (!Row8<T>::finite(top)) {
        amax = 0.f;
#pragma unroll
        for (int i = 0; i < PER; i++)
          if (from[i] >= 0) amax = y[i].finite_amax(amax);
        top = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));
        __syncthreads();           // every thread has read wtop
        if (lane == 0) wtop[head & 1][warp] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kAppendThreads / 32; w++) top = max(top, wtop[head & 1][w]);
        amax = __uint_as_float(top);
      }
      to.settle(amax, fresh);
      const Divide div(to.now);
#pragma unroll
      for (int i = 0; i < PER; i++) {
        const int at = tid + i * kAppendThreads, t = at / per_row;
        uint2* p = reinterpret_cast<uint2*>(to.codes + t * a.c_token + (at & (per_row - 1)) * 8);
        if (from[i] >= 0) {
          float v[8];
          y[i].get(v);
          *p = div.codes(v);
        } else if (to.regrade && t < n_tok) {
          regrade8(p, __fdiv_rn(to.old, to.now));
        }
      }
      if (tid == 0) *to.scale = to.now;   // read by every thread before the barrier above
    }
    __syncthreads();   // owner, wtop and run_end belong to the next run
  }
}

template <typename T, int CTAS>
cudaError_t launch_per(const CacheAppendArgs& a, dim3 grid, cudaStream_t s) {
  const dim3 block(kAppendThreads);
  switch (((a.hd / 8) << a.log_t) / kAppendThreads) {
    case 0: case 1: return launch_pdl(cache_append_kernel<T, 1, CTAS>, grid, block, 0, s, a);
    case 2: return launch_pdl(cache_append_kernel<T, 2, CTAS>, grid, block, 0, s, a);
    case 4: return launch_pdl(cache_append_kernel<T, 4, CTAS>, grid, block, 0, s, a);
    case 8: return launch_pdl(cache_append_kernel<T, 8, CTAS>, grid, block, 0, s, a);
    case 16: return launch_pdl(cache_append_kernel<T, 16, CTAS>, grid, block, 0, s, a);
    default: return cudaErrorInvalidValue;
  }
}

template <typename T>
cudaError_t launch_rows(CacheAppendArgs a, cudaStream_t s) {
  // Heads per CTA: as many as leave several CTAs for every SM; with more, a CTA has loads on their way while it rounds.
  // Rows per CTA: as few (8 to 64, or a block's) as give about one wave of CTAs, four per SM, so that the runs of a
  // round spread: 144 rows in 32 runs take 7.4 us with 64 rows per CTA and 4.8 us with 16, 512 rows in 64 runs 6.9 and
  // 11.9 us (5 layers x 8 heads).
  const long long blocks = (a.n_rows + (1 << a.log_t) - 1) >> a.log_t;
  a.heads = a.n_kv;
  while (a.heads > 1 && blocks * 2 * a.n_layers * ((a.n_kv + a.heads - 1) / a.heads) < 2048) a.heads = (a.heads + 1) / 2;
  const long long per_row = 2LL * a.n_layers * ((a.n_kv + a.heads - 1) / a.heads);
  a.rows_per_cta = 8;
  while (a.rows_per_cta < std::max(64, 1 << a.log_t) && per_row * a.n_rows > 608LL * a.rows_per_cta) a.rows_per_cta *= 2;
  const long long row_ctas = (a.n_rows + a.rows_per_cta - 1) / a.rows_per_cta;
  const dim3 grid((unsigned)row_ctas, 2 * ((a.n_kv + a.heads - 1) / a.heads), a.n_layers);
  return a.rows_per_cta >= std::max(64, 1 << a.log_t) ? launch_per<T, 5>(a, grid, s) : launch_per<T, 4>(a, grid, s);
}

}  // namespace

cudaError_t launch_cache_append(int dtype, const CacheAppendArgs& a, cudaStream_t s) {
  switch (dtype) {
    case DFLASH_F32: return launch_rows<float>(a, s);
    case DFLASH_BF16: return launch_rows<__nv_bfloat16>(a, s);
    case DFLASH_F16: return launch_rows<__half>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace dfl
