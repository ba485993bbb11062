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
// A run is the rows of one block. Two kernels, by the rows of a call:
//  * few rows (rounds: short runs): one warp per (run, head and side, layer), latency-bound. Every row has a
//    warp; 32 slots in one load tell it whether a run starts there and where it ends.
//  * many rows (prompts: whole blocks): one CTA per (run, head and side, layer), HBM-bound. A block's rows
//    stay in registers between the amax and the rounding, so they are read once.
#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>

#include "cache.h"
#include "common.cuh"

namespace dfl {

namespace {

constexpr int kAppendThreads = 256;
constexpr int kFewRows = 2048;     // up to here a warp per run, above a CTA

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

constexpr int kWarpUnits = 8;      // warps per CTA of the few-rows kernel: heads and sides of one row
constexpr int kHeld = 4;           // eighths of a row that a lane of it holds at once

template <typename T>
__global__ void __launch_bounds__(kWarpUnits * 32) cache_append_few_kernel(const __grid_constant__ CacheAppendArgs a) {
  __shared__ int owners[kWarpUnits][128];   // last row of the call for each token of the block, -1: none
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int unit = blockIdx.y * kWarpUnits + warp;
  const int head = unit >> 1, side = unit & 1, layer = a.layer0 + blockIdx.z;
  const int n_tok = 1 << a.log_t;
  int* owner = owners[warp];
  pdl_launch_dependents();
  pdl_wait();
  if (head >= a.n_kv) return;
  for (int row = blockIdx.x * a.rows_per_cta; row < min(a.n_rows, (int)(blockIdx.x + 1) * a.rows_per_cta); row++) {
    // lane l: the row l - 1 further on
    auto block_of = [&](int r) { return r >= 0 && r < a.n_rows ? block_at(a, r) : -1; };
    int b = block_of(row - 1 + lane);
    const int block = __shfl_sync(0xffffffffu, b, 1), prev = __shfl_sync(0xffffffffu, b, 0);
    if (block < 0 || prev == block || (row > 0 && prev < 0 && !starts_run(a, row, block))) continue;
    Target to(a, layer, block, head, side);
    for (int t = lane; t < n_tok; t += 32) owner[t] = -1;
    __syncwarp();
    // its rows: up to the first one of another block
    int end = row;
    for (int r0 = row - 1;; r0 += 32) {
      if (r0 >= row) b = block_of(r0 + lane);
      const bool mine = r0 + lane >= row;
      const unsigned other = __ballot_sync(0xffffffffu, mine && b >= 0 && b != block);
      const int stop = other ? __ffs(other) - 1 : 32;
      if (mine && lane < stop && b == block) atomicMax(&owner[a.slots[r0 + lane] & (n_tok - 1)], r0 + lane);
      end = r0 + stop;
      if (other || end >= a.n_rows) break;
    }
    end = min(end, a.n_rows);
    __syncwarp();
    const T* src = static_cast<const T*>(a.rows[side]) + blockIdx.z * a.row_layer[side] + head * a.row_head[side];
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
}

// PER: eighths of a row per thread, block_tokens * head_dim / 8 / 256 (at least 1). A CTA takes the runs that
// start among its block_tokens rows (a prompt has one), for `heads` heads of one side and layer: the rows of the
// next head are on their way while one head's are rounded.
template <typename T, int PER>
__global__ void __launch_bounds__(kAppendThreads, PER * sizeof(T) <= 8 ? 4 : 1)
    cache_append_kernel(const __grid_constant__ CacheAppendArgs a) {
  __shared__ int owner[128];       // last row of the call for each token of the block, -1: none
  __shared__ uint32_t wtop[2][kAppendThreads / 32];
  __shared__ int starts[128], n_starts, run_end;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int side = blockIdx.y & 1, head0 = (blockIdx.y >> 1) * a.heads, head1 = min(a.n_kv, head0 + a.heads);
  const int layer = a.layer0 + blockIdx.z, n_tok = 1 << a.log_t, per_row = a.hd / 8;
  if (tid == 0) n_starts = 0;
  pdl_launch_dependents();
  pdl_wait();
  __syncthreads();
  {
    const int row = (blockIdx.x << a.log_t) + tid;
    if (tid < n_tok && row < a.n_rows) {
      const int b = block_at(a, row);
      if (b >= 0 && starts_run(a, row, b)) starts[atomicAdd(&n_starts, 1)] = row;
    }
  }
  __syncthreads();
  const int runs = n_starts;
  const T* src = static_cast<const T*>(a.rows[side]) + blockIdx.z * a.row_layer[side];
  for (int u = 0; u < runs; u++) {
    const int row = starts[u], block = block_at(a, row);
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

template <typename T>
cudaError_t launch_rows(CacheAppendArgs a, cudaStream_t s) {
  // heads per CTA: as many as leave several CTAs for every SM
  const long long blocks = ((a.n_rows + (1 << a.log_t) - 1) >> a.log_t) * 2LL * a.n_layers;
  a.heads = a.n_kv;
  while (a.heads > 1 && blocks * ((a.n_kv + a.heads - 1) / a.heads) < 2048) a.heads = (a.heads + 1) / 2;
  const unsigned layers = a.n_layers;
  // a row per CTA, or as many as leave about three CTAs for every SM: most rows start no run
  const int units = (2 * a.n_kv + kWarpUnits - 1) / kWarpUnits;
  a.rows_per_cta = (int)std::max(1LL, std::min(8LL, (long long)a.n_rows * units * a.n_layers / 456));
  if (a.n_rows <= kFewRows)
    return launch_pdl(cache_append_few_kernel<T>, dim3((a.n_rows + a.rows_per_cta - 1) / a.rows_per_cta, units, layers), dim3(kWarpUnits * 32), 0, s, a);
  const dim3 grid((a.n_rows + (1 << a.log_t) - 1) >> a.log_t, 2 * ((a.n_kv + a.heads - 1) / a.heads), layers), block(kAppendThreads);
  switch (((a.hd / 8) << a.log_t) / kAppendThreads) {
    case 0: case 1: return launch_pdl(cache_append_kernel<T, 1>, grid, block, 0, s, a);
    case 2: return launch_pdl(cache_append_kernel<T, 2>, grid, block, 0, s, a);
    case 4: return launch_pdl(cache_append_kernel<T, 4>, grid, block, 0, s, a);
    case 8: return launch_pdl(cache_append_kernel<T, 8>, grid, block, 0, s, a);
    case 16: return launch_pdl(cache_append_kernel<T, 16>, grid, block, 0, s, a);
    default: return cudaErrorInvalidValue;
  }
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
