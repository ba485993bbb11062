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
// One CTA per (run of rows of one block, head and side, layer). HBM-bound for prompts: a run of 64
// rows x 128 columns is read once (16 KB of bf16) and leaves as 8 KB.
#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>

#include "cache.h"
#include "common.cuh"

namespace dfl {

namespace {

constexpr int kAppendThreads = 256;

template <typename T>
struct Row8;   // 8 consecutive elements of a row, as fp32
template <>
struct Row8<float> {
  __device__ static void load(const float* p, float (&x)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};
template <>
struct Row8<__nv_bfloat16> {
  __device__ static void load(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
};
template <>
struct Row8<__half> {
  __device__ static void load(const __half* p, float (&x)[8]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
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

// x / scale: scale is a power of two unless the caller wrote another one into the cache
struct Divide {
  float s, inv;
  bool exact;
  __device__ explicit Divide(float scale) : s(scale), inv(1.f / scale) {
    const uint32_t u = __float_as_uint(scale);
    exact = (u & 0x7fffffu) == 0 && (u >> 23) > 0 && (u >> 23) < 254;
  }
  __device__ float operator()(float x) const { return exact ? x * inv : __fdiv_rn(x, s); }
};

__device__ __forceinline__ uint2 to_codes(const float (&x)[8], const Divide& div) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; i++)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(div(x[2 * i]), div(x[2 * i + 1])), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

__device__ __forceinline__ void from_codes(uint2 c, float (&x)[8]) {
  const uint32_t u[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u[i / 2] >> (16 * (i & 1))), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
}

template <typename T>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const __grid_constant__ CacheAppendArgs a) {
  __shared__ int owner[128];       // last row of the call for each token of the block, -1: none
  __shared__ float wmax[kAppendThreads / 32];
  __shared__ int run_end;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int head = blockIdx.y >> 1, side = blockIdx.y & 1, layer = a.layer0 + blockIdx.z;
  const int n_tok = 1 << a.log_t, per_row = a.hd / 8;
  pdl_launch_dependents();
  pdl_wait();
  // rows of a block out of range are skipped like negative slots
  auto block_at = [&](int row) {
    const int s = a.slots[row];
    const int b = s < 0 ? -1 : s >> a.log_t;
    if (s >= 0 && !in_bounds(b < a.n_blocks, a.err)) return -1;
    return b;
  };
  const T* src = static_cast<const T*>(a.rows[side]) + blockIdx.z * a.row_layer[side] + head * a.row_head[side];
  const int row_end = min(a.n_rows, (int)(blockIdx.x + 1) * a.rows_per_cta);
  for (int row = blockIdx.x * a.rows_per_cta; row < row_end; row++) {
    // a run starts at a row whose block differs from that of the last row before it that has one
    const int block = block_at(row);
    if (block < 0) continue;
    int before = row - 1;
    while (before >= 0 && block_at(before) < 0) before--;
    if (before >= 0 && block_at(before) == block) continue;
    // its end: the first later row with another block
    for (int t = tid; t < n_tok; t += kAppendThreads) owner[t] = -1;
    if (tid == 0) run_end = a.n_rows;
    __syncthreads();
    for (int r0 = row; r0 < a.n_rows; r0 += kAppendThreads) {
      const int r = r0 + tid;
      const int b = r < a.n_rows ? block_at(r) : -1;
      if (b >= 0 && b != block) atomicMin(&run_end, r);
      if (__syncthreads_or(b >= 0 && b != block)) break;
    }
    const int end = run_end;
    for (int r = row + tid; r < end; r += kAppendThreads)
      if (block_at(r) == block) atomicMax(&owner[a.slots[r] & (n_tok - 1)], r);
    __syncthreads();
    // amax over the rows that count
    float amax = 0.f;
    for (int i = tid; i < n_tok * per_row; i += kAppendThreads) {
      const int r = owner[i / per_row];
      if (r < 0) continue;
      float x[8];
      Row8<T>::load(src + r * a.row_row[side] + (i % per_row) * 8, x);
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float m = fabsf(x[j]);
        if (m <= 3.402823466e38f) amax = fmaxf(amax, m);   // finite (false for NaN too)
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0) wmax[warp] = amax;
    __syncthreads();
    amax = wmax[0];
#pragma unroll
    for (int w = 1; w < kAppendThreads / 32; w++) amax = fmaxf(amax, wmax[w]);
    float* sp = a.scales[side] + ((int64_t)layer * a.n_blocks + block) * a.n_kv + head;
    const float old = *sp;
    const bool fresh = owner[0] >= 0;
    const float fit = scale_for(amax), scale = fresh ? fit : fmaxf(old, fit);
    const Divide div(scale);
    uint8_t* dst = a.codes[side] + layer * a.c_layer + block * a.c_block + head * a.c_head;
    const bool regrade = !fresh && scale > old;
    const float ratio = __fdiv_rn(old, scale);
    for (int i = tid; i < n_tok * per_row; i += kAppendThreads) {
      const int t = i / per_row, c8 = (i % per_row) * 8, r = owner[t];
      uint2* at = reinterpret_cast<uint2*>(dst + t * a.c_token + c8);
      float x[8];
      if (r >= 0) {
        Row8<T>::load(src + r * a.row_row[side] + c8, x);
        *at = to_codes(x, div);
      } else if (regrade) {
        from_codes(*at, x);
#pragma unroll
        for (int j = 0; j < 8; j++) x[j] *= ratio;
        *at = to_codes(x, Divide(1.f));
      }
    }
    __syncthreads();   // every thread has read the old scale, owner and wmax
    if (tid == 0) *sp = scale;
  }
}

}  // namespace

cudaError_t launch_cache_append(int dtype, const CacheAppendArgs& a, cudaStream_t s) {
  const dim3 grid((a.n_rows + a.rows_per_cta - 1) / a.rows_per_cta, a.n_kv * 2, a.n_layers), block(kAppendThreads);
  switch (dtype) {
    case DFLASH_F32: return launch_pdl(cache_append_kernel<float>, grid, block, 0, s, a);
    case DFLASH_BF16: return launch_pdl(cache_append_kernel<__nv_bfloat16>, grid, block, 0, s, a);
    case DFLASH_F16: return launch_pdl(cache_append_kernel<__half>, grid, block, 0, s, a);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace dfl
