// Attention of a few query rows per request over the paged 8-bit context cache (include/dflash.h,
// dflash_cache_attention):
//   out_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(scale * q_i . k_j - max_j)
// over the cached keys that row i sees and, when given, the own rows of its request.
//
// One warp per (query row, query head): 32 keys at a time, one per lane, with an online softmax.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "cache.h"
#include "common.cuh"

namespace dfl {

namespace {

constexpr int kSimpleWarps = 4;

__device__ __forceinline__ float row_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float row_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void row_store(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void row_store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float code_f(uint8_t c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

template <typename T, int HD>
__global__ void __launch_bounds__(kSimpleWarps * 32) cache_attn_simple_kernel(const __grid_constant__ CacheAttnArgs a) {
  __shared__ float qs[kSimpleWarps][HD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.z, i = blockIdx.y, head = blockIdx.x * kSimpleWarps + warp;
  pdl_launch_dependents();
  pdl_wait();
  int row0, n;
  if (a.row_start) {
    row0 = a.row_start[b];
    n = min(a.row_start[b + 1] - row0, a.max_q);
  } else {
    row0 = b * a.max_q;
    n = a.max_q;
  }
  const int req = a.requests ? a.requests[b] : b;
  if (i >= n || row0 < 0 || row0 + n > a.n_rows || head >= a.n_kv * a.grp || req < 0 || req >= a.table_rows) return;
  const int kvh = head / a.grp, len = max(a.lens[req], 0), n_tok = 1 << a.log_t;
  const bool own = a.k_own != nullptr;
  const long long at = own ? (long long)len + i : (long long)len - n + i;
  long long lo = 0, hi = len;
  if (a.causal) {
    if (at + 1 < hi) hi = at + 1 < 0 ? 0 : at + 1;
    if (a.window > 0 && at + 1 - a.window > lo) lo = at + 1 - a.window;
  } else if (a.window > 0 && (long long)len - a.window > lo) {
    lo = (long long)len - a.window;
  }
  const T* q = static_cast<const T*>(a.q) + (int64_t)(row0 + i) * a.q_row + (int64_t)head * a.q_head;
  for (int c = lane; c < HD; c += 32) qs[warp][c] = row_f(q[c]) * a.scale_log2;
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[HD / 32] = {};
  const long long n_own = own ? n : 0;
  for (long long j0 = lo; j0 < hi + n_own; j0 += 32) {
    const long long j = j0 + lane;
    float s = -INFINITY, vs = 0.f;
    const uint8_t* vc = nullptr;
    const T* vr = nullptr;
    if (j < hi) {
      const int blk = a.table[(int64_t)req * a.table_blocks + (j >> a.log_t) % a.table_blocks];
      if (in_bounds(blk >= 0 && blk < a.n_blocks, a.err)) {
        const int64_t off = blk * a.c_block + kvh * a.c_head + (j & (n_tok - 1)) * a.c_token;
        vc = a.v + off;
        vs = a.v_scale[(int64_t)blk * a.n_kv + kvh];
        s = 0.f;
        for (int c = 0; c < HD; c++) s = fmaf(qs[warp][c], code_f(a.k[off + c]), s);
        s *= a.k_scale[(int64_t)blk * a.n_kv + kvh];
      }
    } else if (j < hi + n_own) {
      const int jo = (int)(j - hi);
      if (!a.causal || (jo <= i && (a.window <= 0 || jo > i - a.window))) {
        const T* kr = static_cast<const T*>(a.k_own) + (int64_t)(row0 + jo) * a.ko_row + (int64_t)kvh * a.ko_head;
        vr = static_cast<const T*>(a.v_own) + (int64_t)(row0 + jo) * a.vo_row + (int64_t)kvh * a.vo_head;
        s = 0.f;
        for (int c = 0; c < HD; c++) s = fmaf(qs[warp][c], row_f(kr[c]), s);
      }
    }
    float cm = s;
    for (int x = 16; x > 0; x >>= 1) cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, x));
    const float mn = fmaxf(m, cm);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float alpha = exp2f(m - base);
    const float p = vc || vr ? exp2f(s - base) : 0.f;
    l = l * alpha + warp_sum(p);
    m = mn;
    for (int c = 0; c < HD / 32; c++) o[c] *= alpha;
    for (int src = 0; src < 32; src++) {
      const float ps = __shfl_sync(0xffffffffu, p, src), sc = __shfl_sync(0xffffffffu, vs, src);
      const uint8_t* c8 = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(vc), src));
      const T* cr = reinterpret_cast<const T*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(vr), src));
      if (c8)
        for (int c = 0; c < HD / 32; c++) o[c] = fmaf(ps, code_f(c8[c * 32 + lane]) * sc, o[c]);
      else if (cr)
        for (int c = 0; c < HD / 32; c++) o[c] = fmaf(ps, row_f(cr[c * 32 + lane]), o[c]);
    }
  }
  T* out = static_cast<T*>(a.out) + (int64_t)(row0 + i) * a.o_row + (int64_t)head * a.o_head;
  for (int c = 0; c < HD / 32; c++) row_store(out + c * 32 + lane, l == 0.f ? 0.f : o[c] / l);
}

template <typename T>
cudaError_t launch_simple(const CacheAttnArgs& a, cudaStream_t s) {
  const dim3 grid((a.n_kv * a.grp + kSimpleWarps - 1) / kSimpleWarps, a.max_q, a.n_req), block(kSimpleWarps * 32);
  switch (a.hd) {
    case 64: return launch_pdl(cache_attn_simple_kernel<T, 64>, grid, block, 0, s, a);
    case 128: return launch_pdl(cache_attn_simple_kernel<T, 128>, grid, block, 0, s, a);
    case 256: return launch_pdl(cache_attn_simple_kernel<T, 256>, grid, block, 0, s, a);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_cache_attn(int dtype, const CacheAttnArgs& a, cudaStream_t s) {
  return dtype == DFLASH_BF16 ? launch_simple<__nv_bfloat16>(a, s) : launch_simple<__half>(a, s);
}

}  // namespace dfl
