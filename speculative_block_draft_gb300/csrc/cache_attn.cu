// Attention of a few query rows per request over the paged 8-bit context cache (include/dflash.h,
// dflash_cache_attention):
//   out_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(scale * q_i . k_j)
// over the cached keys that row i sees and, when given, the own rows of its request.
//
// First kernel: 128 cached keys at a time on the fifth-generation tensor cores, straight from the
// e4m3 codes as the copy engine brings them (no conversion in between):
//   S[key][row]  = K Q^T   M = 128 keys,  N = query rows, K = head_dim   (kind::f8f6f4)
//   O[d][row]   += V^T P   M = head_dim,  N = query rows, K = 128 keys
// Keys are the tensor-memory lanes of S, so a thread owns a key: few rows fill every lane, a row's
// softmax needs no exchange between threads while its reference stays (below), and a thread's
// probabilities are contiguous bytes of the second product's operand. Queries and probabilities
// are not 8-bit values, so both enter as sums of 8-bit terms: a value's nearest code, the nearest code of what that
// leaves, and so on. Queries are e4m3 terms of a row scaled to its largest element: two hold bf16's 8 significant
// bits, three f16's 11, both down to a step of 2^-18 of that element. The first product adds them up in one accumulator.
// Probabilities are three e5m2 terms (split8), which hold 11 significant bits over 30 powers of two. They are further
// columns of the second product (cheaper: an MMA of up to 64 columns takes the time of one of 64), added when O is read.
//
//   t_ij = s_ij * q_scale_i * k_scale * scale * log2(e) + log2(v_scale)    (scales of the key's block)
//   w_ij = 2^(t_ij - m_i)                       = p_ij * v_scale / 2^m_i
//   O_i = sum_j w_ij * vcode_j,  L_i = sum_j w_ij / v_scale,  out_i = O_i / L_i
// The reference m_i of a row is set so that its largest weight so far is 2^kTop, and moves only when a
// weight would pass 2^kMax (kept below 57344, the largest code): then L and O are rescaled.
// What the terms must hold: L counts a weight w in full and O counts its terms, so what is lost of the small weights adds
// up over the keys, and rows with one large weight and very many small ones are the rule (the first token of a context, with
// a small value). So the step at which a weight ends has to lie far below the largest weight over the number of keys.
// It is 2^-20 (split8), half of it at most is lost: 2^-30 of the largest weight for each key, 2^-13 of it
// over 2^17 keys. (Weights as two or three e4m3 terms, which end at 2^-9, lost the tail: 40% of a row over 16384 keys
// of which one held 0.8.)
//
// What bounds it: the cache's bytes, in the steady state (32 requests, 8 KV heads of 128 columns: 7.1 TB/s with 5
// rows per KV head, 6.8 with 25 rows, 6.5 with 40, 5.6 with 45, from the difference of 16384 and 8192
// keys each), and besides some 12 us (5 rows) to 18 us (25) of start, first references, output and second kernel,
// which short contexts feel.
//
// Work is split by key tiles, not by requests: all tiles of all (request, KV head, row chunk) in one
// line, an equal run of them for each CTA. A run may begin or end inside a (request, head, chunk); those
// pieces are left as (O, m, L) for the second kernel, which joins them and attends over the own rows
// in fp32. (Joined instead by the CTA whose piece comes last: 54.8 us against 42.7 for 32 requests x 5 rows over 512 to
// 2048 keys, 47.6 against 27.9 for 4 x 8 rows over 2000 to 9000. Its four warps have the rows' latency to themselves.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>

#include "cache.h"
#include "common.cuh"
#include "tc05.cuh"

namespace dfl {

namespace {

constexpr int kTile = 128;               // keys per tile
constexpr int kThreads = 256;            // warp 0: copies, 1: MMAs, 2 and 3: queries; warps 4-7: softmax
constexpr int kSoftmax0 = 128;           // first softmax thread
// With two CTAs per SM a thread starts with 128 registers; the softmax warps take over part of the others'.
constexpr int kStartRegs = 128, kOtherRegs = 96, kSoftmaxRegs = 160;
static_assert(kOtherRegs + kSoftmaxRegs <= 2 * kStartRegs, "the shares come out of what the CTA was launched with");
constexpr int kConstRing = 16;           // tiles whose key constants are kept
// Key and value tiles in flight. Four for few rows, bound by the bytes: 32 single tokens over 512 to 16384 keys take
// 89.7 us, 91.4 with six, 91.9 with three. Three for more rows, whose first tiles then come sooner: 4 requests x 8 rows
// over 2000 to 9000 keys 26.5 us, 28.0 with four; with 256 columns (16 x 9 rows) 47.5 us, 47.0 with four.
constexpr int kMaxStages = 4;
constexpr int kPPanel = kTile * 128;     // probabilities: 128 keys x up to 128 columns a panel
constexpr int kPTerms = 3;               // terms of a probability
constexpr float kTop = 9.f, kMax = 15.5f;
constexpr float kLast = 64.f;            // its last term is stored times this
constexpr float kUnset = -1e30f;         // reference of a piece whose row has seen no key
// Built for two CTAs per SM, with 128 registers per thread: 16 requests x 9 rows of 5 query heads, 128 columns, 71 us
// with two CTAs and 90 us with one. With 256 columns shared memory holds one, and more registers help from 48 rows on
// (66 us against 72; 24 rows 29.4 against 27.8).
__host__ __device__ constexpr bool two_per_sm(int hd, int rp) { return rp <= (hd == 256 ? 40 : 48); }
constexpr int kRowArrays = 64;           // rows of the per-row arrays in shared memory

__device__ __forceinline__ float row_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float row_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void row_store(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void row_store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---- geometry ------------------------------------------------------------------------------------
struct Request {
  int req, row0, n;        // table row, first query row, query rows (0: nothing to do)
  int len, lo;             // cached tokens; first position that any row sees
  int s0, tiles;           // first position of tile 0 (a block boundary), key tiles
  int chunks;
};

// First visible position of row i of the request, and one past its last (cached keys). Lengths end below 2^31 - 2^16,
// so positions of rows fit 32 bits.
__device__ __forceinline__ void row_range(const CacheAttnArgs& a, const Request& r, int i, int& lo, int& hi) {
  // a ring holds its last blocks; the newest one, of however few tokens, has a scale of its own, so that what is left of
  // the one it replaced does not count
  const int T = 1 << a.log_t;
  lo = max(0, ((r.len + T - 1) & -T) - a.held);
  hi = r.len;
  if (a.causal) {
    const int at = a.k_own ? r.len + i : r.len - r.n + i;
    hi = min(hi, at + 1);
    if (a.window > 0 && at >= a.window) lo = max(lo, at + 1 - a.window);   // a window may be as large as an int
  } else if (a.window > 0) {
    lo = max(lo, r.len - a.window);
  }
  hi = max(hi, 0);
}

// r / grp, for r < DFLASH_CACHE_MAX_Q * grp: by the rounded-up 2^32 / grp, exact while that times grp is below 2^32.
__device__ __forceinline__ int by_group(const CacheAttnArgs& a, int r) { return a.grp == 1 ? r : (int)__umulhi((unsigned)r, a.grp_mul); }

// What a call says about request b: first query row, query rows, cached tokens, table row.
__device__ __forceinline__ int4 read_request(const CacheAttnArgs& a, int b) {
  int row0 = b * a.max_q, n = a.max_q;
  const int req = a.requests ? a.requests[b] : b;
  if (a.row_start) {
    row0 = a.row_start[b];
    n = a.row_start[b + 1] - row0;
    if (!in_bounds(n <= a.max_q, a.err)) n = a.max_q;
  }
  const bool known = req >= 0 && req < a.table_rows;
  const int len = a.lens[known ? req : 0];
  if (!in_bounds(n >= 0 && row0 >= 0 && row0 <= a.n_rows - n && known, a.err)) n = 0;
  return make_int4(row0, n, n > 0 ? min(max(len, 0), 0x7fff0000) : 0, req);
}

__device__ __forceinline__ Request request_of(const CacheAttnArgs& a, int4 w) {
  Request r;
  r.row0 = w.x;
  r.n = w.y;
  r.len = w.z;
  r.req = w.w;
  int hi;
  row_range(a, r, 0, r.lo, hi);
  r.s0 = r.lo & ~((1 << a.log_t) - 1);
  r.tiles = r.n > 0 && r.lo < r.len ? (r.len - r.s0 + kTile - 1) / kTile : 0;
  r.chunks = a.p.chunks == 1 ? 1 : (r.n * a.grp + a.p.rc - 1) / a.p.rc;
  return r;
}

// A CTA's run is units [first, last) of all; CTA c of g gets an equal share. A (request, KV head, row chunk) is
// `setup` units, which stand for its queries, its first references and its output, then its key tiles. They count
// nothing where there is a CTA for every tile.
__device__ __forceinline__ int unit_begin(int c, int total, int g) {
  const int each = total / g;
  return c * each + min(c, total - each * g);
}

// The tiles of one (request, KV head, row chunk) that a CTA's run holds.
struct Segment {
  Request r;
  int b, pair, head, chunk;   // pair: over all requests, heads and chunks (with gaps)
  int t0, t1;
};

// A place in the ring of key and value tiles, in order.
struct Ring {
  int slot = 0, fill = 0;                 // fill: how often the slot has been filled before
  __device__ void next(int n) {
    if (++slot == n) {
      slot = 0;
      fill++;
    }
  }
};

struct Walk {
  int u, u_end, b;
  __device__ bool next(const CacheAttnArgs& a, const int* before, const int4* words, Segment& s) {
    if (u >= u_end) return false;
    while (u >= before[b + 1]) b++;
    s.b = b;
    s.r = request_of(a, words[b]);
    const int setup = before[a.n_req + 1];
    const unsigned rem = u - before[b], units = s.r.tiles + setup, chunks = s.r.chunks, p = rem / units;
    const int at = rem - p * units, n = min((int)units - at, u_end - u);
    s.head = p / chunks;
    s.chunk = p - s.head * chunks;
    s.pair = (b * a.n_kv + s.head) * a.p.chunks + s.chunk;
    s.t0 = max(at - setup, 0);
    s.t1 = at + n - setup;
    u += n;
    return s.t1 > s.t0;                                // false only at the run's end
  }
};

// ---- tensor-core pieces --------------------------------------------------------------------------
// kind::f8f6f4, M = 128, e4m3 x e4m3 (bits 10-12: the second operand's format, 0 = e4m3, 1 = e5m2) -> fp32
__device__ __forceinline__ constexpr uint32_t idesc_scores(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | (8u << 24); }
// e4m3 x e5m2; the major bits (15, 16) say that the operands' rows run along the contraction (MN-major).
__device__ __forceinline__ constexpr uint32_t idesc_weights(int n) {
  return (1u << 4) | (1u << 10) | (3u << 15) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

// Shared-memory descriptor: swizzle 2 = 128 B, 4 = 64 B; sbo: bytes between groups of 8 rows (keys or
// query rows), lbo: bytes between pieces of one swizzle width along an MN-major row.
__device__ __forceinline__ constexpr uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t swizzle) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)swizzle << 61);
}

__device__ __forceinline__ void umma_f8_warp(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// A load of 8 columns: the registers may be used once tmem_wait8 has returned.
__device__ __forceinline__ void tmem_start8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_wait8(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}

// Two fp32 lanes per instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
               "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
               "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
               "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, int u, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(u), "r"(bar)
      : "memory");
}

// Barrier of the four softmax warps; `any` returns whether any thread's predicate holds.
__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync.aligned 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool softmax_any(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.aligned.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

// Wait for phase `parity` of an mbarrier for at most `ns`; on giving up, set the error bit and return false. (As
// mbar_wait_bounded, in few instructions: the loops here have a dozen waits. The limit is the launch's, not a word in memory:
// with one, 32 requests x 5 rows took 41.6 us instead of 40.3, a token over 1024 keys 8.4 instead of 8.2.)
__device__ __forceinline__ bool wait_bar(const uint64_t* bar, int parity, unsigned* err, unsigned ns) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 t0, t1;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE;\n\t"
      "mov.u32 t0, %%globaltimer_lo;\n\t"
      "AGAIN:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE;\n\t"
      "mov.u32 t1, %%globaltimer_lo;\n\t"
      "sub.u32 t1, t1, t0;\n\t"
      "setp.lt.u32 q, t1, %3;\n\t"
      "@q bra AGAIN;\n\t"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"((uint32_t)parity & 1), "r"(ns)
      : "memory");
  if (!ok && err) atomicOr(err, kErrTimeoutCache);
  return ok;
}
// The same by a converged warp, for all its lanes.
__device__ __forceinline__ bool wait_bar_warp(const uint64_t* bar, int parity, unsigned* err, unsigned ns) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, err, ns));
}
// What a CTA must see finished before it leaves: its copies and its products. 1 s, whatever the launch's limit.
__device__ __forceinline__ bool wait_last(const uint64_t* bar, int parity) { return wait_bar(bar, parity, nullptr, kWaitNs); }

// log2 and reciprocal of a scale, exact for the powers of two that the append writes.
__device__ __forceinline__ void scale_terms(float v, float& lg, float& inv) {
  const uint32_t u = __float_as_uint(v);
  if ((u & 0x7fffffu) == 0 && u < 0x7f000000u) {       // 2^-64 <= v <= 2^126
    lg = (float)((int)(u >> 23) - 127);
    inv = __uint_as_float((254u << 23) - u);
  } else {
    lg = log2f(v);
    inv = 1.f / v;
  }
}

// Sums or maxima over the warp of 8 values per lane: lane l returns that of value (l >> 2) & 7 (lanes of a quad agree).
// Nine shuffles instead of forty (and a redux.sync per value took 70 cycles each).
template <typename F>
__device__ __forceinline__ float reduce8(const float (&v)[8], F f) {
  const int lane = threadIdx.x & 31;
  float a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; i++) a[i] = f(lane & 16 ? v[i + 4] : v[i], __shfl_xor_sync(0xffffffffu, lane & 16 ? v[i] : v[i + 4], 16));
#pragma unroll
  for (int i = 0; i < 2; i++) b[i] = f(lane & 8 ? a[i + 2] : a[i], __shfl_xor_sync(0xffffffffu, lane & 8 ? a[i] : a[i + 2], 8));
  float c = f(lane & 4 ? b[1] : b[0], __shfl_xor_sync(0xffffffffu, lane & 4 ? b[0] : b[1], 4));
  c = f(c, __shfl_xor_sync(0xffffffffu, c, 2));
  return f(c, __shfl_xor_sync(0xffffffffu, c, 1));
}

// 2^k >= 2^-64 with amax <= 448 * 2^k (amax finite): a row's largest value lands in (224, 448].
__device__ __forceinline__ float row_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int k = (int)(u >> 23) - 135 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __int_as_float((max(k, kMinScaleExp) + 127) << 23);
}

// Four values as TERMS words of four e4m3 codes (the first in the low byte), from f16: magnitudes <= 448. The
// rounding to f16 is at the last term's level (2^-12).
template <int TERMS>
__device__ __forceinline__ void split4(float2 x, float2 y, uint32_t (&c)[TERMS]) {
  uint32_t u, v;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(x.y), "f"(x.x));
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(y.y), "f"(y.x));
#pragma unroll
  for (int t = 0; t < TERMS; t++) {
    if (t + 1 < TERMS) {
      asm("{.reg .b16 p, q;\n\t.reg .b32 b, d;\n\t"
          "cvt.rn.satfinite.e4m3x2.f16x2 p, %1;\n\t"
          "cvt.rn.satfinite.e4m3x2.f16x2 q, %2;\n\t"
          "mov.b32 %0, {p, q};\n\t"
          "cvt.rn.f16x2.e4m3x2 b, p;\n\t"
          "cvt.rn.f16x2.e4m3x2 d, q;\n\t"
          "sub.rn.f16x2 %1, %1, b;\n\t"
          "sub.rn.f16x2 %2, %2, d;}"
          : "=r"(c[t]), "+r"(u), "+r"(v));
    } else {
      asm("{.reg .b16 p, q;\n\t"
          "cvt.rn.satfinite.e4m3x2.f16x2 p, %1;\n\t"
          "cvt.rn.satfinite.e4m3x2.f16x2 q, %2;\n\t"
          "mov.b32 %0, {p, q};}"
          : "=r"(c[t]) : "r"(u), "r"(v));
    }
  }
}

// Eight weights w >= 0, <= 2^kMax, as three groups of eight e5m2 codes. e5m2 is the upper byte of f16: with h the f16 nearest to w,
//   c0 = h to 3 significant bits, c1 = h - c0 to 3, c2 = 64 (h - c0 - c1) to 3
// where adding 0x80 to an f16's bits and dropping the low byte rounds to the nearest (halves away from 0; the differences are
// exact). Each term leaves at most a sixteenth of what the one before left, half a step of the first being an eighth of its
// power of two, so c0 + c1 + c2 / 64 is h: all its 11 bits. Below 2^-14 an f16 and the first two codes have steps of
// 2^-24 and 2^-16; then the last code, of up to 2^-17 times 64, ends the sum within 2^-21. A NaN stays one.
__device__ __forceinline__ void split8(const float2 (&w)[4], uint2 (&c)[kPTerms]) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; i++) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h[i]) : "f"(w[i].y), "f"(w[i].x));
#pragma unroll
  for (int t = 0; t + 1 < kPTerms; t++) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; i++) r[i] = h[i] + 0x00800080u;
    c[t].x = __byte_perm(r[0], r[1], 0x7531);
    c[t].y = __byte_perm(r[2], r[3], 0x7531);
#pragma unroll
    for (int i = 0; i < 4; i++) asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(h[i]) : "r"(r[i] & 0xff00ff00u));
  }
  constexpr uint32_t kLast2 = 0x54005400u;             // kLast, twice
  static_assert(kLast == 64.f, "as in kLast2");
#pragma unroll
  for (int i = 0; i < 4; i++) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h[i]) : "r"(kLast2));
  asm("{.reg .b16 p, q;\n\tcvt.rn.satfinite.e5m2x2.f16x2 p, %1;\n\tcvt.rn.satfinite.e5m2x2.f16x2 q, %2;\n\tmov.b32 %0, {p, q};}"
      : "=r"(c[kPTerms - 1].x) : "r"(h[0]), "r"(h[1]));
  asm("{.reg .b16 p, q;\n\tcvt.rn.satfinite.e5m2x2.f16x2 p, %1;\n\tcvt.rn.satfinite.e5m2x2.f16x2 q, %2;\n\tmov.b32 %0, {p, q};}"
      : "=r"(c[kPTerms - 1].y) : "r"(h[2]), "r"(h[3]));
}

// ---- shared memory -----------------------------------------------------------------------------------
struct alignas(16) RowState {            // per query row of the CTA's chunk
  float4 key[kConstRing][kTile / 16];    // per tile and block: k_scale * scale * log2(e), log2(v_scale), 1 / v_scale, there or not
  float neg_m[kRowArrays];               // minus the reference
  float qs[2][kRowArrays];               // the row's query scale; by turns for the segments, as the queries
  float f[kRowArrays], by[kRowArrays];   // factor of a moved reference, minus its step; 1 / L at the end
  float red[4][kRowArrays];              // per softmax warp: maxima, sums
  uint32_t moved[2];                     // rows 0-31, 32-63 whose reference moved
  int unset[kRowArrays];                 // the row has seen no key (its reference is 0)
  int64_t out[kRowArrays];               // its element offset in the output
};

// MMA columns of the scores and of the weights (multiples of 16), and rows of the queries' terms
__host__ __device__ constexpr int score_columns(int rp) { return (rp + 15) / 16 * 16; }
__host__ __device__ constexpr int weight_columns(int rp) { return (kPTerms * rp + 15) / 16 * 16; }
__host__ __device__ constexpr int weight_panels(int rp) { return weight_columns(rp) > 128 ? 2 : 1; }
__host__ __device__ constexpr int query_rows(int terms, int rp) { return (terms * rp + 15) / 16 * 16; }
__host__ __device__ constexpr int panels_of(int hd) { return hd == 256 ? 2 : 1; }
__host__ __device__ constexpr int stage_bytes(int hd) { return kTile * hd; }

__host__ __device__ inline size_t attn_fixed_smem(int hd, int terms, int rp, int n_req) {
  return (size_t)2 * query_rows(terms, rp) * 128 * panels_of(hd) + weight_panels(rp) * kPPanel + sizeof(RowState) + (2 * kMaxStages + 12) * 8 + 80 + 20 * (size_t)(n_req + 1);
}

// ---- the first kernel ----------------------------------------------------------------------------------
// The queries of a segment as e4m3 terms in shared memory (rows of 128 bytes, swizzled as the MMA reads them; a
// second panel for the columns from 128), by `threads` >= 64 threads. A row is scaled so that its largest value
// lies in (224, 448]; qs gets the scale.
template <typename T, int HD, int TERMS, int RP>
__device__ __forceinline__ void prepare_queries(const CacheAttnArgs& a, const Segment& sg, uint8_t* q_s, float* qs, int tid, int threads) {
  constexpr int kPerRow = HD / 8, kAhead = 5;          // lanes of a row; rows in flight per lane
  constexpr int N = query_rows(TERMS, RP);
  const int r0 = sg.chunk * a.p.rc, rows = min(a.p.rc, sg.r.n * a.grp - r0);
  const int c8 = (tid % kPerRow) * 8, at_once = threads / kPerRow;
  if (tid < RP && tid >= rows) qs[tid] = 0.f;          // padding: whatever is there counts nothing
  for (int first = tid / kPerRow; first - tid / kPerRow < rows; first += kAhead * at_once) {
    uint4 v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; u++) {
      const int r = first + u * at_once;
      v[u] = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const int i = by_group(a, r0 + r), row = sg.r.row0 + i, head = sg.head * a.grp + r0 + r - i * a.grp;
        v[u] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + row * a.q_row + head * a.q_head + c8);
      }
    }
#pragma unroll 1
    for (int u = 0; u < kAhead; u++) {
      const int r = first + u * at_once;
      const uint4 now = v[0];                          // the rows move down: one copy of this code
#pragma unroll
      for (int w = 0; w + 1 < kAhead; w++) v[w] = v[w + 1];
      if (r - tid / kPerRow >= rows) break;            // for the whole warp, and no lane has a row
      const T* e = reinterpret_cast<const T*>(&now);
      float x[8], amax = 0.f;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        x[j] = row_f(e[j]);
        const float m = fabsf(x[j]);
        if (m <= 3.402823466e38f) amax = fmaxf(amax, m);
        else x[j] = __int_as_float(0x7fffffff);        // an infinite query has no softmax
      }
#pragma unroll
      for (int o = kPerRow / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const float sc = row_scale(amax), inv = __uint_as_float((254u << 23) - __float_as_uint(sc));
      if (r < rows) {
        uint32_t c[2][TERMS];
#pragma unroll
        for (int j = 0; j < 2; j++)
          split4<TERMS>(make_float2(x[4 * j] * inv, x[4 * j + 1] * inv), make_float2(x[4 * j + 2] * inv, x[4 * j + 3] * inv), c[j]);
#pragma unroll
        for (int t = 0; t < TERMS; t++) {
          const int n = t * RP + r;
          uint8_t* to = q_s + (c8 >> 7) * (N * 128) + n * 128 + ((((c8 & 127) >> 4) ^ (n & 7)) << 4) + (c8 & 8);
          *reinterpret_cast<uint2*>(to) = make_uint2(c[0][t], c[1][t]);
        }
        if (c8 == 0) qs[r] = sc;
      }
    }
  }
}

// RP: query rows of a chunk, padded to the next of 8, 16, 24, 32, 40, 48 (bf16) and 64 (bf16). It is known here so that
// the loops over the rows have no branches: with one, every eight rows would wait for their own loads (32 requests x 25
// rows 81 us; 64 without, and with weights split in two). 25 rows padded to 40 instead of 32 take 53.1 us against 49.5, 45 rows to 64 instead of 48 100
// against 90.
template <typename T, int HD, int RP>
__global__ void __launch_bounds__(kThreads, two_per_sm(HD, RP) ? 2 : 1)
    cache_attn_kernel(const __grid_constant__ CacheAttnArgs a, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap) {
  constexpr int TERMS = __is_same(T, __nv_bfloat16) ? 2 : 3;   // of a query
  constexpr int PANELS = panels_of(HD), STAGE = stage_bytes(HD);
  constexpr int ROWB = HD < 128 ? HD : 128;            // bytes of a key in a panel
  constexpr int PANEL = kTile * 128;                   // bytes between panels (HD = 256)
  constexpr int CH = RP / 8;                           // chunks of 8 rows
  constexpr int NS = score_columns(RP), N = weight_columns(RP), NQ = query_rows(TERMS, RP);
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  constexpr int q_bytes = NQ * 128 * PANELS;
  const int S = a.p.stages;
  uint8_t* ring = sm;
  uint8_t* q_s = ring + (size_t)S * STAGE;             // two buffers, by turns for the segments
  uint8_t* p_s = q_s + 2 * q_bytes;
  RowState& rs = *reinterpret_cast<RowState*>(p_s + weight_panels(RP) * kPPanel);
  uint64_t* bars = reinterpret_cast<uint64_t*>(&rs + 1);
  uint64_t *full = bars, *empty = bars + kMaxStages, *s_full = bars + 2 * kMaxStages, *s_free = s_full + 2, *q_full = s_full + 4,
           *q_free = s_full + 6, *p_full = s_full + 8, *p_free = s_full + 9, *drained = s_full + 10, *q_first = s_full + 11;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_full + 12);
  // Set when a softmax wait gave up, by turns for the stretches between two points where all softmax threads look
  // (just behind a barrier), so that all of them see the same and leave together
  volatile int* dead = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint64_t* scan = reinterpret_cast<uint64_t*>(tmem_slot + 4);   // warp sums
  int4* words = reinterpret_cast<int4*>(tmem_slot + 20);
  int* before = reinterpret_cast<int*>(words + a.n_req);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; i++) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), 1);
    }
    for (int i = 0; i < 2; i++) {
      mbar_init(smem_u32(&s_full[i]), 2);              // the MMAs, and the warp that issued them
      mbar_init(smem_u32(&s_free[i]), 4);
      mbar_init(smem_u32(&q_full[i]), 2);              // the two query warps
      mbar_init(smem_u32(&q_free[i]), 2);              // the MMAs, and the softmax warps
    }
    mbar_init(smem_u32(p_full), 4);
    mbar_init(smem_u32(p_free), 1);
    mbar_init(smem_u32(drained), 1);
    mbar_init(smem_u32(q_first), kThreads / 32 - 1);
    dead[0] = dead[1] = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), (uint32_t)a.p.tmem_cols);
    tmem_relinquish();
  }
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  // units before each request: one prefix sum over the requests, a few of them per thread, of the key tiles (low half)
  // and the setups (high half)
  {
    const int per = (a.n_req + kThreads - 1) / kThreads, b0 = threadIdx.x * per;
    auto work = [&](int b) -> uint64_t {
      const Request r = request_of(a, words[b]);
      const unsigned pairs = r.tiles > 0 ? r.chunks * a.n_kv : 0;
      return (uint64_t)pairs << 32 | pairs * r.tiles;
    };
    uint64_t mine = 0;
#pragma unroll 1
    for (int j = 0; j < per; j++)
      if (b0 + j < a.n_req) {
        words[b0 + j] = read_request(a, b0 + j);
        mine += work(b0 + j);
      }
    uint64_t s = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t v = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += v;
    }
    if (lane == 31) scan[warp] = s;
    __syncthreads();
    uint64_t at = s - mine, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; w++) {
      at += w < warp ? scan[w] : 0;
      all += scan[w];
    }
    const int setup = (uint32_t)all > (uint32_t)a.grid ? a.p.setup : 0;
#pragma unroll 1
    for (int j = 0; j < per; j++)
      if (b0 + j < a.n_req) {
        before[b0 + j] = (int)((uint32_t)at + setup * (uint32_t)(at >> 32));
        at += per > 1 ? work(b0 + j) : mine;
      }
    if (threadIdx.x == 0) {
      before[a.n_req] = (int)((uint32_t)all + setup * (uint32_t)(all >> 32));
      before[a.n_req + 1] = setup;
    }
  }
  __syncthreads();
  const int total = before[a.n_req], ctas = min(a.grid, total);
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.n_req; b += kThreads) a.words[b] = words[b];   // for the second kernel
  Walk walk{0, 0, 0};
  if ((int)blockIdx.x < ctas) {
    walk.u = unit_begin(blockIdx.x, total, ctas);
    walk.u_end = unit_begin(blockIdx.x + 1, total, ctas);
    int lo = 0, hi = a.n_req;                          // the request that holds the first unit
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before[mid] <= walk.u) lo = mid;
      else hi = mid;
    }
    walk.b = lo;
  }
  // Ring order: K of a tile one step ahead of V of the one before: K0 K1 V0 K2 V1 .. V(n-1) per segment.
  const uint32_t tmem_o = tmem + 2 * NS;
  Segment sg;

  constexpr bool kSplitRegs = RP > 8 && two_per_sm(HD, RP);
  // queries of the first segment: all warps but the copy warp, which starts on the keys
  if (warp > 0) {
    Walk w = walk;
    if (w.next(a, before, words, sg)) prepare_queries<T, HD, TERMS, RP>(a, sg, q_s, rs.qs[0], threadIdx.x - 32, kThreads - 32);
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(q_first));
  }
  if (warp < 4) {
    if (kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 0) {
      // ---- copies: one per block of the tile (and 128-byte panel), each by a lane of its own, which also leaves the
      // block's scales for the softmax -----------------------------------------------------------------------
      Ring at;
      int g = 0;
      bool ok = (int)blockIdx.x != a.stall - 1;          // test hook: nothing fills this CTA's tiles
      const int nb = kTile >> a.log_t;
      while (ok && walk.next(a, before, words, sg)) {
        const int* table = a.table + (int64_t)sg.r.req * a.table_blocks;
        const int idx0 = (sg.r.s0 >> a.log_t) + lane;
        auto entry_of = [&](int t) {                     // this lane's block of tile t (as it is), -1: none
          const int idx = idx0 + t * nb;
          return lane < nb && t >= sg.t0 && t < sg.t1 && ((long long)idx << a.log_t) < sg.r.len ? table[idx % a.table_blocks] : -1;
        };
        struct Block {
          int e;
          float ks, vs;
        };
        auto block_of = [&](int e) {                     // -1 if it is not there; its scales
          Block b{-1, 0.f, 0.f};
          if (e != -1 && in_bounds(e >= 0 && e < a.n_blocks, a.err)) {
            b.e = e;
            b.ks = a.k_scale[(int64_t)e * a.n_kv + sg.head];
            b.vs = a.v_scale[(int64_t)e * a.n_kv + sg.head];
          }
          return b;
        };
        auto copy = [&](const CUtensorMap* map, const Block& b, bool key) {
          const int slot = at.slot;
          if (at.fill > 0) ok = wait_bar_warp(&empty[slot], at.fill + 1, a.err, a.wait_ns);
          if (!ok) return;
          const uint32_t bar = smem_u32(&full[slot]);
          const int n = __popc(__ballot_sync(0xffffffffu, b.e >= 0));
          if (b.e >= 0) {
            const uint32_t dst = smem_u32(ring + (size_t)slot * STAGE) + ((uint32_t)(lane * ROWB) << a.log_t);
#pragma unroll
            for (int p = 0; p < PANELS; p++) tma_load_5d(dst + p * PANEL, map, p * 128, 0, sg.head, b.e, a.layer, bar);
          }
          // The constants, behind the copies: their loads may still be under way. The softmax has read those that they
          // replace: the ring of tiles is deeper than the copies run ahead. This stage was free, so the scores of the
          // tile S / 2 back were issued, and the two score buffers let that happen when those of two tiles before it
          // had been read, its constants with them.
          if (key && lane < nb) {
            float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
            if (b.e >= 0) {
              scale_terms(fmaxf(b.vs, __int_as_float((kMinScaleExp + 127) << 23)), c.y, c.z);
              c.x = b.ks * a.scale_log2;
              c.w = 1.f;
            }
            rs.key[g % kConstRing][lane] = c;
          }
          __syncwarp();
          // the only arrival of the fill, so none of its bytes can end it before
          if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)n * ((uint32_t)HD << a.log_t));
          __syncwarp();
          at.next(S);
          if (key) g++;
        };
        // entries three tiles ahead, scales two ahead of the values: K of tile t + 1, then V of tile t
        Block cur{-1, 0.f, 0.f}, nxt = cur;
        int far = -1;
#pragma unroll 1
        for (int t = sg.t0 - 3; ok && t < sg.t1; t++) {
          const Block after = block_of(far);
          far = entry_of(t + 3);
#pragma unroll 1
          for (int side = 0; ok && side < 2; side++) {
            if (side == 0 ? t + 1 < sg.t0 || t + 1 >= sg.t1 : t < sg.t0) continue;
            copy(side == 0 ? &kmap : &vmap, side == 0 ? nxt : cur, side == 0);
          }
          cur = nxt;
          nxt = after;
        }
      }
      // no copy may be in flight when the CTA leaves: the last fill of every stage has landed
      for (int i = 0; i < S; i++) {
        const int fills = at.fill + (i < at.slot);
        if (fills > 0) wait_last(&full[i], fills - 1);
      }
    } else if (warp == 1) {
      // ---- MMAs ---------------------------------------------------------------------------------------------
      const uint32_t id_s = idesc_scores(NS);
      const uint32_t ring_a = smem_u32(ring);
      const uint64_t qd0 = smem_desc(smem_u32(q_s), 16, 1024, 2), pd = smem_desc(smem_u32(p_s), 16, 1024, 2);
      Ring at;                                           // consumed in the order of the copies
      int g = 0, n_seg = 0, pv_done = 0;                 // g: tiles so far
      bool ok = true;
      auto wait = [&](uint64_t* bar, int parity) { return wait_bar_warp(bar, parity, a.err, a.wait_ns); };
      while (ok && walk.next(a, before, words, sg)) {
        const int n = sg.t1 - sg.t0;
        const uint64_t qd = qd0 + (uint64_t)((n_seg & 1) * (q_bytes >> 4));
        ok = n_seg == 0 ? wait(q_first, 0) : wait(&q_full[n_seg & 1], (n_seg - 1) >> 1);
        auto scores = [&](int t) {                       // tile t of the segment
          const int slot = at.slot, gg = g + t;
          ok = ok && wait(&full[slot], at.fill);
          if (ok && gg >= 2) ok = wait(&s_free[gg & 1], (gg >> 1) + 1);
          if (!ok) return;
          tc05_fence_after();
          const uint64_t kd = HD == 64 ? smem_desc(ring_a + slot * STAGE, 16, 512, 4) : smem_desc(ring_a + slot * STAGE, 16, 1024, 2);
          const uint32_t d = tmem + (uint32_t)((gg & 1) * NS);
#pragma unroll
          for (int ks = 0; ks < HD / 32; ks++) {
            const uint64_t ka = kd + (uint64_t)((ks / 4) * (PANEL >> 4) + (ks % 4) * 2);
            const uint64_t qa = qd + (uint64_t)((ks / 4) * (NQ * 8) + (ks % 4) * 2);
#pragma unroll
            for (int i = 0; i < TERMS; i++) umma_f8_warp(d, ka, qa + (uint64_t)(i * RP * 8), id_s, ks > 0 || i > 0);
          }
          umma_commit_warp(smem_u32(&empty[slot]));
          umma_commit_warp(smem_u32(&s_full[gg & 1]));
          if (t + 1 == n) umma_commit_warp(smem_u32(&q_free[n_seg & 1]));
          if (lane == 0) mbar_arrive(smem_u32(&s_full[gg & 1]));   // passes the copy warp's constants on
          __syncwarp();
          at.next(S);
        };
#pragma unroll 1
        for (int t = -1; ok && t < n; t++) {
          if (t + 1 < n) scores(t + 1);
          if (t < 0) continue;
          const int slot = at.slot, gg = g + t;
          ok = ok && wait(&full[slot], at.fill) && wait(p_full, gg);
          if (!ok) break;
          tc05_fence_after();
          const uint32_t va = ring_a + slot * STAGE;
          const uint64_t vd = HD == 64 ? smem_desc(va, STAGE, 512, 4) : smem_desc(va, 16, 1024, 2);
#pragma unroll
          for (int p = 0; p < PANELS; p++)
#pragma unroll
            for (int ks = 0; ks < 4; ks++)
#pragma unroll
              for (int n0 = 0; n0 < N; n0 += 128)        // a panel of weights each
                umma_f8_warp(tmem_o + p * N + n0, vd + (uint64_t)((p * PANEL + ks * 32 * ROWB) >> 4),
                             pd + (uint64_t)((n0 / 128 * kPPanel + ks * 32 * 128) >> 4), idesc_weights(N - n0 < 128 ? N - n0 : 128), t > 0 || ks > 0);
          umma_commit_warp(smem_u32(&empty[slot]));
          umma_commit_warp(smem_u32(p_free));
          pv_done = gg + 1;
          at.next(S);
        }
        g += n;
        n_seg++;
      }
      // nothing of this CTA may still run on the tensor core when its memory is freed. After a wait that gave up
      // there may be scores without a probability product: their commits have a barrier of their own
      if (pv_done > 0 && !wait_last(p_free, pv_done - 1)) atomicOr(a.err, kErrTimeoutCache);
      if (!ok) {
        umma_commit_warp(smem_u32(drained));
        wait_last(drained, 0);
      }
    } else {
      // ---- queries of the later segments, while the one before is at work ---------------------------------------
      bool ok = true;
#pragma unroll 1
      for (int k = 0; ok && walk.next(a, before, words, sg); k++) {
        if (k == 0) continue;
        if (k >= 2) ok = wait_bar_warp(&q_free[k & 1], (k >> 1) + 1, a.err, a.wait_ns);
        if (!ok) break;
        prepare_queries<T, HD, TERMS, RP>(a, sg, q_s + (k & 1) * q_bytes, rs.qs[k & 1], threadIdx.x - 64, 64);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&q_full[k & 1]));
      }
    }
  } else {
    if (kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---- softmax ------------------------------------------------------------------------------------------
    const int quarter = warp & 3, key = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t p_row = smem_u32(p_s) + key * 128;
    int base = 0, g = 0, look = 0, n_seg = 0;
    bool gone = false;
    auto wait = [&](uint64_t* bar, int parity) {
      if (!wait_bar(bar, parity, a.err, a.wait_ns)) dead[look & 1] = 1;
      __syncwarp();
    };
    while (!gone && walk.next(a, before, words, sg)) {
      const int n_tiles = sg.t1 - sg.t0, r0 = sg.chunk * a.p.rc, rows = min(a.p.rc, sg.r.n * a.grp - r0);
      if (key < RP) {
        rs.neg_m[key] = 0.f;
        rs.unset[key] = key < rows;
        const int i = by_group(a, r0 + key);
        rs.out[key] = (sg.r.row0 + i) * a.o_row + (sg.head * a.grp + r0 + key - i * a.grp) * a.o_head;   // where key < rows
      }
      const float* row_qs = rs.qs[n_seg & 1];
      wait(n_seg == 0 ? q_first : &q_full[n_seg & 1], n_seg == 0 ? 0 : (n_seg - 1) >> 1);   // the query scales
      softmax_sync();

      int lo_all, hi_all, dummy;                       // keys that every row sees
      row_range(a, sg.r, by_group(a, r0), dummy, hi_all);
      row_range(a, sg.r, by_group(a, r0 + rows - 1), lo_all, dummy);
      const int at0 = a.k_own ? sg.r.len : sg.r.len - sg.r.n;   // position of the request's first row
      bool unset_any = true;                           // some row has seen no key
      float2 l[CH * 4];
#pragma unroll
      for (int r = 0; r < CH * 4; r++) l[r] = make_float2(0.f, 0.f);
      int pos = sg.r.s0 + sg.t0 * kTile + key;

#pragma unroll 1
      for (int t = 0; t < n_tiles; t++, pos += kTile) {
        const int gg = g + t;
        wait(&s_full[gg & 1], gg >> 1);
        tc05_fence_after();
        const float4 kc = rs.key[gg % kConstRing][key >> a.log_t];
        const float2 ka = make_float2(kc.x, kc.x), vb2 = make_float2(kc.y, kc.y), inv2 = make_float2(kc.z, kc.z);
        const bool seen = kc.w != 0.f && pos >= sg.r.lo && pos < sg.r.len;   // by some row
        const bool whole = seen && pos >= lo_all && pos < hi_all;             // by every row
        // Edges: which rows see this key. A key that no row sees must not reach the product: its code bytes may be
        // anything, and 0 * NaN is NaN. Nor may a NaN value reach the rows that do not see its key: there it becomes
        // 0 and the weight becomes NaN for the rows that do.
        const bool edge = __any_sync(0xffffffffu, !whole);
        uint32_t sees[2] = {~0u, ~0u};                   // rows 0-31, 32-63
        bool v_nan = false;
        if (!whole) {
          // row i of the request sees it from i = pos - at0 on, and with a window for so many rows
          uint64_t bits = 0;
          if (seen) {
            const int i0 = a.causal ? min(max(pos - at0, 0), sg.r.n) : 0;
            const int i1 = a.causal && a.window > 0 ? (int)min((long long)pos - at0 + a.window, (long long)sg.r.n) : sg.r.n;
            const int ra = min(max(i0 * a.grp - r0, 0), RP), rb = min(max(i1 * a.grp - r0, ra), RP);
            bits = (rb == 64 ? ~0ull : (1ull << rb) - 1) & ~(ra == 64 ? ~0ull : (1ull << ra) - 1);
          }
          sees[0] = (uint32_t)bits, sees[1] = (uint32_t)(bits >> 32);
          const int sq = base + (t + 1 < n_tiles ? 2 * t + 2 : 2 * n_tiles - 1), slot = sq % S;
          if (!wait_bar(&full[slot], sq / S, a.err, a.wait_ns)) dead[look & 1] = 1;
#pragma unroll 4
          for (int c = 0; c < HD / 16; c++) {
            uint4* at = reinterpret_cast<uint4*>(ring + (size_t)slot * STAGE + (c >> 3) * PANEL + key * ROWB + (c & 7) * 16);
            uint4 w = make_uint4(0, 0, 0, 0), bad = w;
            if (seen) {
              w = *at;
              bad = make_uint4(__vcmpeq4(w.x & 0x7f7f7f7fu, 0x7f7f7f7fu), __vcmpeq4(w.y & 0x7f7f7f7fu, 0x7f7f7f7fu),
                               __vcmpeq4(w.z & 0x7f7f7f7fu, 0x7f7f7f7fu), __vcmpeq4(w.w & 0x7f7f7f7fu, 0x7f7f7f7fu));
              if (!(bad.x | bad.y | bad.z | bad.w)) continue;
              v_nan = true;
            }
            *at = make_uint4(w.x & ~bad.x, w.y & ~bad.y, w.z & ~bad.z, w.w & ~bad.w);
          }
        }
        __syncwarp();
        // x = t - m of this key for each row
        float2 x[CH * 4];
        bool high = false;                               // an x above kMax
        const uint32_t ts = tmem + lanes + (uint32_t)((gg & 1) * NS);
        uint32_t s8[CH][8];
#pragma unroll
        for (int ch = 0; ch < CH; ch++) tmem_start8(ts + ch * 8, s8[ch]);
#pragma unroll
        for (int ch = 0; ch < CH; ch++) tmem_wait8(s8[ch]);
        tc05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s_free[gg & 1]));
#pragma unroll
        for (int ch = 0; ch < CH; ch++) {
          const float4* qp = reinterpret_cast<const float4*>(row_qs + ch * 8);
          const float4* mp = reinterpret_cast<const float4*>(&rs.neg_m[ch * 8]);
          const float4 q0 = qp[0], q1 = qp[1], m0 = mp[0], m1 = mp[1];
          const float2 q2[4] = {{q0.x, q0.y}, {q0.z, q0.w}, {q1.x, q1.y}, {q1.z, q1.w}};
          const float2 m2[4] = {{m0.x, m0.y}, {m0.z, m0.w}, {m1.x, m1.y}, {m1.z, m1.w}};
          float top = -INFINITY;
#pragma unroll
          for (int j = 0; j < 4; j++) {
            const float2 sc = make_float2(__uint_as_float(s8[ch][2 * j]), __uint_as_float(s8[ch][2 * j + 1]));
            // the scales first: their product with a sum may be finite where the query's alone is not
            const float2 v = fma2(sc, mul2(q2[j], ka), add2(vb2, m2[j]));
            x[ch * 4 + j] = v;
            top = fmaxf(top, fmaxf(v.x, v.y));
          }
          high |= top > kMax;
        }
        if (edge) {
          high = false;
          const float nan = __int_as_float(0x7fffffff);
#pragma unroll
          for (int r = 0; r < CH * 4; r++) {
            const uint32_t two = sees[r / 16] >> (2 * r % 32);
            if (v_nan) x[r] = make_float2(nan, nan);
            if (!(two & 1)) x[r].x = -INFINITY;
            if (!(two & 2)) x[r].y = -INFINITY;
            high |= fmaxf(x[r].x, x[r].y) > kMax;
          }
        }
        // the probabilities of the tile before have been read, and its part of O is there
        if (gg > 0) wait(p_free, gg - 1);
        const bool move = softmax_any(high || unset_any);
        gone = dead[look++ & 1];
        if (gone) break;
        if (move) {
          // New references: the largest x of a row over the tile goes to kTop where it passed kMax or is the row's first.
          // All rows are reduced, without branches between the chunks: their shuffles overlap.
#pragma unroll
          for (int ch = 0; ch < CH; ch++) {
            const float v8[8] = {x[4 * ch].x, x[4 * ch].y, x[4 * ch + 1].x, x[4 * ch + 1].y, x[4 * ch + 2].x, x[4 * ch + 2].y, x[4 * ch + 3].x, x[4 * ch + 3].y};
            const float mx = reduce8(v8, [](float p, float q) { return fmaxf(p, q); });
            if ((lane & 3) == 0) rs.red[quarter][ch * 8 + (lane >> 2)] = mx;
          }
          softmax_sync();
          bool still = false;
          float by = 0.f;                                // the reference grows by this
          if (key < RP) {
            const float mx = fmaxf(fmaxf(rs.red[0][key], rs.red[1][key]), fmaxf(rs.red[2][key], rs.red[3][key]));
            const bool first = rs.unset[key] && mx > -INFINITY;
            if (first || mx > kMax) by = mx - kTop;
            rs.f[key] = first ? 0.f : ex2(-by);
            rs.by[key] = -by;
            rs.neg_m[key] -= by;
            if (first) rs.unset[key] = 0;
            still = rs.unset[key];
          }
          const uint32_t moved = __ballot_sync(0xffffffffu, by != 0.f);
          if (lane == 0 && quarter < 2) rs.moved[quarter] = moved;
          unset_any = softmax_any(still);
#pragma unroll
          for (int r = 0; r < CH * 4; r++) {
            l[r] = mul2(l[r], *reinterpret_cast<const float2*>(&rs.f[2 * r]));
            x[r] = add2(x[r], *reinterpret_cast<const float2*>(&rs.by[2 * r]));
          }
          if (t > 0) {
            tc05_fence_after();
#pragma unroll 1
            for (int r0 = 0; r0 < RP; r0 += 8) {
              if (!((rs.moved[r0 >> 5] >> (r0 & 31)) & 0xffu)) continue;
#pragma unroll 1
              for (int p = 0; p < PANELS; p++) {
                const uint32_t to = tmem_o + lanes + (uint32_t)(p * N + r0 * kPTerms);
                uint32_t o8[kPTerms][8];
#pragma unroll
                for (int i = 0; i < kPTerms; i++) tmem_start8(to + i * 8, o8[i]);
#pragma unroll
                for (int i = 0; i < kPTerms; i++) {
                  tmem_wait8(o8[i]);
                  float o[8];
#pragma unroll
                  for (int j = 0; j < 8; j++) o[j] = __uint_as_float(o8[i][j]) * rs.f[r0 + j];
                  tmem_st8(to + i * 8, o);
                }
              }
            }
            tmem_wait_st();
          }
          softmax_sync();                                // f, by and moved have been read
        }
        __syncwarp();
#pragma unroll
        for (int ch = 0; ch < CH; ch++) {
          float2 w[4];
#pragma unroll
          for (int j = 0; j < 4; j++) {
            w[j] = make_float2(ex2(x[ch * 4 + j].x), ex2(x[ch * 4 + j].y));
            l[ch * 4 + j] = fma2(w[j], inv2, l[ch * 4 + j]);
          }
          // columns of the product: per chunk of rows, its terms side by side
          uint2 c[kPTerms];
          split8(w, c);
#pragma unroll
          for (int i = 0; i < kPTerms; i++) {
            const int o = (ch * kPTerms + i) * 8;
            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(p_row + (uint32_t)((o >> 7) * kPPanel + (((o >> 4 & 7) ^ (key & 7)) << 4) + (o & 8))),
                         "r"(c[i].x), "r"(c[i].y)
                         : "memory");
          }
        }
        fence_proxy_async();
        tc05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(p_full));
      }
      base += 2 * n_tiles;
      g += n_tiles;
      if (gone) break;

      // ---- end of the segment: L over the keys, then O -------------------------------------------------------
#pragma unroll
      for (int ch = 0; ch < CH; ch++) {
        const float v8[8] = {l[4 * ch].x, l[4 * ch].y, l[4 * ch + 1].x, l[4 * ch + 1].y, l[4 * ch + 2].x, l[4 * ch + 2].y, l[4 * ch + 3].x, l[4 * ch + 3].y};
        const float sum = reduce8(v8, [](float p, float q) { return p + q; });
        if ((lane & 3) == 0) rs.red[quarter][ch * 8 + (lane >> 2)] = sum;
      }
      wait(p_free, g - 1);
      softmax_sync();
      gone = dead[look++ & 1];
      if (gone) break;
      if (threadIdx.x == kSoftmax0) mbar_arrive(smem_u32(&q_free[n_seg & 1]));
      const bool direct = sg.t0 == 0 && sg.t1 == sg.r.tiles && !a.k_own;
      const size_t slot = (size_t)blockIdx.x + sg.pair;
      if (threadIdx.x == kSoftmax0) {                  // which CTAs hold the pair's tiles
        if (sg.t0 == 0) a.held_by[sg.pair].x = blockIdx.x;
        if (sg.t1 == sg.r.tiles) a.held_by[sg.pair].y = blockIdx.x;
      }
      if (key < RP) {
        const float L = (rs.red[0][key] + rs.red[1][key]) + (rs.red[2][key] + rs.red[3][key]);
        rs.f[key] = L == 0.f ? 0.f : 1.f / L;
        // a row whose scores were all NaN has no reference, but a sum that the second kernel has to see
        if (!direct) a.part_ml[slot * RP + key] = make_float2(rs.unset[key] && L == 0.f ? kUnset : -rs.neg_m[key], L);
      }
      softmax_sync();
      tc05_fence_after();
      float* part = a.part_o + slot * RP * HD + key;
      T* out = static_cast<T*>(a.out) + key;
#pragma unroll 1
      for (int p = 0; p < PANELS; p++) {
#pragma unroll 1
        for (int ch = 0; ch < rows; ch += 8) {
          uint32_t part8[kPTerms][8];
          float o8[8];
#pragma unroll
          for (int i = 0; i < kPTerms; i++) tmem_start8(tmem_o + lanes + (uint32_t)(p * N + ch * kPTerms + i * 8), part8[i]);
#pragma unroll
          for (int i = 0; i < kPTerms; i++) {
            tmem_wait8(part8[i]);
#pragma unroll
            for (int j = 0; j < 8; j++) o8[j] = i == 0 ? __uint_as_float(part8[i][j]) : fmaf(__uint_as_float(part8[i][j]), i + 1 < kPTerms ? 1.f : 1.f / kLast, o8[j]);
          }
          if (key < HD) {
            const int left = rows - ch;
            if (direct) {
#pragma unroll
              for (int j = 0; j < 8; j++)
                if (j < left) row_store(out + rs.out[ch + j] + p * 128, o8[j] * rs.f[ch + j]);
            } else {
              float* to = part + ch * HD + p * 128;
#pragma unroll
              for (int j = 0; j < 8; j++)
                if (j < left) to[j * HD] = o8[j];
            }
          }
        }
      }
      tc05_fence_before();
      softmax_sync();                                  // rs belongs to the next segment now
      n_seg++;
    }
  }

  // Only now: CTAs that wait beside this one slow its end (one request, 8 rows: 15.5 us against 14.8), and one that took
  // the tensor memory before a CTA of this kernel would wait for it, and it for this one.
  pdl_launch_dependents();
  tc05_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc05_fence_after();
    tmem_dealloc(tmem, (uint32_t)a.p.tmem_cols);
  }
}

// ---- the second kernel: join the pieces of a row, own rows, output ---------------------------------------------
// Latency-bound: two dependent rounds of loads (the call's numbers; then queries, own rows and pieces together). A CTA
// takes some rows of one (request, KV head, chunk), a row in HD / 8 lanes of eight columns each, so that the own
// rows' K/V are read once for all of them (a warp per row, each reading them all, took 18 us instead of 6 for 32
// requests x 5 rows of 5 query heads).
constexpr int kOwnTile = 16;                           // own rows in shared memory at a time
__host__ __device__ constexpr int join_rows(int hd, int warps) { return warps * 256 / hd; }

// kAtOnce: pieces in flight, eight where a row has many (one request x 8 rows over 2048 keys: 14.4 us, 15.1 with four),
// else four for the occupancy (32 requests x 5 rows: 41.0 us, 45.7 with eight). WARPS: four where they hold a chunk's
// rows (one token over 1024 keys: 8.1 us, 8.5 with eight), else eight (4 requests x 8 rows: 25.7 us, 27.5 with four).
template <typename T, int HD, int WARPS, int kAtOnce>
__global__ void __launch_bounds__(WARPS * 32) cache_attn_join_kernel(const __grid_constant__ CacheAttnArgs a) {
  constexpr int LPR = HD / 8;                          // lanes of a row
  constexpr int kStep = LPR / 8;                       // lanes between the scores of neighbouring own rows
  constexpr int kLoads = kOwnTile * LPR / (WARPS * 32) > 0 ? kOwnTile * LPR / (WARPS * 32) : 1;
  __shared__ uint4 own[2][kOwnTile][LPR];              // K, V
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LPR;
  const int pair = blockIdx.x, per_req = a.n_kv * a.p.chunks, b = pair / per_req, in_req = pair - b * per_req;
  const int head = in_req / a.p.chunks, chunk = in_req - head * a.p.chunks;
  const int2 by = a.held_by[pair];
  const Request rq = request_of(a, a.words[b]);
  const int rows = min(a.p.rc, rq.n * a.grp - chunk * a.p.rc), r_cta = blockIdx.y * join_rows(HD, WARPS);
  if (r_cta >= rows) return;
  // CTAs that hold tiles of these rows (within the grid even if one gave up before it left its number)
  const int c0 = rq.tiles > 0 ? max(by.x, 0) : 0, c1 = rq.tiles > 0 ? min(by.y, a.grid - 1) : -1;
  if (c0 == c1 && !a.k_own) return;                    // written by the first kernel
  const int r = min(r_cta + warp * (32 / LPR) + lane / LPR, rows - 1);    // spare lanes repeat the last row
  const bool live = r == r_cta + warp * (32 / LPR) + lane / LPR;
  const int rr = chunk * a.p.rc + r, i = by_group(a, rr), qh = head * a.grp + rr - i * a.grp, row = rq.row0 + i;
  const int n_own = a.k_own ? rq.n : 0;
  // own rows of a tile: this thread's pieces on their way, then into shared memory
  uint4 kw[kLoads], vw[kLoads];
  auto fetch = [&](int j) {
#pragma unroll
    for (int u = 0; u < kLoads; u++) {
      const int at = threadIdx.x + u * WARPS * 32, jr = at / LPR, c = at % LPR;
      kw[u] = vw[u] = make_uint4(0, 0, 0, 0);
      if (jr < kOwnTile && j + jr < n_own) {
        kw[u] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.k_own) + (rq.row0 + j + jr) * a.ko_row + head * a.ko_head + c * 8);
        vw[u] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.v_own) + (rq.row0 + j + jr) * a.vo_row + head * a.vo_head + c * 8);
      }
    }
  };
  auto unpack = [](uint4 w, float (&v)[8]) {
    const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int x = 0; x < 8; x++) v[x] = row_f(e[x]);
  };
  float q[8];
  if (n_own > 0) {
    fetch(0);
    unpack(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + row * a.q_row + qh * a.q_head + sub * 8), q);
#pragma unroll
    for (int x = 0; x < 8; x++) q[x] = fabsf(q[x]) <= 3.402823466e38f ? q[x] : __int_as_float(0x7fffffff);   // as in the first kernel
  }
  float m = -INFINITY, L = 0.f, o[8];
#pragma unroll
  for (int c = 0; c < 8; c++) o[c] = 0.f;
  for (int c = c0; c <= c1; c += kAtOnce) {
    float2 ml[kAtOnce];
    float4 w[kAtOnce][2];
    float top = m;
#pragma unroll
    for (int u = 0; u < kAtOnce; u++) {
      ml[u] = make_float2(kUnset, 0.f);
      if (c + u <= c1) {
        const size_t at = ((size_t)(c + u) + pair) * a.p.rp + r;
        ml[u] = __ldcg(&a.part_ml[at]);
        const float4* p = reinterpret_cast<const float4*>(a.part_o + at * HD + sub * 8);
        w[u][0] = __ldcg(p);
        w[u][1] = __ldcg(p + 1);
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; u++)
      if (ml[u].x != kUnset) top = fmaxf(top, ml[u].x);
    const float so = m == top ? 1.f : ex2(m - top);
    L *= so;
#pragma unroll
    for (int x = 0; x < 8; x++) o[x] *= so;
#pragma unroll
    for (int u = 0; u < kAtOnce; u++) {
      if (ml[u].x == kUnset) continue;
      const float sn = ml[u].x == top ? 1.f : ex2(ml[u].x - top);
      const float v[8] = {w[u][0].x, w[u][0].y, w[u][0].z, w[u][0].w, w[u][1].x, w[u][1].y, w[u][1].z, w[u][1].w};
      L = fmaf(ml[u].y, sn, L);
#pragma unroll
      for (int x = 0; x < 8; x++) o[x] = fmaf(v[x], sn, o[x]);
    }
    m = top;
  }
  const int j1 = a.causal ? i + 1 : n_own, j0 = a.causal && a.window > 0 ? max(0, i + 1 - a.window) : 0;   // own rows it sees
  for (int t0 = 0; t0 < n_own; t0 += kOwnTile) {
    if (t0 > 0) {
      __syncthreads();                                 // the tile before has been read
      fetch(t0);
    }
#pragma unroll
    for (int u = 0; u < kLoads; u++) {
      const int at = threadIdx.x + u * WARPS * 32;
      if (at < kOwnTile * LPR) {
        own[0][at / LPR][at % LPR] = kw[u];
        own[1][at / LPR][at % LPR] = vw[u];
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int j = t0; j < min(t0 + kOwnTile, n_own); j += 8) {
      float s8[8];
#pragma unroll
      for (int u = 0; u < 8; u++) {
        float k[8];
        unpack(own[0][j - t0 + u][sub], k);
        s8[u] = 0.f;
#pragma unroll
        for (int x = 0; x < 8; x++) s8[u] = fmaf(q[x], k[x], s8[u]);
      }
      // over the row's lanes; lane l of them: the score of row j + l / kStep
      float h4[4], h2[2];
      constexpr int D = LPR / 2;
#pragma unroll
      for (int x = 0; x < 4; x++) h4[x] = (sub & D ? s8[x + 4] : s8[x]) + __shfl_xor_sync(0xffffffffu, sub & D ? s8[x] : s8[x + 4], D);
#pragma unroll
      for (int x = 0; x < 2; x++) h2[x] = (sub & (D / 2) ? h4[x + 2] : h4[x]) + __shfl_xor_sync(0xffffffffu, sub & (D / 2) ? h4[x] : h4[x + 2], D / 2);
      float s = (sub & (D / 4) ? h2[1] : h2[0]) + __shfl_xor_sync(0xffffffffu, sub & (D / 4) ? h2[0] : h2[1], D / 4);
#pragma unroll
      for (int d = kStep / 2; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      const int mine = j + sub / kStep;
      s = mine >= j0 && mine < j1 ? s * a.scale_log2 : -INFINITY;
      float top = s;
#pragma unroll
      for (int d = kStep; d < LPR; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      top = fmaxf(top, m);
      const float base = top == -INFINITY ? 0.f : top;
      const float p = ex2(s - base), so = ex2(m - base);
      float sum = p;
#pragma unroll
      for (int d = kStep; d < LPR; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      L = fmaf(L, so, sum);
#pragma unroll
      for (int x = 0; x < 8; x++) o[x] *= so;
#pragma unroll
      for (int u = 0; u < 8; u++) {
        const float pu = __shfl_sync(0xffffffffu, p, (lane - sub) + u * kStep);
        if (j + u < j0 || j + u >= j1) continue;       // a masked row's values may be anything
        float v[8];
        unpack(own[1][j - t0 + u][sub], v);
#pragma unroll
        for (int x = 0; x < 8; x++) o[x] = fmaf(pu, v[x], o[x]);
      }
      m = top;
    }
  }
  if (!live) return;
  const float inv = L == 0.f ? 0.f : 1.f / L;
  uint4 w;
  T* e = reinterpret_cast<T*>(&w);
#pragma unroll
  for (int x = 0; x < 8; x++) row_store(&e[x], o[x] * inv);
  *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + row * a.o_row + qh * a.o_head + sub * 8) = w;
}

template <typename T, int HD, int WARPS>
cudaError_t launch_join(const CacheAttnArgs& a, cudaStream_t s) {
  const dim3 grid(a.n_req * a.n_kv * a.p.chunks, (a.p.rc + join_rows(HD, WARPS) - 1) / join_rows(HD, WARPS));
  const bool many = a.grid >= 4 * (int)grid.x;         // pieces of a row: about the CTAs per (request, KV head, chunk)
  return launch_pdl(many ? cache_attn_join_kernel<T, HD, WARPS, 8> : cache_attn_join_kernel<T, HD, WARPS, 4>, grid, dim3(WARPS * 32), 0, s, a);
}

template <typename T, int HD, int RP>
cudaError_t launch(const CacheAttnArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t s) {
  static std::atomic<int> smem_set[kMaxDevices];
  cudaError_t e = ensure_smem_limit(cache_attn_kernel<T, HD, RP>, a.p.smem, smem_set);
  if (e != cudaSuccess) return e;
  if (RP > 8 && two_per_sm(HD, RP)) {   // the softmax warps would wait for registers that the CTA does not have
    static const int regs = [] {
      cudaFuncAttributes at{};
      return cudaFuncGetAttributes(&at, cache_attn_kernel<T, HD, RP>) == cudaSuccess ? at.numRegs : 0;
    }();
    if (regs < kStartRegs) return cudaErrorInvalidConfiguration;
  }
  e = launch_pdl(cache_attn_kernel<T, HD, RP>, dim3(a.grid), dim3(kThreads), a.p.smem, s, a, kmap, vmap);
  if (e != cudaSuccess) return e;
  return a.p.rc <= join_rows(HD, 4) ? launch_join<T, HD, 4>(a, s) : launch_join<T, HD, 8>(a, s);
}

template <typename T, int HD>
cudaError_t launch_rows(const CacheAttnArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t s) {
  switch (a.p.rp) {
    case 8: return launch<T, HD, 8>(a, kmap, vmap, s);
    case 16: return launch<T, HD, 16>(a, kmap, vmap, s);
    case 24: return launch<T, HD, 24>(a, kmap, vmap, s);
    case 32: return launch<T, HD, 32>(a, kmap, vmap, s);
    case 40: return launch<T, HD, 40>(a, kmap, vmap, s);
    case 48:
      if constexpr (__is_same(T, __nv_bfloat16)) return launch<T, HD, 48>(a, kmap, vmap, s);
      break;
    case 64:
      if constexpr (__is_same(T, __nv_bfloat16)) return launch<T, HD, 64>(a, kmap, vmap, s);
  }
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t launch_hd(const CacheAttnArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t s) {
  switch (a.hd) {
    case 64: return launch_rows<T, 64>(a, kmap, vmap, s);
    case 128: return launch_rows<T, 128>(a, kmap, vmap, s);
    case 256: return launch_rows<T, 256>(a, kmap, vmap, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

CacheAttnPlan plan_cache_attn(int dtype, int hd, int grp, int max_q, int n_req) {
  CacheAttnPlan p{};
  const int terms = dtype == DFLASH_BF16 ? 2 : 3;
  // so many that two score buffers and the output fit tensor memory, and two buffers of queries shared memory
  const int limit = dtype == DFLASH_BF16 ? 64 : 40, rows = grp * max_q;
  p.chunks = (rows + limit - 1) / limit;
  p.rc = (rows + p.chunks - 1) / p.chunks;
  p.rp = p.rc <= 8 ? 8 : p.rc <= 16 ? 16 : p.rc <= 24 ? 24 : p.rc <= 32 ? 32 : p.rc <= 40 ? 40 : p.rc <= 48 ? 48 : 64;   // the kernels there are
  const int cols = 2 * score_columns(p.rp) + panels_of(hd) * weight_columns(p.rp);
  p.tmem_cols = 32;
  while (p.tmem_cols < cols) p.tmem_cols *= 2;
  const size_t fixed = attn_fixed_smem(hd, terms, p.rp, n_req) + 1024;
  constexpr size_t kPerSm = 227 * 1024;
  // two CTAs per SM where registers and tensor memory allow it and each can hold its key and value tiles (one: 72 us
  // against 53 for 32 requests x 5 rows, 36.5 against 30 for 4 x 8)
  const size_t half = kPerSm / 2 - 1024;
  // 32 requests x 5 rows over 512 to 2048 keys: 50.0 us if it counts nothing, 47.1 as 2 tiles, 46.5 as 3, 46.2 as 4; 16 x 9
  // causal rows over 500 to 8192: 70.9, 57.5, 55.7, 55.6, with 256 columns 66.4, 54.9, 53.4, 47.7; one request's 264
  // tiles: 15.5 us up to 3, 17.7 as 4.
  p.setup = hd == 256 ? 4 : 3;
  const size_t stages = hd == 256 || p.rp == 8 ? kMaxStages : 3;
  p.ctas_per_sm = two_per_sm(hd, p.rp) && p.tmem_cols <= 256 && fixed + stages * stage_bytes(hd) <= half ? 2 : 1;
  const size_t room = (p.ctas_per_sm == 2 ? half : kPerSm) - fixed;
  p.stages = (int)std::min<size_t>(stages, room / stage_bytes(hd));
  p.smem = fixed + (size_t)p.stages * stage_bytes(hd);
  return p;
}

cudaError_t launch_cache_attn(int dtype, const CacheAttnArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                              cudaStream_t s) {
  return dtype == DFLASH_BF16 ? launch_hd<__nv_bfloat16>(a, kmap, vmap, s) : launch_hd<__half>(a, kmap, vmap, s);
}

}  // namespace dfl
