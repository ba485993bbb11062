// Block tables and slots of the paged context cache, from the requests' lengths (include/dflash.h,
// dflash_pool_reserve / dflash_pool_truncate). Whole-number work on a few kilobytes: what bounds it
// is the latency of a launch and of two dependent reads (lengths, then free blocks), so each call is
// one launch, and every CTA recomputes the prefix sums over the requests (one request per thread)
// instead of waiting for another CTA's.
//
//   need_i  = blocks(len_i + n_i) - blocks(len_i),  blocks(x) = min(ceil(x / T), table_blocks if ring)
//   sum_i   = need_0 + .. + need_i (requests whose table holds them)
//   granted = holds and (need_i == 0 or sum_i <= free_count)
//   block number g of the call (g counted over granted requests in order) = free_list[free_count - 1 - g]
//   slot(row at position p of request i) = block(p / T) * T + p % T
#include <algorithm>

#include "cache.h"
#include "common.cuh"

namespace dfl {

namespace {

constexpr int kPoolThreads = 1024;                  // one request per thread
static_assert(kPoolThreads == DFLASH_POOL_MAX_REQUESTS, "one request per thread");

struct PoolArgs {
  dflash_pool p;
  int n_req, n_slots, log_t;
  const int32_t* requests;
  const int32_t* n;        // n_new, or new_len
  int32_t *slots, *row_start, *granted;
};

// Inclusive prefix sum of one value per thread over the CTA; total receives the whole sum. Sums stay
// below 2^31: a request brings at most DFLASH_POOL_MAX_NEW = 2^20 rows, and there are 1024 at most.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  __syncthreads();   // an earlier scan's sums have been read
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  int w = warp_sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = warp > 0 ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
  return s + before;
}

__device__ __forceinline__ int blocks_of(long long len, const PoolArgs& a) {
  const long long b = (len + a.p.block_tokens - 1) >> a.log_t;
  return (int)(a.p.ring && b > a.p.table_blocks ? a.p.table_blocks : (b < 0x7fffffff ? b : 0x7fffffff));
}

// The table row of this thread's request; -1 if there is none, it is out of range, or an earlier
// request of the call names the same row.
__device__ __forceinline__ int request_row(const PoolArgs& a, int* rows) {
  const int i = threadIdx.x;
  int r = i < a.n_req ? (a.requests ? a.requests[i] : i) : -1;
  if (r < 0 || r >= a.p.table_rows) r = -1;
  if (a.requests) {
    rows[i] = r;
    __syncthreads();
    if (r >= 0) {
      bool twice = false;
      for (int j = 0; j < i; j++) twice |= rows[j] == r;
      if (twice) r = -1;
    }
  }
  return r;
}

__global__ void __launch_bounds__(kPoolThreads) pool_reserve_kernel(const __grid_constant__ PoolArgs a) {
  __shared__ int sums[32];
  __shared__ int start[kPoolThreads + 1];          // rows before each request
  __shared__ int rows[kPoolThreads], lens[kPoolThreads], had[kPoolThreads], first[kPoolThreads], upto[kPoolThreads];
  __shared__ bool last;
  const int i = threadIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  const int r = request_row(a, rows);
  const int avail = min(max(*a.p.free_count, 0), a.p.n_blocks);
  int len = 0, n = 0, need = 0, before = 0;
  bool holds = false;
  if (r >= 0) {
    len = a.p.lens[r];
    n = a.n[i];
    const long long after = (long long)len + n;
    holds = len >= 0 && n >= 0 && n <= DFLASH_POOL_MAX_NEW && after < 0x7fffffffLL &&
            (a.p.ring || after <= ((long long)a.p.table_blocks << a.log_t));
    if (holds) {
      before = blocks_of(len, a);
      need = blocks_of(after, a) - before;
    }
  }
  int total;
  const int sum = block_scan(need, sums, total);
  const bool ok = holds && (need == 0 || sum <= avail);
  if (!ok) need = n = 0;
  const int taken = block_scan(need, sums, total) - need;
  const int total_blocks = total;
  const int my_end = block_scan(n, sums, total);
  const int total_rows = total;
  rows[i] = r;
  lens[i] = len;
  had[i] = before;
  first[i] = taken;
  upto[i] = len + n;
  start[i] = my_end - n;
  if (i == 0) start[kPoolThreads] = total_rows;
  __syncthreads();
  // every CTA has read the pool's state once all have taken a ticket: the last one writes the new
  // state below (the slots do not depend on it), and puts the ticket back
  if (i == 0) last = gridDim.x == 1 || atom_add_acq_rel_gpu(static_cast<int*>(a.p.scratch), 1) == (int)gridDim.x - 1;
  // Four rows next to one another per thread: mostly of one request and block, so one search and one table entry (1024
  // requests x 512 rows 13.8 us a round trip with the truncation, 16.2 with one). One where a CTA has a thread for each
  // (32 requests x 8 rows 6.7 us, 7.2 with four).
  const int T = a.p.block_tokens, tb = a.p.table_blocks, n_out = max(total_rows, a.n_slots), per = n_out > kPoolThreads ? 4 : 1;
  for (long long row0 = (long long)per * (blockIdx.x * kPoolThreads + i); row0 < n_out; row0 += (long long)per * gridDim.x * kPoolThreads) {
    // the request of the first row: the last one whose rows start at or before it and that has rows
    int lo = 0, hi = kPoolThreads, known = -1, known_of = -1, block = -1;   // block: entry `known` of request `known_of`
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= row0) lo = mid;
      else hi = mid;
    }
#pragma unroll
    for (int u = 0; u < 4; u++) {
      const long long at_row = row0 + u;
      if (u >= per || at_row >= n_out) break;
      const int row = (int)at_row;
      int slot = -1;
      if (row < total_rows) {
        while (start[lo + 1] <= row) lo++;             // ends: the last start is total_rows
        const int pos = lens[lo] + row - start[lo];
        const int idx = pos >> a.log_t, at = a.p.ring ? idx % tb : idx;
        const bool starts = (pos & (T - 1)) == 0 && idx == at && at >= had[lo];
        if (at != known || lo != known_of || starts) {
          int32_t* entry = a.p.table + (size_t)rows[lo] * tb + at;
          if (at < had[lo]) {
            block = *entry;
          } else {
            block = a.p.free_list[avail - 1 - (first[lo] + at - had[lo])];
            if (starts) *entry = block;                // the first row of a new block notes it
          }
          known = at, known_of = lo;
        }
        const bool kept = !a.p.ring || idx + tb > ((upto[lo] - 1) >> a.log_t);
        if (kept && block >= 0 && block < a.p.n_blocks) slot = block * T + (pos & (T - 1));
      }
      if (row < a.n_slots) a.slots[row] = slot;
    }
  }
  __syncthreads();
  if (last) {
    if (i < a.n_req) {
      a.granted[i] = ok ? 1 : 0;
      a.row_start[i + 1] = my_end;
      if (ok) a.p.lens[r] = len + n;
    }
    if (i == 0) {
      a.row_start[0] = 0;
      *a.p.free_count = avail - total_blocks;
      *static_cast<int*>(a.p.scratch) = 0;
    }
  }
}

__global__ void __launch_bounds__(kPoolThreads) pool_truncate_kernel(const __grid_constant__ PoolArgs a) {
  __shared__ int sums[32];
  __shared__ int rows[kPoolThreads], from[kPoolThreads], start[kPoolThreads + 1];
  __shared__ bool last;
  const int i = threadIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  const int r = request_row(a, rows);
  const int count = min(max(*a.p.free_count, 0), a.p.n_blocks);
  int after = 0, gone = 0, keep = -1;
  if (r >= 0) {
    const int len = a.p.lens[r], n = a.n[i];
    if (len > 0 && n >= 0 && n < len) {
      keep = n;
      after = blocks_of(keep, a);
      gone = max(0, min(blocks_of(len, a), a.p.table_blocks) - after);
    }
  }
  int total;
  const int end = block_scan(gone, sums, total);
  __syncthreads();
  rows[i] = r;
  from[i] = after;
  start[i] = end - gone;
  if (i == 0) start[kPoolThreads] = total;
  __syncthreads();
  // as in the reservation, the last CTA to have read the lengths and the count writes the new ones
  if (i == 0) last = gridDim.x == 1 || atom_add_acq_rel_gpu(static_cast<int*>(a.p.scratch), 1) == (int)gridDim.x - 1;
  for (int g = blockIdx.x * kPoolThreads + i; g < total; g += gridDim.x * kPoolThreads) {
    int lo = 0, hi = kPoolThreads;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= g) lo = mid;
      else hi = mid;
    }
    int32_t* entry = a.p.table + (size_t)rows[lo] * a.p.table_blocks + from[lo] + g - start[lo];
    const int to = count + total - 1 - g;
    if (to < a.p.n_blocks) a.p.free_list[to] = *entry;
    *entry = -1;
  }
  __syncthreads();
  if (last) {
    if (keep >= 0) a.p.lens[r] = keep;
    if (i == 0) {
      *a.p.free_count = min(count + total, a.p.n_blocks);
      *static_cast<int*>(a.p.scratch) = 0;
    }
  }
}

__global__ void __launch_bounds__(DFLASH_MAX_BATCH) pool_numbers_kernel(const __grid_constant__ PoolNumbers v, int32_t* d_req, int32_t* d_n) {
  pdl_launch_dependents();
  pdl_wait();
  const int i = threadIdx.x;
  if (i < v.n_req) {
    d_req[i] = v.req[i];
    if (d_n) d_n[i] = v.n[i];
  }
}

__global__ void __launch_bounds__(256) pool_init_kernel(int n_blocks, int32_t* free_list, int32_t* free_count) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < n_blocks) free_list[i] = n_blocks - 1 - i;
  if (i == 0) *free_count = n_blocks;
}

int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) l++;
  return l;
}

bool pool_ok(const dflash_pool* p, int n_req) {
  return p && n_req >= 0 && n_req <= DFLASH_POOL_MAX_REQUESTS && block_tokens_ok(p->block_tokens) && p->n_blocks > 0 &&
         (long long)p->n_blocks * p->block_tokens < (1LL << 31) && p->table_rows > 0 && p->table_blocks > 0 &&
         (p->ring == 0 || p->ring == 1) && p->lens && p->table && p->free_list && p->free_count && p->scratch;
}

}  // namespace

cudaError_t launch_pool_numbers(const PoolNumbers& v, int32_t* d_req, int32_t* d_n, cudaStream_t s) {
  return launch_pdl(pool_numbers_kernel, dim3(1), dim3(DFLASH_MAX_BATCH), 0, s, v, d_req, d_n);
}

cudaError_t launch_pool_init(int n_blocks, int32_t* free_list, int32_t* free_count, cudaStream_t s) {
  pool_init_kernel<<<(n_blocks + 255) / 256, 256, 0, s>>>(n_blocks, free_list, free_count);
  return cudaGetLastError();
}

}  // namespace dfl

using namespace dfl;

extern "C" int dflash_pool_reserve(const dflash_pool* p, int n_requests, const int32_t* requests, const int32_t* n_new,
                                   int32_t* slots, int n_slots, int32_t* row_start, int32_t* granted, void* stream) {
  if (!pool_ok(p, n_requests) || n_slots < 0) return DFLASH_EINVAL;
  if (!requests && n_requests > p->table_rows) return DFLASH_EINVAL;
  if (n_requests == 0 && n_slots == 0) return DFLASH_OK;
  if ((n_requests > 0 && (!n_new || !granted)) || !row_start || (n_slots > 0 && !slots)) return DFLASH_EINVAL;
  PoolArgs a{};
  a.p = *p;
  a.n_req = n_requests;
  a.n_slots = n_slots;
  a.log_t = log2_of(p->block_tokens);
  a.requests = requests;
  a.n = n_new;
  a.slots = slots;
  a.row_start = row_start;
  a.granted = granted;
  // a CTA for every four rows per thread: its prefix sums cost about as much as those
  const int grid = std::min(152, std::max(1, n_slots / (4 * kPoolThreads)));
  return launch_pdl(pool_reserve_kernel, dim3(grid), dim3(kPoolThreads), 0, static_cast<cudaStream_t>(stream), a) ==
                 cudaSuccess
             ? DFLASH_OK
             : DFLASH_ECUDA;
}

extern "C" int dflash_pool_truncate(const dflash_pool* p, int n_requests, const int32_t* requests,
                                    const int32_t* new_len, void* stream) {
  if (!pool_ok(p, n_requests)) return DFLASH_EINVAL;
  if (!requests && n_requests > p->table_rows) return DFLASH_EINVAL;
  if (n_requests == 0) return DFLASH_OK;
  if (!new_len) return DFLASH_EINVAL;
  PoolArgs a{};
  a.p = *p;
  a.n_req = n_requests;
  a.log_t = log2_of(p->block_tokens);
  a.requests = requests;
  a.n = new_len;
  // a CTA for every 4096 table entries that might be released
  const int grid = (int)std::min<int64_t>(32, std::max<int64_t>(1, (int64_t)n_requests * p->table_blocks / (4 * kPoolThreads)));
  return launch_pdl(pool_truncate_kernel, dim3(grid), dim3(kPoolThreads), 0, static_cast<cudaStream_t>(stream), a) ==
                 cudaSuccess
             ? DFLASH_OK
             : DFLASH_ECUDA;
}
