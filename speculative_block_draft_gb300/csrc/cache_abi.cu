// C entry points of the paged 8-bit context cache (include/dflash.h): argument checks and the
// host-side handle. The kernels are in cache_append.cu and cache_attn.cu, the block tables in pool.cu.
#include <math.h>

#include <algorithm>
#include <new>

#include "cache.h"
#include "tensor_map.h"

using namespace dfl;

struct dflash_cache {
  dflash_cache_config cfg;
  int device = 0, log_t = 0;
  unsigned* err = nullptr;      // error bits
  int n_sm = 148;
  int4* requests = nullptr;     // [max_requests]
  int2* held_by = nullptr;      // [requests x KV heads x row chunks]
  float2* part_ml = nullptr;    // attention pieces: rows of (reference, sum), then of head_dim floats
  float* part_o = nullptr;
  int64_t part_rows = 0;
  unsigned wait_ns = kWaitNs;
  int stall = 0;                // the next attention call's CacheAttnArgs::stall
  CUtensorMap kmap{}, vmap{};
};

namespace {

bool multiple_of_16(int64_t v) { return v % 16 == 0; }
bool aligned_16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

bool valid(const dflash_cache_config* c) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return false;
  if (c->n_layers < 1 || c->n_layers > 65535 || c->n_blocks < 1 || !block_tokens_ok(c->block_tokens)) return false;
  if ((int64_t)c->n_blocks * c->block_tokens >= (1LL << 31)) return false;
  if (c->n_kv_heads < 1 || c->n_kv_heads > 4096) return false;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return false;
  if (!aligned_16(c->k) || !aligned_16(c->v)) return false;
  if (c->layer_stride < (c->n_layers > 1) || c->block_stride < (c->n_blocks > 1) || c->head_stride < (c->n_kv_heads > 1) ||
      c->token_stride < c->head_dim)
    return false;
  if (!multiple_of_16(c->layer_stride) || !multiple_of_16(c->block_stride) || !multiple_of_16(c->head_stride) ||
      !multiple_of_16(c->token_stride))
    return false;
  // strides are tensor-map strides, below 2^40
  if (c->layer_stride >= (1LL << 40) || c->block_stride >= (1LL << 40) || c->head_stride >= (1LL << 40) ||
      c->token_stride >= (1LL << 40))
    return false;
  if (c->n_q_heads == 0 && c->max_requests == 0 && c->max_q == 0) return true;
  return c->n_q_heads >= 1 && c->n_q_heads % c->n_kv_heads == 0 && c->n_q_heads / c->n_kv_heads <= 4096 && c->max_requests >= 1 &&
         c->max_requests <= DFLASH_CACHE_MAX_REQUESTS && c->max_q >= 1 && c->max_q <= DFLASH_CACHE_MAX_Q;
}

// Rows of attention pieces that a call within the limits can leave: one per query row, padded, of each
// (request, KV head), and the CTAs' own. A chunk of rows is padded by at most 15 (49 rows as 64) and a share of one
// row, and there is one for every 40 rows at most; a CTA's chunk holds at most 64 rows, and an SM two CTAs.
int64_t piece_rows(const dflash_cache_config& f, int n_sm) {
  const int64_t rows = (int64_t)(f.n_q_heads / f.n_kv_heads) * f.max_q;
  return (int64_t)2 * n_sm * 64 + (int64_t)f.max_requests * f.n_kv_heads * (rows + 16 * ((rows + 39) / 40));
}

size_t round_256(size_t v) { return (v + 255) & ~(size_t)255; }

// Workspace: error word | requests | their pieces' CTAs | (m, L) of the pieces | O of the pieces.
size_t carve(dflash_cache* c, uint8_t* base) {
  const dflash_cache_config& f = c->cfg;
  size_t at = 256;
  c->err = reinterpret_cast<unsigned*>(base);
  if (f.max_requests) {
    c->part_rows = piece_rows(f, c->n_sm);
    c->requests = reinterpret_cast<int4*>(base + at);
    at += round_256(16 * (size_t)f.max_requests);
    c->held_by = reinterpret_cast<int2*>(base + at);
    at += round_256(8 * (size_t)f.max_requests * f.n_kv_heads * (((size_t)(f.n_q_heads / f.n_kv_heads) * f.max_q + 39) / 40));
    c->part_ml = reinterpret_cast<float2*>(base + at);
    at += round_256(8 * (size_t)c->part_rows);
    c->part_o = reinterpret_cast<float*>(base + at);
    at += round_256(4 * (size_t)c->part_rows * f.head_dim);
  }
  return at;
}

// Codes as [layer][block][head][token][column]; one copy brings the tokens of a block and head, 128 columns (64
// for head_dim 64) wide, in the swizzle that the MMA reads.
int make_code_map(const dflash_cache_config& f, void* base, CUtensorMap* map) {
  EncodeTiled encode = tensor_map_encoder();
  if (!encode) return DFLASH_ECUDA;
  const cuuint64_t dims[5] = {(cuuint64_t)f.head_dim, (cuuint64_t)f.block_tokens, (cuuint64_t)f.n_kv_heads, (cuuint64_t)f.n_blocks,
                              (cuuint64_t)f.n_layers};
  auto stride = [](int64_t s) { return (cuuint64_t)(s > 0 ? s : 16); };   // 0 only where there is one of it
  const cuuint64_t strides[4] = {stride(f.token_stride), stride(f.head_stride), stride(f.block_stride), stride(f.layer_stride)};
  const cuuint32_t box[5] = {(cuuint32_t)(f.head_dim < 128 ? f.head_dim : 128), (cuuint32_t)f.block_tokens, 1, 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            f.head_dim == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DFLASH_OK : DFLASH_EINVAL;
}

bool on_device(const dflash_cache* c) {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && dev == c->device;
}

// strides of rows of 2-byte or 4-byte elements: whole 16-byte steps
bool rows_ok(const dflash_rows& r, int elem) {
  return r.data && aligned_16(r.data) && r.layer_stride * elem % 16 == 0 && r.row_stride * elem % 16 == 0 &&
         r.head_stride * elem % 16 == 0;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? DFLASH_OK : DFLASH_ECUDA; }

}  // namespace

extern "C" {

size_t dflash_cache_workspace_bytes(const dflash_cache_config* cfg) {
  if (!valid(cfg)) return 0;
  dflash_cache c;
  c.cfg = *cfg;
  int dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&c.n_sm, cudaDevAttrMultiProcessorCount, dev);
  return carve(&c, nullptr);
}

int dflash_cache_create(const dflash_cache_config* cfg, void* workspace, size_t workspace_bytes, void* stream,
                        dflash_cache** out) {
  if (!out) return DFLASH_EINVAL;
  *out = nullptr;
  if (!valid(cfg) || !workspace || (reinterpret_cast<uintptr_t>(workspace) & 255)) return DFLASH_EINVAL;
  if (workspace_bytes < dflash_cache_workspace_bytes(cfg)) return DFLASH_ECAPACITY;
  dflash_cache* c = new (std::nothrow) dflash_cache();
  if (!c) return DFLASH_EINVAL;
  c->cfg = *cfg;
  while ((1 << c->log_t) < cfg->block_tokens) c->log_t++;
  int st = DFLASH_OK;
  if (cudaGetDevice(&c->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&c->n_sm, cudaDevAttrMultiProcessorCount, c->device) != cudaSuccess)
    st = DFLASH_ECUDA;
  if (st == DFLASH_OK) {
    carve(c, static_cast<uint8_t*>(workspace));
    if (cfg->max_requests) {
      st = make_code_map(*cfg, cfg->k, &c->kmap);
      if (st == DFLASH_OK) st = make_code_map(*cfg, cfg->v, &c->vmap);
    }
  }
  if (st == DFLASH_OK && cudaMemsetAsync(c->err, 0, 256, static_cast<cudaStream_t>(stream)) != cudaSuccess) st = DFLASH_ECUDA;
  if (st != DFLASH_OK) {
    delete c;
    return st;
  }
  *out = c;
  return DFLASH_OK;
}

void dflash_cache_destroy(dflash_cache* c) { delete c; }

int dflash_cache_check_errors(dflash_cache* c, void* stream) {
  if (!c) return DFLASH_EINVAL;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return DFLASH_ECUDA;
  unsigned word = 0;
  if (cudaMemcpy(&word, c->err, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return DFLASH_ECUDA;
  if (!word) return DFLASH_OK;
  const unsigned zero = 0;
  if (cudaMemcpy(c->err, &zero, 4, cudaMemcpyHostToDevice) != cudaSuccess) return DFLASH_ECUDA;
  return (word & kErrBounds) ? DFLASH_EBOUNDS : DFLASH_ETIMEOUT;
}

int dflash_cache_set_wait_limit(dflash_cache* c, unsigned limit_us) {
  if (!c) return DFLASH_EINVAL;
  c->wait_ns = limit_us ? std::min(limit_us, 4000000u) * 1000u : kWaitNs;
  return DFLASH_OK;
}

int dflash_cache_debug_stall(dflash_cache* c, int cta) {
  if (!c) return DFLASH_EINVAL;
  c->stall = cta < 0 ? 0 : cta + 1;
  return DFLASH_OK;
}

int dflash_cache_append(dflash_cache* c, int layer, int n_layers, int n_rows, const int32_t* slots,
                        const dflash_rows* k, const dflash_rows* v, int dtype, void* stream) {
  if (!c || !k || !v || n_rows < 0 || layer < 0 || n_layers < 0 || (int64_t)layer + n_layers > c->cfg.n_layers)
    return DFLASH_EINVAL;
  if (dtype != DFLASH_F32 && dtype != DFLASH_BF16 && dtype != DFLASH_F16) return DFLASH_EINVAL;
  if (n_rows == 0 || n_layers == 0) return DFLASH_OK;
  const int elem = dtype == DFLASH_F32 ? 4 : 2;
  if (!slots || !rows_ok(*k, elem) || !rows_ok(*v, elem) || !on_device(c)) return DFLASH_EINVAL;
  const dflash_cache_config& f = c->cfg;
  CacheAppendArgs a{};
  a.codes[0] = static_cast<uint8_t*>(f.k);
  a.codes[1] = static_cast<uint8_t*>(f.v);
  a.scales[0] = f.k_scale;
  a.scales[1] = f.v_scale;
  const dflash_rows* r[2] = {k, v};
  for (int s = 0; s < 2; s++) {
    a.rows[s] = r[s]->data;
    a.row_layer[s] = r[s]->layer_stride;
    a.row_row[s] = r[s]->row_stride;
    a.row_head[s] = r[s]->head_stride;
  }
  a.c_layer = f.layer_stride;
  a.c_block = f.block_stride;
  a.c_head = f.head_stride;
  a.c_token = f.token_stride;
  a.layer0 = layer;
  a.n_layers = n_layers;
  a.n_rows = n_rows;
  a.n_blocks = f.n_blocks;
  a.n_kv = f.n_kv_heads;
  a.hd = f.head_dim;
  a.log_t = c->log_t;
  a.slots = slots;
  a.err = c->err;
  return status_of(launch_cache_append(dtype, a, static_cast<cudaStream_t>(stream)));
}

int dflash_cache_attention(dflash_cache* c, const dflash_attention* p, void* stream) {
  if (!c || !p) return DFLASH_EINVAL;
  const dflash_cache_config& f = c->cfg;
  if (f.max_requests == 0) return DFLASH_EINVAL;
  if (p->layer < 0 || p->layer >= f.n_layers || p->n_requests < 0 || p->n_rows < 0 || p->max_q < 0 || p->window < 0 ||
      (p->causal != 0 && p->causal != 1) || (p->dtype != DFLASH_BF16 && p->dtype != DFLASH_F16) ||
      !(p->scale == p->scale) || isinf(p->scale))
    return DFLASH_EINVAL;
  if (p->n_requests == 0 || p->max_q == 0 || p->n_rows == 0) return DFLASH_OK;
  if (p->n_requests > f.max_requests || p->max_q > f.max_q) return DFLASH_ECAPACITY;
  if (p->table_rows < 1 || p->table_blocks < 1 || !p->lens || !p->table) return DFLASH_EINVAL;
  if (!p->requests && p->n_requests > p->table_rows) return DFLASH_EINVAL;
  if (!p->row_start && (int64_t)p->n_requests * p->max_q > p->n_rows) return DFLASH_EINVAL;
  if (!rows_ok(p->q, 2) || !rows_ok(p->out, 2)) return DFLASH_EINVAL;
  if ((p->k_own.data == nullptr) != (p->v_own.data == nullptr)) return DFLASH_EINVAL;
  if (p->k_own.data && (!rows_ok(p->k_own, 2) || !rows_ok(p->v_own, 2))) return DFLASH_EINVAL;
  if (!on_device(c)) return DFLASH_EINVAL;
  CacheAttnArgs a{};
  const int64_t scales = (int64_t)p->layer * f.n_blocks * f.n_kv_heads;
  a.k_scale = f.k_scale + scales;
  a.v_scale = f.v_scale + scales;
  a.layer = p->layer;
  a.n_blocks = f.n_blocks;
  a.n_kv = f.n_kv_heads;
  a.hd = f.head_dim;
  a.log_t = c->log_t;
  a.grp = f.n_q_heads / f.n_kv_heads;
  a.grp_mul = (unsigned)(((1ull << 32) + a.grp - 1) / a.grp);
  a.n_req = p->n_requests;
  a.n_rows = p->n_rows;
  a.max_q = p->max_q;
  a.table_rows = p->table_rows;
  a.table_blocks = p->table_blocks;
  a.held = (int)std::min<int64_t>((int64_t)p->table_blocks << c->log_t, 0x7fffffff);
  a.causal = p->causal;
  a.window = p->window;
  a.requests = p->requests;
  a.lens = p->lens;
  a.table = p->table;
  a.row_start = p->row_start;
  a.q = p->q.data;
  a.out = const_cast<void*>(p->out.data);
  a.k_own = p->k_own.data;
  a.v_own = p->v_own.data;
  a.q_row = p->q.row_stride;
  a.q_head = p->q.head_stride;
  a.o_row = p->out.row_stride;
  a.o_head = p->out.head_stride;
  a.ko_row = p->k_own.row_stride;
  a.ko_head = p->k_own.head_stride;
  a.vo_row = p->v_own.row_stride;
  a.vo_head = p->v_own.head_stride;
  a.scale_log2 = p->scale * 1.4426950408889634f;
  a.err = c->err;
  a.wait_ns = c->wait_ns;
  a.p = plan_cache_attn(p->dtype, f.head_dim, a.grp, p->max_q, p->n_requests);
  // key tiles are counted in 32 bits: a request has at most as many as its table row names, and one more
  const int64_t pairs = (int64_t)p->n_requests * f.n_kv_heads * a.p.chunks;
  const int64_t tiles = pairs * ((((int64_t)p->table_blocks << c->log_t) + 127) / 128 + 1);
  if (tiles + pairs * a.p.setup >= (1LL << 31)) return DFLASH_EINVAL;
  a.grid = (int)std::min<int64_t>((int64_t)a.p.ctas_per_sm * c->n_sm, tiles);
  if ((a.grid + pairs) * a.p.rp > c->part_rows) return DFLASH_ECAPACITY;
  a.words = c->requests;
  a.held_by = c->held_by;
  a.part_o = c->part_o;
  a.part_ml = c->part_ml;
  a.stall = c->stall;
  c->stall = 0;
  return status_of(launch_cache_attn(p->dtype, a, c->kmap, c->vmap, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
