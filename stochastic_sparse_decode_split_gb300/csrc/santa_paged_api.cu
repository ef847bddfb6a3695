// santa_paged_api.cu -- C ABI of the paged cache: host-side validation (all of
// it before any launch), workspace layout and the launches.
#include <limits.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <atomic>

#include "../../include/santa.h"
#include "santa_launch.h"
#include "santa_paged.cuh"

static_assert(SANTA_CACHE_DEVERR_PAGE == santa::ERR_PAGE && SANTA_CACHE_DEVERR_CHUNK == santa::ERR_CHUNK &&
                  SANTA_CACHE_DEVERR_POSITION == santa::ERR_POSITION,
              "device error bits");

namespace {

constexpr size_t ALIGN = 256, HEADER = 256;   // as in santa_api.cu: the error word opens the workspace

size_t up(size_t x) { return (x + ALIGN - 1) / ALIGN * ALIGN; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Multiprocessor count of the current device (152 where there is none), kept per device.
int sms() {
  static std::atomic<int> kept[64];
  int dev = -1, n = 0;
  if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64 && (n = kept[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (dev < 0 || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    (void)cudaGetLastError();
    return 152;
  }
  if (dev < 64) kept[dev].store(n, std::memory_order_relaxed);
  return n;
}

santa_status_t check(const santa_paged_t* p) {
  if (!p) return SANTA_ERR_INVALID_ARG;
  if (p->batch < 1 || p->batch > 65535 || p->n_q_heads < 1 || p->n_kv_heads < 1) return SANTA_ERR_INVALID_ARG;
  if (p->n_q_heads > 65535 || p->n_q_heads % p->n_kv_heads) return SANTA_ERR_INVALID_ARG;
  if (p->nk < 1 || p->nk > SANTA_MAX_NK || p->max_q < 1 || p->total_q < 1 || p->total_q > SANTA_MAX_TOKENS)
    return SANTA_ERR_INVALID_ARG;
  if (!p->q_offsets && p->total_q != (int64_t)p->batch * p->max_q) return SANTA_ERR_INVALID_ARG;
  if (p->n_pages < 1 || p->max_pages < 1) return SANTA_ERR_INVALID_ARG;
  if (p->page_size < 16 || p->page_size > 256 || (p->page_size & (p->page_size - 1))) return SANTA_ERR_UNSUPPORTED;
  if ((int64_t)p->n_pages * p->page_size > INT32_MAX || (int64_t)p->max_pages * p->page_size < p->nk)
    return SANTA_ERR_INVALID_ARG;
  if (p->dtype < SANTA_BF16 || p->dtype > SANTA_FP32) return SANTA_ERR_UNSUPPORTED;
  if (p->cache_dtype != p->dtype && p->cache_dtype != SANTA_E4M3) return SANTA_ERR_UNSUPPORTED;
  if (p->head_dim != 64 && p->head_dim != 128) return SANTA_ERR_UNSUPPORTED;
  if (p->n_q_heads / p->n_kv_heads > SANTA_MAX_GROUP) return SANTA_ERR_UNSUPPORTED;
  if ((p->causal != 0 && p->causal != 1) || p->window < 0 || (p->window && !p->causal)) return SANTA_ERR_INVALID_ARG;
  if (!(p->scale == p->scale) || isinf(p->scale)) return SANTA_ERR_INVALID_ARG;
  if (p->total_q * p->n_q_heads > INT32_MAX) return SANTA_ERR_UNSUPPORTED;   // a CTA per output row at most
  return SANTA_OK;
}

santa_status_t check_cache(const santa_paged_t* p, const void* K, const void* V, const float* ks, const float* vs,
                           const void* ws, size_t ws_bytes, size_t need) {
  if (!p->page_table || !aligned(p->page_table, 4) || !aligned(p->kv_lens, 4) || !aligned(p->q_offsets, 8))
    return SANTA_ERR_INVALID_ARG;
  if (!K || !V || !aligned(K, 16) || !aligned(V, 16)) return SANTA_ERR_INVALID_ARG;
  if (p->cache_dtype == SANTA_E4M3 ? (!ks || !vs || !aligned(ks, 16) || !aligned(vs, 16)) : (ks || vs))
    return SANTA_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, ALIGN) || ws_bytes < need) return SANTA_ERR_WORKSPACE;
  return SANTA_OK;
}

santa::PagedArgs args(const santa_paged_t* p) {
  santa::PagedArgs a;
  memset(&a, 0, sizeof a);
  a.dtype = p->dtype;
  a.e4m3 = p->cache_dtype == SANTA_E4M3;
  a.D = p->head_dim;
  a.B = p->batch;
  a.H = p->n_q_heads;
  a.Hkv = p->n_kv_heads;
  a.G = p->n_q_heads / p->n_kv_heads;
  while ((1 << a.page_shift) < p->page_size) ++a.page_shift;
  a.n_pages = p->n_pages;
  a.max_pages = p->max_pages;
  a.table = p->page_table;
  a.kv_lens = p->kv_lens;
  a.q_offsets = p->q_offsets;
  a.nk = (int)p->nk;
  a.max_q = (int)std::min<int64_t>(p->max_q, p->total_q);   // as an upper bound it may be above
  a.total_q = p->total_q;
  a.causal = p->causal;
  a.window = p->window < p->nk ? p->window : 0;   // one that no key is outside of is none
  a.sl2 = (float)((p->scale > 0.f ? (double)p->scale : 1.0 / sqrt((double)p->head_dim)) * 1.4426950408889634);
  a.num_sms = sms();
  return a;
}

// Which kernel: up to 16 query rows per sequence and KV head the one for few
// rows; more than that it takes 16 by 16, reading the cache again for each, and
// starts in 6 us where the kernel for chunks (tiles of 128 rows) takes 13 to
// 26.  So it also has the calls whose 16-row tiles meet at most 3 * 2^13 blocks
// of 16 keys in all.  Measured, few rows against chunks: at that border (8
// sequences of 8191 keys, 2 KV heads of 64, 40 rows) 20.2 against 23.3 us, with
// 4096 keys and 96 rows 20.5 against 20.9; at two thirds of it (64 rows) 17.0
// against 19.5, e4m3 19.1 against 24.0, and for heads of 128 (4 sequences of
// 4096 keys, 8 KV heads, 32 rows) 22.1 against 28.9, e4m3 25.1 against 32.4; at
// four thirds (128 rows) 29.4 against 21.9, heads of 128 (one sequence of 16384
// keys, 64 rows) 39 against 31.9.
bool few_rows(const santa::PagedArgs& a) {
  const int64_t rows = (int64_t)a.max_q * a.G, span = a.window ? std::min<int64_t>(a.nk, (int64_t)a.window + a.max_q) : a.nk;
  return rows <= 16 || (rows + 15) / 16 <= 3 * 8192 * 16 / span / ((int64_t)a.B * a.Hkv);
}

// The attention's plan, and its workspace: header, the chunk attention's notes
// of shared items, the pieces' sums.
struct Plan {
  size_t share, part_o, part_ml, total;
};
Plan plan(santa::PagedArgs& a) {
  const bool few = few_rows(a);
  const size_t rows = (few ? santa::plan_paged_tokens(a) : (size_t)santa::plan_paged_chunk(a)) * a.rows;
  Plan p;
  p.share = HEADER;
  p.part_o = p.share + (few ? 0 : up((size_t)a.splits * sizeof(santa::ChunkShare)));
  p.part_ml = p.part_o + up(rows * a.D * sizeof(float));
  p.total = p.part_ml + up(rows * 2 * sizeof(float));
  return p;
}

}  // namespace

extern "C" {

size_t santa_paged_workspace_size(const santa_paged_t* p) {
  if (check(p) != SANTA_OK) return 0;
  santa::PagedArgs a = args(p);
  return plan(a).total;
}

santa_status_t santa_kv_append(const santa_paged_t* p, const santa_append_t* ap, void* K, void* V, float* k_scale,
                               float* v_scale, void* workspace, size_t ws_bytes, santa_stream_t stream) {
  santa_status_t st = check(p);
  if (st != SANTA_OK) return st;
  if (!ap) return SANTA_ERR_INVALID_ARG;
  st = check_cache(p, K, V, k_scale, v_scale, workspace, ws_bytes, HEADER);
  if (st != SANTA_OK) return st;
  const int64_t es = p->dtype == SANTA_FP32 ? 4 : 2, D = p->head_dim;
  auto rows_ok = [&](const void* x, int64_t stride, int64_t heads) {
    return x && aligned(x, 16) && stride >= heads * D && (stride * es) % 16 == 0;
  };
  if (!rows_ok(ap->k, ap->k_stride, p->n_kv_heads) || !rows_ok(ap->v, ap->v_stride, p->n_kv_heads)) return SANTA_ERR_INVALID_ARG;
  if (ap->q) {
    if (!rows_ok(ap->q, ap->q_stride, p->n_q_heads) || !ap->q_out || !aligned(ap->q_out, 16)) return SANTA_ERR_INVALID_ARG;
    if (ap->q_out == ap->q && ap->q_stride != p->n_q_heads * D) return SANTA_ERR_INVALID_ARG;
  } else if (ap->q_out || ap->q_norm) {
    return SANTA_ERR_INVALID_ARG;
  }
  if (!aligned(ap->q_norm, 16) || !aligned(ap->k_norm, 16)) return SANTA_ERR_INVALID_ARG;
  if ((ap->q_norm || ap->k_norm) && !(ap->eps >= 0.f && !isinf(ap->eps))) return SANTA_ERR_INVALID_ARG;
  if (ap->rope) {
    if (!aligned(ap->rope, 16) || ap->rope_positions < 1 || ap->rotated < 16 || ap->rotated > D ||
        (ap->interleaved != 0 && ap->interleaved != 1))
      return SANTA_ERR_INVALID_ARG;
    if (ap->rotated % 16) return SANTA_ERR_UNSUPPORTED;
  } else if (ap->rotated) {
    return SANTA_ERR_INVALID_ARG;
  }
  santa::PagedArgs a = args(p);
  a.err = static_cast<int*>(workspace);
  a.stream = (cudaStream_t)stream;
  santa::AppendArgs x;
  memset(&x, 0, sizeof x);
  x.q = ap->q;
  x.k = ap->k;
  x.v = ap->v;
  x.q_stride = ap->q_stride;
  x.k_stride = ap->k_stride;
  x.v_stride = ap->v_stride;
  x.q_out = ap->q_out;
  x.q_norm = ap->q_norm;
  x.k_norm = ap->k_norm;
  x.eps = ap->eps;
  x.rope = ap->rope;
  x.rope_positions = ap->rope_positions;
  x.rotated = ap->rope ? ap->rotated : 0;
  x.interleaved = ap->rope ? ap->interleaved : 0;
  x.K = K;
  x.V = V;
  x.ks = k_scale;
  x.vs = v_scale;
  return santa::launch_kv_append(a, x) == cudaSuccess ? SANTA_OK : SANTA_ERR_CUDA;
}

santa_status_t santa_paged_attention(const santa_paged_t* p, const void* q, const void* K, const void* V,
                                     const float* k_scale, const float* v_scale, void* out, float* lse,
                                     void* workspace, size_t ws_bytes, santa_stream_t stream) {
  santa_status_t st = check(p);
  if (st != SANTA_OK) return st;
  if (p->dtype == SANTA_FP32) return SANTA_ERR_UNSUPPORTED;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4)) return SANTA_ERR_INVALID_ARG;
  santa::PagedArgs a = args(p);
  const Plan l = plan(a);
  st = check_cache(p, K, V, k_scale, v_scale, workspace, ws_bytes, l.total);
  if (st != SANTA_OK) return st;
  const bool few = few_rows(a);
  if (few && (int64_t)a.B * a.tiles * a.Hkv > INT32_MAX / a.splits) return SANTA_ERR_UNSUPPORTED;   // one CTA per split
  unsigned char* w = static_cast<unsigned char*>(workspace);
  a.q = q;
  a.K = K;
  a.V = V;
  a.ks = k_scale;
  a.vs = v_scale;
  a.out = out;
  a.lse = lse;
  a.wide = aligned(out, 32);
  a.err = reinterpret_cast<int*>(w);
  a.share = reinterpret_cast<santa::ChunkShare*>(w + l.share);
  a.part_o = reinterpret_cast<float*>(w + l.part_o);
  a.part_ml = reinterpret_cast<float*>(w + l.part_ml);
  a.stream = (cudaStream_t)stream;
  return (few ? santa::launch_paged_tokens(a) : santa::launch_paged_chunk(a)) == cudaSuccess ? SANTA_OK : SANTA_ERR_CUDA;
}

santa_status_t santa_kv_read(const santa_paged_t* p, const void* K, const void* V, const float* k_scale,
                             const float* v_scale, const int64_t* kv_offsets, int64_t rows, void* K_out, void* V_out,
                             void* workspace, size_t ws_bytes, santa_stream_t stream) {
  santa_status_t st = check(p);
  if (st != SANTA_OK) return st;
  st = check_cache(p, K, V, k_scale, v_scale, workspace, ws_bytes, HEADER);
  if (st != SANTA_OK) return st;
  if ((rows != 0 && (!K_out || !V_out)) || !aligned(K_out, 16) || !aligned(V_out, 16) || !aligned(kv_offsets, 8))
    return SANTA_ERR_INVALID_ARG;
  if (rows < 0 || (!kv_offsets && rows < p->batch * p->nk)) return SANTA_ERR_INVALID_ARG;
  santa::PagedArgs a = args(p);
  a.K = K;
  a.V = V;
  a.ks = k_scale;
  a.vs = v_scale;
  a.err = static_cast<int*>(workspace);
  a.stream = (cudaStream_t)stream;
  return santa::launch_kv_read(a, kv_offsets, rows, K_out, V_out) == cudaSuccess ? SANTA_OK : SANTA_ERR_CUDA;
}

}  // extern "C"
