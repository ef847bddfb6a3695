// santa_paged_api.cu -- C ABI of the paged cache: host-side validation (all of
// it before any launch), workspace layout and the launches.
#include <limits.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <atomic>

#include "../../include/santa.h"
#include "santa_join.cuh"
#include "santa_launch.h"
#include "santa_paged.cuh"

static_assert(SANTA_CACHE_DEVERR_PAGE == santa::ERR_PAGE && SANTA_CACHE_DEVERR_CHUNK == santa::ERR_CHUNK &&
                  SANTA_CACHE_DEVERR_POSITION == santa::ERR_POSITION &&
                  SANTA_CACHE_DEVERR_PREFIX == santa::ERR_PREFIX,
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
bool few_rows(const santa::PagedArgs& a, int64_t span, int64_t blocks = 3 * 8192) {
  const int64_t rows = (int64_t)a.max_q * a.G;
  return rows <= 16 || (rows + 15) / 16 <= blocks * 16 / span / ((int64_t)a.B * a.Hkv);
}
int64_t span_of(const santa::PagedArgs& a) { return a.window ? std::min<int64_t>(a.nk, (int64_t)a.window + a.max_q) : a.nk; }
bool few_rows(const santa::PagedArgs& a) { return few_rows(a, span_of(a)); }

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

// Differential heads: the kernel for few rows takes eight rows of both maps at a
// time.  It has the calls of at most two such tiles per sequence (its cache is
// then read at most twice, mostly from the L2), and those whose tiles meet at most
// 9216 blocks of 16 keys.  Measured, few rows against chunks, 32 and 8 heads of
// 128: two tiles (4 tokens) at 8192 keys 19.8 against 25.0 us, e4m3 22.1 against
// 28.2, at 32768 keys 38.7 against 48.1, e4m3 42.9 against 63.2; 4096 blocks (2048
// keys, 16 tokens) 18.1 against 24.5, e4m3 20.3 against 25.0; 8192 (8192 keys, 8
// tokens) 25.0 against 25.6, e4m3 27.8 against 28.6; 16384 (16 tokens) 38.4
// against 31.2, e4m3 41.9 against 33.7; 16 and 2 heads of 64, 16384 blocks (32768
// keys, 8 tokens) 23.7 against 21.4.
//
// A pass over prefixes, whose chunks run beside the other pass, has borders of
// its own.  Measured, few rows against chunks, one group, 1 to 300 keys of their
// own: 28 and 4 heads of 128 over 16 bits, 8192 blocks (8 sequences, 8192 keys)
// 22.3 against 22.2 us, 14336 (16 sequences) 25.1 against 24.4, 28672 (32) 35.2
// against 30.5; 32 and 8 heads, e4m3, 8192 (16, 4096 keys) 22.7 against 22.2,
// 16384 (16, 8192 keys) 31.2 against 26.1.  Differential, 32 and 8 heads of 128,
// 16 bits, 1024 blocks (4 sequences, 2048 keys) 17.0 against 17.6, 2048 (4 and
// 4096) 19.7 against 18.9, (8 and 2048) 20.3 against 17.9, 4096 (8 and 4096) 23.7
// against 19.3; e4m3, 4096 (16 and 2048) 26.9 against 28.3, 8192 (16 and 4096) 33.7
// against 32.6, two tiles (4 and 32768) 45.6 against 63.2; 16 and 2 heads of 64,
// 4096 (16 and 4096) 18.3 against 18.8, 8192 (16 and 8192) 21.3 against 19.9, two
// tiles (2 and 32768) 17.2 against 19.4.
int64_t border(const santa::JoinArgs& a) {
  if (a.phase == 1) return !a.diff ? 12288 : a.e4m3 || a.D == 64 ? 5120 : 1920;
  return a.diff ? 9216 : 3 * 8192;
}
bool few_diff(const santa::JoinArgs& a, int64_t span) {
  const int64_t rows = (int64_t)a.max_q * a.G, any = a.phase == 1 && !a.e4m3 && a.D == 128 ? 8 : 16;
  return rows <= any || (rows + 7) / 8 <= border(a) * 16 / span / ((int64_t)a.B * (a.Hkv / 2));
}

// ---- attention in passes: a shared prefix, differential heads

santa_status_t check_join(const santa_paged_t* p, const santa_prefix_t* x, bool diff) {
  santa_status_t st = check(p);
  if (st != SANTA_OK) return st;
  if (p->dtype == SANTA_FP32) return SANTA_ERR_UNSUPPORTED;
  if (diff && (p->n_kv_heads % 2)) return SANTA_ERR_INVALID_ARG;
  if (!x) return SANTA_OK;
  if (x->n_groups < 1 || x->n_groups > p->batch || x->max_group < 1) return SANTA_ERR_INVALID_ARG;
  if (x->max_prefix < 1 || x->max_own < 1) return SANTA_ERR_INVALID_ARG;
  if (p->window && p->window < p->nk) return SANTA_ERR_UNSUPPORTED;   // what a group sees of its prefix would differ by token
  return SANTA_OK;
}

// A pass's kernel and the sizes of its sums; `span` keys, that may begin inside a block.
void plan_pass(santa::JoinArgs& a, int64_t span, bool inside) {
  if (a.diff) {
    a.chunk = !few_diff(a, span);
    if (a.chunk) a.tokens = santa::CHUNK_ROWS / a.G;
    else santa::plan_diff_tokens(a, (int)span, inside);
  } else {
    a.chunk = !few_rows(a, span, border(a));
    if (a.chunk) a.tokens = 2 * (santa::CHUNK_ROWS / a.G);
    else santa::plan_tokens(a, (int)span, inside, 32);   // sums are joined in any case: finer splits cost little
  }
  a.heads = santa::x_items(a);
  if (a.chunk) {
    a.one_map = a.diff && !a.e4m3 && a.D == 128;
    if (a.diff && (a.e4m3 || a.D == 128)) a.heads *= 2;   // an item for each value head, or (one_map) for each map
    a.rows = (a.one_map ? 1 : 2) * santa::CHUNK_ROWS;
    a.tiles = (a.max_q + a.tokens - 1) / a.tokens;
    const int64_t items = (int64_t)a.B * a.heads * a.tiles, blocks = (span + santa::BKEYS - 1) / santa::BKEYS + inside;
    a.splits = (int)std::min<int64_t>(a.num_sms, items * blocks);
    a.sources = (int)(a.splits / items) + 1;   // of a pass that has the GPU for itself
  } else {
    a.sources = a.splits;
  }
}

// CTAs of a pass of chunks over the prefixes when the pass behind it is one of
// few rows: that one, which HBM bounds, then runs on the other SMs from the
// start on, under the start, the products and the stores of the first.  The
// division is the best of a few by an estimate of both: a block of 256 rows and
// 128 keys is 1.9 us of an SM (e4m3 3.4, differential 2.5; 128 rows of a
// differential map with both value heads 1.2; heads of 64 0.7 of that, one tile of
// rows half, e4m3 three quarters; from prefixes of 65536 and 131072 keys heads of
// 64 come to 0.77 over 16 bits and of differential e4m3 blocks, to 0.98 of 256
// e4m3 rows), and 15 us are start and end; the other pass's
// CTAs take 4 us and their keys (half of what may be) at 45 GB/s per SM; what it
// has not done when the first is over it does on all SMs.  Several prefixes count
// as 0.75 of their bound each (between half of it and all: of their lengths the
// host knows the bound alone), and the first pass keeps at least 9 sixteenths.
// Measured, 64 sequences of 100 to 2000 keys behind 32768, 32 and 8 heads of 128:
// 118 us on all SMs one after the other, 99 with 120, 91 with 90, 92 with 76, 100
// with 60; e4m3 108 on all, 98 with 112, 86 with 96, 92 with 80; 16 behind 8192, 28
// and 4 heads: 27.5 on all, 20.9 with 104, 19.6 with 88, 20.4 with 64; differential,
// 32 behind 16384, e4m3: 64 on all, 52 with 112 or 104, 57 with 88.
int prefix_ctas(const santa::JoinArgs& p, const santa::JoinArgs& own) {
  const double tiles = std::min((double)p.B * p.tiles, (double)p.total_q / p.tokens + 0.5 * p.B);
  const double blocks = tiles * p.heads * p.max_prefix / santa::BKEYS * (p.B > 1 ? 0.75 : 1.0);
  const bool one = !p.diff && p.max_q <= p.tokens / 2;
  const double first = blocks * (p.e4m3 ? (p.diff ? 2.5 : 3.4) : p.one_map ? 1.2 : 1.9) * (p.D == 64 ? 0.7 : 1.0) * (!one ? 1.0 : p.e4m3 ? 0.75 : 0.5);
  constexpr int per_sm = 2;   // CTAs of the other pass
  const double ctas = (double)own.B * own.tiles * own.heads * own.splits, row = p.e4m3 ? p.D + 4.0 : 2.0 * p.D;
  const double each = 4 + 0.5 * own.max_own / own.splits * 2 * row * (p.diff ? 2 : 1) * per_sm / 45e3;
  const int items = (int)std::min<int64_t>((int64_t)p.tiles * p.heads, p.num_sms);
  int best = p.splits;
  double least = 1e30;
  for (int sixteenths = 9; sixteenths <= 16; ++sixteenths) {   // more only where it gives more
    int x = std::min(p.splits, p.num_sms * sixteenths / 16);
    if (p.B == 1 && items < x) x = std::min(p.splits, (x + items - 1) / items * items);   // as many for each item
    const int rest = p.num_sms - x;
    const double t1 = 15 + first / x, t2 = rest ? each * std::max(1.0, ctas / (rest * per_sm)) : 1e9;
    const double all = each * std::max(1.0, ctas / (p.num_sms * per_sm));
    const double t = t2 <= t1 ? t1 : std::min(t2, t1 + std::max(each, all * (rest ? 1 - t1 / t2 : 1)));
    if (t < 0.97 * least) {
      least = t;
      best = x;
    }
  }
  return best;
}

struct JoinPlan {
  santa::JoinArgs prefix, own;
  size_t total;
};

// Lays one pass's sums out from byte `at` of the workspace on.
void lay_out(santa::JoinArgs& a, unsigned char* ws, size_t& at) {
  const size_t wide = a.diff ? 2 * a.D : a.D, all = (size_t)a.total_q * a.H;
  auto take = [&](size_t bytes) {
    unsigned char* const p = ws + at;
    at += up(bytes);
    return p;
  };
  if (a.chunk) {
    const size_t rows = (size_t)a.splits * 2 * a.rows, cols = a.one_map ? wide : wide * santa::x_items(a) / a.heads;
    a.part_o = reinterpret_cast<float*>(take(rows * cols * sizeof(float)));
    a.part_ml = reinterpret_cast<float*>(take(rows * 2 * sizeof(float)));
    a.row_o = reinterpret_cast<float*>(take(all * wide * sizeof(float)));
    a.row_ml = reinterpret_cast<float*>(take(all * 2 * (wide / cols) * sizeof(float)));
    a.notes = reinterpret_cast<santa::PieceNote*>(take((size_t)a.total_q * a.heads * sizeof(santa::PieceNote)));
  } else {
    const size_t rows = (size_t)a.B * a.tiles * a.heads * a.splits * a.rows * (a.diff ? 2 : 1);
    a.part_o = reinterpret_cast<float*>(take(rows * wide * sizeof(float)));
    a.part_ml = reinterpret_cast<float*>(take(rows * 2 * (a.diff ? 2 : 1) * sizeof(float)));
  }
}

JoinPlan join_plan(const santa_paged_t* p, const santa_prefix_t* x, bool diff, void* ws) {
  JoinPlan l;
  memset(&l, 0, sizeof l);
  static_cast<santa::PagedArgs&>(l.own) = args(p);
  l.own.diff = diff;
  l.own.seqs = l.own.B;
  l.own.seq_q = l.own.max_q;
  l.prefix = l.own;
  if (x) {
    l.own.phase = 2;
    l.own.n_groups = x->n_groups;
    l.own.group_q = (int)std::min<int64_t>((int64_t)x->max_group * l.own.max_q, p->total_q);
    l.own.group_offsets = x->group_offsets;
    l.own.prefix_lens = x->prefix_lens;
    l.own.max_prefix = (int)std::min(x->max_prefix, p->nk);   // upper bounds may be above what there can be
    l.own.max_own = (int)std::min(x->max_own, p->nk);
    l.prefix = l.own;
    l.prefix.phase = 1;
    l.prefix.B = x->n_groups;
    l.prefix.max_q = l.own.group_q;
    plan_pass(l.prefix, l.own.max_prefix, false);
    plan_pass(l.own, l.own.max_own, true);
    if (l.prefix.chunk && !l.own.chunk) l.prefix.splits = prefix_ctas(l.prefix, l.own);
  } else {
    plan_pass(l.own, span_of(l.own), l.own.window != 0);
  }
  size_t at = HEADER;
  unsigned char* const w = static_cast<unsigned char*>(ws);
  if (x) lay_out(l.prefix, w, at);
  lay_out(l.own, w, at);
  l.total = at;
  return l;
}

// Whether the grid of a pass has a number, of two of them as well.
bool fits(const santa::JoinArgs& a) { return a.chunk || (int64_t)a.B * a.tiles * a.heads <= INT32_MAX / 2 / a.splits; }

santa_status_t join(const santa_paged_t* p, const santa_prefix_t* x, const santa_diff_t* d, const void* q, const void* K,
                    const void* V, const float* ks, const float* vs, void* out, float* lse, void* ws, size_t ws_bytes,
                    santa_stream_t stream) {
  santa_status_t st = check_join(p, x, d != nullptr);
  if (st != SANTA_OK) return st;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4)) return SANTA_ERR_INVALID_ARG;
  if (x && (!x->prefix_lens || !aligned(x->prefix_lens, 4) || !aligned(x->group_offsets, 4) || (!x->group_offsets && x->n_groups != 1)))
    return SANTA_ERR_INVALID_ARG;
  if (d && (!d->lambda || !aligned(d->lambda, 4) || !aligned(d->norm, 16) || d->lambda_stride < 0 ||
            (d->lambda_stride && d->lambda_stride < p->n_q_heads / 2) || (d->norm && !(d->eps >= 0.f && !isinf(d->eps))) ||
            !(d->gain == d->gain) || isinf(d->gain)))
    return SANTA_ERR_INVALID_ARG;
  JoinPlan l = join_plan(p, x, d != nullptr, ws);
  st = check_cache(p, K, V, ks, vs, ws, ws_bytes, l.total);
  if (st != SANTA_OK) return st;
  if ((x && !fits(l.prefix)) || !fits(l.own)) return SANTA_ERR_UNSUPPORTED;   // their sum has a number, too
  for (santa::JoinArgs* a : {&l.prefix, &l.own}) {
    a->q = q;
    a->K = K;
    a->V = V;
    a->ks = ks;
    a->vs = vs;
    a->out = out;
    a->lse = lse;
    a->err = static_cast<int*>(ws);
    a->stream = (cudaStream_t)stream;
    if (d) {
      a->lambda = d->lambda;
      a->lambda_stride = d->lambda_stride;
      a->norm = d->norm;
      a->eps = d->eps;
      a->gain = d->gain;
    }
  }
  const bool both = x && !l.prefix.chunk && !l.own.chunk;   // in one launch
  auto launch = [&](const santa::JoinArgs& a, bool behind) {
    const santa::JoinArgs* const first = both ? &l.prefix : nullptr;
    if (a.diff && a.chunk) return a.one_map ? santa::launch_diff_wide(a, behind) : santa::launch_diff_chunk(a, behind);
    if (a.diff) return santa::launch_diff_tokens(first, a, behind);
    return a.chunk ? santa::launch_join_chunk(a, behind) : santa::launch_join_tokens(first, a, behind);
  };
  cudaError_t e = x && !both ? launch(l.prefix, false) : cudaSuccess;
  if (e == cudaSuccess) e = launch(l.own, x && !both);
  if (e == cudaSuccess) e = santa::launch_join(l.prefix, l.own);
  return e == cudaSuccess ? SANTA_OK : SANTA_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t santa_shared_workspace_size(const santa_paged_t* p, const santa_prefix_t* x) {
  if (!x || check_join(p, x, false) != SANTA_OK) return 0;
  return join_plan(p, x, false, nullptr).total;
}

size_t santa_diff_workspace_size(const santa_paged_t* p, const santa_prefix_t* x) {
  if (check_join(p, x, true) != SANTA_OK) return 0;
  return join_plan(p, x, true, nullptr).total;
}

santa_status_t santa_shared_attention(const santa_paged_t* p, const santa_prefix_t* x, const void* q, const void* K, const void* V,
                                      const float* k_scale, const float* v_scale, void* out, float* lse, void* workspace,
                                      size_t ws_bytes, santa_stream_t stream) {
  if (!x) return SANTA_ERR_INVALID_ARG;
  return join(p, x, nullptr, q, K, V, k_scale, v_scale, out, lse, workspace, ws_bytes, stream);
}

santa_status_t santa_diff_attention(const santa_paged_t* p, const santa_prefix_t* x, const santa_diff_t* d, const void* q,
                                    const void* K, const void* V, const float* k_scale, const float* v_scale, void* out, float* lse,
                                    void* workspace, size_t ws_bytes, santa_stream_t stream) {
  if (!d) return SANTA_ERR_INVALID_ARG;
  return join(p, x, d, q, K, V, k_scale, v_scale, out, lse, workspace, ws_bytes, stream);
}

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
