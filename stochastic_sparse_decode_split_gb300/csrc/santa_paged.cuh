// santa_paged.cuh -- what the paged-cache kernels share: the batch's
// description, the mask as ranges of keys, and the division of a tile's keys
// into splits.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "santa_common.cuh"

// For what the host computes as the kernels do.
#define SANTA_HD __host__ __device__ __forceinline__

namespace santa {

constexpr int ERR_PAGE = 16;       // a page-table entry outside the pool
constexpr int ERR_CHUNK = 32;      // bad q_offsets / kv_offsets, or more new tokens than keys
constexpr int ERR_POSITION = 64;   // a position past the rotation table

// A v_scale is divided by: one below the smallest that santa_kv_append writes
// (its floor of the magnitudes, 2^-60, by 448) counts as that; a negative one,
// a NaN or an infinity makes its row of values NaN.
constexpr float V_SCALE_LEAST = 8.673617379884035e-19f / 448.f;
__device__ __forceinline__ bool odd_scale(float v) { return !(v >= 0.f && v <= 3.402823466e38f); }

// Probabilities that enter their product in fp16 are taken relative to a
// maximum lowered by this much (base 2).  With the largest at 1, those below
// 2^-14 (the weights of a context of tens of thousands of keys) would be held in
// steps of 2^-24, and those below 2^-25 be lost, however many they are.  At 2^15
// nothing overflows for the kernel for few rows, at 2^7 for chunks, whose
// probabilities grow by 2^8 before the maximum follows; the rounding of one then
// is at most 2^-40 or 2^-32 of the largest.  bf16 has the range without.
constexpr float TOKENS_BIAS = 15.f, CHUNK_BIAS = 7.f;
template <typename M16> __host__ __device__ constexpr float fp16_bias(float bias) { return std::is_same<M16, fp16_t>::value ? bias : 0.f; }
// The natural logarithm of sum l relative to maximum m (base 2), which is `bias` below the true one.
__device__ __forceinline__ float log_sum(float m, float l, float bias) {
  return (m + bias) * 0.6931471805599453f + __logf(l * __int_as_float((127 - (int)bias) << 23));
}

constexpr int PG_BLK = 16;         // keys per block: no block crosses a page (the smallest page is one block)

// Everything the paged kernels need, validated and carved out of the workspace.
struct PagedArgs {
  int dtype, e4m3, D;   // 0 bf16, 1 fp16, 2 fp32 tokens; e4m3 cache or the tokens' type
  int B, H, Hkv, G;
  int page_shift, n_pages, max_pages;
  const int32_t* table;
  const int32_t* kv_lens;
  const int64_t* q_offsets;
  int nk, max_q;
  long long total_q;
  int causal, window;
  float sl2;            // score scale in base-2 units (scale * log2 e)
  const void* q;
  const void* K;
  const void* V;
  const float* ks;
  const float* vs;
  void* out;
  float* lse;
  int wide;             // `out` is 32-byte aligned
  int* err;
  // attention: packed rows (token * G + head of the group) are cut into tiles
  // of `rows` of them (`tokens` whole tokens when the tiles keep tokens
  // together, else 0); tiles per sequence at most.  Few rows: most splits of a
  // tile and key blocks per split; chunks: `splits` CTAs
  int rows, tokens, tiles, splits, split_blk;
  float* part_o;        // [pieces, rows, D] unnormalised sums
  float* part_ml;       // [pieces, rows, 2] maximum (base 2) and sum; a negative sum marks a bad page
  struct ChunkShare* share;   // [splits] chunk attention: the shared items
  int num_sms;
  cudaStream_t stream;
};

// An item of the chunk attention that several CTAs share: its pieces are
// slot `slot` of CTA `first` and slot 0 of the following ones (count 0: none).
struct ChunkShare {
  int b, kvh, tile, first, slot, count;
};

// One sequence: its new tokens' first row and number, its keys.  `ok` false:
// its lengths were refused (the error word says why; n = 0 where its token
// rows are not to be trusted).
struct Seq {
  long long q0;
  int n, kv;
  bool ok;
  int from;   // keys before this one are another pass's (0 but in a pass over what a sequence does not share)
};

SANTA_HD Seq paged_seq(const PagedArgs& a, int b, bool flag) {
  Seq s;
  int e = 0;
  if (a.q_offsets) {
    const long long lo = a.q_offsets[b], hi = a.q_offsets[b + 1];
    const bool fine = lo >= 0 && hi >= lo && hi <= a.total_q && hi - lo <= a.max_q;
    s.q0 = fine ? lo : 0;
    s.n = fine ? (int)(hi - lo) : 0;
    if (!fine) e |= ERR_CHUNK;
  } else {
    s.q0 = (long long)b * a.max_q;
    s.n = a.max_q;
  }
  const int kv = a.kv_lens ? a.kv_lens[b] : a.nk;
  const bool fine = kv >= 0 && kv <= a.nk;
  s.kv = fine ? kv : 0;
  if (!fine) e |= ERR_NK_BOUND;
  s.ok = e == 0;
  s.from = 0;
#ifdef __CUDA_ARCH__
  if (e && flag) flag_error(a.err, e);
#endif
  return s;
}

// The sequence of token row t (false: padding, or offsets that do not hold it).
SANTA_HD bool paged_seq_of(const PagedArgs& a, long long t, int& b) {
  if (!a.q_offsets) {
    b = (int)(t / a.max_q);
    return b < a.B;
  }
  int lo = 0, hi = a.B;   // the last b with q_offsets[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.q_offsets[mid] <= t) lo = mid;
    else hi = mid;
  }
  b = lo;
  return a.q_offsets[b] <= t && t < a.q_offsets[b + 1];
}

// Keys [lo, hi) that the token at position `pos` sees.
SANTA_HD void visible_keys(const PagedArgs& a, int kv, int pos, int& lo, int& hi) {
  hi = a.causal ? min(max(pos + 1, 0), kv) : kv;
  lo = a.window ? min(max(pos - a.window + 1, 0), hi) : 0;
}
// The kernels take the batch's description as a type A, PagedArgs or one made
// from it (santa_join.cuh), and ask for these; so does what the host computes.
SANTA_HD void visible_keys(const PagedArgs& a, const Seq& s, int pos, int& lo, int& hi) { visible_keys(a, s.kv, pos, lo, hi); }
SANTA_HD int item_heads(const PagedArgs& a) { return a.Hkv; }   // items of a tile: one per KV head
SANTA_HD const int32_t* page_row(const PagedArgs& a, int b) { return a.table + (long long)b * a.max_pages; }

// The key blocks of a tile whose first and last token are i0 and i1 (of n):
// blk blocks of `keys` keys from block blk_lo on.
struct TileKeys {
  int blk_lo, blk;
};
template <typename A>
SANTA_HD TileKeys tile_keys(const A& a, const Seq& s, int i0, int i1, int keys) {
  int lo0, hi0, lo1, hi1;
  visible_keys(a, s, s.kv - s.n + i0, lo0, hi0);
  visible_keys(a, s, s.kv - s.n + i1, lo1, hi1);
  TileKeys t;
  t.blk_lo = lo0 / keys;
  t.blk = hi1 > lo0 ? (hi1 + keys - 1) / keys - t.blk_lo : 0;
  return t;
}

// First and last token of tile `tile` (the rows of a tile need not start at a
// token's first head unless the tiles keep tokens together).
SANTA_HD void tile_tokens(const PagedArgs& a, int n, int tile, int& i0, int& i1) {
  if (a.tokens) {
    i0 = tile * a.tokens;
    i1 = min(n, i0 + a.tokens) - 1;
  } else {
    i0 = tile * a.rows / a.G;
    i1 = min(n - 1, (tile * a.rows + a.rows - 1) / a.G);
  }
}

// Raises a kernel's dynamic shared memory limit, once per device (`done`: one bit each).
inline cudaError_t raise_smem(const void* kernel, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

constexpr int PG_CHUNK_KEYS = 128;   // keys per block of the chunk attention

// The two attention kernels: their plan (the number of pieces whose sums go
// through memory) and their launches, merge included.
size_t plan_paged_tokens(PagedArgs& a);                // few rows per KV head (mma.sync)
cudaError_t launch_paged_tokens(const PagedArgs& a);
int plan_paged_chunk(PagedArgs& a);                    // many (tcgen05.mma)
cudaError_t launch_paged_chunk(const PagedArgs& a);

struct AppendArgs {
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  void* q_out;
  const void *q_norm, *k_norm;
  float eps;
  const float* rope;
  long long rope_positions;
  int rotated, interleaved;
  void *K, *V;
  float *ks, *vs;
};
cudaError_t launch_kv_append(const PagedArgs& a, const AppendArgs& p);
cudaError_t launch_kv_read(const PagedArgs& a, const int64_t* kv_offsets, long long rows, void* K_out, void* V_out);

}  // namespace santa
