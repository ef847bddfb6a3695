// santa_paged_tokens.cu -- attention over a paged cache for few query rows per
// KV head: the merge of split tiles, the plan and the launches (the kernel is
// in santa_tokens.cuh).
#include "santa_join.cuh"
#include "santa_tokens.cuh"

namespace santa {

namespace {

// One warp per output row of a split tile, or WPR = 4 where there are more than
// eight splits: their sums under a running maximum, eight requested at a time
// (76 splits a row: 17 us with one warp).  Rows of tiles that were not split are
// written already.  What it looks up of the batch is none of the attention
// kernel's output, and so is read while that still runs; but no thread ends
// before it has waited, or the merge could be over, and the stream's next
// kernel begin, while the attention still writes.
template <typename T, int D, int WPR>
__global__ void __launch_bounds__(128) paged_merge_kernel(PagedArgs a) {
  __shared__ float s_o[WPR][D], s_ml[WPR][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = WPR == 1 ? 0 : warp;
  const long long w = (long long)blockIdx.x * (4 / WPR) + warp / WPR;   // the row
  const long long t = w / a.H;
  const int h = (int)(w - t * a.H);
  int b;
  if (t >= a.total_q || !paged_seq_of(a, t, b)) return wait_for_predecessor();
  const Seq s = paged_seq(a, b, false);
  const int i = (int)(t - s.q0), kvh = h / a.G, g = h % a.G;
  if (i >= s.n) return wait_for_predecessor();
  const int tile = (i * a.G + g) / a.rows, r = (i * a.G + g) % a.rows;
  int i0, i1;
  tile_tokens(a, s.n, tile, i0, i1);
  const int splits = max(1, (tile_keys(a, s, i0, i1, PG_BLK).blk + a.split_blk - 1) / a.split_blk);
  if (splits == 1) return wait_for_predecessor();
  const long long base = (((long long)b * a.tiles + tile) * a.Hkv + kvh) * a.splits;
  constexpr int E = D / 32, U = 8;
  float m = -INFINITY, l = 0.f, o[E] = {};
  bool bad = false;
  wait_for_predecessor();
  for (int k0 = part * U; k0 < splits; k0 += WPR * U) {
    float2 ml[U], y[U][E / 2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + u >= splits) continue;
      const long long at = (base + k0 + u) * a.rows + r;
      ml[u] = *reinterpret_cast<const float2*>(a.part_ml + 2 * at);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) y[u][e] = *reinterpret_cast<const float2*>(a.part_o + at * D + lane * E + 2 * e);
    }
    float mn = m;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k0 + u < splits) mn = fmaxf(mn, ml[u].x);
    const float mu = mn > -INFINITY ? mn : 0.f, f0 = fast_exp2(m - mu);
    m = mn;
    l *= f0;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= f0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + u >= splits) continue;
      bad |= ml[u].y < 0.f;
      const float f = fast_exp2(ml[u].x - mu);
      l = fmaf(ml[u].y, f, l);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        o[2 * e] = fmaf(y[u][e].x, f, o[2 * e]);
        o[2 * e + 1] = fmaf(y[u][e].y, f, o[2 * e + 1]);
      }
    }
  }
  if (WPR > 1) {   // a row's warps: the whole CTA came here
    if (bad) l = -1.f;
    if (lane == 0) {
      s_ml[part][0] = m;
      s_ml[part][1] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[part][lane * E + e] = o[e];
    __syncthreads();
    if (part) return;
    float mn = m;
#pragma unroll
    for (int u = 1; u < WPR; ++u) mn = fmaxf(mn, s_ml[u][0]);
    const float mu = mn > -INFINITY ? mn : 0.f, f0 = fast_exp2(m - mu);
    m = mn;
    l = bad ? 0.f : l * f0;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= f0;
#pragma unroll
    for (int u = 1; u < WPR; ++u) {
      const float f = fast_exp2(s_ml[u][0] - mu);
      bad |= s_ml[u][1] < 0.f;
      l = fmaf(s_ml[u][1], f, l);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(s_o[u][lane * E + e], f, o[e]);
    }
  }
  const bool empty = bad || l == 0.f;
  const float inv = empty ? 0.f : __fdividef(1.f, l);
  const long long at = t * a.H + h;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + at * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) dst[e / 2] = empty ? 0u : Pack<T>::pack(o[e] * inv, o[e + 1] * inv);
  if (a.lse && lane == 0) a.lse[at] = empty ? -INFINITY : log_sum(m, l, a.e4m3 ? TOKENS_BIAS : fp16_bias<T>(TOKENS_BIAS));
}

template <typename T, bool E4M3, int D, int R>
cudaError_t tokens_inst(const PagedArgs& a) {
  auto kern = paged_tokens_kernel<T, E4M3, D, R>;
  constexpr int smem = (int)smem_bytes<E4M3, D, R>();
  static std::atomic<unsigned long long> raised{0};
  const cudaError_t e = raise_smem((const void*)kern, smem, raised);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)((long long)a.B * a.tiles * a.Hkv * a.splits), NT, smem, a.stream>>>(a);
  return cudaGetLastError();
}
template <typename T, bool E4M3>
cudaError_t tokens_shape(const PagedArgs& a) {
  if (a.D == 128) return a.rows == 8 ? tokens_inst<T, E4M3, 128, 8>(a) : tokens_inst<T, E4M3, 128, 16>(a);
  return a.rows == 8 ? tokens_inst<T, E4M3, 64, 8>(a) : tokens_inst<T, E4M3, 64, 16>(a);
}
template <typename T>
cudaError_t tokens_type(const PagedArgs& a) {
  return a.e4m3 ? tokens_shape<T, true>(a) : tokens_shape<T, false>(a);
}

template <typename T>
cudaError_t merge_type(const PagedArgs& a, const cudaLaunchConfig_t& cfg) {
  if (a.D == 128)
    return a.splits > 8 ? cudaLaunchKernelEx(&cfg, paged_merge_kernel<T, 128, 4>, a) : cudaLaunchKernelEx(&cfg, paged_merge_kernel<T, 128, 1>, a);
  return a.splits > 8 ? cudaLaunchKernelEx(&cfg, paged_merge_kernel<T, 64, 4>, a) : cudaLaunchKernelEx(&cfg, paged_merge_kernel<T, 64, 1>, a);
}

}  // namespace

// Splits: enough CTAs for two on every SM.  Sequences differ in length, and a
// CTA's share is the longest's, so long tiles are cut finer, into up to four
// CTAs for every place, while a split keeps 1024 keys.  But not into a few more
// CTAs than places, which would take two rounds: eight sequences of 8191 keys,
// 3 tiles and 2 heads of 64, 28.6 us as 384 CTAs, 20.2 as 288 (with lengths from
// 300 on 17.2 and 20.0); at 1.7 rounds (512, lengths from 300 on, e4m3) 33.4
// us, 41.9 as 256.
void plan_splits(PagedArgs& a, long long pieces, long long places, int blks, int fine_blks) {
  long long want = std::max<long long>(1, places / pieces);
  const long long fine = std::min<long long>(4 * places / pieces, fine_blks / 64);
  if (2 * fine * pieces >= 3 * places) want = std::max(want, fine);
  a.split_blk = (int)std::max<long long>(NW, (blks + want - 1) / want);
  a.splits = (blks + a.split_blk - 1) / a.split_blk;
}
void plan_tokens(PagedArgs& a, int span, int more_blocks, int round) {
  a.rows = a.max_q * a.G <= 8 ? 8 : 16;
  a.tokens = 0;
  a.tiles = (int)(((long long)a.max_q * a.G + a.rows - 1) / a.rows);
  const int blks = (span + PG_BLK - 1) / PG_BLK + more_blocks;
  plan_splits(a, (long long)a.B * a.Hkv * a.tiles, 2ll * a.num_sms, blks, blks + round);
}

size_t plan_paged_tokens(PagedArgs& a) {
  plan_tokens(a, a.window ? (int)std::min<long long>(a.nk, (long long)a.window + a.max_q) : a.nk, a.window ? 1 : 0);
  return a.splits == 1 ? 0 : (size_t)a.B * a.Hkv * a.tiles * a.splits;
}

cudaError_t launch_paged_tokens(const PagedArgs& a) {
  const cudaError_t e = a.dtype == 0 ? tokens_type<bf16_t>(a) : tokens_type<fp16_t>(a);
  if (e != cudaSuccess || a.splits == 1) return e;
  // the merge waits for the kernel's end (programmatic dependent launch: its own start overlaps it)
  cudaLaunchConfig_t cfg = {};
  const int per = a.splits > 8 ? 1 : 4;   // rows per CTA
  cfg.gridDim = dim3((unsigned)((a.total_q * a.H + per - 1) / per));
  cfg.blockDim = dim3(128);
  cfg.stream = a.stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return a.dtype == 0 ? merge_type<bf16_t>(a, cfg) : merge_type<fp16_t>(a, cfg);
}

}  // namespace santa
