// santa_paged_chunk.cu -- attention of a chunk of new tokens over a paged cache:
// the merge of the items that CTAs shared, the plan and the launches (the kernel
// is in santa_chunk.cuh).
#include "santa_chunk.cuh"

namespace santa {

namespace {

// The items that CTAs shared: CTA c of the attention left a note of the one
// whose last piece it had.  Two rows per warp, 32 per CTA; one pass over the
// pieces under a running maximum, four of each row requested at a time.
template <typename T, int D>
__global__ void __launch_bounds__(512, 2) chunk_merge_kernel(PagedArgs a) {
  const int lane = threadIdx.x & 31, row0 = blockIdx.y * 32 + (threadIdx.x >> 5) * 2;
  const int per = TROWS / a.G, sub = row0 / TROWS;
  wait_for_predecessor();
  const ChunkShare r = a.share[blockIdx.x];
  if (r.count == 0 || row0 % TROWS >= per * a.G) return;
  const Seq s = paged_seq(a, r.b, false);
  const int tok0 = r.tile * a.tokens + sub * per;
  if (tok0 + row0 % TROWS / a.G >= s.n) return;
  constexpr int E = D / 32, U = 4, R = 2;
  float m[R], l[R], o[R][E];
  bool bad[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
    bad[i] = false;
#pragma unroll
    for (int e = 0; e < E; ++e) o[i][e] = 0.f;
  }
  for (int k0 = 0; k0 < r.count; k0 += U) {
    float2 ml[U][R], y[U][R][E / 2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + u >= r.count) continue;
      const long long at = ((long long)(r.first + k0 + u) * 2 + (k0 + u == 0 ? r.slot : 0)) * a.rows + row0;
      // a row past the tile's last one reads what its lane computed for nothing, or nobody wrote: it is not stored
#pragma unroll
      for (int i = 0; i < R; ++i) {
        ml[u][i] = *reinterpret_cast<const float2*>(a.part_ml + 2 * (at + i));
#pragma unroll
        for (int e = 0; e < E / 2; ++e) y[u][i][e] = *reinterpret_cast<const float2*>(a.part_o + (at + i) * D + lane * E + 2 * e);
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float mn = m[i];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (k0 + u < r.count) mn = fmaxf(mn, ml[u][i].x);
      const float mu = mn > -INFINITY ? mn : 0.f, f0 = fast_exp2(m[i] - mu);
      m[i] = mn;
      l[i] *= f0;
#pragma unroll
      for (int e = 0; e < E; ++e) o[i][e] *= f0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k0 + u >= r.count) continue;
        bad[i] |= ml[u][i].y < 0.f;
        const float f = fast_exp2(ml[u][i].x - mu);
        l[i] = fmaf(ml[u][i].y, f, l[i]);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          o[i][2 * e] = fmaf(y[u][i][e].x, f, o[i][2 * e]);
          o[i][2 * e + 1] = fmaf(y[u][i][e].y, f, o[i][2 * e + 1]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int in_tile = row0 % TROWS + i, tok = tok0 + in_tile / a.G;
    if (in_tile >= per * a.G || tok >= s.n) continue;
    const bool empty = bad[i] || l[i] == 0.f;
    const float inv = empty ? 0.f : __fdividef(1.f, l[i]);
    const long long at = (s.q0 + tok) * a.H + (long long)r.kvh * a.G + in_tile % a.G;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + at * D + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = empty ? 0u : pack2h<T>(o[i][e] * inv, o[i][e + 1] * inv);
    if (a.lse && lane == 0) a.lse[at] = empty ? -INFINITY : log_sum(m[i], l[i], a.e4m3 ? CHUNK_BIAS : fp16_bias<T>(CHUNK_BIAS));
  }
}

template <typename T, bool E4M3, int D>
cudaError_t chunk_inst(const PagedArgs& a) {
  using Gm = ChunkGeom<E4M3, D>;
  auto kern = paged_chunk_kernel<T, E4M3, D, PagedArgs, false>;
  static std::atomic<unsigned long long> raised{0};
  const cudaError_t e = raise_smem((const void*)kern, (int)Gm::SMEM, raised);
  if (e != cudaSuccess) return e;
  CUtensorMap tq, tk, tv;
  memset(&tq, 0, sizeof tq);
  memset(&tk, 0, sizeof tk);
  memset(&tv, 0, sizeof tv);
  if (!encode(&tq, a.q, 2, D, a.H, a.total_q, 64, a.G, TROWS / a.G) || !encode_cache<E4M3, D>(&tk, a, a.K) ||
      !encode_cache<E4M3, D>(&tv, a, a.V))
    return cudaErrorInvalidValue;
  kern<<<(unsigned)a.splits, Gm::THREADS, Gm::SMEM, a.stream>>>(tq, tk, tv, a);
  const cudaError_t launched = cudaGetLastError();
  if (launched != cudaSuccess || !chunk_may_share(a)) return launched;
  // the merge waits for the kernel's end (programmatic dependent launch: its own start overlaps it)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.splits, a.rows / 32);
  cfg.blockDim = dim3(512);
  cfg.stream = a.stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_merge_kernel<T, D>, a);
}
template <typename T>
cudaError_t chunk_type(const PagedArgs& a) {
  if (a.D == 128) return a.e4m3 ? chunk_inst<T, true, 128>(a) : chunk_inst<T, false, 128>(a);
  return a.e4m3 ? chunk_inst<T, true, 64>(a) : chunk_inst<T, false, 64>(a);
}

}  // namespace

// One CTA per SM at most (`splits` of them), and two pieces' sums of each: at
// most its first and its last item are shared.  Returns their number.
int plan_paged_chunk(PagedArgs& a) {
  a.rows = 2 * TROWS;
  a.tokens = 2 * (TROWS / a.G);
  a.tiles = (a.max_q + a.tokens - 1) / a.tokens;
  a.splits = (int)std::min<long long>(a.num_sms, (long long)a.B * a.Hkv * a.tiles * chunk_blocks(a));
  return chunk_may_share(a) ? 2 * a.splits : 0;
}

cudaError_t launch_paged_chunk(const PagedArgs& a) {
  return a.dtype == 0 ? chunk_type<bf16_t>(a) : chunk_type<fp16_t>(a);
}

}  // namespace santa
