// santa_join.cu -- the end of an attention in passes: every row's sums, of what
// its group shares and of what its sequence has of its own, become one result;
// for differential heads the difference of two, and its norm.
//
// Bound by the reads of the pieces (D + 2 floats each, which the passes have
// just left in the L2) and, for single tokens, by the chain of look-ups before
// them; those of the batch are made while the last pass still runs.
#include <type_traits>

#include "santa_join.cuh"

namespace santa {

namespace {

template <typename T> __device__ __forceinline__ uint32_t pack16(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack16<bf16_t>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <> __device__ __forceinline__ uint32_t pack16<fp16_t>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <typename T> __device__ __forceinline__ float2 unpack16(uint32_t r);
template <> __device__ __forceinline__ float2 unpack16<bf16_t>(uint32_t r) {
  return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 unpack16<fp16_t>(uint32_t r) {
  __half2 h;
  memcpy(&h, &r, 4);
  return __half22float2(h);
}

// Where the sums of one row in one pass are: `count` pieces; piece k at row
// at0 (k = 0) or at1 + k step of arrays whose rows have `width` columns.
struct Source {
  const float *o, *ml;
  long long at0, at1, step;
  int count, width, column, parts, part;
};

// Of row `i` of the pass's sequence vb, whose tokens are s: query head `head`
// (its KV item `item`, g-th of the group, differential map e), columns from
// `column` on.
template <int D, bool DIFF>
__device__ __forceinline__ Source find(const JoinArgs& a, int vb, const Seq& s, int i, int unit, int e, int column, long long row_at) {
  Source r;
  const int x = unit / a.G, g = unit - x * a.G;   // KV head (differential: pair of them), place in its group
  constexpr int W = DIFF ? 2 * D : D;
  const int dv = a.chunk ? W * x_items(a) / a.heads : W, parts = DIFF && a.e4m3 ? 2 : W / dv;
  r.parts = parts;
  r.part = parts == 2 ? column / D : 0;
  if (!a.chunk) {
    const int rows = a.rows * (DIFF ? 2 : 1), pr = i * a.G + g, tile = pr / a.rows;
    int i0, i1;
    tile_tokens(a, s.n, tile, i0, i1);
    r.count = max(1, (tile_keys(a, s, i0, i1, PG_BLK).blk + a.split_blk - 1) / a.split_blk);
    r.o = a.part_o;
    r.ml = a.part_ml;
    r.width = W;
    r.column = column;
    r.at0 = r.at1 = ((((long long)vb * a.tiles + tile) * x_items(a) + x) * a.splits) * rows + e * a.rows + pr % a.rows;
    r.step = rows;
    return r;
  }
  const int per = CHUNK_ROWS / a.G, tile = i / a.tokens, in = i - tile * a.tokens;
  const int row = (DIFF ? e : in / per) * CHUNK_ROWS + in % per * a.G + g;
  const int item = W == dv ? x : 2 * x + r.part;
  const PieceNote n = a.notes[((long long)vb * a.tiles + tile) * a.heads + item];
  if (n.count == 0) {
    r.count = 1;
    r.o = a.row_o;
    r.ml = a.row_ml;
    r.width = W;
    r.column = column;
    r.at0 = row_at;
    r.at1 = r.step = 0;
    return r;
  }
  r.count = n.count;
  r.o = a.part_o;
  r.ml = a.part_ml;
  r.width = dv;
  r.column = column % dv;
  r.parts = 1;
  r.part = 0;
  r.at0 = ((long long)n.first * 2 + n.slot) * a.rows + row;
  r.at1 = (long long)n.first * 2 * a.rows + row;
  r.step = 2ll * a.rows;
  return r;
}

// One warp per output row, or WPR = 4 where a row has many pieces: a running
// maximum, U pieces requested at a time.
template <typename T, int D, bool DIFF, int WPR>
__global__ void __launch_bounds__(128) join_kernel(JoinArgs p, JoinArgs a) {
  constexpr int W = DIFF ? 2 * D : D, E = W / 32, NE = DIFF ? 2 : 1, U = DIFF ? 4 : 8;
  __shared__ float s_o[WPR][NE][W], s_ml[WPR][NE][32][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = WPR == 1 ? 0 : warp;
  const int units = DIFF ? a.H / 2 : a.H, column = lane * E;
  const long long w = (long long)blockIdx.x * (4 / WPR) + warp / WPR, t = w / units;
  const int unit = (int)(w - t * units);
  int b;
  if (t >= a.total_q || !paged_seq_of(a, t, b)) return wait_for_predecessor();
  const Seq s = paged_seq(a, b, false);
  const int i = (int)(t - s.q0);
  if (i >= s.n) return wait_for_predecessor();
  Seq sp = {};
  int g = 0;
  if (p.n_groups) {
    g = group_of(a, b);
    sp = paged_seq(p, g, false);
  }
  const bool prefix = s.ok && sp.kv > 0;
  wait_for_predecessor();
  float m[NE], l[NE], o[NE][E];
  bool bad = false;
#pragma unroll
  for (int e = 0; e < NE; ++e) {
    m[e] = -INFINITY;
    l[e] = 0.f;
#pragma unroll
    for (int c = 0; c < E; ++c) o[e][c] = 0.f;
    if (!s.ok) continue;
    const long long row_at = t * a.H + (DIFF ? 2 * unit + e : unit);
    const Source own = find<D, DIFF>(a, b, s, i, unit, e, column, row_at);
    Source pre = own;
    pre.count = 0;
    if (prefix) pre = find<D, DIFF>(p, g, sp, (int)(t - sp.q0), unit, e, column, row_at);
    const int count = own.count + pre.count;
#pragma unroll 1
    for (int k0 = part * U; k0 < count; k0 += WPR * U) {
      float2 ml[U];
      float y[U][E];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u;
        if (k >= count) continue;
        const bool first = k < pre.count;
        const Source& r = first ? pre : own;
        const int kk = first ? k : k - pre.count;
        const long long at = kk == 0 ? r.at0 : r.at1 + kk * r.step;
        ml[u] = *reinterpret_cast<const float2*>(r.ml + (at * r.parts + r.part) * 2);
        const float* const src = r.o + at * r.width + r.column;
#pragma unroll
        for (int c = 0; c < E; c += 2) *reinterpret_cast<float2*>(&y[u][c]) = *reinterpret_cast<const float2*>(src + c);
      }
      float mn = m[e];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (k0 + u < count) mn = fmaxf(mn, ml[u].x);
      const float mu = mn > -INFINITY ? mn : 0.f, f0 = fast_exp2(m[e] - mu);
      m[e] = mn;
      l[e] *= f0;
#pragma unroll
      for (int c = 0; c < E; ++c) o[e][c] *= f0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k0 + u >= count) continue;
        bad |= ml[u].y < 0.f;
        const float f = fast_exp2(ml[u].x - mu);
        l[e] = fmaf(ml[u].y, f, l[e]);
#pragma unroll
        for (int c = 0; c < E; ++c) o[e][c] = fmaf(y[u][c], f, o[e][c]);
      }
    }
  }
  if (WPR > 1) {   // a row's warps: the whole CTA came here
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      s_ml[part][e][lane][0] = m[e];
      s_ml[part][e][lane][1] = bad ? -1.f : l[e];
#pragma unroll
      for (int c = 0; c < E; ++c) s_o[part][e][column + c] = o[e][c];
    }
    __syncthreads();
    if (part) return;
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      float mn = m[e];
#pragma unroll
      for (int u = 1; u < WPR; ++u) mn = fmaxf(mn, s_ml[u][e][lane][0]);
      const float mu = mn > -INFINITY ? mn : 0.f, f0 = fast_exp2(m[e] - mu);
      m[e] = mn;
      l[e] *= f0;
#pragma unroll
      for (int c = 0; c < E; ++c) o[e][c] *= f0;
#pragma unroll
      for (int u = 1; u < WPR; ++u) {
        const float f = fast_exp2(s_ml[u][e][lane][0] - mu), lu = s_ml[u][e][lane][1];
        bad |= lu < 0.f;
        l[e] = fmaf(lu, f, l[e]);
#pragma unroll
        for (int c = 0; c < E; ++c) o[e][c] = fmaf(s_o[u][e][column + c], f, o[e][c]);
      }
    }
  }
  bad = __any_sync(FULL, bad) || !s.ok;
  float y[E];
  bool empty = false;
#pragma unroll
  for (int e = 0; e < NE; ++e) {
    const bool none = bad || l[e] == 0.f;
    empty |= none;
    if (a.lse && lane == 0) {
      // the sum's exponent goes to the maximum's side, so that the logarithm's argument is near 1
      const int ex = (int)(__float_as_uint(l[e]) >> 23) - 127;
      const float near1 = __uint_as_float((__float_as_uint(l[e]) & 0x7fffffu) | 0x3f800000u);
      const float v = l[e] <= 3.402823466e38f ? (m[e] + (float)ex) * 0.6931471805599453f + __logf(near1) : l[e];
      a.lse[t * a.H + (DIFF ? 2 * unit + e : unit)] = none ? -INFINITY : v;
    }
    float f = none ? 0.f : __fdividef(1.f, l[e]);
    if (DIFF && e == 1) f *= -a.lambda[t * a.lambda_stride + unit];
#pragma unroll
    for (int c = 0; c < E; ++c) y[c] = e == 0 ? o[e][c] * f : fmaf(o[e][c], f, y[c]);
  }
  if (DIFF) {
    float f = a.gain;
    if (a.norm) {
      float sq = 0.f;
#pragma unroll
      for (int c = 0; c < E; ++c) sq = fmaf(y[c], y[c], sq);
#pragma unroll
      for (int x = 16; x; x >>= 1) sq += __shfl_xor_sync(FULL, sq, x);
      f *= 1.f / sqrtf(sq * (1.f / W) + a.eps);
    }
#pragma unroll
    for (int c = 0; c < E; c += 2) {
      float2 wt = make_float2(1.f, 1.f);
      if (a.norm) wt = unpack16<T>(reinterpret_cast<const uint32_t*>(a.norm)[(column + c) / 2]);
      y[c] *= f * wt.x;
      y[c + 1] *= f * wt.y;
    }
  }
  uint32_t* const dst = reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + (t * units + unit) * W + column);
#pragma unroll
  for (int c = 0; c < E; c += 2) dst[c / 2] = empty ? 0u : pack16<T>(y[c], y[c + 1]);
}

template <typename T, int D, bool DIFF>
cudaError_t rows(const JoinArgs& p, const JoinArgs& a) {
  const long long n = a.total_q * (DIFF ? a.H / 2 : a.H);
  if ((p.n_groups ? p.sources : 0) + a.sources > 8)
    return launch_pass(join_kernel<T, D, DIFF, 4>, (unsigned)n, 128, 0, a.stream, true, p, a);
  return launch_pass(join_kernel<T, D, DIFF, 1>, (unsigned)((n + 3) / 4), 128, 0, a.stream, true, p, a);
}
template <typename T>
cudaError_t shape(const JoinArgs& p, const JoinArgs& a) {
  if (a.D == 128) return a.diff ? rows<T, 128, true>(p, a) : rows<T, 128, false>(p, a);
  return a.diff ? rows<T, 64, true>(p, a) : rows<T, 64, false>(p, a);
}

}  // namespace

cudaError_t launch_join(const JoinArgs& prefixes, const JoinArgs& own) {
  return own.dtype == 0 ? shape<bf16_t>(prefixes, own) : shape<fp16_t>(prefixes, own);
}

}  // namespace santa
