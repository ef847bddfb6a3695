// santa_join.cu -- the end of an attention in passes: every row's sums, of what
// its group shares and of what its sequence has of its own, become one result;
// for differential heads the difference of two, and its norm.
//
// Bound by the reads of the pieces (D + 2 floats each, which the passes have
// just left in the L2) and, for single tokens, by the chain of look-ups before
// them; those of the batch are made while the last pass still runs.
#include <algorithm>
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

// A set of rows is up to R query heads of one token and KV head (differential:
// one pair of heads, whose two maps follow each other).  In a pass of few rows
// every lane looks for the row of head lane % R: its first piece and their
// number; in one of chunks for the place of the set's note and the first row.
struct Place {
  unsigned at;
  int count;
};
template <int D, bool DIFF, int R>
__device__ __forceinline__ Place locate(const JoinArgs& a, int vb, const Seq& s, int i, int x, int g0, int lane) {
  Place l;
  if (!a.chunk) {
    const int shift = a.rows == 16 ? 4 : a.rows == 8 ? 3 : 2, pr = i * a.G + g0 + lane % R, tile = pr >> shift;
    const unsigned i0 = (unsigned)(tile << shift) / (unsigned)a.G, i1 = (unsigned)((tile << shift) + a.rows - 1) / (unsigned)a.G;
    const int blk = tile_keys(a, s, (int)i0, min((int)i1, s.n - 1), PG_BLK).blk;
    l.count = max(1, (int)((unsigned)(blk + a.split_blk - 1) / (unsigned)a.split_blk));
    const unsigned piece = ((unsigned)vb * a.tiles + tile) * x_items(a) + x;
    l.at = (piece * a.splits << (DIFF ? shift + 1 : shift)) + (unsigned)(pr - (tile << shift));
    return l;
  }
  const unsigned per = CHUNK_ROWS / (unsigned)a.G, tile = (unsigned)i / (unsigned)a.tokens, in = i - tile * a.tokens, sub = DIFF ? 0 : in / per;
  const int part = a.heads == x_items(a) || a.one_map ? 0 : lane >> 4;   // columns of the second value head
  l.at = ((unsigned)s.q0 + tile * a.tokens) * a.heads + (a.heads == x_items(a) ? x : 2 * x + part);
  l.count = (int)(sub * CHUNK_ROWS + (in - sub * per) * a.G) + g0;
  return l;
}

// Where a pass left the sums of a set for this lane's columns: piece k at row
// `at` (k = 0) or at + next + k step of arrays of `width` columns, the set's
// further rows `rise` behind (few rows: looked up among the lanes).
struct Sums {
  const float *o, *ml;
  unsigned at, next, step, rise;
  int count, width, ml_step, map;   // map: from the first to the second map
};
template <int D, bool DIFF>
__device__ __forceinline__ Sums sums(const JoinArgs& a, const Place& l, const PieceNote& n, int column, unsigned row_at, bool there) {
  Sums f;
  constexpr int W = DIFF ? 2 * D : D;
  if (!a.chunk) {
    const int halves = DIFF && a.e4m3 ? 2 : 1;
    f.o = a.part_o + column;
    f.ml = a.part_ml + (halves == 2 && column >= D ? 2 : 0);
    f.width = W;
    f.ml_step = 2 * halves;
    f.at = l.at;
    f.count = l.count;
    f.next = f.rise = 0;
    f.step = a.rows * (DIFF ? 2 : 1);
    f.map = a.rows;
  } else {
    const bool whole = n.count == 0, halves = DIFF && a.heads != x_items(a) && !a.one_map;
    const int dv = halves ? D : W;
    f.o = whole ? a.row_o + column : a.part_o + (halves && column >= D ? column - D : column);
    f.ml = whole ? a.row_ml + (halves && column >= D ? 2 : 0) : a.part_ml;
    f.width = whole ? W : dv;
    f.ml_step = whole && halves ? 4 : 2;
    f.at = whole ? row_at : (unsigned)((n.first * 2 + n.slot) * a.rows + l.count);
    f.count = max(n.count, 1);
    f.next = 0u - (unsigned)(n.slot * a.rows);
    f.step = 2 * a.rows;
    f.rise = whole && DIFF ? 2 : 1;
    f.map = whole ? 1 : a.one_map ? 0 : CHUNK_ROWS;   // one_map: each map has pieces of its own
  }
  if (!there) f.count = 0;
  return f;
}

__device__ __forceinline__ int last_at_most(const int64_t* v, int n, long long t, int lane) {   // the last of n with v[i] <= t; the same in every lane
  int lo = 0;
  for (int stride = 1;;) {
    for (stride = 1; (long long)stride * 32 < n - lo; stride *= 32);
    const int i = lo + lane * stride;
    const unsigned hit = __ballot_sync(FULL, i < n && v[i] <= t);
    if (hit) lo += (31 - __clz(hit)) * stride;
    if (stride == 1) return lo;
    n = min(n, lo + stride);
  }
}

// Whether another group holds a sequence of group g as well, which offsets that
// decrease somewhere can bring about: both then have left sums, and notes, at the
// same rows.  The same in every lane.  A call, which one group does without: inlined
// it costs the join's loops registers.
__device__ __noinline__ bool overlapped(const JoinArgs& a, int g, int lane) {
  const int first = a.group_offsets[g], last = a.group_offsets[g + 1];
  bool hit = false;
#pragma unroll 4
  for (int k = lane; k < a.n_groups; k += 32) {
    const int lo = a.group_offsets[k], hi = a.group_offsets[k + 1];
    hit |= k != g && lo < hi && lo < last && hi > first;
  }
  return __any_sync(FULL, hit);
}

// WARPS warps of a CTA share the pieces of a set, or (WARPS = 1) each of its
// four warps has sets of its own.  A CTA has `sets` sets of a token, whose
// look-ups are made once for them: one round for the sequence (32 offsets at a
// time), one for its lengths, one for the notes, then U pieces of the set's rows at
// a time.
template <int WARPS> constexpr int join_threads() { return WARPS == 1 ? 128 : WARPS * 32; }

template <typename T, int D, bool DIFF, int WARPS, int RS, int U>
__global__ void __launch_bounds__(join_threads<WARPS>(), WARPS == 16 ? 1 : WARPS == 1 && DIFF ? (D == 128 ? 5 : 6) : WARPS == 4 && U == 4 ? 3 : 4) join_kernel(const __grid_constant__ Passes ps, int sets, int ctas) {
  constexpr int W = DIFF ? 2 * D : D, E = W / 32, ROWS = DIFF ? 2 : RS;
  static_assert(!DIFF || RS == 1, "a pair at a time");
  const JoinArgs &p = ps.p[0], &a = ps.p[1];
  __shared__ float s_o[WARPS][ROWS][W], s_ml[WARPS][ROWS][32][2];
  __shared__ int s_bad[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = WARPS == 1 ? 0 : warp, column = lane * E;
  const int units = DIFF ? a.H / 2 : a.H, per_x = (int)((unsigned)(a.G + RS - 1) / RS), all = x_items(a) * per_x;   // sets of a token
  const unsigned t = blockIdx.x / (unsigned)ctas;
  const int set0 = (int)(blockIdx.x - t * ctas) * sets, set_end = min(all, set0 + sets);
  int b;
  if (a.q_offsets) {
    b = last_at_most(a.q_offsets, a.B, t, lane);
    if (!(a.q_offsets[b] <= t && t < a.q_offsets[b + 1])) return wait_for_predecessor();
  } else {
    b = (int)(t / (unsigned)a.max_q);
    if (b >= a.B) return wait_for_predecessor();
  }
  Seq s = paged_seq(a, b, false);
  const int i = (int)(t - s.q0);
  if (i >= s.n) return wait_for_predecessor();
  Seq sp = {};
  int g = 0;
  if (p.n_groups) {
    g = group_of(a, b);
    sp = paged_seq(p, g, false);
    if (p.n_groups > 1 && overlapped(p, g, lane)) s.ok = false;
  }
  const bool prefix = s.ok && sp.kv > 0;
  const int ip = prefix ? (int)(t - sp.q0) : 0;
  const int first = set0 + (WARPS == 1 ? warp : 0);
  Place own = {}, pre = {};
  auto look = [&](int set) {
    const int x = (int)((unsigned)set / (unsigned)per_x), g0 = (set - x * per_x) * RS;
    own = locate<D, DIFF, RS>(a, b, s, i, x, g0, lane);
    if (prefix) pre = locate<D, DIFF, RS>(p, g, sp, ip, x, g0, lane);
  };
  // the notes of the next set are on their way while this one's sums are read
  constexpr int NE = DIFF && D == 128 ? 2 : 1;
  PieceNote own_note[NE] = {}, pre_note[NE] = {};
  auto notes = [&] {   // one_map: one for each map
    if (a.chunk && s.ok) {
      own_note[0] = a.notes[own.at];
      if (NE == 2 && a.one_map) own_note[NE - 1] = a.notes[own.at + 1];
    }
    if (p.chunk && prefix) {
      pre_note[0] = p.notes[pre.at];
      if (NE == 2 && p.one_map) pre_note[NE - 1] = p.notes[pre.at + 1];
    }
  };
  if (first < set_end) look(first);
  wait_for_predecessor();
  if (first < set_end) notes();
#pragma unroll 1
  for (int set = first; set < set_end; set += WARPS == 1 ? 4 : 1) {   // `own`, `pre` and the notes are this set's
    const int x = (int)((unsigned)set / (unsigned)per_x), g0 = (set - x * per_x) * RS, rows = DIFF ? 2 : min(RS, a.G - g0), unit0 = x * a.G + g0;
    const unsigned row_at = t * (unsigned)a.H + (DIFF ? 2 * unit0 : unit0);
    Sums f0[NE], f1[NE];
    f0[0] = sums<D, DIFF>(p, pre, pre_note[0], column, row_at, prefix);
    f1[0] = sums<D, DIFF>(a, own, own_note[0], column, row_at, s.ok);
    if constexpr (NE == 2) {
      f0[1] = f0[0];
      f1[1] = f1[0];
      if (p.one_map) f0[1] = sums<D, DIFF>(p, pre, pre_note[1], column, row_at, prefix);
      if (a.one_map) f1[1] = sums<D, DIFF>(a, own, own_note[1], column, row_at, s.ok);
    }
    const int next = set + (WARPS == 1 ? 4 : 1);
    float m[ROWS], l[ROWS], o[ROWS][E];
    unsigned at0[ROWS], at1[ROWS];
    int n0[ROWS], n1[ROWS], most = 0;
    bool bad = !s.ok;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int c = 0; c < E; ++c) o[r][c] = 0.f;
      if (DIFF) {
        const int e = NE == 2 ? r : 0;
        at0[r] = f0[e].at + r * f0[e].map;
        at1[r] = f1[e].at + r * f1[e].map;
        n0[r] = f0[e].count;
        n1[r] = f1[e].count;
      } else {
        const int from = p.chunk ? lane : r, from1 = a.chunk ? lane : r;   // few rows: the lane that looked for it
        at0[r] = __shfl_sync(FULL, f0[0].at, from) + r * f0[0].rise;
        at1[r] = __shfl_sync(FULL, f1[0].at, from1) + r * f1[0].rise;
        n0[r] = __shfl_sync(FULL, f0[0].count, from);
        n1[r] = __shfl_sync(FULL, f1[0].count, from1);
        if (r >= rows) n0[r] = n1[r] = 0;
      }
      most = max(most, n0[r] + n1[r]);
    }
    if (next < set_end) {
      look(next);
      notes();
    }
    // the pieces of both passes, one after the other, under a running maximum
#pragma unroll 1
    for (int k0 = part * U; k0 < most; k0 += WARPS * U) {
      float2 ml[U][ROWS];
      float y[U][ROWS][E];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          ml[u][r] = make_float2(-INFINITY, 0.f);
#pragma unroll
          for (int c = 0; c < E; ++c) y[u][r][c] = 0.f;
          const int k = k0 + u;
          if (k >= n0[r] + n1[r]) continue;
          const bool in0 = k < n0[r];
          const int kk = in0 ? k : k - n0[r];
          const Sums &x0 = f0[NE == 2 ? r : 0], &x1 = f1[NE == 2 ? r : 0];
          const unsigned at = (in0 ? at0[r] : at1[r]) + (kk == 0 ? 0u : (in0 ? x0.next : x1.next) + (unsigned)kk * (in0 ? x0.step : x1.step));
          ml[u][r] = *reinterpret_cast<const float2*>((in0 ? x0.ml : x1.ml) + (size_t)at * (in0 ? x0.ml_step : x1.ml_step));
          const float* const src = (in0 ? x0.o : x1.o) + (size_t)at * (in0 ? x0.width : x1.width);
          if constexpr (E == 2) *reinterpret_cast<float2*>(y[u][r]) = *reinterpret_cast<const float2*>(src);
#pragma unroll
          for (int c = 0; c + 3 < E; c += 4) *reinterpret_cast<float4*>(&y[u][r][c]) = *reinterpret_cast<const float4*>(src + c);
        }
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        float mn = m[r];
#pragma unroll
        for (int u = 0; u < U; ++u) mn = fmaxf(mn, ml[u][r].x);
        const float mu = mn > -INFINITY ? mn : 0.f, old = fast_exp2(m[r] - mu);
        m[r] = mn;
        l[r] *= old;
#pragma unroll
        for (int c = 0; c < E; ++c) o[r][c] *= old;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          bad |= ml[u][r].y < 0.f;
          const float w = fast_exp2(ml[u][r].x - mu);
          l[r] = fmaf(ml[u][r].y, w, l[r]);
#pragma unroll
          for (int c = 0; c < E; ++c) o[r][c] = fmaf(y[u][r][c], w, o[r][c]);
        }
      }
    }
    bad = __any_sync(FULL, bad);
    if (WARPS > 1) {
      if (set > first) __syncthreads();
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        s_ml[part][r][lane][0] = m[r];
        s_ml[part][r][lane][1] = l[r];
#pragma unroll
        for (int c = 0; c < E; ++c) s_o[part][r][column + c] = o[r][c];
      }
      if (lane == 0) s_bad[part] = bad;
      __syncthreads();
#pragma unroll
      for (int u = 0; u < WARPS; ++u) bad |= s_bad[u] != 0;
    }
    float y[E];
    bool empty = false;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int e = DIFF ? r : 0, unit = DIFF ? unit0 : unit0 + r;
      if (r >= rows || (WARPS > 1 && (DIFF ? 0 : r % WARPS) != part)) continue;   // one warp has a row's end
      float mm = m[r], ll = l[r], z[E];
#pragma unroll
      for (int c = 0; c < E; ++c) z[c] = o[r][c];
      if (WARPS > 1) {
        mm = -INFINITY;
        ll = 0.f;
#pragma unroll
        for (int u = 0; u < WARPS; ++u) mm = fmaxf(mm, s_ml[u][r][lane][0]);
        const float mu = mm > -INFINITY ? mm : 0.f;
#pragma unroll
        for (int c = 0; c < E; ++c) z[c] = 0.f;
#pragma unroll
        for (int u = 0; u < WARPS; ++u) {
          const float w = fast_exp2(s_ml[u][r][lane][0] - mu);
          ll = fmaf(s_ml[u][r][lane][1], w, ll);
#pragma unroll
          for (int c = 0; c < E; ++c) z[c] = fmaf(s_o[u][r][column + c], w, z[c]);
        }
      }
      const bool none = bad || ll == 0.f;
      empty = (e && empty) || none;
      if (a.lse && lane == 0) {
        // the sum's exponent goes to the maximum's side, so that the logarithm's argument is near 1
        const int ex = (int)(__float_as_uint(ll) >> 23) - 127;
        const float near1 = __uint_as_float((__float_as_uint(ll) & 0x7fffffu) | 0x3f800000u);
        const float v = ll <= 3.402823466e38f ? (mm + (float)ex) * 0.6931471805599453f + __logf(near1) : ll;
        a.lse[(size_t)t * a.H + (DIFF ? 2 * unit + e : unit)] = none ? -INFINITY : v;
      }
      float f = none ? 0.f : __fdividef(1.f, ll);
      if (DIFF && e == 1) f *= -a.lambda[t * a.lambda_stride + unit];
#pragma unroll
      for (int c = 0; c < E; ++c) y[c] = e == 0 ? z[c] * f : fmaf(z[c], f, y[c]);
      if (DIFF && e == 0) continue;
      if (DIFF) {
        float k = a.gain;
        if (a.norm) {
          float sq = 0.f;
#pragma unroll
          for (int c = 0; c < E; ++c) sq = fmaf(y[c], y[c], sq);
#pragma unroll
          for (int v = 16; v; v >>= 1) sq += __shfl_xor_sync(FULL, sq, v);
          k *= 1.f / sqrtf(sq * (1.f / W) + a.eps);
        }
#pragma unroll
        for (int c = 0; c < E; c += 2) {
          float2 wt = make_float2(1.f, 1.f);
          if (a.norm) wt = unpack16<T>(reinterpret_cast<const uint32_t*>(a.norm)[(column + c) / 2]);
          y[c] *= k * wt.x;
          y[c + 1] *= k * wt.y;
        }
      }
      uint32_t w[E / 2];
#pragma unroll
      for (int c = 0; c < E; c += 2) w[c / 2] = empty ? 0u : pack16<T>(y[c], y[c + 1]);
      T* const dst = static_cast<T*>(a.out) + ((size_t)t * units + unit) * W + column;
      if constexpr (E == 2) *reinterpret_cast<uint32_t*>(dst) = w[0];
      else if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// How many warps share a set of rows, and how many sets a CTA has.
template <typename T, int D, bool DIFF, int WARPS, int RS, int U>
cudaError_t sized(const JoinArgs& p, const JoinArgs& a) {
  const int all = x_items(a) * ((a.G + RS - 1) / RS), least = WARPS == 1 ? 4 : 1;
  const long long want = std::max<long long>(1, a.total_q * all / least / (12ll * a.num_sms));   // CTAs for about two rounds
  const int ctas = (int)((all + least - 1) / least / std::min<long long>(want, (all + least - 1) / least));
  const int sets = ((all + ctas - 1) / ctas + least - 1) / least * least, n = (all + sets - 1) / sets;
  return launch_pass(join_kernel<T, D, DIFF, WARPS, RS, U>, (unsigned)(a.total_q * n), join_threads<WARPS>(), 0, a.stream, true, Passes{{p, a}}, sets, n);
}
template <typename T, int D, bool DIFF>
cudaError_t rows(const JoinArgs& p, const JoinArgs& a) {
  const int sources = (p.n_groups ? p.sources : 0) + a.sources;
  const long long n = a.total_q * (DIFF ? a.H / 2 : a.H);
  constexpr int RS = DIFF ? 1 : 4;
  if (sources > 16 && n <= 2ll * a.num_sms) return sized<T, D, DIFF, 16, 1, DIFF ? 2 : 4>(p, a);
  if (sources <= 4) return sized<T, D, DIFF, 1, RS, DIFF ? 1 : 2>(p, a);
  // few rows: what a warp has to read in one round rather than two, with more registers (sixteen tokens behind
  // 8192 keys 21.5 -> 20.8 us; 64 behind 32768 the other way round, 87.7 -> 92.0; differential, 16 rows 8.3 -> 8.1,
  // 512 44.9 -> 47.9)
  return n <= (DIFF ? 2ll : 12ll) * a.num_sms ? sized<T, D, DIFF, 4, RS, 4>(p, a) : sized<T, D, DIFF, 4, RS, 2>(p, a);
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
