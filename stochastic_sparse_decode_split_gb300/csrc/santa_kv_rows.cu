// santa_kv_rows.cu -- new tokens written into a paged cache (norm, rotation,
// e4m3) and a paged cache read back as packed rows.
//
// Both move every byte once and compute little, so HBM bounds them at large
// sizes and the launch at small ones.
#include <algorithm>
#include <type_traits>

#include "santa_launch.h"
#include "santa_paged.cuh"

namespace santa {

namespace {

constexpr float E4M3_MAX = 448.f;
constexpr float AMAX_FLOOR = 8.673617379884035e-19f;   // 2^-60

// Eight consecutive elements of storage type T, 16-byte aligned, rounded once.
template <typename T> __device__ __forceinline__ void store8(T* p, const float (&f)[8]);
template <> __device__ __forceinline__ void store8<bf16_t>(bf16_t* p, const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <> __device__ __forceinline__ void store8<fp16_t>(fp16_t* p, const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <> __device__ __forceinline__ void store8<float>(float* p, const float (&f)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

// The larger of two values, NaN if either is.
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

// Two values as e4m3 (lo in the low byte), to nearest, saturating at 448.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four consecutive elements as they are stored, and as float pairs.
template <typename T> struct Four;
template <typename T> struct Four16 {
  typedef uint2 raw;
  static __device__ __forceinline__ raw load(const T* p) {
    raw r;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));   // q_out may be q
    return r;
  }
};
template <> struct Four<bf16_t> : Four16<bf16_t> {
  static __device__ __forceinline__ void widen(const uint2& r, f2x (&f)[2]) {
    f[0] = pack2(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u));
    f[1] = pack2(__uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
  }
  static __device__ __forceinline__ void store(bf16_t* p, const f2x (&f)[2]) {
    const float2 a = unpack2(f[0]), b = unpack2(f[1]);
    uint2 w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(a.y), "f"(a.x));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(b.y), "f"(b.x));
    *reinterpret_cast<uint2*>(p) = w;
  }
};
template <> struct Four<fp16_t> : Four16<fp16_t> {
  static __device__ __forceinline__ void widen(const uint2& r, f2x (&f)[2]) {
    __half2 a, b;
    memcpy(&a, &r.x, 4);
    memcpy(&b, &r.y, 4);
    const float2 x = __half22float2(a), y = __half22float2(b);
    f[0] = pack2(x.x, x.y);
    f[1] = pack2(y.x, y.y);
  }
  static __device__ __forceinline__ void store(fp16_t* p, const f2x (&f)[2]) {
    const float2 a = unpack2(f[0]), b = unpack2(f[1]);
    uint2 w;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(a.y), "f"(a.x));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(b.y), "f"(b.x));
    *reinterpret_cast<uint2*>(p) = w;
  }
};
template <> struct Four<float> {
  typedef uint4 raw;
  static __device__ __forceinline__ raw load(const float* p) {
    raw r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
  }
  static __device__ __forceinline__ void widen(const uint4& r, f2x (&f)[2]) {
    f[0] = pack2(__uint_as_float(r.x), __uint_as_float(r.y));
    f[1] = pack2(__uint_as_float(r.z), __uint_as_float(r.w));
  }
  static __device__ __forceinline__ void store(float* p, const f2x (&f)[2]) {
    const float2 a = unpack2(f[0]), b = unpack2(f[1]);
    *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y);
  }
};
__device__ __forceinline__ f2x mul2(f2x a, f2x b) {
  f2x d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// A warp takes one token and a run of groups of RPW rows of it, a row being one
// head: `qg` groups of queries (blockIdx.y < qparts), or `kvg` of keys and the
// same of values.  LPR lanes hold a row, eight elements each in two pieces of
// four.  For half pairs the pieces are the two members of four pairs, elements
// 4 j and rotated / 2 + 4 j on; else eight elements in a row.  So a lane turns
// its own four pairs, under one cos and sin each that it keeps over its rows.
// Groups in a run are neighbours in memory: their loads and stores differ by
// constants, which matters here (address arithmetic was two fifths of the
// instructions when a warp's groups were strided, at 200 instructions a group).
//
// The first rows are requested before the token's sequence, position and page
// are looked up: those are four to five loads that wait on one another.
//
// As many warps as their registers allow without spilling: 32 per SM in 16
// bits, 28 over e4m3, 20 in float32.  8192 tokens of 32 and 8 heads of 128:
// 33.9 us in bf16 (36.5 with 24 warps), 32.7 over e4m3 (35.0; 34.0 with 32 and
// a few spills), 5.6 TB/s; twice the rows in flight per warp and fewer warps
// were slower (34.8 to 38.5).  In float32 62.3 us, 6.5 TB/s; 57.6 over e4m3.
template <typename T, int D, bool E4M3, bool INTER>
__global__ void __launch_bounds__(128, sizeof(T) == 4 ? 5 : E4M3 ? 7 : 8) kv_append_kernel(PagedArgs a, AppendArgs p, int qparts, int qg, int kvg) {
  using F = Four<T>;
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  constexpr int U = 4;   // groups in flight; of a key-value run two of each
  const int lane = threadIdx.x & 31, sub = lane % LPR, rr = lane / LPR;
  const long long t = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (t >= a.total_q) {
    // CTAs past the tokens look the sequences over: one without tokens, or
    // whose offsets no token finds, would be refused by nobody
    const long long i = ((long long)blockIdx.x - (a.total_q + 3) / 4) * 128 + threadIdx.x;
    if (blockIdx.y == 0 && i >= 0 && i < a.B) {
      const Seq s = paged_seq(a, (int)i, true);
      if (s.ok && s.n > s.kv) flag_error(a.err, ERR_CHUNK);
    }
    return;
  }
  const bool is_q = (int)blockIdx.y < qparts;
  const int part = is_q ? blockIdx.y : blockIdx.y - qparts;
  const int heads = is_q ? a.H : a.Hkv;
  const int g0 = part * (is_q ? qg : kvg), g1 = min(g0 + (is_q ? qg : kvg), (heads + RPW - 1) / RPW);

  const int half = p.rotated >> 1;
  const bool turns = 8 * sub < p.rotated;
  const int off0 = !INTER && turns ? 4 * sub : 8 * sub, off1 = !INTER && turns ? half + 4 * sub : 8 * sub + 4;
  int h = g0 * RPW + rr;   // this lane's head of the batch's first group
  const T* src = (is_q ? static_cast<const T*>(p.q) + t * p.q_stride : static_cast<const T*>(p.k) + t * p.k_stride) + h * D;
  const T* srv = is_q ? src + 2 * RPW * D : static_cast<const T*>(p.v) + t * p.v_stride + h * D;
  typename F::raw in[U][2];
  auto request = [&](int g) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int uu = is_q ? u : u & 1;
      if (g + uu < g1 && h + uu * RPW < heads) {
        const T* s = u < 2 ? src + u * RPW * D : srv + (u - 2) * RPW * D;
        in[u][0] = F::load(s + off0);
        in[u][1] = F::load(s + off1);
      }
    }
  };
  request(g0);

  int b;
  if (!paged_seq_of(a, t, b)) return;
  const Seq s = paged_seq(a, b, false);
  if (!s.ok || s.n > s.kv) return;
  const int pos = s.kv - s.n + (int)(t - s.q0);
  if (p.rotated && pos >= p.rope_positions) {
    if (lane == 0) flag_error(a.err, ERR_POSITION);
    return;
  }
  const int slot = pos & ((1 << a.page_shift) - 1);
  f2x c[2], sn[2], neg[2];
  if (turns) {
    const float4* t4 = reinterpret_cast<const float4*>(p.rope + ((long long)pos * half + 4 * sub) * 2);
    const float4 x = __ldg(t4), y = __ldg(t4 + 1);
    c[0] = pack2(x.x, x.z);
    c[1] = pack2(y.x, y.z);
    sn[0] = pack2(x.y, x.w);
    sn[1] = pack2(y.y, y.w);
    neg[0] = pack2(-x.y, -x.w);
    neg[1] = pack2(-y.y, -y.w);
  }
  const T* const weight = static_cast<const T*>(is_q ? p.q_norm : p.k_norm);
  f2x wt[2][2];
  if (weight) {
    F::widen(*reinterpret_cast<const typename F::raw*>(weight + off0), wt[0]);
    F::widen(*reinterpret_cast<const typename F::raw*>(weight + off1), wt[1]);
  }
  // Norm and rotation of one group's row (in the lanes that hold it).
  auto norm_turn = [&](f2x (&x)[2][2]) {
    if (weight) {
      f2x ss2 = mul2(x[0][0], x[0][0]);
      ss2 = ffma2(x[0][1], x[0][1], ss2);
      ss2 = ffma2(x[1][0], x[1][0], ss2);
      ss2 = ffma2(x[1][1], x[1][1], ss2);
      const float2 sp = unpack2(ss2);
      float ss = sp.x + sp.y;
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(FULL, ss, o);
      const float inv = rsqrtf(ss * (1.f / D) + p.eps);
      const f2x inv2 = pack2(inv, inv);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i >> 1][i & 1] = mul2(mul2(x[i >> 1][i & 1], inv2), wt[i >> 1][i & 1]);
    }
    if (!turns) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (INTER) {   // two neighbouring pairs
        const float2 cc = unpack2(c[i]), ss = unpack2(sn[i]), e = unpack2(x[i][0]), f = unpack2(x[i][1]);
        x[i][0] = pack2(fmaf(e.x, cc.x, -(e.y * ss.x)), fmaf(e.y, cc.x, e.x * ss.x));
        x[i][1] = pack2(fmaf(f.x, cc.y, -(f.y * ss.y)), fmaf(f.y, cc.y, f.x * ss.y));
      } else {       // first and second members of two pairs
        const f2x A = x[0][i], B = x[1][i];
        x[0][i] = ffma2(A, c[i], mul2(B, neg[i]));
        x[1][i] = ffma2(B, c[i], mul2(A, sn[i]));
      }
    }
  };

  if (is_q) {
    T* dst = static_cast<T*>(p.q_out) + (t * a.H + h) * D;
    for (int g = g0; g < g1;) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (g + u >= g1) break;
        f2x x[2][2];
        F::widen(in[u][0], x[0]);
        F::widen(in[u][1], x[1]);
        norm_turn(x);
        if (h + u * RPW < heads) {
          F::store(dst + u * RPW * D + off0, x[0]);
          F::store(dst + u * RPW * D + off1, x[1]);
        }
      }
      g += U;
      if (g >= g1) break;
      h += U * RPW;
      src += U * RPW * D;
      srv += U * RPW * D;
      dst += U * RPW * D;
      request(g);
    }
    return;
  }
  const int pid = a.table[(long long)b * a.max_pages + (pos >> a.page_shift)];
  if ((unsigned)pid >= (unsigned)a.n_pages) {
    if (lane == 0) flag_error(a.err, ERR_PAGE);
    return;
  }
  const long long at = ((((long long)pid << a.page_shift) + slot) * a.Hkv + h) * D;
  unsigned char *kc = static_cast<unsigned char*>(p.K) + at, *vc = static_cast<unsigned char*>(p.V) + at;
  T *kd = static_cast<T*>(p.K) + at, *vd = static_cast<T*>(p.V) + at;
  const long long sat = (((long long)pid * a.Hkv) << a.page_shift) + slot;
  for (int g = g0; g < g1;) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int uu = u & 1, hh = h + uu * RPW;
      if (g + uu >= g1) continue;
      const bool live = hh < heads, is_v = u >= 2;
      if (is_v && !E4M3) {   // as they are
        if (live) {
          *reinterpret_cast<typename F::raw*>(vd + uu * RPW * D + off0) = in[u][0];
          *reinterpret_cast<typename F::raw*>(vd + uu * RPW * D + off1) = in[u][1];
        }
        continue;
      }
      f2x x[2][2];
      F::widen(in[u][0], x[0]);
      F::widen(in[u][1], x[1]);
      if (!is_v) norm_turn(x);
      if (E4M3) {
        float m = AMAX_FLOOR;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = unpack2(x[i >> 1][i & 1]);
          m = max_nan(m, max_nan(fabsf(f.x), fabsf(f.y)));
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(FULL, m, o));
        const float inv = __fdiv_rn(E4M3_MAX, m);
        const f2x inv2 = pack2(inv, inv);
        uint32_t code[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 e = unpack2(mul2(x[i][0], inv2)), f = unpack2(mul2(x[i][1], inv2));
          code[i] = e4m3x2(e.x, e.y) | e4m3x2(f.x, f.y) << 16;
        }
        if (live) {
          unsigned char* dst = (is_v ? vc : kc) + uu * RPW * D;
          *reinterpret_cast<uint32_t*>(dst + off0) = code[0];
          *reinterpret_cast<uint32_t*>(dst + off1) = code[1];
          if (sub == 0) (is_v ? p.vs : p.ks)[sat + ((long long)hh << a.page_shift)] = __fdiv_rn(m, E4M3_MAX);
        }
      } else if (live) {
        F::store(kd + uu * RPW * D + off0, x[0]);
        F::store(kd + uu * RPW * D + off1, x[1]);
      }
    }
    g += 2;
    if (g >= g1) break;
    h += 2 * RPW;
    src += 2 * RPW * D;
    srv += 2 * RPW * D;
    kc += 2 * RPW * D;
    vc += 2 * RPW * D;
    kd += 2 * RPW * D;
    vd += 2 * RPW * D;
    request(g);
  }
}

// Packed rows of one sequence: a CTA takes 16 keys (one block, inside one
// page) of K or V at a time; their bytes are contiguous on both sides, which is
// all the order that HBM needs: 8 sequences of up to 32768 keys, 8 heads of 128,
// e4m3 to bf16, 221 us, 6.1 TB/s (0.90 of a copy's rate); three short ones 2.3 us.
template <typename T, bool E4M3>
__global__ void __launch_bounds__(256) kv_read_kernel(PagedArgs a, const int64_t* kv_offsets, long long rows,
                                                      T* __restrict__ K_out, T* __restrict__ V_out) {
  const int b = blockIdx.y, tid = threadIdx.x;
  const int kv = a.kv_lens ? a.kv_lens[b] : a.nk;
  const long long r0 = kv_offsets ? kv_offsets[b] : (long long)b * a.nk;
  const long long r1 = kv_offsets ? kv_offsets[b + 1] : r0 + a.nk;
  int e = 0;
  if (kv < 0 || kv > a.nk) e |= ERR_NK_BOUND;
  else if (r0 < 0 || r1 < r0 || r1 > rows || r1 - r0 < kv) e |= ERR_CHUNK;
  if (e) {
    if (tid == 0 && blockIdx.x == 0) flag_error(a.err, e);
    return;
  }
  const long long key0 = (long long)blockIdx.x * PG_BLK;
  if (key0 >= kv) return;
  const int n = min(PG_BLK, kv - (int)key0);
  const int pid = a.table[(long long)b * a.max_pages + (int)(key0 >> a.page_shift)];
  const bool page_ok = (unsigned)pid < (unsigned)a.n_pages;
  if (!page_ok && tid == 0) flag_error(a.err, ERR_PAGE);
  const int slot = (int)key0 & ((1 << a.page_shift) - 1);
  const long long row = ((long long)pid << a.page_shift) + slot;
  const int rowlen = a.Hkv * a.D;
  const bool is_v = blockIdx.z != 0;
  T* const dst = (is_v ? V_out : K_out) + (r0 + key0) * rowlen;
  constexpr int U = 4;
  if (E4M3) {
    const unsigned char* const src = static_cast<const unsigned char*>(is_v ? a.V : a.K) + row * rowlen;
    const float* const sc = (is_v ? a.vs : a.ks) + (((long long)pid * a.Hkv) << a.page_shift) + slot;
    const int vecs = n * rowlen / 16, per_row = rowlen / 16, per_head = a.D / 16;
    for (int i0 = tid; i0 < vecs; i0 += 256 * U) {
      uint4 w[U];
      float f[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + 256 * u;
        w[u] = make_uint4(0u, 0u, 0u, 0u);
        f[u] = 0.f;
        if (i < vecs && page_ok) {
          w[u] = ld_stream(src + (long long)i * 16);
          const int rr = i / per_row, hh = (i - rr * per_row) / per_head;
          f[u] = __ldg(sc + (hh << a.page_shift) + rr);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + 256 * u;
        if (i >= vecs) break;
        const uint32_t ww[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
        float x[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t h2;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(ww[j / 2] >> (16 * (j & 1)))));
          __half2 h;
          memcpy(&h, &h2, 4);
          const float2 y = __half22float2(h);
          x[2 * j] = y.x * f[u];
          x[2 * j + 1] = y.y * f[u];
        }
        float lo[8], hi[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          lo[j] = x[j];
          hi[j] = x[8 + j];
        }
        store8<T>(dst + (long long)i * 16, lo);
        store8<T>(dst + (long long)i * 16 + 8, hi);
      }
    }
  } else {
    const T* const src = static_cast<const T*>(is_v ? a.V : a.K) + row * rowlen;
    constexpr int EPV = 16 / (int)sizeof(T);
    const int vecs = n * rowlen / EPV;
    for (int i0 = tid; i0 < vecs; i0 += 256 * U) {
      uint4 w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + 256 * u;
        w[u] = make_uint4(0u, 0u, 0u, 0u);
        if (i < vecs && page_ok) w[u] = ld_stream(src + (long long)i * EPV);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + 256 * u;
        if (i < vecs) *reinterpret_cast<uint4*>(dst + (long long)i * EPV) = w[u];
      }
    }
  }
}

template <typename T, int D, bool E4M3>
cudaError_t append_inst(const PagedArgs& a, const AppendArgs& p) {
  constexpr int RPW = 32 / (D / 8);
  const int gq = p.q ? (a.H + RPW - 1) / RPW : 0, gkv = (a.Hkv + RPW - 1) / RPW;
  // few tokens: a warp per group, all of a token's rows at once; many: up to
  // eight groups of queries, or four of keys and values, share a warp's
  // look-ups and angles
  const bool many = a.total_q * (gq + 2 * gkv) >= 64ll * a.num_sms;
  const int qparts = many ? (gq + 7) / 8 : gq, kvparts = many ? (gkv + 3) / 4 : gkv;
  const int qg = qparts ? (gq + qparts - 1) / qparts : 1, kvg = (gkv + kvparts - 1) / kvparts;
  const dim3 grid((unsigned)((a.total_q + 3) / 4 + (a.B + 127) / 128), (unsigned)(qparts + kvparts));
  if (p.interleaved) kv_append_kernel<T, D, E4M3, true><<<grid, 128, 0, a.stream>>>(a, p, qparts, qg, kvg);
  else kv_append_kernel<T, D, E4M3, false><<<grid, 128, 0, a.stream>>>(a, p, qparts, qg, kvg);
  return cudaGetLastError();
}

template <typename T>
cudaError_t append_type(const PagedArgs& a, const AppendArgs& p) {
  if (a.D == 128) return a.e4m3 ? append_inst<T, 128, true>(a, p) : append_inst<T, 128, false>(a, p);
  return a.e4m3 ? append_inst<T, 64, true>(a, p) : append_inst<T, 64, false>(a, p);
}

template <typename T>
cudaError_t read_type(const PagedArgs& a, const int64_t* off, long long rows, void* K, void* V) {
  const dim3 grid((unsigned)((a.nk + PG_BLK - 1) / PG_BLK), (unsigned)a.B, 2);
  if (a.e4m3) kv_read_kernel<T, true><<<grid, 256, 0, a.stream>>>(a, off, rows, (T*)K, (T*)V);
  else kv_read_kernel<T, false><<<grid, 256, 0, a.stream>>>(a, off, rows, (T*)K, (T*)V);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const PagedArgs& a, const AppendArgs& p) {
  return a.dtype == 0 ? append_type<bf16_t>(a, p) : a.dtype == 1 ? append_type<fp16_t>(a, p) : append_type<float>(a, p);
}

cudaError_t launch_kv_read(const PagedArgs& a, const int64_t* kv_offsets, long long rows, void* K_out, void* V_out) {
  return a.dtype == 0   ? read_type<bf16_t>(a, kv_offsets, rows, K_out, V_out)
         : a.dtype == 1 ? read_type<fp16_t>(a, kv_offsets, rows, K_out, V_out)
                        : read_type<float>(a, kv_offsets, rows, K_out, V_out);
}

}  // namespace santa
