// santa_kv_rows.cu -- new tokens written into a paged cache (norm, rotation,
// e4m3) and a paged cache read back as packed rows.
//
// Both move every byte once and compute little, so HBM bounds them at large
// sizes and the launch at small ones.
#include <algorithm>

#include "santa_launch.h"
#include "santa_paged.cuh"

namespace santa {

namespace {

constexpr float E4M3_MAX = 448.f;
constexpr float AMAX_FLOOR = 8.673617379884035e-19f;   // 2^-60

// Eight consecutive elements of storage type T, 16-byte aligned.
template <typename T> struct Eight;
template <typename T> struct Eight16 {
  static __device__ __forceinline__ void load(const T* p, float (&f)[8]) {
    Elem<T>::widen(*reinterpret_cast<const uint4*>(p), f);
  }
};
template <> struct Eight<bf16_t> : Eight16<bf16_t> {
  static __device__ __forceinline__ void store(bf16_t* p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Eight<fp16_t> : Eight16<fp16_t> {
  static __device__ __forceinline__ void store(fp16_t* p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Eight<float> {
  static __device__ __forceinline__ void load(const float* p, float (&f)[8]) {
    const float4 x = *reinterpret_cast<const float4*>(p), y = *reinterpret_cast<const float4*>(p + 4);
    f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
    f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&f)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
  }
};

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

// One warp handles `iters` groups of RPW rows of one token, a row being one
// head of q, k or v in that order; LPR lanes hold a row, eight elements each.
// The token's angles stay in registers over the groups.
template <typename T, int D, bool E4M3>
__global__ void __launch_bounds__(256) kv_append_kernel(PagedArgs a, AppendArgs p, int warps_per_token, int iters) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31;
  const long long w = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const long long t = w / warps_per_token;
  const int part = (int)(w - t * warps_per_token);
  if (t >= a.total_q) return;
  int b;
  if (!paged_seq_of(a, t, b)) return;
  const Seq s = paged_seq(a, b, lane == 0);
  if (!s.ok) return;
  if (s.n > s.kv) {
    if (lane == 0) flag_error(a.err, ERR_CHUNK);
    return;
  }
  const int pos = s.kv - s.n + (int)(t - s.q0);
  const bool turns = p.rope != nullptr && p.rotated > 0;
  if (turns && pos >= p.rope_positions) {
    if (lane == 0) flag_error(a.err, ERR_POSITION);
    return;
  }
  const int page_i = pos >> a.page_shift, slot = pos & ((1 << a.page_shift) - 1);
  const int pid = a.table[(long long)b * a.max_pages + page_i];
  const bool page_ok = (unsigned)pid < (unsigned)a.n_pages;
  if (!page_ok && lane == 0) flag_error(a.err, ERR_PAGE);
  const long long row = ((long long)pid << a.page_shift) + slot;

  // this lane's eight elements d0 .. d0 + 7 of every row it handles, and
  // their rotation: x' = x c + y s with y the partner element (the partner
  // lane's for half pairs, the neighbour for interleaved ones)
  const int sub = lane % LPR, d0 = sub * 8, half = p.rotated >> 1;
  const bool in_rot = turns && d0 < p.rotated;
  const bool upper = !p.interleaved && d0 >= half;
  float c[8], sn[8];
  int partner = lane;
  if (in_rot) {
    const float2* tb = reinterpret_cast<const float2*>(p.rope) + (long long)pos * half;
    if (p.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 cs = __ldg(tb + d0 / 2 + i);
        c[2 * i] = c[2 * i + 1] = cs.x;
        sn[2 * i] = -cs.y;
        sn[2 * i + 1] = cs.y;
      }
    } else {
      partner = upper ? lane - half / 8 : lane + half / 8;
      const float4* t4 = reinterpret_cast<const float4*>(tb + (upper ? d0 - half : d0));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 cs = __ldg(t4 + i);
        c[2 * i] = cs.x;
        sn[2 * i] = upper ? cs.y : -cs.y;
        c[2 * i + 1] = cs.z;
        sn[2 * i + 1] = upper ? cs.w : -cs.w;
      }
    }
  }

  const int nq = p.q ? a.H : 0, total = nq + 2 * a.Hkv;
  const T* const qp = static_cast<const T*>(p.q) + t * p.q_stride;
  const T* const kp = static_cast<const T*>(p.k) + t * p.k_stride;
  const T* const vp = static_cast<const T*>(p.v) + t * p.v_stride;
  constexpr int U = 4;   // rows in flight per lane
  for (int it = 0; it < iters; it += U) {
    float x[U][8];
    int r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      r[u] = it + u < iters ? (part * iters + it + u) * RPW + lane / LPR : total;
      if (r[u] < total) {
        const T* src = r[u] < nq ? qp + r[u] * D : r[u] < nq + a.Hkv ? kp + (r[u] - nq) * D : vp + (r[u] - nq - a.Hkv) * D;
        Eight<T>::load(src + d0, x[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (__all_sync(FULL, r[u] >= total)) break;
      const bool live = r[u] < total, is_q = r[u] < nq, is_k = !is_q && r[u] < nq + a.Hkv;
      const void* wt = is_q ? p.q_norm : is_k ? p.k_norm : nullptr;
      if (p.q_norm || p.k_norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = live ? fmaf(x[u][i], x[u][i], ss) : 0.f;
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(FULL, ss, o);
        if (live && wt) {
          const float inv = rsqrtf(ss * (1.f / D) + p.eps);
          float g[8];
          Eight<T>::load(static_cast<const T*>(wt) + d0, g);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[u][i] = x[u][i] * inv * g[i];
        }
      }
      if (turns) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = p.interleaved ? x[u][i ^ 1] : __shfl_sync(FULL, x[u][i], partner);
        if (in_rot && live && (is_q || is_k)) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[u][i] = x[u][i] * c[i] + y[i] * sn[i];
        }
      }
      if (E4M3) {
        float m = AMAX_FLOOR;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max_nan(m, live ? fabsf(x[u][i]) : 0.f);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(FULL, m, o));
        if (live && !is_q && page_ok) {
          const float inv = __fdiv_rn(E4M3_MAX, m);
          uint32_t lo = 0, hi = 0;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            lo |= e4m3x2(x[u][2 * i] * inv, x[u][2 * i + 1] * inv) << (16 * i);
            hi |= e4m3x2(x[u][2 * i + 4] * inv, x[u][2 * i + 5] * inv) << (16 * i);
          }
          const int kvh = is_k ? r[u] - nq : r[u] - nq - a.Hkv;
          unsigned char* dst = static_cast<unsigned char*>(is_k ? p.K : p.V) + (row * a.Hkv + kvh) * D + d0;
          *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
          if (sub == 0) (is_k ? p.ks : p.vs)[((((long long)pid * a.Hkv) + kvh) << a.page_shift) + slot] = __fdiv_rn(m, E4M3_MAX);
        }
      }
      if (live) {
        if (is_q) {
          Eight<T>::store(static_cast<T*>(p.q_out) + (t * a.H + r[u]) * D + d0, x[u]);
        } else if (!E4M3 && page_ok) {
          const int kvh = is_k ? r[u] - nq : r[u] - nq - a.Hkv;
          Eight<T>::store(static_cast<T*>(is_k ? p.K : p.V) + (row * a.Hkv + kvh) * D + d0, x[u]);
        }
      }
    }
  }
}

// Packed rows of one sequence: a CTA takes 16 keys (one block, inside one
// page) of K or V at a time; their bytes are contiguous on both sides.
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
        Eight<T>::store(dst + (long long)i * 16, lo);
        Eight<T>::store(dst + (long long)i * 16 + 8, hi);
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
  const int groups = ((p.q ? a.H : 0) + 2 * a.Hkv + RPW - 1) / RPW;
  // few tokens: one group per warp, all of a token's rows at once; many: a
  // warp keeps the token's angles over up to eight groups
  const int iters = a.total_q * groups >= 64ll * a.num_sms ? std::min(8, groups) : 1;
  const int wpt = (groups + iters - 1) / iters;
  const long long ctas = (a.total_q * wpt * 32 + 255) / 256;
  kv_append_kernel<T, D, E4M3><<<(unsigned)ctas, 256, 0, a.stream>>>(a, p, wpt, iters);
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
