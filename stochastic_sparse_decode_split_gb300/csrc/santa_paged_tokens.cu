// santa_paged_tokens.cu -- exact attention over a paged cache for few query
// rows per KV head (single tokens, a handful of proposed ones), and the merge
// of split tiles.
//
// out = softmax(scale q K^T + mask) V in one pass over the keys.  Every K and
// V row is used for at most 16 query rows, so HBM bounds the kernel: what
// matters is bytes in flight and an even share for every SM.  A tile (16 or 8
// query rows of one sequence and KV head) is cut into splits of whole
// 16-key blocks; a CTA's four warps take its blocks in turn, each with its own
// ring of cp.async stages (no barrier inside the loop; a stage is refilled as
// soon as it is left).  Scores come from the tensor cores as S^T = K q^T (16
// keys x 8 rows), the running softmax is kept in base 2, and O^T = V^T P^T
// accumulates in registers.
//
// Measured: 16 sequences of 1024 to 32768 keys, 28 and 4 heads of 128, fp16:
// 103 us, 6.3 TB/s (0.93 of a copy's rate); two of 131072 over e4m3, 32 and 8
// heads: 103 us, 5.4 TB/s (0.79: more instructions per byte); one token over
// 1000 keys 5.8 us, the two launches and their chain of look-ups.
//
// e4m3 caches: codes widen to fp16 exactly, on the way from shared memory to
// the tensor cores.  Queries become fp16 under a power of two per row that
// brings the row's largest magnitude to [2^10, 2^11): exact for bf16 values
// down to 2^-24 of it (smaller ones lose bits that 32-bit sums do not see
// either).  A key's score is multiplied by its k_scale; its v_scale enters as
// log2 v_scale beside the score, so that P = 2^(s + log2 v_scale - m) stays in
// range whatever the scales are, and the sum of the softmax collects
// P / v_scale.
#include <algorithm>
#include <type_traits>

#include "santa_launch.h"
#include "santa_paged.cuh"
#include "santa_tma.cuh"

namespace santa {

namespace {

constexpr int NW = 4, NT = NW * 32;   // warps and threads per CTA

__device__ __forceinline__ uint32_t movm(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
template <typename T> struct Pack;
template <> struct Pack<bf16_t> {
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float2 unpack(uint32_t r) {
    return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
  }
};
template <> struct Pack<fp16_t> {
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float2 unpack(uint32_t r) {
    __half2 h;
    memcpy(&h, &r, 4);
    return __half22float2(h);
  }
};
// Two e4m3 codes (the low 16 bits) as fp16, exact.
__device__ __forceinline__ uint32_t widen8(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
// 16 bytes global -> shared, `bytes` of them read (0: zeros, nothing is read).
__device__ __forceinline__ void cp16z(uint32_t dst, const void* src, int bytes, unsigned long long pol) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes),
               "l"(pol)
               : "memory");
}

template <bool E4M3, int D>
struct Geom {
  static constexpr int ROWB = D * (E4M3 ? 1 : 2);      // bytes of a row
  static constexpr int CH = ROWB / 16;                 // its 16-byte chunks
  static constexpr int KB = PG_BLK * ROWB;             // a block of K (or V)
  static constexpr int STAGE = 2 * KB + (E4M3 ? 2 * PG_BLK * 4 : 0);
  // Stages per warp.  16-bit caches: 96 KiB of ring per CTA and two CTAs per
  // SM; e4m3, where more is computed per byte: 66 KiB and three.
  static constexpr int NS = KB >= 4096 ? 3 : !E4M3 ? 6 : KB >= 2048 ? 4 : 7;
  static constexpr int RING = NW * NS * STAGE;
  // offset of chunk c of row r in a block: eight rows at one chunk fall on
  // eight bank groups (128-byte lines, chunk index xor line number)
  static __device__ __forceinline__ uint32_t at(int r, int c) {
    if (ROWB == 256) return swz128_offset(r, c);
    if (ROWB == 128) return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
    const int line = r >> 1;
    return (uint32_t)(line * 128 + ((((r & 1) * 4 + c) ^ (line & 7)) << 4));
  }
  // at(r + j JROWS, c) from at(r, c), for r < JROWS, the rows that a warp's
  // copy covers: the line moves on, and the swizzle only in its higher bits.
  static constexpr int JROWS = 32 / CH;
  static __device__ __forceinline__ uint32_t at_next(uint32_t at0, int j) {
    return ROWB == 256 ? (at0 ^ (uint32_t)((2 * j & 7) << 4)) + 256u * j : (at0 ^ (uint32_t)((4 * j & 7) << 4)) + 512u * j;
  }
};

template <bool E4M3, int D, int R>
constexpr size_t smem_bytes() {
  const size_t ring = Geom<E4M3, D>::RING, merge = (size_t)NW * R * D * 4;
  return (ring > merge ? ring : merge) + 128;
}

// R: query rows per tile (8 or 16).
template <typename T, bool E4M3, int D, int R>
__global__ void __launch_bounds__(NT, E4M3 ? 3 : 2) paged_tokens_kernel(PagedArgs a) {
  using Gm = Geom<E4M3, D>;
  using M16 = typename std::conditional<E4M3, fp16_t, T>::type;   // the products' type
  constexpr int NS = Gm::NS, NB = R / 8;
  constexpr float BIAS = fp16_bias<M16>(TOKENS_BIAS);
  extern __shared__ __align__(128) unsigned char smem_raw[];
  __shared__ float s_m[NW][R], s_l[NW][R];
  __shared__ int s_bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g8 = lane >> 2, t4 = lane & 3;
  allow_dependents();

  // ---- which tile, which of its splits
  unsigned x = blockIdx.x;
  const int split = x % a.splits;
  x /= a.splits;
  const int kvh = x % a.Hkv;
  x /= a.Hkv;
  const int tile = x % a.tiles, b = x / a.tiles;
  const Seq s = paged_seq(a, b, tid == 0 && split == 0 && kvh == 0 && tile == 0);
  const int row0 = tile * R, nrows = min(R, s.n * a.G - row0);
  if (nrows <= 0) return;
  int i0, i1;
  tile_tokens(a, s.n, tile, i0, i1);
  const TileKeys tk = tile_keys(a, s, i0, i1, PG_BLK);
  const int splits = max(1, (tk.blk + a.split_blk - 1) / a.split_blk);
  if (split >= splits) return;
  const int blk0 = tk.blk_lo + split * a.split_blk;
  const int nblk = min(a.split_blk, tk.blk - split * a.split_blk);
  const int mine = nblk > warp ? (nblk - warp + NW - 1) / NW : 0;
  const int first_pos = s.kv - s.n;
  if (tid == 0) s_bad = 0;
  __syncthreads();

  // ---- the warp's ring
  const uint32_t ring = ((smem_addr(smem_raw) + 127u) & ~127u) + (uint32_t)(warp * NS * Gm::STAGE);
  const unsigned long long pol = evict_first_policy();
  const long long step = (long long)a.Hkv * Gm::ROWB;   // from row to row of a page
  const long long lane_off = lane / Gm::CH * step + lane % Gm::CH * 16;
  const uint32_t lane_at = Gm::at(lane / Gm::CH, lane % Gm::CH);
  uint32_t put = 0, get = 0;   // offsets of the next block's stage
  int pids = 0;        // lane l: page of the warp's block (k & ~31) + l
  auto issue = [&](int k) {
    if ((k & 31) == 0) {
      const int kk = k + lane;
      pids = 0;
      if (kk < mine) pids = a.table[(long long)b * a.max_pages + (((blk0 + warp + NW * kk) * PG_BLK) >> a.page_shift)];
    }
    const int pid = __shfl_sync(FULL, pids, k & 31);
    if (k < mine) {
      const bool ok = (unsigned)pid < (unsigned)a.n_pages;
      if (!ok && lane == 0) {
        s_bad = 1;
        flag_error(a.err, ERR_PAGE);
      }
      const int key0 = (blk0 + warp + NW * k) * PG_BLK;
      const int slot = key0 & ((1 << a.page_shift) - 1);
      const int live = ok ? min(PG_BLK, s.kv - key0) : 0;
      const long long row = ok ? ((long long)pid << a.page_shift) + slot : 0;
      const uint32_t dst = ring + put;
      const long long off = (row * a.Hkv + kvh) * Gm::ROWB;
      const unsigned char* kp = static_cast<const unsigned char*>(a.K) + off;
      const unsigned char* vp = static_cast<const unsigned char*>(a.V) + off;
      if (live == PG_BLK) {   // addresses by additions: 103.5 -> 102.9 us where HBM bounds, 39.9 -> 39.2 with 16 rows
        kp += lane_off;
        vp += lane_off;
#pragma unroll
        for (int j = 0; j < Gm::KB / 512; ++j) {
          const uint32_t to = dst + Gm::at_next(lane_at, j);
          cp_async16_hint(to, kp, pol);
          cp_async16_hint(to + Gm::KB, vp, pol);
          kp += Gm::JROWS * step;
          vp += Gm::JROWS * step;
        }
      } else {
#pragma unroll 1
        for (int j = 0; j < Gm::KB / 512; ++j) {
          const int q = lane + 32 * j, r = q / Gm::CH, c = q % Gm::CH;
          const long long o = r < live ? r * step + c * 16 : 0;
          cp16z(dst + Gm::at(r, c), kp + o, r < live ? 16 : 0, pol);
          cp16z(dst + Gm::KB + Gm::at(r, c), vp + o, r < live ? 16 : 0, pol);
        }
      }
      if (E4M3 && lane < 8) {
        const int i = (lane & 3) * 4;   // four scales; a row past the last key may hold anything
        const float* sp = (lane < 4 ? a.ks : a.vs) + ((((ok ? (long long)pid : 0) * a.Hkv) + kvh) << a.page_shift) + slot + i;
        cp16z(dst + 2 * Gm::KB + lane * 16, sp, max(0, min(16, (live - i) * 4)), pol);
      }
    }
    cp_async_commit();
    put = put + Gm::STAGE == NS * Gm::STAGE ? 0 : put + Gm::STAGE;
  };
#pragma unroll
  for (int k = 0; k < NS; ++k) issue(k);

  // ---- query fragments (the B operand: k = d, n = row); rows past the last read as zero
  const T* const qp = static_cast<const T*>(a.q);
  uint32_t bq[NB][D / 16][2];
  float sl[NB][2];      // score factor of rows 8 nb + 2 t4 + hh
  int lo_[NB][2], hi_[NB][2];   // the keys they see
  int lo_all = 0, hi_all = INT32_MAX;   // keys that every row sees
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int r = 8 * nb + g8, pr = row0 + r;
    const long long tok = s.q0 + pr / a.G;
    const uint32_t* q2 = reinterpret_cast<const uint32_t*>(qp + (tok * a.H + (long long)kvh * a.G + pr % a.G) * D);
    float mx = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      // 16-bit caches: d = 16 ks + 2 t4 (+1) and + 8; e4m3: d = 16 ks + 4 t4 (+1) and + 2 (see the K fragments)
      const int w0 = E4M3 ? 8 * ks + 2 * t4 : 8 * ks + t4, w1 = E4M3 ? w0 + 1 : w0 + 4;
      bq[nb][ks][0] = r < nrows ? __ldg(q2 + w0) : 0u;
      bq[nb][ks][1] = r < nrows ? __ldg(q2 + w1) : 0u;
      if (E4M3) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 f = Pack<T>::unpack(bq[nb][ks][e]);
          mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
    }
    float up = 1.f, down = 1.f;
    if (E4M3) {
      mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
      const int ex = (int)(__float_as_uint(mx) >> 23);   // biased exponent of the row's largest magnitude
      if (ex > 11 && ex < 255) {
        // 2^(137 - ex) in two factors' worth of range: both it and its inverse are normal floats for ex in 11 .. 254
        up = __uint_as_float((uint32_t)(127 + 10 + 127 - ex) << 23);
        down = __uint_as_float((uint32_t)(ex - 10) << 23);
      }
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 f = Pack<T>::unpack(bq[nb][ks][e]);
          bq[nb][ks][e] = Pack<M16>::pack(f.x * up, f.y * up);
        }
    }
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int rr = 8 * nb + 2 * t4 + hh;
      sl[nb][hh] = a.sl2 * __shfl_sync(FULL, down, (2 * t4 + hh) * 4);
      visible_keys(a, s.kv, first_pos + (row0 + min(rr, nrows - 1)) / a.G, lo_[nb][hh], hi_[nb][hh]);
      lo_all = max(lo_all, lo_[nb][hh]);
      hi_all = min(hi_all, hi_[nb][hh]);
    }
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo_all = max(lo_all, __shfl_xor_sync(FULL, lo_all, o));
    hi_all = min(hi_all, __shfl_xor_sync(FULL, hi_all, o));
  }

  // ---- the pass over the keys
  float rm[NB][2], rl[NB][2], oacc[NB][D / 16][4];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    rm[nb][0] = rm[nb][1] = -INFINITY;
    rl[nb][0] = rl[nb][1] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) oacc[nb][i][0] = oacc[nb][i][1] = oacc[nb][i][2] = oacc[nb][i][3] = 0.f;
  }
  const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8, lhalf = lane >> 4;        // K: matrices (rows 0-7, 8-15) x (chunk, next)
  const int vrow = (lane & 7) + ((lane >> 4) & 1) * 8, vhalf = (lane >> 3) & 1;  // 16-bit V^T
  // U blocks at a time: one maximum, one rescaling for all of their keys
  auto take = [&](auto blocks, int k) {
    constexpr int U = decltype(blocks)::value;
    cp_async_wait<NS - U>();
    __syncwarp();
    uint32_t kb[U];
    int key0[U];
    bool whole = true;   // every row sees every key; the same in every lane
#pragma unroll
    for (int u = 0; u < U; ++u) {
      kb[u] = ring + get;
      get = get + Gm::STAGE == NS * Gm::STAGE ? 0 : get + Gm::STAGE;
      key0[u] = (blk0 + warp + NW * (k + u)) * PG_BLK;
      whole &= key0[u] >= lo_all && key0[u] + PG_BLK <= hi_all;
    }
    float acc[U][NB][2][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) acc[u][nb][e][0] = acc[u][nb][e][1] = acc[u][nb][e][2] = acc[u][nb][e][3] = 0.f;
      if (E4M3) {
#pragma unroll
        for (int c = 0; c < D / 16; c += 2) {
          uint32_t f[4];
          ldmatrix_x4(kb[u] + Gm::at(lrow, c + lhalf), f);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t fa[4] = {widen8(f[2 * e]), widen8(f[2 * e + 1]), widen8(f[2 * e] >> 16), widen8(f[2 * e + 1] >> 16)};
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) Mma<M16>::run(acc[u][nb][e], fa, bq[nb][c + e][0], bq[nb][c + e][1]);
          }
        }
      } else {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t f[4];
          ldmatrix_x4(kb[u] + Gm::at(lrow, ks * 2 + lhalf), f);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) Mma<M16>::run(acc[u][nb][ks & 1], f, bq[nb][ks][0], bq[nb][ks][1]);
        }
      }
    }
    // a v_scale that is none makes the values NaN, not the softmax: vnan is added to its probabilities
    float ksc[U][2], lv[U][2], rv[U][2], vnan[U][2];
    if (E4M3) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float v;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(ksc[u][j]) : "r"(kb[u] + 2 * Gm::KB + (g8 + 8 * j) * 4));
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(kb[u] + 2 * Gm::KB + 64 + (g8 + 8 * j) * 4));
          vnan[u][j] = 0.f;
          if (odd_scale(v)) {
            vnan[u][j] = __int_as_float(0x7fffffff);
            v = 1.f;
          }
          v = fmaxf(v, V_SCALE_LEAST);
          asm("lg2.approx.f32 %0, %1;" : "=f"(lv[u][j]) : "f"(v));
          asm("rcp.approx.f32 %0, %1;" : "=f"(rv[u][j]) : "f"(v));
        }
    }
    float p[U][NB][2][2];   // [nb][key g8 + 8 j][row hh]
    float alpha[NB][2];
    auto softmax = [&](auto all) {
      constexpr bool ALL = decltype(all)::value;   // every row sees every key of the blocks
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          bool vis[U][2];
          float sc[U][2], m = -INFINITY;
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int key = key0[u] + g8 + 8 * j;
              vis[u][j] = ALL || (key >= lo_[nb][hh] && key < hi_[nb][hh]);
              const float v = (acc[u][nb][0][2 * j + hh] + acc[u][nb][1][2 * j + hh]) * sl[nb][hh];
              sc[u][j] = E4M3 ? fmaf(v, ksc[u][j], lv[u][j]) : v;
              if (!ALL && !vis[u][j]) sc[u][j] = -INFINITY;
              m = fmaxf(m, sc[u][j]);
            }
          m = fmaxf(m, __shfl_xor_sync(FULL, m, 4));
          m = fmaxf(m, __shfl_xor_sync(FULL, m, 8));
          m = fmaxf(m, __shfl_xor_sync(FULL, m, 16));
          const float mn = fmaxf(rm[nb][hh], m - BIAS), mu = mn > -INFINITY ? mn : 0.f;
          alpha[nb][hh] = fast_exp2(rm[nb][hh] - mu);
          rm[nb][hh] = mn;
          float sum = 0.f;
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float& pj = p[u][nb][j][hh];
              pj = ALL || vis[u][j] ? fast_exp2(sc[u][j] - mu) : 0.f;
              sum += E4M3 ? (ALL || vis[u][j] ? pj * rv[u][j] : 0.f) : pj;
              if (E4M3 && (ALL || vis[u][j])) pj += vnan[u][j];
            }
          rl[nb][hh] = fmaf(rl[nb][hh], alpha[nb][hh], sum);
        }
    };
    if (whole) softmax(std::true_type());
    else softmax(std::false_type());
    bool moved = false;   // most blocks leave the maxima where they are
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) moved |= alpha[nb][0] != 1.f || alpha[nb][1] != 1.f;
    if (__any_sync(FULL, moved)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            oacc[nb][i][hh] *= alpha[nb][hh];
            oacc[nb][i][2 + hh] *= alpha[nb][hh];
          }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t vb = kb[u] + Gm::KB;
      // A masked key's value is multiplied by zero below, which a NaN or an
      // infinity would survive: blocks that not every row sees in full are
      // looked over, and such a block is added up without the tensor cores.
      bool odd = false;
      if (!whole) {
#pragma unroll
        for (int j = 0; j < Gm::KB / 512; ++j) {
          const uint4 v = lds128(vb + (lane + 32 * j) * 16);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (E4M3) {
#pragma unroll
              for (int e = 0; e < 4; ++e) odd |= ((w[i] >> (8 * e)) & 0x7fu) == 0x7fu;
            } else {
              const uint32_t ex = std::is_same<T, bf16_t>::value ? 0x7f80u : 0x7c00u;
              odd |= (w[i] & ex) == ex || ((w[i] >> 16) & ex) == ex;
            }
          }
        }
        odd = __any_sync(FULL, odd);
      }
      if (odd) {
#pragma unroll 1
        for (int key = 0; key < PG_BLK; ++key) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const float pk = __shfl_sync(FULL, key & 8 ? p[u][nb][1][hh] : p[u][nb][0][hh], (key & 7) * 4 + t4);
              if (key0[u] + key < lo_[nb][hh] || key0[u] + key >= hi_[nb][hh]) continue;
#pragma unroll
              for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  float v;
                  if (E4M3) {
                    uint32_t byte;
                    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(byte) : "r"(vb + Gm::at(key, i) + 2 * g8 + e));
                    v = Pack<fp16_t>::unpack(widen8(byte)).x;
                  } else {
                    const int d = 16 * i + g8 + 8 * e;
                    uint16_t hw;
                    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(hw) : "r"(vb + Gm::at(key, d >> 3) + (d & 7) * 2));
                    v = Pack<T>::unpack(hw).x;
                  }
                  oacc[nb][i][2 * e + hh] = fmaf(pk, v, oacc[nb][i][2 * e + hh]);
                }
            }
        }
        continue;
      }
      // P^T as the B operand (k = key, n = row); over 16-bit caches and for
      // tiles of eight rows split into a 16-bit head and the rounding of the
      // rest, which that HBM-bound loop has room for (with 16 rows it cost 6 %)
      constexpr bool REST = !E4M3 && R == 8;
      uint32_t ph[NB][2], pl[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t h = Pack<M16>::pack(p[u][nb][j][0], p[u][nb][j][1]);
          ph[nb][j] = movm(h);
          if (REST) {
            const float2 back = Pack<M16>::unpack(h);
            pl[nb][j] = movm(Pack<M16>::pack(p[u][nb][j][0] - back.x, p[u][nb][j][1] - back.y));
          }
        }
      if (E4M3) {
#pragma unroll
        for (int c = 0; c < D / 16; c += 2) {
          // matrices (keys 0-7, 8-15) x (chunk c, c + 1), transposed in pairs
          // of codes: a register holds d = 16 c + 2 g8 (+1) of keys 2 t4 (+1)
          uint32_t f[4];
          ldsm4_trans(vb + Gm::at(lrow, c + lhalf), f);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t lo = __byte_perm(f[2 * e], 0, 0x3120), hi = __byte_perm(f[2 * e + 1], 0, 0x3120);
            const uint32_t fa[4] = {widen8(lo), widen8(lo >> 16), widen8(hi), widen8(hi >> 16)};
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) Mma<M16>::run(oacc[nb][c + e], fa, ph[nb][0], ph[nb][1]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t f[4];
          ldsm4_trans(vb + Gm::at(vrow, 2 * i + vhalf), f);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            Mma<M16>::run(oacc[nb][i], f, ph[nb][0], ph[nb][1]);
            if (REST) Mma<M16>::run(oacc[nb][i], f, pl[nb][0], pl[nb][1]);
          }
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < U; ++u) issue(k + NS + u);   // into the stages that these blocks leave
  };
  // Two at a time over e4m3 with tiles of eight rows, whose loop is bound by
  // the latency of its instructions and has the registers (two sequences of
  // 131072 keys 100.0 -> 98.9 us, one of 32768 17.8 -> 16.7); with 16 rows it
  // would spill, and in 16 bits HBM bounds.
  constexpr int U = E4M3 && R == 8 ? 2 : 1;
  int k = 0;
#pragma unroll 1
  for (; k + U <= mine; k += U) take(std::integral_constant<int, U>(), k);
  if (U > 1 && k < mine) take(std::integral_constant<int, 1>(), k);
  cp_async_wait_all();

  // ---- the warps' partials, merged in shared memory (over the rings)
  __syncthreads();
  float* const s_o = reinterpret_cast<float*>(smem_raw + ((128u - (smem_addr(smem_raw) & 127u)) & 127u));   // [NW][R][D]
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      float l = rl[nb][hh];
      l += __shfl_xor_sync(FULL, l, 4);
      l += __shfl_xor_sync(FULL, l, 8);
      l += __shfl_xor_sync(FULL, l, 16);
      const int r = 8 * nb + 2 * t4 + hh;
      if (g8 == 0) {
        s_m[warp][r] = rm[nb][hh];
        s_l[warp][r] = l;
      }
      float* po = s_o + (warp * R + r) * D;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const int d = 16 * i + (E4M3 ? 2 * g8 : g8);
        po[d] = oacc[nb][i][hh];
        po[d + (E4M3 ? 1 : 8)] = oacc[nb][i][2 + hh];
      }
    }
  __syncthreads();
  const bool bad = s_bad != 0;
  const long long part = ((((long long)b * a.tiles + tile) * a.Hkv + kvh) * a.splits + split) * R;
  for (int i = tid; i < nrows * (D / 4); i += NT) {
    const int r = i / (D / 4), d = i % (D / 4) * 4;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) m = fmaxf(m, s_m[w][r]);
    const float mu = m > -INFINITY ? m : 0.f;
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = fast_exp2(s_m[w][r] - mu);
      const float4 y = *reinterpret_cast<const float4*>(s_o + (w * R + r) * D + d);
      l = fmaf(s_l[w][r], f, l);
      o.x = fmaf(y.x, f, o.x);
      o.y = fmaf(y.y, f, o.y);
      o.z = fmaf(y.z, f, o.z);
      o.w = fmaf(y.w, f, o.w);
    }
    if (splits == 1) {
      const float inv = bad || l == 0.f ? 0.f : __fdividef(1.f, l);
      const int pr = row0 + r;
      const long long at = (s.q0 + pr / a.G) * a.H + (long long)kvh * a.G + pr % a.G;
      uint2 w;
      w.x = bad || l == 0.f ? 0u : Pack<T>::pack(o.x * inv, o.y * inv);
      w.y = bad || l == 0.f ? 0u : Pack<T>::pack(o.z * inv, o.w * inv);
      *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + at * D + d) = w;
      if (a.lse && d == 0) a.lse[at] = bad || l == 0.f ? -INFINITY : log_sum(m, l, BIAS);
    } else {
      *reinterpret_cast<float4*>(a.part_o + (part + r) * D + d) = o;
      if (d == 0) {
        a.part_ml[2 * (part + r)] = m;
        a.part_ml[2 * (part + r) + 1] = bad ? -1.f : l;   // a sum is never negative: the mark of a bad page
      }
    }
  }
}

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
size_t plan_paged_tokens(PagedArgs& a) {
  a.rows = a.max_q * a.G <= 8 ? 8 : 16;
  a.tokens = 0;
  a.tiles = (int)(((long long)a.max_q * a.G + a.rows - 1) / a.rows);
  const long long pieces = (long long)a.B * a.Hkv * a.tiles;
  const int span = a.window ? (int)std::min<long long>(a.nk, (long long)a.window + a.max_q) : a.nk;
  const int blks = (span + PG_BLK - 1) / PG_BLK + (a.window ? 1 : 0);
  const long long places = 2ll * a.num_sms;
  long long want = std::max<long long>(1, places / pieces);
  const long long fine = std::min<long long>(4 * places / pieces, blks / 64);
  if (2 * fine * pieces >= 3 * places) want = std::max(want, fine);
  a.split_blk = (int)std::max<long long>(NW, (blks + want - 1) / want);
  a.splits = (blks + a.split_blk - 1) / a.split_blk;
  return a.splits == 1 ? 0 : (size_t)pieces * a.splits;
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
