// santa_diff_tokens.cu -- differential heads over a paged cache for few query
// rows per pair of KV heads (single tokens, a handful of proposed ones).
//
// As the kernel of santa_tokens.cuh, whose notes on rings, fragments and e4m3
// hold here, with both heads of a pair at once: S_e^T = K_e q_e^T for the first
// and the second map (e = 0, 1), a running softmax of each, and O_e^T +=
// [V_0 V_1]^T P_e^T, so that every K and V row is read once; HBM bounds it.  A
// block is 16 keys of four heads; a tile is eight query rows of each map, or,
// where a sequence has no more than four of them (PACK), four of each, which
// then share the eight columns of a product: half the exponentials and products
// with V.  The sums of the two maps stay apart (their difference is taken where
// all pieces of a row are known, in santa_join.cu).  Over an e4m3 cache the two
// value heads' scales differ, so each map has a maximum and probabilities for
// each.
//
// Measured: 16 sequences of 1024 to 32768 keys, 28 and 4 heads of 128, fp16: 102
// us, 5.5 TB/s (0.82 of a copy's rate; CTAs' starts and ends, the join 8 us);
// two of 131072 over e4m3, 32 and 8 heads: 107 us, 4.9 TB/s (142 with each map
// in columns of its own: bound by its instructions); one token over 1000 keys
// 8.3 us, two launches and their chains of look-ups.
#include <type_traits>

#include "santa_join.cuh"
#include "santa_tokens.cuh"

namespace santa {

namespace {

// Stages are large, and CTAs start, merge and end: with one CTA of four warps
// per SM and three stages a warp, 16 sequences of 1024 to 32768 keys took 119 us,
// with two of two warps 109, with two of three warps and two stages 102.
template <bool E4M3, int D>
struct DiffGeom {
  using Gm = Geom<E4M3, D>;
  static constexpr int STAGE = 4 * Gm::KB + (E4M3 ? 4 * PG_BLK * 4 : 0);   // K_0, K_1, V_0, V_1, their scales
  static constexpr int WARPS = STAGE >= 16384 ? 3 : 4;                     // of a CTA
  static constexpr int NS = STAGE >= 16384 ? 2 : STAGE >= 8192 ? 3 : 6;    // stages per warp
  static constexpr int CTAS = 2;                                           // per SM
  static constexpr int RING = WARPS * NS * STAGE, THREADS = WARPS * 32;
  static constexpr int SMEM = RING + 128;
};
static_assert(DiffGeom<true, 128>::WARPS * 16 * 256 * 4 <= DiffGeom<true, 128>::RING && DiffGeom<true, 64>::WARPS * 16 * 128 * 4 <= DiffGeom<true, 64>::RING, "the merge lies over the rings");

template <typename T, bool E4M3, int D, bool PACK>
__device__ __forceinline__ void diff_tokens(const JoinArgs& a, unsigned x, bool behind) {
  using Gm = Geom<E4M3, D>;
  using Dg = DiffGeom<E4M3, D>;
  using M16 = typename std::conditional<E4M3, fp16_t, T>::type;
  constexpr int NW = Dg::WARPS, NT = Dg::THREADS, NS = Dg::NS, R = PACK ? 4 : 8, NB = PACK ? 1 : 2, F = E4M3 ? 2 : 1, NI = 2 * D / 16, W = 2 * D;   // F: maxima of a map
  constexpr float BIAS = fp16_bias<M16>(TOKENS_BIAS);
  extern __shared__ __align__(128) unsigned char smem_raw[];
  __shared__ float s_m[NW][2][R][F], s_l[NW][2][R][F];
  __shared__ int s_bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g8 = lane >> 2, t4 = lane & 3;
  allow_dependents();
  auto done = [&] {   // not over before the pass that it may have started under
    if (behind) wait_for_predecessor();
  };

  // ---- which tile, which of its splits
  const int split = x % a.splits;
  x /= a.splits;
  const int pair = x % a.heads;
  x /= a.heads;
  const int tile = x % a.tiles, b = x / a.tiles;
  const Seq s = paged_seq(a, b, tid == 0 && split == 0 && pair == 0 && tile == 0);
  const int row0 = tile * R, nrows = min(R, s.n * a.G - row0);
  if (nrows <= 0) return done();
  int i0, i1;
  tile_tokens(a, s.n, tile, i0, i1);
  const TileKeys tk = tile_keys(a, s, i0, i1, PG_BLK);
  const int32_t* const pages = page_row(a, b);
  const int splits = max(1, (tk.blk + a.split_blk - 1) / a.split_blk);
  if (split >= splits) return done();
  const int blk0 = tk.blk_lo + split * a.split_blk;
  const int nblk = min(a.split_blk, tk.blk - split * a.split_blk);
  const int mine = nblk > warp ? (nblk - warp + NW - 1) / NW : 0;
  const int first_pos = s.kv - s.n;
  if (tid == 0) s_bad = 0;
  __syncthreads();

  // ---- the warp's ring
  const uint32_t ring = ((smem_addr(smem_raw) + 127u) & ~127u) + (uint32_t)(warp * NS * Dg::STAGE);
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
      if (kk < mine) pids = pages[((blk0 + warp + NW * kk) * PG_BLK) >> a.page_shift];
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
      const long long off = (row * a.Hkv + 2 * pair) * Gm::ROWB;
      const unsigned char* kp = static_cast<const unsigned char*>(a.K) + off;
      const unsigned char* vp = static_cast<const unsigned char*>(a.V) + off;
      if (live == PG_BLK) {
        kp += lane_off;
        vp += lane_off;
#pragma unroll
        for (int j = 0; j < Gm::KB / 512; ++j) {
          const uint32_t to = dst + Gm::at_next(lane_at, j);
          cp_async16_hint(to, kp, pol);
          cp_async16_hint(to + Gm::KB, kp + Gm::ROWB, pol);
          cp_async16_hint(to + 2 * Gm::KB, vp, pol);
          cp_async16_hint(to + 3 * Gm::KB, vp + Gm::ROWB, pol);
          kp += Gm::JROWS * step;
          vp += Gm::JROWS * step;
        }
      } else {
#pragma unroll 1
        for (int j = 0; j < Gm::KB / 512; ++j) {
          const int q = lane + 32 * j, r = q / Gm::CH, c = q % Gm::CH, bytes = r < live ? 16 : 0;
          const long long o = r < live ? r * step + c * 16 : 0;
          const uint32_t to = dst + Gm::at(r, c);
          cp16z(to, kp + o, bytes, pol);
          cp16z(to + Gm::KB, kp + o + Gm::ROWB, bytes, pol);
          cp16z(to + 2 * Gm::KB, vp + o, bytes, pol);
          cp16z(to + 3 * Gm::KB, vp + o + Gm::ROWB, bytes, pol);
        }
      }
      if (E4M3 && lane < 16) {
        const int i = (lane & 3) * 4, head = 2 * pair + ((lane >> 2) & 1);   // four scales; a row past the last key may hold anything
        const float* sp = (lane < 8 ? a.ks : a.vs) + ((((ok ? (long long)pid : 0) * a.Hkv) + head) << a.page_shift) + slot + i;
        cp16z(dst + 4 * Gm::KB + lane * 16, sp, max(0, min(16, (live - i) * 4)), pol);
      }
    }
    cp_async_commit();
    put = put + Dg::STAGE == NS * Dg::STAGE ? 0 : put + Dg::STAGE;
  };
#pragma unroll
  for (int k = 0; k < NS; ++k) issue(k);

  // ---- query fragments of both maps; rows past the last read as zero
  const T* const qp = static_cast<const T*>(a.q);
  // columns of the products: 8 nb + c is row c of map nb, or row c % 4 of map c / 4
  uint32_t bq[NB][D / 16][2];
  float sl[NB][2];     // score factor of columns 2 t4 + hh
  int lo_[2], hi_[2];  // the keys they see
  int lo_all = 0, hi_all = INT32_MAX;   // keys that every row sees
  {
    const int pr = row0 + g8 % R;
    const bool there = g8 % R < nrows;
    const long long tok = s.q0 + pr / a.G;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int e = PACK ? g8 / 4 : nb;
      const uint32_t* q2 = reinterpret_cast<const uint32_t*>(qp + (tok * a.H + 2 * ((long long)pair * a.G + pr % a.G) + e) * D);
      float mx = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const int w0 = E4M3 ? 8 * ks + 2 * t4 : 8 * ks + t4, w1 = E4M3 ? w0 + 1 : w0 + 4;
        bq[nb][ks][0] = there ? __ldg(q2 + w0) : 0u;
        bq[nb][ks][1] = there ? __ldg(q2 + w1) : 0u;
        if (E4M3) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 f = Pack<T>::unpack(bq[nb][ks][i]);
            mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
      }
      float up = 1.f, down = 1.f;
      if (E4M3) {
        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
        const int ex = (int)(__float_as_uint(mx) >> 23);
        if (ex > 11 && ex < 255) {
          up = __uint_as_float((uint32_t)(127 + 10 + 127 - ex) << 23);
          down = __uint_as_float((uint32_t)(ex - 10) << 23);
        }
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 f = Pack<T>::unpack(bq[nb][ks][i]);
            bq[nb][ks][i] = Pack<M16>::pack(f.x * up, f.y * up);
          }
      }
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) sl[nb][hh] = a.sl2 * __shfl_sync(FULL, down, (2 * t4 + hh) * 4);
    }
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      visible_keys(a, s, first_pos + (row0 + min((2 * t4 + hh) % R, nrows - 1)) / a.G, lo_[hh], hi_[hh]);
      lo_all = max(lo_all, lo_[hh]);
      hi_all = min(hi_all, hi_[hh]);
    }
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo_all = max(lo_all, __shfl_xor_sync(FULL, lo_all, o));
    hi_all = min(hi_all, __shfl_xor_sync(FULL, hi_all, o));
  }

  // ---- the pass over the keys
  float rm[NB][F][2], rl[NB][F][2], oacc[NB][NI][4];
#pragma unroll
  for (int e = 0; e < NB; ++e) {
#pragma unroll
    for (int f = 0; f < F; ++f) {
      rm[e][f][0] = rm[e][f][1] = -INFINITY;
      rl[e][f][0] = rl[e][f][1] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) oacc[e][i][0] = oacc[e][i][1] = oacc[e][i][2] = oacc[e][i][3] = 0.f;
  }
  const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8, lhalf = lane >> 4;        // K: matrices (rows 0-7, 8-15) x (chunk, next)
  const int vrow = (lane & 7) + ((lane >> 4) & 1) * 8, vhalf = (lane >> 3) & 1;  // 16-bit V^T
#pragma unroll 1
  for (int k = 0; k < mine; ++k) {
    cp_async_wait<NS - 1>();
    __syncwarp();
    const uint32_t kb = ring + get, vb = kb + 2 * Gm::KB, sc = kb + 4 * Gm::KB;
    get = get + Dg::STAGE == NS * Dg::STAGE ? 0 : get + Dg::STAGE;
    const int key0 = (blk0 + warp + NW * k) * PG_BLK;
    const bool whole = key0 >= lo_all && key0 + PG_BLK <= hi_all;   // every row sees every key; the same in every lane
    float lv[2][2], rv[2][2], vnan[2][2];   // [value head][key g8 + 8 j]
    if (E4M3) {
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float v;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(sc + 128 + 64 * f + (g8 + 8 * j) * 4));
          vnan[f][j] = 0.f;
          if (odd_scale(v)) {
            vnan[f][j] = __int_as_float(0x7fffffff);
            v = 1.f;
          }
          v = fmaxf(v, V_SCALE_LEAST);
          asm("lg2.approx.f32 %0, %1;" : "=f"(lv[f][j]) : "f"(v));
          asm("rcp.approx.f32 %0, %1;" : "=f"(rv[f][j]) : "f"(v));
        }
    }
    float p[NB][F][2][2];   // [columns][maximum][key g8 + 8 j][column hh]
    float alpha[NB][F][2];
    bool moved = false;     // most blocks leave the maxima where they are
    float acc[2][2][4];
    const bool second = t4 >> 1;   // PACK: the lane's columns are the second map's
#pragma unroll
    for (int e = 0; e < 2; ++e) {   // scores with K_e; PACK: of all columns, half of which are taken
      const int nb = PACK ? 0 : e;
      const uint32_t ke = kb + e * Gm::KB;
#pragma unroll
      for (int i = 0; i < 2; ++i) acc[e][i][0] = acc[e][i][1] = acc[e][i][2] = acc[e][i][3] = 0.f;
      if (E4M3) {
#pragma unroll
        for (int c = 0; c < D / 16; c += 2) {
          uint32_t f[4];
          ldmatrix_x4(ke + Gm::at(lrow, c + lhalf), f);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t fa[4] = {widen8(f[2 * i]), widen8(f[2 * i + 1]), widen8(f[2 * i] >> 16), widen8(f[2 * i + 1] >> 16)};
            Mma<M16>::run(acc[e][i], fa, bq[nb][c + i][0], bq[nb][c + i][1]);
          }
        }
      } else {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t f[4];
          ldmatrix_x4(ke + Gm::at(lrow, ks * 2 + lhalf), f);
          Mma<M16>::run(acc[e][ks & 1], f, bq[nb][ks][0], bq[nb][ks][1]);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < NB; ++e) {
      float ksc[2] = {1.f, 1.f};
      if (E4M3) {
#pragma unroll
        for (int j = 0; j < 2; ++j) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(ksc[j]) : "r"(sc + 64 * (PACK ? (int)second : e) + (g8 + 8 * j) * 4));
      }
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          bool vis[2];
          float y[2], m = -INFINITY;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int key = key0 + g8 + 8 * j;
            vis[j] = whole || (key >= lo_[hh] && key < hi_[hh]);
            const float v0 = acc[e][0][2 * j + hh] + acc[e][1][2 * j + hh], v1 = acc[1][0][2 * j + hh] + acc[1][1][2 * j + hh];
            const float v = (PACK && second ? v1 : v0) * sl[e][hh];
            y[j] = E4M3 ? fmaf(v, ksc[j], lv[f][j]) : v;
            if (!vis[j]) y[j] = -INFINITY;
            m = fmaxf(m, y[j]);
          }
          m = fmaxf(m, __shfl_xor_sync(FULL, m, 4));
          m = fmaxf(m, __shfl_xor_sync(FULL, m, 8));
          m = fmaxf(m, __shfl_xor_sync(FULL, m, 16));
          const float mn = fmaxf(rm[e][f][hh], m - BIAS), mu = mn > -INFINITY ? mn : 0.f;
          alpha[e][f][hh] = fast_exp2(rm[e][f][hh] - mu);
          moved |= alpha[e][f][hh] != 1.f;
          rm[e][f][hh] = mn;
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float& pj = p[e][f][j][hh];
            pj = vis[j] ? fast_exp2(y[j] - mu) : 0.f;
            sum += E4M3 ? (vis[j] ? pj * rv[f][j] : 0.f) : pj;
            if (E4M3 && vis[j]) pj += vnan[f][j];
          }
          rl[e][f][hh] = fmaf(rl[e][f][hh], alpha[e][f][hh], sum);
        }
    }
    if (__any_sync(FULL, moved)) {
#pragma unroll
      for (int e = 0; e < NB; ++e)
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            oacc[e][i][hh] *= alpha[e][F == 2 ? i / (NI / 2) : 0][hh];
            oacc[e][i][2 + hh] *= alpha[e][F == 2 ? i / (NI / 2) : 0][hh];
          }
    }
    // A masked key's value is multiplied by zero below, which a NaN or an
    // infinity would survive: blocks that not every row sees in full are
    // looked over, and such a block is added up without the tensor cores.
    bool odd = false;
    if (!whole) {
#pragma unroll 1
      for (int j = 0; j < 2 * Gm::KB / 512; ++j) {
        const uint4 v = lds128(vb + (lane + 32 * j) * 16);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (E4M3) {
#pragma unroll
            for (int q = 0; q < 4; ++q) odd |= ((w[i] >> (8 * q)) & 0x7fu) == 0x7fu;
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
        for (int e = 0; e < NB; ++e)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            float pk[F];
#pragma unroll
            for (int f = 0; f < F; ++f) pk[f] = __shfl_sync(FULL, key & 8 ? p[e][f][1][hh] : p[e][f][0][hh], (key & 7) * 4 + t4);
            if (key0 + key < lo_[hh] || key0 + key >= hi_[hh]) continue;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
              const int f = i / (NI / 2), c = i % (NI / 2);
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                float v;
                if (E4M3) {
                  uint32_t byte;
                  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(byte) : "r"(vb + f * Gm::KB + Gm::at(key, c) + 2 * g8 + q));
                  v = Pack<fp16_t>::unpack(widen8(byte)).x;
                } else {
                  const int d = 16 * c + g8 + 8 * q;
                  uint16_t hw;
                  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(hw) : "r"(vb + f * Gm::KB + Gm::at(key, d >> 3) + (d & 7) * 2));
                  v = Pack<T>::unpack(hw).x;
                }
                oacc[e][i][2 * q + hh] = fmaf(pk[F == 2 ? f : 0], v, oacc[e][i][2 * q + hh]);
              }
            }
          }
      }
      __syncwarp();
      issue(k + NS);
      continue;
    }
    // P^T as the B operand (k = key, n = row); over 16-bit caches split into a
    // 16-bit head and the rounding of the rest: the difference of the maps
    // leaves less of the result than of its rounding
    constexpr bool REST = !E4M3;
    uint32_t ph[NB][F][2], pl[NB][2];
#pragma unroll
    for (int e = 0; e < NB; ++e)
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t h = Pack<M16>::pack(p[e][f][j][0], p[e][f][j][1]);
          ph[e][f][j] = movm(h);
          if (REST) {
            const float2 back = Pack<M16>::unpack(h);
            pl[e][j] = movm(Pack<M16>::pack(p[e][f][j][0] - back.x, p[e][f][j][1] - back.y));
          }
        }
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const uint32_t vf = vb + f * Gm::KB;
      if (E4M3) {
#pragma unroll
        for (int c = 0; c < D / 16; c += 2) {
          uint32_t x4[4];
          ldsm4_trans(vf + Gm::at(lrow, c + lhalf), x4);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t lo = __byte_perm(x4[2 * i], 0, 0x3120), hi = __byte_perm(x4[2 * i + 1], 0, 0x3120);
            const uint32_t fa[4] = {widen8(lo), widen8(lo >> 16), widen8(hi), widen8(hi >> 16)};
#pragma unroll
            for (int e = 0; e < NB; ++e) Mma<M16>::run(oacc[e][f * (NI / 2) + c + i], fa, ph[e][F - 1 ? f : 0][0], ph[e][F - 1 ? f : 0][1]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t x4[4];
          ldsm4_trans(vf + Gm::at(vrow, 2 * i + vhalf), x4);
#pragma unroll
          for (int e = 0; e < NB; ++e) {
            Mma<M16>::run(oacc[e][f * (NI / 2) + i], x4, ph[e][0][0], ph[e][0][1]);
            if (REST) Mma<M16>::run(oacc[e][f * (NI / 2) + i], x4, pl[e][0], pl[e][1]);
          }
        }
      }
    }
    __syncwarp();
    issue(k + NS);   // into the stage that this block leaves
  }
  cp_async_wait_all();

  // ---- the warps' partials, merged in shared memory (over the rings)
  __syncthreads();
  float* const s_o = reinterpret_cast<float*>(smem_raw + ((128u - (smem_addr(smem_raw) & 127u)) & 127u));   // [NW][2][R][W]
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int r = (2 * t4 + hh) % R, e = PACK ? t4 >> 1 : nb;
#pragma unroll
      for (int f = 0; f < F; ++f) {
        float l = rl[nb][f][hh];
        l += __shfl_xor_sync(FULL, l, 4);
        l += __shfl_xor_sync(FULL, l, 8);
        l += __shfl_xor_sync(FULL, l, 16);
        if (g8 == 0) {
          s_m[warp][e][r][f] = rm[nb][f][hh];
          s_l[warp][e][r][f] = l;
        }
      }
      float* po = s_o + ((warp * 2 + e) * R + r) * W;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int d = 16 * i + (E4M3 ? 2 * g8 : g8);
        po[d] = oacc[nb][i][hh];
        po[d + (E4M3 ? 1 : 8)] = oacc[nb][i][2 + hh];
      }
    }
  __syncthreads();
  const bool bad = s_bad != 0;
  const long long part = ((((long long)b * a.tiles + tile) * a.heads + pair) * a.splits + split) * 2 * R;
  for (int i = tid; i < 2 * nrows * (W / 4); i += NT) {
    const int d = i % (W / 4) * 4, er = i / (W / 4), e = er >= nrows, r = er - e * nrows, f = F == 2 ? d / D : 0;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) m = fmaxf(m, s_m[w][e][r][f]);
    const float mu = m > -INFINITY ? m : 0.f;
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float g = fast_exp2(s_m[w][e][r][f] - mu);
      const float4 y = *reinterpret_cast<const float4*>(s_o + ((w * 2 + e) * R + r) * W + d);
      l = fmaf(s_l[w][e][r][f], g, l);
      o.x = fmaf(y.x, g, o.x);
      o.y = fmaf(y.y, g, o.y);
      o.z = fmaf(y.z, g, o.z);
      o.w = fmaf(y.w, g, o.w);
    }
    const long long at = part + e * R + r;
    *reinterpret_cast<float4*>(a.part_o + at * W + d) = o;
    if (d == f * D) {
      float* const ml = a.part_ml + (at * F + f) * 2;
      ml[0] = m;
      ml[1] = bad ? -1.f : l;   // a sum is never negative: the mark of a bad page
    }
  }
  done();
}

template <typename T, bool E4M3, int D, bool PACK>
__global__ void __launch_bounds__(DiffGeom<E4M3, D>::THREADS, DiffGeom<E4M3, D>::CTAS) diff_tokens_kernel(const __grid_constant__ JoinArgs a) {
  diff_tokens<T, E4M3, D, PACK>(a, blockIdx.x, blockIdx.x == 0);
}
// Both passes, `first` CTAs of the one over the prefixes.
template <typename T, bool E4M3, int D, bool PACK>
__global__ void __launch_bounds__(DiffGeom<E4M3, D>::THREADS, DiffGeom<E4M3, D>::CTAS) diff_both_kernel(const __grid_constant__ Passes p, unsigned first) {
  if (blockIdx.x < first) diff_tokens<T, E4M3, D, false>(p.p[0], blockIdx.x, false);
  else diff_tokens<T, E4M3, D, PACK>(p.p[1], blockIdx.x - first, false);
}

template <typename T, bool E4M3, int D, bool PACK>
cudaError_t inst(const JoinArgs* p, const JoinArgs& a, bool behind) {
  constexpr int smem = DiffGeom<E4M3, D>::SMEM;
  const void* const kern = p ? (const void*)diff_both_kernel<T, E4M3, D, PACK> : (const void*)diff_tokens_kernel<T, E4M3, D, PACK>;
  static std::atomic<unsigned long long> raised[2] = {{0}, {0}};
  const cudaError_t e = raise_smem(kern, smem, raised[p != nullptr]);
  if (e != cudaSuccess) return e;
  if (!p) return launch_pass(diff_tokens_kernel<T, E4M3, D, PACK>, (unsigned)tokens_grid(a), DiffGeom<E4M3, D>::THREADS, smem, a.stream, behind, a);
  const unsigned first = (unsigned)tokens_grid(*p);
  return launch_pass(diff_both_kernel<T, E4M3, D, PACK>, first + (unsigned)tokens_grid(a), DiffGeom<E4M3, D>::THREADS, smem, a.stream, false, Passes{{*p, a}}, first);
}
template <typename T, bool E4M3, int D>
cudaError_t rows(const JoinArgs* p, const JoinArgs& a, bool behind) {
  return a.rows == 4 ? inst<T, E4M3, D, true>(p, a, behind) : inst<T, E4M3, D, false>(p, a, behind);
}
template <typename T>
cudaError_t type(const JoinArgs* p, const JoinArgs& a, bool behind) {
  if (a.D == 128) return a.e4m3 ? rows<T, true, 128>(p, a, behind) : rows<T, false, 128>(p, a, behind);
  return a.e4m3 ? rows<T, true, 64>(p, a, behind) : rows<T, false, 64>(p, a, behind);
}

}  // namespace

void plan_diff_tokens(JoinArgs& a, int span, int more_blocks) {
  a.rows = a.phase != 1 && (long long)a.max_q * a.G <= 4 ? 4 : 8;   // a group has more rows than its sequences
  a.tokens = 0;
  a.tiles = (int)(((long long)a.max_q * a.G + a.rows - 1) / a.rows);
  const int blks = (span + PG_BLK - 1) / PG_BLK + more_blocks;
  plan_splits(a, (long long)a.B * (a.Hkv / 2) * a.tiles, 2ll * a.num_sms, blks, blks + 32);
}

cudaError_t launch_diff_tokens(const JoinArgs* prefixes, const JoinArgs& a, bool behind) {
  return a.dtype == 0 ? type<bf16_t>(prefixes, a, behind) : type<fp16_t>(prefixes, a, behind);
}

}  // namespace santa
