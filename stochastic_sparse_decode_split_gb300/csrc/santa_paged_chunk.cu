// santa_paged_chunk.cu -- exact attention of a chunk of new tokens over a paged
// cache: both products on the fifth-generation tensor cores, sums in tensor
// memory.
//
// A CTA takes two tiles of 128 query rows of one sequence and KV head (the
// group's heads of consecutive tokens: a K or V row in shared memory serves
// all of them) and the key blocks, 128 keys each, of its split.  With 256 rows
// per 64 KiB of K and V the products bound the kernel, then the exponentials,
// then the L2; HBM does not.  Roles, one CTA per SM:
//   warps 0-3, 4-7  softmax of tile 0 and 1: one thread per row.  S comes out
//                   of tensor memory, P goes back over it in 16 bits, the sum
//                   O is rescaled only when the maximum has grown by 2^8
//                   (probabilities stay below 256, the result is the same)
//   warp 8          issues the products: S_t = Q_t K^T and O_t += P_t V, so
//                   that one tile's products run during the other's softmax
//   warp 9          TMA: pages of K and V into two stages each (128-byte swizzle)
//   warps 10, 11    16-bit caches: V rows past the last key become zeros, and
//                   in blocks that not every row sees NaN and infinities, whose
//                   product with a masked probability would not be zero, are
//                   taken out and given back at the end to the rows that see them
//   warps 12-15     e4m3 caches: codes widen to fp16 in place (TMA brings them
//                   into the stage's upper half); the scales are staged beside
// Order of the products: S of block j + 1 is issued after O += P V of block j
// of the same tile and overwrites the columns P was read from; products issued
// by one thread execute in order.  That S is complete therefore says that the
// previous O is too, which is when the softmax may rescale O.
#include <algorithm>
#include <cstring>
#include <mutex>
#include <type_traits>

#include <cudaTypedefs.h>

#include "santa_launch.h"
#include "santa_paged.cuh"
#include "santa_tcgen05.cuh"

namespace santa {

namespace {

constexpr int BKEYS = PG_CHUNK_KEYS;   // keys per block
constexpr int TROWS = 128;             // rows per tile (lanes of tensor memory)
constexpr float RESCALE = 8.f;         // growth of the maximum (base 2) that O is rescaled for
constexpr unsigned long long WAIT_NS = 1000000000ull;

template <bool E4M3, int D>
struct ChunkGeom {
  static constexpr int THREADS = E4M3 ? 512 : 384;
  static constexpr int HALF = TROWS * 128;              // 128 rows x 64 elements of 16 bits
  static constexpr int TILE = HALF * (D / 64);          // a tile of Q, a block of K or V
  static constexpr int OFF_K = 2 * TILE, OFF_V = OFF_K + 2 * TILE, OFF_SC = OFF_V + 2 * TILE;
  static constexpr int SC_STAGE = 3 * BKEYS * 4;        // k_scale, log2 v_scale, 1 / v_scale
  static constexpr int BYTES = OFF_SC + (E4M3 ? 4 * SC_STAGE : 0);
  static constexpr size_t SMEM = BYTES + 1024;
};

// Barriers.
enum { Q_FULL, Q_READY, K_FULL, K_READY = K_FULL + 2, K_EMPTY = K_READY + 2, V_FULL = K_EMPTY + 2, V_READY = V_FULL + 2,
       V_EMPTY = V_READY + 2, S_FULL = V_EMPTY + 2, P_FULL = S_FULL + 2, O_DONE = P_FULL + 2, N_BAR = O_DONE + 2 };

// Waits for a phase, for a second at most; after one wait has run out in the
// CTA (`dead`), no other waits.
__device__ __forceinline__ void wait_phase(uint32_t bar, unsigned parity, int* err, volatile int* dead) {
  if (mbar_try_wait(bar, parity)) return;
  const unsigned long long t0 = global_ns();
  for (;;) {
    if (mbar_try_wait(bar, parity)) return;
    if (*dead) return;
    if (global_ns() - t0 > WAIT_NS) break;
  }
  *dead = 1;
  flag_error(err, ERR_TIMEOUT);
}

template <typename T> __device__ __forceinline__ uint32_t pack2h(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2h<bf16_t>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <> __device__ __forceinline__ uint32_t pack2h<fp16_t>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <typename T> __device__ __forceinline__ float2 unpack2h(uint32_t r);
template <> __device__ __forceinline__ float2 unpack2h<bf16_t>(uint32_t r) {
  return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 unpack2h<fp16_t>(uint32_t r) {
  __half2 h;
  memcpy(&h, &r, 4);
  return __half22float2(h);
}
__device__ __forceinline__ f2x add2(f2x a, f2x b) {
  f2x d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2x mul2(f2x a, f2x b) {
  f2x d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void tma_load_hint(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"((uint64_t)tm), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// NaN or infinity among the eight 16-bit elements of a chunk.
template <typename T>
__device__ __forceinline__ bool odd16(const uint4& v) {
  const uint32_t ex = std::is_same<T, bf16_t>::value ? 0x7f80u : 0x7c00u;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  bool odd = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) odd |= (w[i] & ex) == ex || ((w[i] >> 16) & ex) == ex;
  return odd;
}
template <typename T>
__device__ __forceinline__ uint32_t without_odd16(uint32_t w) {
  const uint32_t ex = std::is_same<T, bf16_t>::value ? 0x7f80u : 0x7c00u;
  if ((w & ex) == ex) w &= 0xffff0000u;
  if (((w >> 16) & ex) == ex) w &= 0xffffu;
  return w;
}

// T: type of q and out; the products' type is T, or fp16 over an e4m3 cache.
template <typename T, bool E4M3, int D>
__global__ void __launch_bounds__(ChunkGeom<E4M3, D>::THREADS, 1)
paged_chunk_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, PagedArgs a) {
  using Gm = ChunkGeom<E4M3, D>;
  using M16 = typename std::conditional<E4M3, fp16_t, T>::type;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) unsigned long long s_bar[N_BAR];
  __shared__ uint32_t s_tm;
  __shared__ int s_dead, s_bad, s_odd;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  allow_dependents();

  // ---- which pair of tiles, which split (tiles fastest: the CTAs that run
  // together share K and V in the L2; a causal chunk's last, longest, first)
  unsigned x = blockIdx.x;
  const int tile = a.tiles - 1 - (int)(x % a.tiles);
  x /= a.tiles;
  const int split = x % a.splits;
  x /= a.splits;
  const int kvh = x % a.Hkv, b = x / a.Hkv;
  const Seq s = paged_seq(a, b, tid == 0 && split == 0 && kvh == 0 && tile == 0);
  const int per = TROWS / a.G;                       // tokens per tile of 128 rows
  const int tok0 = tile * a.tokens;
  if (tok0 >= s.n) return;
  int i0, i1;
  tile_tokens(a, s.n, tile, i0, i1);
  const TileKeys tk = tile_keys(a, s, i0, i1, BKEYS);
  if (split >= tk.splits) return;
  const int blk0 = tk.blk_lo + split * a.split_blk;
  const int nblk = min(a.split_blk, tk.blk - split * a.split_blk);
  const int first_pos = s.kv - s.n;
  const bool two = tok0 + per < s.n;                 // the second tile holds tokens

  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_addr(s_bar);
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  if (tid == 0) {
    s_dead = s_bad = s_odd = 0;
    for (int i = 0; i < N_BAR; ++i) {
      const int count = i == Q_READY ? (two ? 8 : 4)
                        : i == K_READY || i == K_READY + 1 ? 4
                        : i == V_READY || i == V_READY + 1 ? (E4M3 ? 4 : 2)
                        : i == P_FULL || i == P_FULL + 1 ? 4 : 1;
      mbar_init(bar(i), (unsigned)count);
    }
    mbar_fence_init();
  }
  if (warp == 8) tm_alloc(smem_addr(&s_tm), 512);
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tm = s_tm;
  volatile int* const dead = &s_dead;
  const uint32_t tmS = tm, tmO = tm + 256;           // tile t: S (and P) at 128 t, O at 256 + 128 t

  if (warp >= 8) {
    // registers: 256 x 208 + 128 x 88 of the launch's 384 x 168, 256 x 176 + 256 x 80 of 512 x 128
    if (E4M3) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8) {
      // -------------------------------------------------------- the products
      if (lane == 0 && nblk > 0) {
        constexpr uint32_t shS = mma_shape(std::is_same<M16, bf16_t>::value, BKEYS, false);
        constexpr uint32_t shO = mma_shape(std::is_same<M16, bf16_t>::value, D, true);
        auto product_s = [&](int t, int st) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t o = (uint32_t)((k >> 2) * Gm::HALF + (k & 3) * 32);
            mma_ss(tmS + 128 * t, smem_operand(base + t * Gm::TILE + o, 16),
                   smem_operand(base + Gm::OFF_K + st * Gm::TILE + o, 16), shS, k != 0);
          }
          mma_commit(bar(S_FULL + t));
        };
        auto product_o = [&](int t, int st, bool add) {
#pragma unroll
          for (int k = 0; k < BKEYS / 16; ++k)
            mma_ts(tmO + 128 * t, tmS + 128 * t + 8 * k, smem_operand(base + Gm::OFF_V + st * Gm::TILE + k * 2048, Gm::HALF),
                   shO, add || k != 0);
        };
        wait_phase(bar(E4M3 ? Q_READY : Q_FULL), 0, a.err, dead);
        wait_phase(bar(E4M3 ? K_READY : K_FULL), 0, a.err, dead);
        tm_fence_after();
        product_s(0, 0);
        if (two) product_s(1, 0);
        mma_commit(bar(K_EMPTY));
        for (int j = 0; j < nblk; ++j) {
          const int st = j & 1, nx = (j + 1) & 1;
          wait_phase(bar(V_READY + st), (j >> 1) & 1, a.err, dead);
          wait_phase(bar(P_FULL), j & 1, a.err, dead);
          tm_fence_after();
          product_o(0, st, j > 0);
          if (j + 1 < nblk) {
            wait_phase(bar((E4M3 ? K_READY : K_FULL) + nx), ((j + 1) >> 1) & 1, a.err, dead);
            tm_fence_after();
            product_s(0, nx);
          }
          if (two) {
            wait_phase(bar(P_FULL + 1), j & 1, a.err, dead);
            tm_fence_after();
            product_o(1, st, j > 0);
          }
          mma_commit(bar(V_EMPTY + st));
          if (j + 1 < nblk) {
            if (two) product_s(1, nx);
            mma_commit(bar(K_EMPTY + nx));
          }
        }
        mma_commit(bar(O_DONE));
        wait_phase(bar(O_DONE), 0, a.err, dead);     // nothing of it is in flight when the CTA ends
      }
      __syncwarp();
    } else if (warp == 9) {
      // ------------------------------------------------------------- the TMA
      const int rows = min(1 << a.page_shift, BKEYS);      // rows per box
      const int boxes = BKEYS / rows;
      constexpr int ROWB = E4M3 ? D : 2 * D;
      if (nblk > 0) {
        if (lane == 0) {
          prefetch_tensormap(&tmK);
          prefetch_tensormap(&tmV);
          // the last token's box may reach past q, where it reads zeros
          mbar_expect_tx(bar(Q_FULL), (unsigned)((two ? 2 : 1) * per * a.G * 2 * D));
          for (int t = 0; t < (two ? 2 : 1); ++t)
            for (int h = 0; h < D / 64; ++h)
              tma_load_hint(base + t * Gm::TILE + h * Gm::HALF, &tmQ, 64 * h, kvh * a.G, (int)(s.q0 + tok0 + t * per),
                            bar(Q_FULL));
        }
        const int32_t* const table = a.table + (long long)b * a.max_pages;
        int next = 0;
        auto page_of = [&](int j) {   // lane l: page of box l of block j (-1: no key there)
          const int key = (blk0 + j) * BKEYS + lane * rows;
          return j < nblk && lane < boxes && key < s.kv ? table[key >> a.page_shift] : INT32_MIN;
        };
        next = page_of(0);
        for (int j = 0; j < nblk; ++j) {
          const int pid = next, st = j & 1;
          next = page_of(j + 1);
          const int key0 = (blk0 + j) * BKEYS;
          const bool ok = pid != INT32_MIN && (unsigned)pid < (unsigned)a.n_pages;
          if (pid != INT32_MIN && !ok) {
            s_bad = 1;
            flag_error(a.err, ERR_PAGE);
          }
          const unsigned bytes = (unsigned)__popc(__ballot_sync(FULL, ok)) * (unsigned)(rows * ROWB);
          const int row = ok ? (pid << a.page_shift) + ((key0 + lane * rows) & ((1 << a.page_shift) - 1)) : 0;
          if (j > 1) wait_phase(bar(K_EMPTY + st), ((j >> 1) - 1) & 1, a.err, dead);
          const uint32_t kd = base + Gm::OFF_K + st * Gm::TILE, vd = base + Gm::OFF_V + st * Gm::TILE;
          if (lane == 0) mbar_expect_tx(bar(K_FULL + st), bytes);
          __syncwarp();
          if (ok) {
            if (E4M3) {
              tma_load_hint(kd + Gm::TILE / 2 + lane * rows * D, &tmK, 0, kvh, row, bar(K_FULL + st));
            } else {
#pragma unroll
              for (int h = 0; h < D / 64; ++h)
                tma_load_hint(kd + h * Gm::HALF + lane * rows * 128, &tmK, 64 * h, kvh, row, bar(K_FULL + st));
            }
          }
          if (j > 1) wait_phase(bar(V_EMPTY + st), ((j >> 1) - 1) & 1, a.err, dead);
          if (lane == 0) mbar_expect_tx(bar(V_FULL + st), bytes);
          __syncwarp();
          if (ok) {
            if (E4M3) {
              tma_load_hint(vd + Gm::TILE / 2 + lane * rows * D, &tmV, 0, kvh, row, bar(V_FULL + st));
            } else {
#pragma unroll
              for (int h = 0; h < D / 64; ++h)
                tma_load_hint(vd + h * Gm::HALF + lane * rows * 128, &tmV, 64 * h, kvh, row, bar(V_FULL + st));
            }
          }
        }
        // the copies are over before the CTA ends, also where a wait ran out
        for (int j = max(0, nblk - 2); j < nblk; ++j) {
          wait_phase(bar(K_FULL + (j & 1)), (j >> 1) & 1, a.err, dead);
          wait_phase(bar(V_FULL + (j & 1)), (j >> 1) & 1, a.err, dead);
        }
        if (*dead)
          for (int i = 0; i < 1000; ++i) __nanosleep(1000);
      }
    } else if (!E4M3 && warp < 12) {
      // ------------------------------------- V: rows past the end, odd values
      int lo0, hi0, lo1, hi1;
      visible_keys(a, s.kv, first_pos + i0, lo0, hi0);
      visible_keys(a, s.kv, first_pos + i1, lo1, hi1);
      for (int j = 0; j < nblk; ++j) {
        const int st = j & 1, key0 = (blk0 + j) * BKEYS, live = min(BKEYS, s.kv - key0);
        wait_phase(bar(V_FULL + st), (j >> 1) & 1, a.err, dead);
        if (key0 < lo1 || key0 + BKEYS > hi0) {
          const uint32_t vd = base + Gm::OFF_V + st * Gm::TILE;
          bool found = false;
          for (int i = tid - 320; i < Gm::TILE / 16; i += 64) {
            const int r = (i >> 3) & (TROWS - 1);   // chunk i of the tile lies in row r of its half
            if (r >= live) {
              sts128(vd + i * 16, make_uint4(0u, 0u, 0u, 0u));
            } else {
              uint4 v = lds128(vd + i * 16);
              if (odd16<T>(v)) {
                v = make_uint4(without_odd16<T>(v.x), without_odd16<T>(v.y), without_odd16<T>(v.z), without_odd16<T>(v.w));
                sts128(vd + i * 16, v);
                found = true;
              }
            }
          }
          if (found) s_odd = 1;
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(V_READY + st));
      }
    } else if (E4M3 && warp >= 12) {
      // ------------------------------------------------- e4m3 codes to fp16
      const int ct = tid - 384;                       // 0 .. 127
      constexpr int CPR = D / 16, PASS = BKEYS * CPR / 128;   // 16-byte chunks of a row; chunks per thread
      const int32_t* const table = a.table + (long long)b * a.max_pages;
      for (int i = 0; i < 2 * nblk; ++i) {
        const int j = i >> 1, st = j & 1, key0 = (blk0 + j) * BKEYS, live = min(BKEYS, s.kv - key0);
        const bool is_v = i & 1;
        if (!is_v) {   // this thread's key's scales, on their way while the codes arrive
          const int key = key0 + ct;
          float ksc = 0.f, vsc = 1.f;
          if (ct < live) {
            const int pid = table[key >> a.page_shift];
            if ((unsigned)pid < (unsigned)a.n_pages) {
              const long long at = ((((long long)pid * a.Hkv) + kvh) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
              ksc = __ldg(a.ks + at);
              vsc = __ldg(a.vs + at);
            }
          }
          if (!(vsc <= 3.402823466e38f)) {   // the values are NaN, the softmax is not: given back at the end
            s_odd = 1;
            vsc = 1.f;
          }
          float lv, rv;
          asm("lg2.approx.f32 %0, %1;" : "=f"(lv) : "f"(vsc));
          asm("rcp.approx.f32 %0, %1;" : "=f"(rv) : "f"(vsc));
          const uint32_t sc = base + Gm::OFF_SC + (j & 3) * Gm::SC_STAGE + ct * 4;
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(sc), "f"(ksc) : "memory");
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(sc + BKEYS * 4), "f"(lv) : "memory");
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(sc + 2 * BKEYS * 4), "f"(rv) : "memory");
        }
        const uint32_t dst = base + (is_v ? Gm::OFF_V : Gm::OFF_K) + st * Gm::TILE, src = dst + Gm::TILE / 2;
        wait_phase(bar((is_v ? V_FULL : K_FULL) + st), (j >> 1) & 1, a.err, dead);
        uint4 w[PASS];
#pragma unroll
        for (int p = 0; p < PASS; ++p) w[p] = lds128(src + (ct + 128 * p) * 16);
        group_sync(1, 128);
#pragma unroll
        for (int p = 0; p < PASS; ++p) {
          const int c = (ct + 128 * p) % CPR, r = (ct + 128 * p) / CPR;
          uint32_t word[4] = {w[p].x, w[p].y, w[p].z, w[p].w}, h[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (r >= live) word[e] = 0u;
            if (is_v) {
              const uint32_t nan = ((word[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
              if (nan) {   // NaN codes come back at the end, too
                s_odd = 1;
                word[e] &= ~((nan >> 7) * 0xffu);
              }
            }
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[2 * e]) : "h"((uint16_t)word[e]));
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[2 * e + 1]) : "h"((uint16_t)(word[e] >> 16)));
          }
          // chunks 2c and 2c + 1 of the row; the upper half's lanes store them
          // the other way round, off the lower half's banks
          const uint32_t row = dst + (uint32_t)((c >> 2) * Gm::HALF + r * 128);
          const int c0 = (2 * c) & 7, swap = (c >> 2) & 1;
          const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
          sts128(row + (((c0 + swap) ^ (r & 7)) << 4), swap ? hi : lo);
          sts128(row + (((c0 + 1 - swap) ^ (r & 7)) << 4), swap ? lo : hi);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar((is_v ? V_READY : K_READY) + st));
      }
    }
  } else {
    // -------------------------------------------------------------- softmax
    if (E4M3) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int t = warp >> 2, row = tid & 127;
    if (t == 0 || two) {
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t mS = tmS + 128 * t + lanes, mO = tmO + 128 * t + lanes;
      const int ta = tok0 + t * per, tb = min(ta + per, s.n) - 1;   // the tile's tokens
      const int tok = min(ta + row / a.G, tb);                      // rows past the last compute it again, for nothing
      const bool live_row = row < per * a.G && ta + row / a.G <= tb;
      int lo, hi, lo_last, hi_last, lo_first, hi_first;
      visible_keys(a, s.kv, first_pos + tok, lo, hi);
      visible_keys(a, s.kv, first_pos + ta, lo_first, hi_first);
      visible_keys(a, s.kv, first_pos + tb, lo_last, hi_last);
      float sl = a.sl2;
      if (E4M3 && nblk > 0) {
        // the row of q in fp16 under a power of two (see santa_paged_tokens.cu)
        wait_phase(bar(Q_FULL), 0, a.err, dead);
        const uint32_t qr = base + t * Gm::TILE + row * 128;
        float mx = 0.f;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = lds128(qr + (c >> 3) * Gm::HALF + (((c & 7) ^ (row & 7)) << 4));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpack2h<T>(w[e]);
            mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
        float up = 1.f;
        const int ex = (int)(__float_as_uint(mx) >> 23);
        if (ex > 11 && ex < 255) {
          up = __uint_as_float((uint32_t)(264 - ex) << 23);
          sl *= __uint_as_float((uint32_t)(ex - 10) << 23);
        }
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint32_t at = qr + (c >> 3) * Gm::HALF + (((c & 7) ^ (row & 7)) << 4);
          const uint4 v = lds128(at);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpack2h<T>(w[e]);
            o[e] = pack2h<fp16_t>(f.x * up, f.y * up);
          }
          sts128(at, make_uint4(o[0], o[1], o[2], o[3]));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Q_READY));
      }
      float m = -INFINITY;          // the maximum that P and O are relative to
      f2x l2 = pack2(0.f, 0.f);
      for (int j = 0; j < nblk; ++j) {
        const int key0 = (blk0 + j) * BKEYS;
        wait_phase(bar(S_FULL + t), j & 1, a.err, dead);
        tm_fence_after();
        uint32_t sr[BKEYS];
#pragma unroll
        for (int c = 0; c < BKEYS; c += 32) tm_ld32(mS + c, sr + c);
        tm_wait_ld();
        if (E4M3) {
          const uint32_t sc = base + Gm::OFF_SC + (j & 3) * Gm::SC_STAGE;
          const f2x sl_2 = pack2(sl, sl);
#pragma unroll
          for (int c = 0; c < BKEYS; c += 4) {
            const uint4 k4 = lds128(sc + c * 4), v4 = lds128(sc + (BKEYS + c) * 4);
            f2x y0 = mul2(pack2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), sl_2);
            f2x y1 = mul2(pack2(__uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3])), sl_2);
            y0 = ffma2(y0, pack2(__uint_as_float(k4.x), __uint_as_float(k4.y)), pack2(__uint_as_float(v4.x), __uint_as_float(v4.y)));
            y1 = ffma2(y1, pack2(__uint_as_float(k4.z), __uint_as_float(k4.w)), pack2(__uint_as_float(v4.z), __uint_as_float(v4.w)));
            const float2 f0 = unpack2(y0), f1 = unpack2(y1);
            sr[c] = __float_as_uint(f0.x);
            sr[c + 1] = __float_as_uint(f0.y);
            sr[c + 2] = __float_as_uint(f1.x);
            sr[c + 3] = __float_as_uint(f1.y);
          }
        }
        if (key0 < lo_last || key0 + BKEYS > hi_first) {
          const int c0 = lo - key0, cn = hi - lo;
#pragma unroll
          for (int c = 0; c < BKEYS; ++c)
            if ((unsigned)(c - c0) >= (unsigned)cn) sr[c] = 0xff800000u;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < BKEYS; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mx[e] = fmaxf(fmaxf(mx[e], __uint_as_float(sr[c + 2 * e])), __uint_as_float(sr[c + 2 * e + 1]));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * (E4M3 ? 1.f : sl);
        const float mn = fmaxf(m, top);
        if (j == 0) {
          m = mn;
        } else if (__any_sync(FULL, mn > m + RESCALE)) {
          const float f = fast_exp2(m - (mn > -INFINITY ? mn : 0.f));
          m = mn;
          const float2 l = unpack2(l2);
          l2 = pack2(l.x * f, l.y * f);
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tm_ld32(mO + c, o);
            tm_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tm_st32(mO + c, o);
          }
        }
        const float neg = m > -INFINITY ? -m : 0.f;
        const f2x neg2 = pack2(neg, neg), sl_2 = pack2(sl, sl);
        const uint32_t sc = base + Gm::OFF_SC + (j & 3) * Gm::SC_STAGE + 2 * BKEYS * 4;
#pragma unroll
        for (int c = 0; c < BKEYS; c += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            f2x y0 = pack2(__uint_as_float(sr[c + e]), __uint_as_float(sr[c + e + 1]));
            f2x y1 = pack2(__uint_as_float(sr[c + e + 2]), __uint_as_float(sr[c + e + 3]));
            y0 = E4M3 ? add2(y0, neg2) : ffma2(y0, sl_2, neg2);
            y1 = E4M3 ? add2(y1, neg2) : ffma2(y1, sl_2, neg2);
            const float2 f0 = unpack2(y0), f1 = unpack2(y1);
            const float p0 = fast_exp2(f0.x), p1 = fast_exp2(f0.y), p2 = fast_exp2(f1.x), p3 = fast_exp2(f1.y);
            if (E4M3) {
              const uint4 r4 = lds128(sc + (c + e) * 4);
              l2 = ffma2(pack2(p0, p1), pack2(__uint_as_float(r4.x), __uint_as_float(r4.y)), l2);
              l2 = ffma2(pack2(p2, p3), pack2(__uint_as_float(r4.z), __uint_as_float(r4.w)), l2);
            } else {
              l2 = add2(l2, pack2(p0, p1));
              l2 = add2(l2, pack2(p2, p3));
            }
            pk[e / 2] = pack2h<M16>(p0, p1);
            pk[e / 2 + 1] = pack2h<M16>(p2, p3);
          }
          tm_st16(mS + c / 2, pk);
        }
        tm_wait_st();
        tm_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(P_FULL + t));
      }
      // ------------------------------------------------------- the result
      if (nblk > 0) {
        wait_phase(bar(O_DONE), 0, a.err, dead);
        tm_fence_after();
      }
      const float2 lp = unpack2(l2);
      const float l = lp.x + lp.y;
      const bool bad = s_bad != 0, odd = s_odd != 0, empty = bad || l == 0.f;
      const long long at = (s.q0 + tok) * a.H + (long long)kvh * a.G + row % a.G;
      const long long part = ((((long long)b * a.tiles + tile) * a.Hkv + kvh) * a.splits + split) * a.rows + t * TROWS + row;
      const bool whole = tk.splits == 1;
      const float inv = whole && !empty ? __fdividef(1.f, l) : 1.f;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        if (nblk > 0) {
          tm_ld32(mO + c, o);
          tm_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        float f[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(o[e]) * inv;
        if (odd && live_row) {
          // what was taken out of V, to the rows that see its key
          for (int key = max(lo, blk0 * BKEYS); key < min(hi, (blk0 + nblk) * BKEYS); ++key) {
            const int pid = a.table[(long long)b * a.max_pages + (key >> a.page_shift)];
            if ((unsigned)pid >= (unsigned)a.n_pages) continue;
            const int slot = key & ((1 << a.page_shift) - 1);
            const long long vr = (((long long)pid << a.page_shift) + slot) * a.Hkv + kvh;
            if (E4M3) {
              const float sc = a.vs[((((long long)pid * a.Hkv) + kvh) << a.page_shift) + slot];
              const unsigned char* v = static_cast<const unsigned char*>(a.V) + vr * D + c;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(sc <= 3.402823466e38f) || (v[e] & 0x7f) == 0x7f) f[e] = __int_as_float(0x7fffffff);
            } else {
              const uint32_t* v = reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.V) + vr * D + c);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float2 y = unpack2h<T>(v[e]);
                if (!(fabsf(y.x) <= 3.402823466e38f)) f[2 * e] += y.x;
                if (!(fabsf(y.y) <= 3.402823466e38f)) f[2 * e + 1] += y.y;
              }
            }
          }
        }
        if (live_row) {
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + at * D + c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint4 w;
              w.x = empty ? 0u : pack2h<T>(f[8 * e], f[8 * e + 1]);
              w.y = empty ? 0u : pack2h<T>(f[8 * e + 2], f[8 * e + 3]);
              w.z = empty ? 0u : pack2h<T>(f[8 * e + 4], f[8 * e + 5]);
              w.w = empty ? 0u : pack2h<T>(f[8 * e + 6], f[8 * e + 7]);
              dst[e] = w;
            }
          } else {
            float4* dst = reinterpret_cast<float4*>(a.part_o + part * D + c);
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
          }
        }
      }
      if (live_row) {
        if (!whole) {
          a.part_ml[2 * part] = m;
          a.part_ml[2 * part + 1] = bad ? -1.f : l;
        } else if (a.lse) {
          a.lse[at] = empty ? -INFINITY : m * 0.6931471805599453f + __logf(l);
        }
      }
    }
    tm_fence_before();
  }
  __syncthreads();
  if (warp == 8) {
    tm_fence_after();
    tm_free(tm, 512);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// A [rows, heads, d] array as a three-dimensional tensor, boxes of bx x by x bz.
bool encode(CUtensorMap* tm, const void* base, int es, int d, int heads, long long rows, int bx, int by, int bz) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)d * es, (cuuint64_t)heads * d * es};
  const cuuint32_t box[3] = {(cuuint32_t)bx, (cuuint32_t)by, (cuuint32_t)bz}, one[3] = {1, 1, 1};
  return enc(tm, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims,
             strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, es == 2 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, bool E4M3, int D>
cudaError_t chunk_inst(const PagedArgs& a) {
  using Gm = ChunkGeom<E4M3, D>;
  auto kern = paged_chunk_kernel<T, E4M3, D>;
  static std::atomic<unsigned long long> raised{0};
  const cudaError_t e = raise_smem((const void*)kern, (int)Gm::SMEM, raised);
  if (e != cudaSuccess) return e;
  const int rows = std::min(1 << a.page_shift, BKEYS);
  const long long pool = (long long)a.n_pages << a.page_shift;
  CUtensorMap tq, tk, tv;
  memset(&tq, 0, sizeof tq);
  memset(&tk, 0, sizeof tk);
  memset(&tv, 0, sizeof tv);
  constexpr int es = E4M3 ? 1 : 2, bx = E4M3 ? D : 64;
  if (!encode(&tq, a.q, 2, D, a.H, a.total_q, 64, a.G, TROWS / a.G) || !encode(&tk, a.K, es, D, a.Hkv, pool, bx, 1, rows) ||
      !encode(&tv, a.V, es, D, a.Hkv, pool, bx, 1, rows))
    return cudaErrorInvalidValue;
  kern<<<(unsigned)((long long)a.B * a.Hkv * a.splits * a.tiles), Gm::THREADS, Gm::SMEM, a.stream>>>(tq, tk, tv, a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t chunk_type(const PagedArgs& a) {
  if (a.D == 128) return a.e4m3 ? chunk_inst<T, true, 128>(a) : chunk_inst<T, false, 128>(a);
  return a.e4m3 ? chunk_inst<T, true, 64>(a) : chunk_inst<T, false, 64>(a);
}

}  // namespace

// Splits: the fewest blocks of keys that one SM works through one after
// another, a CTA's start and end counted as 4 blocks and those of a split,
// whose sums go through memory, as 12 (128 KiB out and in again).
void plan_paged_chunk(PagedArgs& a) {
  const int per = TROWS / a.G;
  a.rows = 2 * TROWS;
  a.tokens = 2 * per;
  a.tiles = (a.max_q + a.tokens - 1) / a.tokens;
  const long long items = (long long)a.B * a.Hkv * a.tiles;
  const int span = a.window ? (int)std::min<long long>(a.nk, (long long)a.window + a.tokens) : a.nk;
  const int blks = (span + BKEYS - 1) / BKEYS + (a.window ? 1 : 0);
  long long best = -1;
  for (int n = 1; n <= std::min(blks, 64); ++n) {
    const int each = (blks + n - 1) / n;
    const long long waves = (items * n + a.num_sms - 1) / a.num_sms, cost = waves * (each + (n > 1 ? 12 : 4));
    if (best < 0 || cost < best) {
      best = cost;
      a.split_blk = each;
    }
  }
  a.splits = (blks + a.split_blk - 1) / a.split_blk;
}

cudaError_t launch_paged_chunk(const PagedArgs& a) {
  return a.dtype == 0 ? chunk_type<bf16_t>(a) : chunk_type<fp16_t>(a);
}

}  // namespace santa
