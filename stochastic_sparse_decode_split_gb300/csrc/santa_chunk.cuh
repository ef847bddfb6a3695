// santa_chunk.cuh -- exact attention of a chunk of new tokens over a paged cache,
// the kernel: both products on the fifth-generation tensor cores, sums in tensor
// memory.
//
// An item is two tiles of 128 query rows of one sequence and KV head (the
// group's heads of consecutive tokens: a K or V row in shared memory serves
// all of them) against its keys, in blocks of 128.  With 256 rows per 64 KiB
// of K and V the products bound the kernel, then the exponentials, then the
// L2; HBM does not.  One CTA per SM; each takes an equal share of the blocks
// of the whole batch, counted from the lengths on the device, so a CTA's share
// may begin or end inside an item, whose sums then go through memory
// (santa_chunk_share.cuh has the division).  Roles:
//   warps 0-3, 4-7  softmax of tile 0 and 1: one thread per row.  S comes out
//                   of tensor memory, P goes back over it in 16 bits, the sum
//                   O is rescaled only when the maximum has grown by 2^8
//                   (probabilities stay within a factor of 256, the result is the same)
//   warp 8          issues the products: S_t = Q_t K^T and O_t += P_t V, so
//                   that one tile's products run during the other's softmax
//   warp 9          TMA: pages of K and V into two stages each (128-byte swizzle).
//                   A box is a page's rows of 128 bytes, and what the unit can
//                   take is 70 cycles a box of 16 rows: bringing later blocks
//                   into the L2 beside it cost more than it gave (with
//                   pages of 16, 1500 tokens of heads of 64 267 -> 214 us
//                   without; of 64, 2048 tokens at 32768 keys 780 -> 761)
//   warps 10, 11    16-bit caches: V rows past the last key (and, behind a prefix,
//                   before the pass's first) become zeros, and
//                   in blocks that not every row sees NaN and infinities, whose
//                   product with a masked probability would not be zero, are
//                   taken out and given back at the end to the rows that see them
//   warps 12-15     e4m3 caches: codes widen to fp16 in place (TMA brings them
//                   into the stage's upper half); the scales are staged beside
// An item whose second tile is empty (few tokens) gives its blocks to the two
// softmax groups in turn, with a sum O each, joined at the end.
//
// A job is one tile (or, of such an item, one group) and one block.  Order of
// the products: S of job k + 2 is issued after O += P V of job k, whose P it
// overwrites; products issued by one thread execute in order.  That S is
// complete therefore says that the O of the same tile is too, which is when
// the softmax may rescale it.
//
// Measured: 2048 tokens at 32768 keys, 32 and 8 heads of 128, bf16: 745 to 774
// us, 1.37 to 1.43 PFLOP/s (0.72 to 0.75 of a library product's rate; the clock
// falls from 1.86 to 1.74 GHz as the tensor cores fill); six chunks of up to 700
// tokens over e4m3 in a window of 4096: 181 us, where for a tile softmax, issue
// of the products and hand-overs follow one another, the other tile in between
// (K left in e4m3, for products of that kind with q as a sum of two or three
// such values, took as long).
#pragma once

#include <algorithm>
#include <cstring>
#include <type_traits>

#include <cudaTypedefs.h>

#include "santa_chunk_share.cuh"
#include "santa_join.cuh"
#include "santa_launch.h"
#include "santa_paged.cuh"
#include "santa_tcgen05.cuh"

namespace santa {

namespace {

constexpr int TROWS = CHUNK_ROWS;           // rows per tile (lanes of tensor memory)
constexpr float RESCALE = 8.f;         // growth of the maximum (base 2) that O is rescaled for
constexpr unsigned long long WAIT_NS = 1000000000ull;

// D: elements of a head; DV: columns of V per item.
template <bool E4M3, int D, int DV = D, bool DIFF = false>
struct ChunkGeom {
  static constexpr int THREADS = E4M3 ? 512 : 384;
  static constexpr int HALF = TROWS * 128;              // 128 rows x 64 elements of 16 bits
  static constexpr int TILE = HALF * (D / 64);          // a tile of Q, a block of K
  static constexpr int VTILE = HALF * (DV / 64);        // a block of V
  static constexpr int OFF_K = 2 * TILE, OFF_V = OFF_K + 2 * TILE, OFF_SC = OFF_V + 2 * VTILE;
  static constexpr int SC_STAGE = (DIFF ? 4 : 3) * BKEYS * 4;   // k_scale, log2 v_scale, 1 / v_scale, the second k_scale
  static constexpr int BYTES = OFF_SC + (E4M3 ? 4 * SC_STAGE : 0);
  static constexpr size_t SMEM = BYTES + 1024;
};

// Columns of V that an item has (see the kernel).
template <bool E4M3, int D, bool DIFF> __host__ __device__ constexpr int diff_columns() { return DIFF && !E4M3 ? 128 : D; }

// Barriers.
enum { Q_FULL, Q_READY, K_FULL, K_READY = K_FULL + 2, K_EMPTY = K_READY + 2, V_FULL = K_EMPTY + 2, V_READY = V_FULL + 2,
       V_EMPTY = V_READY + 2, S_FULL = V_EMPTY + 2, P_FULL = S_FULL + 2, O_FREE = P_FULL + 2, O_DONE = O_FREE + 2, ML_FULL,
       Q_SEEN, PIECE_SEEN, N_BAR };

// Whether a phase is over, without waiting.
__device__ __forceinline__ bool test_phase(uint32_t bar, unsigned parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok)
               : "r"(bar), "r"(parity)
               : "memory");
  return ok != 0;
}

// Waits for a phase, for a second at most; after one wait has run out in the
// CTA (`dead`), no other waits.
__device__ __forceinline__ void wait_phase(uint32_t bar, unsigned parity, int* err, volatile int* dead) {
  if (test_phase(bar, parity)) return;   // 40 cycles; the waiting form takes more also where there is nothing to wait for
  unsigned long long t0 = 0;
  for (unsigned i = 0;; ++i) {
    if (mbar_try_wait(bar, parity)) return;
    if (i % 64 == 63) {
      if (*dead) return;
      if (t0 == 0) t0 = global_ns();
      else if (global_ns() - t0 > WAIT_NS) break;
    }
  }
  *dead = 1;
  flag_error(err, ERR_TIMEOUT);
}
// A value that is the same in every lane, in a register that the compiler
// knows to be uniform (loops and addresses that depend on it then are, too).
__device__ __forceinline__ unsigned uniform(unsigned x) { return __reduce_max_sync(FULL, x); }

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
// Two e4m3 codes (the low 16 bits) as fp16, exact.
__device__ __forceinline__ uint32_t widen8(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
// 32 bytes, 32-byte aligned.
__device__ __forceinline__ void st_global8(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"((uint64_t)tm), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load4(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"((uint64_t)tm), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
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

__device__ __forceinline__ int scan_add(int v, int lane) {   // inclusive, over a warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(FULL, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Fills `sh` but for a barrier at the end; every thread of the CTA calls it,
// NT of them, one item each at a time.  One round of look-ups and one barrier
// where the batch has at most NT tiles.
template <int NT, typename A>
__device__ __forceinline__ void take_share(const A& a, Share& sh, long long* s_sum, int* s_items, int* s_most) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int NWP = NT / 32;
  const long long n = (long long)a.B * a.tiles;
  const Item item = item_at(a, tid, blockIdx.x == 0);
  const int mine = item.w;
  int incl = scan_add(mine, lane), items = __popc(__ballot_sync(FULL, mine > 0)), most = (int)__reduce_max_sync(FULL, (unsigned)mine);
  long long sum = __shfl_sync(FULL, incl, 31);
  for (long long i = tid + NT; i < n + lane; i += NT) {   // whole warps
    const int w = item_weight(a, i, blockIdx.x == 0);
    sum += (long long)__reduce_add_sync(FULL, (unsigned)w);
    items += __popc(__ballot_sync(FULL, w > 0));
    most = max(most, (int)__reduce_max_sync(FULL, (unsigned)w));
  }
  if (tid == 0) {
    sh.b = a.B;
    sh.known = 0;
  }
  if (lane == 0) {
    s_sum[warp] = sum;
    s_items[warp] = items;
    s_most[warp] = most;
  }
  __syncthreads();
  long long total = 0, all = 0, before = 0;
#pragma unroll
  for (int w = 0; w < NWP; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
    all += s_items[w];
    most = max(most, s_most[w]);
  }
  const int heads = item_heads(a);
  const long long T = total * heads;
  const int P = share_ctas(a, T, (int)min((long long)gridDim.x, T), all * heads, most);
  if ((int)blockIdx.x >= P) {
    if (tid == 0) sh.lo = sh.hi = sh.pos = 0;
    return;
  }
  const long long lo = share_begin(T, blockIdx.x, P);
  if (tid == 0) {
    sh.T = T;
    sh.P = P;
    sh.lo = lo;
    sh.hi = share_begin(T, blockIdx.x + 1, P);
    sh.split = item_split(a, T, P, all * heads, most);
  }
  if (n <= NT) {
    share_place(a, sh, lo, before + incl - mine, item);
    return;
  }
  long long base = 0;   // weight of the items before i0
  for (long long i0 = 0; i0 < n && base * heads <= lo; i0 += NT) {
    const Item x = item_at(a, i0 + tid, false);
    incl = scan_add(x.w, lane);
    __syncthreads();
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    before = base;
#pragma unroll
    for (int k = 0; k < NWP; ++k) {
      if (k < warp) before += s_sum[k];
      base += s_sum[k];
    }
    share_place(a, sh, lo, before + incl - x.w, x);
  }
}

// T: type of q and out; the products' type is T, or fp16 over an e4m3 cache.
// A: PagedArgs, or JoinArgs of a pass whose sums are joined later (all of them
// go through memory then: an item that one CTA has whole to its rows).
// DIFF (with JoinArgs): differential heads.  The two tiles are the same 128
// rows of the first and of the second query heads; each has K blocks of its own
// (stage t of K is tile t's), and both use the same columns of V: those of both
// value heads of 64, or, over an e4m3 cache, where their scales differ, those of
// one (heads of 128 over 16 bits: santa_diff_wide.cu).
template <typename T, bool E4M3, int D, typename A, bool DIFF>
__global__ void __launch_bounds__(ChunkGeom<E4M3, D, diff_columns<E4M3, D, DIFF>(), DIFF>::THREADS, 1)
paged_chunk_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, A a) {
  constexpr bool JOIN = !std::is_same<A, PagedArgs>::value;
  static_assert(JOIN || !DIFF, "differential heads are joined");
  constexpr int DV = diff_columns<E4M3, D, DIFF>(), PARTS = DIFF ? 2 * D / DV : 1;   // items per pair of KV heads
  // A row's scores 32 at a time, read from tensor memory once for the maximum and
  // once for the exponentials, in loops: a quarter of the instructions, which
  // a pass of few blocks waits for (they come from HBM, in competition with K and
  // V: the first block's softmax took 7 us), and no spilled registers over e4m3.
  // 64 tokens behind 32768 keys 87.5 -> 85.9 us, six e4m3 chunks in a window
  // of 4096 202.7 -> 187.2.  All 128 at once where a CTA has many blocks of a
  // 16-bit cache: 2048 tokens at 32768 keys 779 against 796 us.
  constexpr bool SHORT = E4M3 || JOIN;
  // Over e4m3 a block of K is loaded and widened before the V of the block before
  // it, whose place is free only behind the product of the V two earlier, when
  // that K's scores are due half a block later: 96 tokens behind three prefixes of
  // up to 20001 keys 123.7 -> 109.4 us, six chunks in a window of 4096 184.9 ->
  // 180.5.  Not over 16 bits, where K needs no widening (757 against 764 us, 2048 tokens
  // at 32768 keys), nor where tiles have K of their own, whose places are freed later.
  constexpr bool AHEAD = E4M3 && !DIFF;
  using Gm = ChunkGeom<E4M3, D, DV, DIFF>;
  using M16 = typename std::conditional<E4M3, fp16_t, T>::type;
  constexpr float BIAS = fp16_bias<M16>(CHUNK_BIAS);
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) unsigned long long s_bar[N_BAR];
  __shared__ Share sh;
  __shared__ long long s_sum[Gm::THREADS / 32];
  __shared__ int s_items[Gm::THREADS / 32], s_most[Gm::THREADS / 32];
  __shared__ float s_ml[2][2][TROWS], s_sl[TROWS];
  __shared__ uint32_t s_tm;
  __shared__ int s_dead, s_bad[4], s_odd[4];   // of piece np: entry np & 3 holds np + 1
  __shared__ Walk s_walk[8];                    // the softmax warps' walks: their registers hold rows of S
  __shared__ Piece s_piece[8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  allow_dependents();

  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_addr(s_bar);
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  if (tid == 0) {
    s_dead = 0;
    for (int i = 0; i < 4; ++i) s_bad[i] = s_odd[i] = 0;
    if (!JOIN) a.share[blockIdx.x].count = 0;
  }
  static_assert(N_BAR <= 64, "a lane of warps 10 and 11 each");
  if (tid >= 320 && tid < 320 + N_BAR) {   // warps that have nothing else to do yet
    const int i = tid - 320;
    const int count = i == Q_READY || i == PIECE_SEEN ? 8
                      : i == K_READY || i == K_READY + 1 ? 4
                      : i == V_READY || i == V_READY + 1 ? (E4M3 ? 4 : 2)
                      : i == P_FULL || i == P_FULL + 1 || i == O_FREE || i == O_FREE + 1 || i == ML_FULL || i == Q_SEEN ? 4 : 1;
    mbar_init(bar(i), (unsigned)count);
    mbar_fence_init();
  }
  if (warp == 8) tm_alloc(smem_addr(&s_tm), 512);
  if (tid == 288) {
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  take_share<Gm::THREADS>(a, sh, s_sum, s_items, s_most);
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tm = uniform(s_tm);
  volatile int* const dead = &s_dead;
  const uint32_t tmS = tm, tmO = tm + 256;           // tile t: S (and P) at 128 t, O at 256 + 128 t
  const int per = TROWS / a.G;                       // tokens per tile of 128 rows

  if (warp >= 8) {
    Walk walk;
    Piece p;
    walk.start(a, sh);
    // registers: 256 x 208 + 128 x 88 of the launch's 384 x 168, 256 x 192 + 256 x 64 of 512 x 128
    if (E4M3) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8) {
      // -------------------------------------------------------- the products
      {
        constexpr uint32_t shS = mma_shape(std::is_same<M16, bf16_t>::value, BKEYS, false);
        constexpr uint32_t shO = mma_shape(std::is_same<M16, bf16_t>::value, DV, true);
        unsigned np = 0, kn = 0, vn = 0;               // pieces, blocks of K and V so far
        unsigned done0 = 0, done1 = 0, used0 = 0, used1 = 0;   // jobs and pieces of each tile so far
        while (uniform(walk.next(a, sh, p))) {
          const int nblk = (int)uniform((unsigned)p.nblk);
          if constexpr (JOIN) {   // the join of this item finds its pieces here
            if (p.last && lane == 0) {
              PieceNote note = {0, 0, 0, 0};
              if (!p.whole) {
                const ChunkShare r = share_note(sh, p, (int)blockIdx.x);
                note.first = r.first;
                note.slot = r.slot;
                note.count = r.count;
              }
              a.notes[(p.s.q0 + p.i0) * item_heads(a) + p.kvh] = note;
            }
          }
          if (nblk == 0) continue;
          const bool two = DIFF || uniform(p.two) != 0;
          const int jobs = two ? 2 * nblk : nblk;
          wait_phase(bar(E4M3 ? Q_READY : Q_FULL), np & 1, a.err, dead);
          // S with block kn of all (differential: of all of tile t), for tile t (one lane)
          auto k_bar = [&](int t) { return bar((E4M3 ? K_READY : K_FULL) + (DIFF ? t : (int)(kn & 1))); };
          auto k_parity = [&] { return (DIFF ? kn : kn >> 1) & 1; };
          auto product_s = [&](auto tile) {
            constexpr int t = decltype(tile)::value;
            const SmemOperand q(base + (two && t ? Gm::TILE : 0), 16), kk(base + Gm::OFF_K + (DIFF ? t : kn & 1) * Gm::TILE, 16);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              const uint32_t o = (uint32_t)((i >> 2) * Gm::HALF + (i & 3) * 32);
              mma_ss(tmS + 128 * t, q.at(o), kk.at(o), shS, i != 0);
            }
            mma_commit(bar(S_FULL + t));
            if (DIFF) mma_commit(bar(K_EMPTY + t));
            else if (!two || t == 1) mma_commit(bar(K_EMPTY + (kn & 1)));
          };
          auto first_s = [&](auto tile) {
            constexpr int t = decltype(tile)::value;
            if (DIFF || !two || t == 0) wait_phase(k_bar(t), k_parity(), a.err, dead);
            tm_fence_after();
            if (elect_one()) product_s(tile);
            __syncwarp();
            kn += !two || t == 1;
          };
          bool v_ok = false, p_ok = false, k_ok = false;   // of the next job: V, P and its next K are there
          // O += P V of job k, of tile t = k & 1, then S of job k + 2, in one
          // run of the electing lane; then a look at what the next job waits
          // for, under the products that are still in the queue.
          auto job = [&](auto tile, int k, unsigned& done, unsigned& used, unsigned& next_done) {
            constexpr int t = decltype(tile)::value;
            const int st = vn & 1;
            const bool first = !two || t == 0, last = !two || t == 1, more = k + 2 < jobs;
            if (first) {
              if (!v_ok) wait_phase(bar(V_READY + st), (vn >> 1) & 1, a.err, dead);
            }
            if ((DIFF || first) && !k_ok && more) wait_phase(k_bar(t), k_parity(), a.err, dead);
            if (k < 2) {                               // the previous piece's sums have been read
              if (used > 0) wait_phase(bar(O_FREE + t), (used - 1) & 1, a.err, dead);
              ++used;
            }
            if (!p_ok) wait_phase(bar(P_FULL + t), done & 1, a.err, dead);
            ++done;
            tm_fence_after();
            const SmemOperand v(base + Gm::OFF_V + st * Gm::VTILE, Gm::HALF);
            if (elect_one()) {
#pragma unroll
              for (int i = 0; i < BKEYS / 16; ++i)
                mma_ts(tmO + 128 * t, tmS + 128 * t + 8 * i, v.at(i * 2048), shO, k > 1 || i != 0);
              if (last) mma_commit(bar(V_EMPTY + st));
              if (more) product_s(tile);
              if (k + 1 == jobs) mma_commit(bar(O_DONE));
            }
            __syncwarp();
            vn += last;
            kn += last && more;
            p_ok = test_phase(bar(P_FULL + 1 - t), next_done & 1);
            if (last) {
              v_ok = test_phase(bar(V_READY + (vn & 1)), (vn >> 1) & 1);
            }
            if (DIFF || last) k_ok = test_phase(k_bar(1 - t), k_parity());
          };
          const std::integral_constant<int, 0> t0;
          const std::integral_constant<int, 1> t1;
          first_s(t0);
          if (jobs > 1) first_s(t1);
          for (int k = 0; k < jobs; k += 2) {
            job(t0, k, done0, used0, done1);
            if (k + 1 < jobs) job(t1, k + 1, done1, used1, done0);
          }
          ++np;
          // the merge of this item finds its pieces here
          if (!JOIN && sh.split && !p.whole && p.last && lane == 0) a.share[blockIdx.x] = share_note(sh, p, (int)blockIdx.x);
        }
        if (np > 0) wait_phase(bar(O_DONE), (np - 1) & 1, a.err, dead);   // nothing is in flight when the CTA ends
      }
      __syncwarp();
    } else if (warp == 9) {
      // ------------------------------------------------------------- the TMA
      const int rows = min(1 << a.page_shift, BKEYS);      // rows per box
      const int boxes = BKEYS / rows;
      constexpr int ROWB = E4M3 ? D : 2 * D, ROWB_V = E4M3 ? DV : 2 * DV;
      unsigned np = 0, n = 0;
      while (walk.next(a, sh, p)) {
        if (p.nblk == 0) continue;
        // heads: of K (differential: of tile 0; tile 1 has the next one), the first of V
        const int pair = p.kvh / PARTS, k_head = DIFF ? 2 * pair : p.kvh, v_head = DIFF ? 2 * pair + (PARTS == 2 ? p.kvh % 2 : 0) : p.kvh;
        const int32_t* const table = page_row(a, p.b);
        // lane l: page of box l of block j (INT32_MIN: no key of this pass there; the row of a sequence behind a
        // prefix need not name the pages that lie wholly inside it, some of which its first block may cover)
        auto page_of = [&](int j) {
          const int key = (p.blk0 + j) * BKEYS + lane * rows;
          const bool there = key < p.s.kv && (!JOIN || key > p.s.from - rows);
          return j < p.nblk && lane < boxes && there ? max(table[key >> a.page_shift], -1) : INT32_MIN;
        };
        auto row_of = [&](int pid, int j) {   // first row of a lane's box
          return (pid << a.page_shift) + (((p.blk0 + j) * BKEYS + lane * rows) & ((1 << a.page_shift) - 1));
        };
        int pid = page_of(0), pid1 = page_of(1), pid2 = AHEAD ? page_of(2) : INT32_MIN;
        for (int j = 0; j < p.nblk; ++j, ++n) {
          const int st = n & 1;
          const bool ok = pid != INT32_MIN && (unsigned)pid < (unsigned)a.n_pages;
          if (pid != INT32_MIN && !ok) {
            s_bad[np & 3] = np + 1;
            flag_error(a.err, ERR_PAGE);
          }
          const unsigned boxes_ok = (unsigned)__popc(__ballot_sync(FULL, ok)) * (unsigned)rows;
          const int row = ok ? row_of(pid, j) : 0;
          const uint32_t vd = base + Gm::OFF_V + st * Gm::VTILE;
          auto load_k = [&](int page, int i, unsigned at) {   // block i of the piece, block `at` of all
            const bool there = page != INT32_MIN && (unsigned)page < (unsigned)a.n_pages;
            const unsigned bytes = (unsigned)__popc(__ballot_sync(FULL, there)) * (unsigned)(rows * ROWB);
            const int first = there ? row_of(page, i) : 0;
#pragma unroll
            for (int t = 0; t < (DIFF ? 2 : 1); ++t) {
              const int ks = DIFF ? t : (int)(at & 1);
              if (at > (DIFF ? 0 : 1)) wait_phase(bar(K_EMPTY + ks), ((DIFF ? at : at >> 1) - 1) & 1, a.err, dead);
              const uint32_t kd = base + Gm::OFF_K + ks * Gm::TILE;
              if (lane == 0) mbar_expect_tx(bar(K_FULL + ks), bytes);
              __syncwarp();
              if (there) {
                if (E4M3) {
                  tma_load(kd + Gm::TILE / 2 + lane * rows * D, &tmK, 0, k_head + t, first, bar(K_FULL + ks));
                } else {
#pragma unroll
                  for (int h = 0; h < D / 64; ++h)
                    tma_load(kd + h * Gm::HALF + lane * rows * 128, &tmK, 64 * h, k_head + t, first, bar(K_FULL + ks));
                }
              }
            }
          };
          if (j == 0 || !AHEAD) load_k(pid, j, n);
          if (j == 0) {
            // Q, once the previous piece's products are over; the last
            // token's box may reach past q, where it reads zeros
            if (np > 0) wait_phase(bar(O_DONE), (np - 1) & 1, a.err, dead);
            if (E4M3 && np > 0) wait_phase(bar(Q_SEEN), (np - 1) & 1, a.err, dead);
            if (lane == 0) {
              const int tiles = DIFF || p.two ? 2 : 1;
              mbar_expect_tx(bar(Q_FULL), (unsigned)(tiles * per * a.G * 2 * D));
              for (int t = 0; t < tiles; ++t)
                for (int h = 0; h < D / 64; ++h) {
                  const uint32_t to = base + t * Gm::TILE + h * Gm::HALF;
                  if (DIFF) tma_load4(to, &tmQ, 64 * h, t, pair * a.G, (int)(p.s.q0 + p.i0), bar(Q_FULL));
                  else tma_load(to, &tmQ, 64 * h, p.kvh * a.G, (int)(p.s.q0 + p.i0 + t * per), bar(Q_FULL));
                }
            }
            __syncwarp();
          }
          if (AHEAD && j + 1 < p.nblk) load_k(pid1, j + 1, n + 1);
          // No piece's sums are complete (its V is not there) before every softmax
          // warp has seen that the previous one's were: see PIECE_SEEN below.
          if (j == 0 && np > 0) wait_phase(bar(PIECE_SEEN), (np - 1) & 1, a.err, dead);
          if (n > 1) wait_phase(bar(V_EMPTY + st), ((n >> 1) - 1) & 1, a.err, dead);
          if (lane == 0) mbar_expect_tx(bar(V_FULL + st), boxes_ok * ROWB_V);
          __syncwarp();
          if (ok) {
            if (E4M3) {
              tma_load(vd + Gm::VTILE / 2 + lane * rows * D, &tmV, 0, v_head, row, bar(V_FULL + st));
            } else {
#pragma unroll
              for (int h = 0; h < DV / 64; ++h)
                tma_load(vd + h * Gm::HALF + lane * rows * 128, &tmV, 64 * h % D, v_head + 64 * h / D, row, bar(V_FULL + st));
            }
          }
          pid = pid1;   // looked up two blocks ahead
          pid1 = AHEAD ? pid2 : page_of(j + 2);
          if (AHEAD) pid2 = page_of(j + 3);
        }
        ++np;
      }
      // the copies are over before the CTA ends, also where a wait ran out
      for (unsigned i = n > 2 ? n - 2 : 0; i < n; ++i) {
        if (!DIFF) wait_phase(bar(K_FULL + (i & 1)), (i >> 1) & 1, a.err, dead);
        wait_phase(bar(V_FULL + (i & 1)), (i >> 1) & 1, a.err, dead);
      }
      if (DIFF && n > 0) {
        wait_phase(bar(K_FULL), (n - 1) & 1, a.err, dead);
        wait_phase(bar(K_FULL + 1), (n - 1) & 1, a.err, dead);
      }
      if (*dead)
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    } else if (!E4M3 && warp < 12) {
      // -------------------- V: rows past the end or another pass's, odd values
      unsigned np = 0, n = 0;
      while (walk.next(a, sh, p)) {
        if (p.nblk == 0) continue;
        int lo0, hi0, lo1, hi1;
        visible_keys(a, p.s, p.s.kv - p.s.n + p.i0, lo0, hi0);
        visible_keys(a, p.s, p.s.kv - p.s.n + p.i1, lo1, hi1);
        for (int j = 0; j < p.nblk; ++j, ++n) {
          const int st = n & 1, key0 = (p.blk0 + j) * BKEYS, live = min(BKEYS, p.s.kv - key0), first = JOIN ? p.s.from - key0 : 0;
          wait_phase(bar(V_FULL + st), (n >> 1) & 1, a.err, dead);
          if (key0 < lo1 || key0 + BKEYS > hi0) {
            const uint32_t vd = base + Gm::OFF_V + st * Gm::VTILE;
            bool found = false;
            for (int i = tid - 320; i < Gm::VTILE / 16; i += 64) {
              const int r = (i >> 3) & (TROWS - 1);   // chunk i of the tile lies in row r of its half
              if (r >= live || r < first) {
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
            if (found) s_odd[np & 3] = np + 1;
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(V_READY + st));
        }
        ++np;
      }
    } else if (E4M3 && warp >= 12) {
      // ------------------------------------------------- e4m3 codes to fp16
      const int ct = tid - 384;                       // 0 .. 127
      constexpr int CPR = D / 16, PASS = BKEYS * CPR / 128;   // 16-byte chunks of a row; chunks per thread
      unsigned np = 0, n = 0;
      while (walk.next(a, sh, p)) {
        if (p.nblk == 0) continue;
        const int32_t* const table = page_row(a, p.b);
        const int pair = p.kvh / PARTS, k_head = DIFF ? 2 * pair : p.kvh, v_head = DIFF ? 2 * pair + (PARTS == 2 ? p.kvh % 2 : 0) : p.kvh;
        constexpr int STEPS = DIFF ? 3 : 2;           // the blocks of K, then V's
        for (int i = 0; i < STEPS * p.nblk; ++i) {
          // in the order in which they are loaded
          const bool is_v = AHEAD ? (i > 0 && i % 2 == 0) || i + 1 == STEPS * p.nblk : i % STEPS == STEPS - 1;
          const int which = AHEAD ? is_v : i % STEPS, j = AHEAD ? (is_v ? i - 1 : i + 1) / 2 : i / STEPS;
          const unsigned at = n + j;
          const int st = at & 1, key0 = (p.blk0 + j) * BKEYS, live = min(BKEYS, p.s.kv - key0), first = JOIN ? p.s.from - key0 : 0;
          if (which == 0) {   // this thread's key's scales, on their way while the codes arrive
            const int key = key0 + ct;
            float ksc = 0.f, ksc1 = 0.f, vsc = 1.f;
            if (ct < live && ct >= first) {
              const int pid = table[key >> a.page_shift];
              if ((unsigned)pid < (unsigned)a.n_pages) {
                auto scale_at = [&](int head) { return ((((long long)pid * a.Hkv) + head) << a.page_shift) + (key & ((1 << a.page_shift) - 1)); };
                ksc = __ldg(a.ks + scale_at(k_head));
                if (DIFF) ksc1 = __ldg(a.ks + scale_at(k_head + 1));
                vsc = __ldg(a.vs + scale_at(v_head));
              }
            }
            if (odd_scale(vsc)) {   // the values are NaN, the softmax is not: given back at the end
              s_odd[np & 3] = np + 1;
              vsc = 1.f;
            }
            vsc = fmaxf(vsc, V_SCALE_LEAST);
            float lv, rv;
            asm("lg2.approx.f32 %0, %1;" : "=f"(lv) : "f"(vsc));
            asm("rcp.approx.f32 %0, %1;" : "=f"(rv) : "f"(vsc));
            const uint32_t sc = base + Gm::OFF_SC + (at & 3) * Gm::SC_STAGE + ct * 4;
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(sc), "f"(ksc) : "memory");
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(sc + BKEYS * 4), "f"(lv) : "memory");
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(sc + 2 * BKEYS * 4), "f"(rv) : "memory");
            if (DIFF) asm volatile("st.shared.f32 [%0], %1;" ::"r"(sc + 3 * BKEYS * 4), "f"(ksc1) : "memory");
          }
          const int stage = DIFF && !is_v ? which : st;
          const uint32_t dst = base + (is_v ? Gm::OFF_V : Gm::OFF_K) + stage * Gm::TILE, src = dst + Gm::TILE / 2;   // DV == D
          wait_phase(bar((is_v ? V_FULL : K_FULL) + stage), (DIFF && !is_v ? at : at >> 1) & 1, a.err, dead);
          const int c = ct % CPR, r0 = ct / CPR;      // this thread's chunk of rows r0, r0 + 128 / CPR, ...
          // chunks 2c and 2c + 1 of a row's 16-bit elements; rows of a thread are 0 modulo 8 apart
          const uint32_t row = dst + (uint32_t)((c >> 2) * Gm::HALF + r0 * 128);
          const uint32_t lo = row + ((((2 * c) & 7) ^ (r0 & 7)) << 4), hi = row + ((((2 * c + 1) & 7) ^ (r0 & 7)) << 4);
          // Four chunks at a time.  With 128 elements a row's codes lie where
          // its own second half goes, and a row's threads are of one warp;
          // with 64 all codes are read before any is overwritten.
#pragma unroll 1
          for (int q0 = 0; q0 < PASS; q0 += 4) {
            uint4 w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) w[q] = lds128(src + (ct + 128 * (q0 + q)) * 16);
            if (PASS == 4) group_sync(1, 128);
            else __syncwarp();
            if (live < BKEYS || first > 0) {   // no key of this pass: whatever was there before
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if (r0 + (q0 + q) * (128 / CPR) >= live || r0 + (q0 + q) * (128 / CPR) < first) w[q] = make_uint4(0u, 0u, 0u, 0u);
            }
            uint32_t nan = 0;     // bit 7 of a byte: some code there is a NaN
#pragma unroll
            for (int q = 0; q < 4; ++q)
              nan |= ((w[q].x & 0x7f7f7f7fu) + 0x01010101u) | ((w[q].y & 0x7f7f7f7fu) + 0x01010101u) |
                     ((w[q].z & 0x7f7f7f7fu) + 0x01010101u) | ((w[q].w & 0x7f7f7f7fu) + 0x01010101u);
            if (is_v && (nan & 0x80808080u)) {        // NaN codes come back at the end, too
              auto clean = [](uint32_t x) { return x & ~(((((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xffu); };
              s_odd[np & 3] = np + 1;
#pragma unroll
              for (int q = 0; q < 4; ++q) w[q] = make_uint4(clean(w[q].x), clean(w[q].y), clean(w[q].z), clean(w[q].w));
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t o = (uint32_t)((q0 + q) * (128 / CPR) * 128);
              sts128(lo + o, make_uint4(widen8(w[q].x), widen8(w[q].x >> 16), widen8(w[q].y), widen8(w[q].y >> 16)));
              sts128(hi + o, make_uint4(widen8(w[q].z), widen8(w[q].z >> 16), widen8(w[q].w), widen8(w[q].w >> 16)));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar((is_v ? V_READY : K_READY) + stage));
        }
        ++np;
        n += p.nblk;
      }
    }
  } else {
    // -------------------------------------------------------------- softmax
    if (E4M3) asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int t = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t mS = tmS + 128 * t + lanes, mO = tmO + 128 * t + lanes;
    unsigned np = 0, jobs = 0, n = 0, joined = 0;      // pieces, this tile's jobs, blocks, pieces whose groups were joined
    int slot = 0;
    Piece& pc = s_piece[warp];
    if (lane == 0) s_walk[warp].start(a, sh);
    for (;;) {
      int more = 0;
      __syncwarp();   // the other lanes have read the last piece
      if (lane == 0) {
        Walk w = s_walk[warp];
        more = w.next(a, sh, pc);
        s_walk[warp] = w;
      }
      more = __shfl_sync(FULL, more, 0);
      __syncwarp();
      if (!more) break;
      const int nblk = pc.nblk, blk0 = pc.blk0;
      const bool two = DIFF || pc.two;
      const int step = two ? 1 : 2;
      int lo, hi, lo_last, hi_first;                   // keys that the row sees; that every row of the tile sees
      // The row's maximum that P and O are relative to.  Infinite for rows past
      // the tile's tokens, which hold other tokens or whatever was there: so
      // they never ask for a rescaling, and the rounding of the others does not
      // depend on them.
      float m;
      {
        const int first_pos = pc.s.kv - pc.s.n;
        const int ta = pc.i0 + (two && !DIFF ? t * per : 0), tb = min(ta + per, pc.s.n) - 1;   // the tile's tokens
        int none;
        visible_keys(a, pc.s, first_pos + min(ta + row / a.G, tb), lo, hi);   // rows past the last compute it again, for nothing
        visible_keys(a, pc.s, first_pos + ta, none, hi_first);
        visible_keys(a, pc.s, first_pos + tb, lo_last, none);
        m = row < (tb - ta + 1) * a.G ? -INFINITY : INFINITY;
      }
      float sl = a.sl2;
      if (E4M3 && nblk > 0) {
        // Group 1 sees every phase of Q_FULL, also of pieces that it has no
        // part in, and the next Q waits until it has: a wait that skipped a
        // phase, or fell two behind, would take one phase for another.
        wait_phase(bar(Q_FULL), np & 1, a.err, dead);
        __syncwarp();
        if (t == 1 && lane == 0) mbar_arrive(bar(Q_SEEN));
        if (t == 0 || two) {
          // the row of q in fp16 under a power of two (see santa_tokens.cuh)
          const uint32_t qr = base + (two ? t * Gm::TILE : 0) + row * 128;
          float mx = 0.f;
#pragma unroll 2   // run once per piece: straight-line code that runs once waits for its instructions
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
#pragma unroll 2
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
          if (!two) s_sl[row] = sl;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(Q_READY));
            if (!two) mbar_arrive(bar(Q_READY));   // for the other group's warp
          }
        } else if (nblk > 1) {
          wait_phase(bar(Q_READY), np & 1, a.err, dead);
          sl = s_sl[row];
        }
      }
      float l = 0.f;                // the row's sum
      const int j_first = two ? 0 : t;
      f2x l2[E4M3 ? 2 : 4];         // chains of additions: one would take longer than the exponentials
#pragma unroll
      for (int e = 0; e < (E4M3 ? 2 : 4); ++e) l2[e] = pack2(0.f, 0.f);
      for (int j = j_first; j < nblk; j += step, ++jobs) {
        const int key0 = (blk0 + j) * BKEYS;
        wait_phase(bar(S_FULL + t), jobs & 1, a.err, dead);
        tm_fence_after();
        // 32 scores at a time: their scales (e4m3), the mask, the largest
        const uint32_t sc = base + Gm::OFF_SC + ((n + j) & 3) * Gm::SC_STAGE;
        const f2x sl_2 = pack2(sl, sl);
        auto scale32 = [&](int c0, uint32_t* x) {
          // a key's three factors from shared memory: 96 loads of 16 bytes per
          // thread, at 128 bytes a cycle 3000 cycles for the eight warps of
          // both tiles, of which one tile waits for 1200 of its 3100
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const uint4 k4 = lds128(sc + ((DIFF ? t * 3 * BKEYS : 0) + c0 + c) * 4), v4 = lds128(sc + (BKEYS + c0 + c) * 4);
            const f2x x0 = mul2(pack2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sl_2);
            const f2x x1 = mul2(pack2(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])), sl_2);
            const float2 y0 = unpack2(ffma2(x0, pack2(__uint_as_float(k4.x), __uint_as_float(k4.y)), pack2(__uint_as_float(v4.x), __uint_as_float(v4.y))));
            const float2 y1 = unpack2(ffma2(x1, pack2(__uint_as_float(k4.z), __uint_as_float(k4.w)), pack2(__uint_as_float(v4.z), __uint_as_float(v4.w))));
            x[c] = __float_as_uint(y0.x);
            x[c + 1] = __float_as_uint(y0.y);
            x[c + 2] = __float_as_uint(y1.x);
            x[c + 3] = __float_as_uint(y1.y);
          }
        };
        const bool partial = key0 < lo_last || key0 + BKEYS > hi_first;
        auto mask32 = [&](int c0, uint32_t* x) {
          const int from = lo - key0 - c0, cn = hi - lo;
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if ((unsigned)(c - from) >= (unsigned)cn) x[c] = 0xff800000u;
        };
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        auto top32 = [&](const uint32_t* x) {
#pragma unroll
          for (int c = 0; c < 32; c += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mx[e] = fmaxf(fmaxf(mx[e], __uint_as_float(x[c + 2 * e])), __uint_as_float(x[c + 2 * e + 1]));
        };
        uint32_t sr[SHORT ? 32 : BKEYS];
        if constexpr (SHORT) {
#pragma unroll 1
          for (int c = 0; c < BKEYS; c += 32) {
            tm_ld32(mS + c, sr);
            tm_wait_ld();
            if (E4M3) scale32(c, sr);
            if (partial) mask32(c, sr);
            top32(sr);
            if (E4M3) {   // the scores as they are now, for the second time
              tm_st16(mS + c, sr);
              tm_st16(mS + c + 16, sr + 16);
            }
          }
          if (E4M3) tm_wait_st();
        } else {
          if (E4M3) {
#pragma unroll
            for (int c = 0; c < BKEYS; c += 32) {
              tm_ld32(mS + c, sr + c);
              tm_wait_ld();
              scale32(c, sr + c);
            }
          } else {
#pragma unroll
            for (int c = 0; c < BKEYS; c += 32) tm_ld32(mS + c, sr + c);
            tm_wait_ld();
          }
          if (partial) {
#pragma unroll
            for (int c = 0; c < BKEYS; c += 32) mask32(c, sr + c);
          }
#pragma unroll
          for (int c = 0; c < BKEYS; c += 32) top32(sr + c);
        }
        const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * (E4M3 ? 1.f : sl) - BIAS);
        if (j == j_first) {
          m = mn;
        } else if (__any_sync(FULL, mn > m + RESCALE)) {
          const float f = fast_exp2(m - (mn > -INFINITY ? mn : 0.f));
          m = mn;
#pragma unroll
          for (int e = 0; e < (E4M3 ? 2 : 4); ++e) l2[e] = mul2(l2[e], pack2(f, f));
#pragma unroll 1
          for (int c = 0; c < DV; c += 16) {
            uint32_t o[16];
            tm_ld16(mO + c, o);
            tm_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tm_st16(mO + c, o);
          }
        }
        const float neg = m > -INFINITY ? -m : 0.f;
        const f2x neg2 = pack2(neg, neg);
        auto weigh32 = [&](int c, const uint32_t* x) {   // P of columns c .. c + 31
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            f2x x0 = pack2(__uint_as_float(x[e]), __uint_as_float(x[e + 1]));
            f2x x1 = pack2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
            const float2 y0 = unpack2(E4M3 ? add2(x0, neg2) : ffma2(x0, sl_2, neg2));
            const float2 y1 = unpack2(E4M3 ? add2(x1, neg2) : ffma2(x1, sl_2, neg2));
            const float p0 = fast_exp2(y0.x), p1 = fast_exp2(y0.y), p2 = fast_exp2(y1.x), p3 = fast_exp2(y1.y);
            if (E4M3) {
              const uint4 r4 = lds128(sc + (2 * BKEYS + c + e) * 4);
              l2[0] = ffma2(pack2(p0, p1), pack2(__uint_as_float(r4.x), __uint_as_float(r4.y)), l2[0]);
              l2[1] = ffma2(pack2(p2, p3), pack2(__uint_as_float(r4.z), __uint_as_float(r4.w)), l2[1]);
            } else {
              f2x &la = l2[(e >> 1) & 3], &lb = l2[((e >> 1) + 1) & 3];
              la = add2(la, pack2(p0, p1));
              lb = add2(lb, pack2(p2, p3));
            }
            pk[e / 2] = pack2h<M16>(p0, p1);
            pk[e / 2 + 1] = pack2h<M16>(p2, p3);
          }
          tm_st16(mS + c / 2, pk);
        };
        if constexpr (SHORT) {
#pragma unroll 1
          for (int c = 0; c < BKEYS; c += 32) {
            tm_ld32(mS + c, sr);
            tm_wait_ld();
            if (!E4M3 && partial) mask32(c, sr);
            weigh32(c, sr);
          }
        } else {
#pragma unroll
          for (int c = 0; c < BKEYS; c += 32) weigh32(c, sr + c);
        }
        tm_wait_st();
        tm_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(P_FULL + t));
      }
      {
        f2x s2 = add2(l2[0], l2[1]);
        if (!E4M3) s2 = add2(s2, add2(l2[E4M3 ? 0 : 2], l2[E4M3 ? 0 : 3]));
        const float2 lp = unpack2(s2);
        l = lp.x + lp.y;
      }
      // ------------------------------------------------------- the result
      const bool join = !two && nblk > 1;          // both groups hold sums of these rows
      const bool mine = t == 0 || two;               // this group writes
      // A wait knows a phase by its parity: once the next one is over as well,
      // the phase looks as if it were still to come.  O_DONE and ML_FULL are
      // waited for by warps that the next piece may not need (group 1 where it
      // is one block of one tile; group 0, whose join the other group's next
      // one could overtake), so each softmax warp says when it is past a
      // piece's waits: the V of the next piece is loaded, and group 1 takes
      // part in the next join, after all eight have.  Group 1 waits also where
      // it has no part, or it could arrive twice in one phase.
      if (!mine && nblk > 0 && np > 0) {
        wait_phase(bar(PIECE_SEEN), (np - 1) & 1, a.err, dead);
        __syncwarp();
      }
      if (join && t == 1) {
        s_ml[joined & 1][0][row] = m;
        s_ml[joined & 1][1][row] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(ML_FULL));
      }
      if (!mine && nblk > 0 && lane == 0) mbar_arrive(bar(PIECE_SEEN));
      if (mine) {
        float f0 = 1.f, f1 = 0.f;                      // weights of the two sums
        if (nblk > 0) {
          wait_phase(bar(O_DONE), np & 1, a.err, dead);
          tm_fence_after();
        }
        if (join) wait_phase(bar(ML_FULL), joined & 1, a.err, dead);
        if (nblk > 0) {
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(PIECE_SEEN));
        }
        if (join) {
          const float m1 = s_ml[joined & 1][0][row], l1 = s_ml[joined & 1][1][row], mm = fmaxf(m, m1), mu = mm > -INFINITY ? mm : 0.f;
          f0 = fast_exp2(m - mu);
          f1 = fast_exp2(m1 - mu);
          l = l * f0 + l1 * f1;
          m = mm;
        }
        const bool bad = nblk > 0 && s_bad[np & 3] == (int)np + 1, odd = nblk > 0 && s_odd[np & 3] == (int)np + 1;
        const bool empty = bad || l == 0.f;
        const int ta = pc.i0 + (two && !DIFF ? t * per : 0), tb = min(ta + per, pc.s.n) - 1, tok = min(ta + row / a.G, tb);
        const int pair = pc.kvh / PARTS, part_v = PARTS == 2 ? pc.kvh % 2 : 0;
        const int kvh = DIFF ? 2 * pair + part_v : pc.kvh;   // the first head of V
        const bool live_row = row < per * a.G && ta + row / a.G <= tb, whole = pc.whole;
        const long long at = (pc.s.q0 + tok) * a.H + (DIFF ? 2 * (pair * a.G + row % a.G) + t : kvh * a.G + row % a.G);
        const long long part = ((long long)blockIdx.x * 2 + slot) * a.rows + (two ? t * TROWS : 0) + row;
        // where the sums go, in a pass that is joined
        float *to_o = nullptr, *to_ml = nullptr;
        if (JOIN || !whole) {
          to_o = a.part_o + part * DV;
          to_ml = a.part_ml + 2 * part;
        }
        if constexpr (JOIN) {
          if (whole) {
            to_o = a.row_o + at * (DV * PARTS) + part_v * DV;
            to_ml = a.row_ml + (at * PARTS + part_v) * 2;
          }
        }
        if (!JOIN && whole && !empty) {
          const float inv = __fdividef(1.f, l);
          f0 *= inv;
          f1 *= inv;
        }
        // all of the row's sums at once, so that the next piece's products may
        // overwrite them while this one is stored; 32 at a time over an e4m3
        // cache, where registers are fewer
        constexpr int EC = E4M3 || SHORT ? 32 : DV;
#pragma unroll 1
        for (int c0 = 0; c0 < DV; c0 += EC) {
          float f[EC];
#pragma unroll
          for (int c = 0; c < EC; c += 32) {
            uint32_t o[32];
            if (nblk > 0) {
              tm_ld32(mO + c0 + c, o);
              tm_wait_ld();
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) f[c + e] = nblk > 0 ? __uint_as_float(o[e]) * f0 : 0.f;
            if (join) {
              tm_ld32(mO + 128 + c0 + c, o);
              tm_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) f[c + e] = fmaf(__uint_as_float(o[e]), f1, f[c + e]);
            }
          }
          if (nblk > 0 && c0 + EC == DV) {
            tm_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(bar(O_FREE + t));
              if (join) mbar_arrive(bar(O_FREE + 1));
            }
          }
          if (live_row) {
            // 32 bytes per lane and store: a lane's row is its own, and half
            // sectors would be written twice
            if (!JOIN && whole) {
              T* const dst = static_cast<T*>(a.out) + at * D + c0;
#pragma unroll
              for (int c = 0; c < EC; c += 16) {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = empty ? 0u : pack2h<T>(f[c + 2 * e], f[c + 2 * e + 1]);
                if (a.wide) st_global8(dst + c, w);
                else {
                  *reinterpret_cast<uint4*>(dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
                  *reinterpret_cast<uint4*>(dst + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                }
              }
            } else {
              float* const dst = to_o + c0;
#pragma unroll
              for (int c = 0; c < EC; c += 8) st_global8(dst + c, reinterpret_cast<const uint32_t*>(f + c));
            }
          }
        }
        if (live_row) {
          if (JOIN || !whole) {
            to_ml[0] = m;
            to_ml[1] = bad ? -1.f : l;
          } else if (a.lse) {
            a.lse[at] = empty ? -INFINITY : log_sum(m, l, BIAS);
          }
        }
        if (odd) {
          // What was taken out of V, to the rows that see its key, in what they
          // have just stored: a lane looks into a key of its own, 32 of them at
          // a time.  Over an e4m3 cache it is NaNs, a bit for each column; keys
          // that every row of the tile sees give theirs to all at once, so that
          // 2^21 keys take well under the second that the other warps wait.  In
          // 16 bits it is what the cleaned blocks held, few at the mask's edges.
          // After the stores, so that the usual way is not longer for it
          // (between the sums and the stores it took 3 %).
          int clean_lo, clean_hi, none;
          visible_keys(a, pc.s, pc.s.kv - pc.s.n + pc.i0, none, clean_hi);
          visible_keys(a, pc.s, pc.s.kv - pc.s.n + pc.i1, clean_lo, none);
          const int32_t* const table = page_row(a, pc.b);
          const int end = min(pc.s.kv, (blk0 + nblk) * BKEYS);
          const bool mark = live_row && (JOIN || !(whole && empty));
          auto give = [&](int c, float y) {   // y is odd: the sum with it is the result's, whatever the scale
            if (!JOIN && whole) {
              uint16_t* const o = static_cast<uint16_t*>(a.out) + at * D + c;
              *o = (uint16_t)pack2h<T>(unpack2h<T>(*o).x + y, 0.f);
            } else {
              to_o[c] += y;
            }
          };
          constexpr int EC_ODD = E4M3 ? 32 : DV;
#pragma unroll 1
          for (int c0 = 0; c0 < DV; c0 += EC_ODD) {
            uint32_t nan_columns = 0;
#pragma unroll 1
            for (int key0 = blk0 * BKEYS; key0 < end; key0 += 32) {
              const int block = key0 & -BKEYS, key = key0 + lane;
              if (!E4M3 && block >= clean_lo && block + BKEYS <= clean_hi) continue;
              const int pid = key < end && (!JOIN || key >= pc.s.from) ? table[key >> a.page_shift] : -1;
              const int in_page = key & ((1 << a.page_shift) - 1);
              long long at_v = 0;
              uint32_t found = 0;   // e4m3: the odd columns; else whether there are any
              if ((unsigned)pid < (unsigned)a.n_pages) {
                at_v = ((((long long)pid << a.page_shift) + in_page) * a.Hkv + kvh) * D + c0;
                const uint4* const v = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(a.V) + at_v * (E4M3 ? 1 : 2));
                if (E4M3) {
#pragma unroll
                  for (int q = 0; q < EC_ODD / 16; ++q) {
                    const uint4 w = v[q];
                    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)   // the bytes' marks side by side: bits 24 to 27 of the product
                      found |= (((((ww[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 0x01020408u >> 24 & 15u) << ((16 * q + 4 * e) & 31);
                  }
                  if (odd_scale(a.vs[((((long long)pid * a.Hkv) + kvh) << a.page_shift) + in_page])) found = ~0u;
                } else {
#pragma unroll 4
                  for (int q = 0; q < DV / 8; ++q) found |= odd16<T>(v[q]);
                }
              }
              if (E4M3 && key0 >= lo_last && key0 + 32 <= hi_first) {
                nan_columns |= __reduce_or_sync(FULL, found);
                continue;
              }
              for (unsigned keys = __ballot_sync(FULL, found != 0); keys; keys &= keys - 1) {
                const int u = __ffs(keys) - 1;
                const uint32_t columns = __shfl_sync(FULL, found, u);
                const long long at_u = __shfl_sync(FULL, at_v, u);
                if (!mark || key0 + u < lo || key0 + u >= hi) continue;
                if (E4M3) {
                  nan_columns |= columns;
                } else {
                  const uint32_t* const v = reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.V) + at_u);
#pragma unroll 1
                  for (int e = 0; e < DV / 2; ++e) {
                    const float2 y = unpack2h<T>(v[e]);
                    if (!(fabsf(y.x) <= 3.402823466e38f)) give(2 * e, y.x);
                    if (!(fabsf(y.y) <= 3.402823466e38f)) give(2 * e + 1, y.y);
                  }
                }
              }
            }
            if (E4M3 && mark)
              for (; nan_columns; nan_columns &= nan_columns - 1) give(c0 + __ffs(nan_columns) - 1, __int_as_float(0x7fffffff));
          }
        }
      }
      if (nblk > 0) ++np;
      n += nblk;
      joined += join;
      slot = 1;
    }
    tm_fence_before();
  }
  __syncthreads();
  if (warp == 8) {
    tm_fence_after();
    tm_free(tm, 512);
  }
  // a pass may start under the one before it, whose sums the join needs as well: it is not over before that one is
  if (JOIN && blockIdx.x == 0) wait_for_predecessor();
}

inline PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> kept{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 fn = kept.load(std::memory_order_relaxed);
  if (fn) return fn;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  kept.store(fn, std::memory_order_relaxed);
  return fn;
}

// Query heads in pairs: [rows, heads, d] with the two of a pair as a dimension of their own, boxes of one of them.
inline bool encode_pairs(CUtensorMap* tm, const void* base, int d, int heads, long long rows, int by, int bz) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)d, 2, (cuuint64_t)heads / 2, (cuuint64_t)rows};
  const cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)d * 4, (cuuint64_t)heads * d * 2};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)by, (cuuint32_t)bz}, one[4] = {1, 1, 1, 1};
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A [rows, heads, d] array as a three-dimensional tensor, boxes of bx x by x bz.
inline bool encode(CUtensorMap* tm, const void* base, int es, int d, int heads, long long rows, int bx, int by, int bz) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)d * es, (cuuint64_t)heads * d * es};
  const cuuint32_t box[3] = {(cuuint32_t)bx, (cuuint32_t)by, (cuuint32_t)bz}, one[3] = {1, 1, 1};
  return enc(tm, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims,
             strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, es == 2 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// K or V of the cache: a box is a page, or 128 rows of one.
template <bool E4M3, int D>
bool encode_cache(CUtensorMap* tm, const PagedArgs& a, const void* pool) {
  return encode(tm, pool, E4M3 ? 1 : 2, D, a.Hkv, (long long)a.n_pages << a.page_shift, E4M3 ? D : 64, 1,
                std::min(1 << a.page_shift, BKEYS));
}

}  // namespace

}  // namespace santa
