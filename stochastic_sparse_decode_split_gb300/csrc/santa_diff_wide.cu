// santa_diff_wide.cu -- differential heads of 128 over a 16-bit cache, many query
// rows: chunks of one map at a time, over the columns of both value heads.
//
// A map's sum O has 2 x 128 columns, and tensor memory holds one of them beside
// two blocks of scores.  So an item is 128 rows of one map against its keys, and
// the two softmax groups of santa_chunk.cuh, whose roles and order of products
// this kernel has, take its blocks in turn and add to the same O.  A row then has
// one maximum that O is relative to, which goes from group to group: at block j
// a group takes it over from the other, which has had block j - 1, raises it if
// its block asks for more than 2^8 above it (then it scales O, once the product
// of block j - 1 is over), and hands it on before the exponentials, so that
// those of both groups overlap.  Each group's l is relative to the maximum that
// it saw last; they join at the item's end, where group t stores the columns of
// value head t.
//
// Against a tile for each map and an item for each value head (whose scores are
// computed twice): 6 units of products instead of 8, half the exponentials.
// 2048 tokens at 16384 keys, 32 and 8 heads, bf16: 760 -> 610 us, 1.27 PFLOP/s
// (0.67 of a library product's rate; the way of a block through its group, and
// V's second half, for which there is a third stage but no fourth, set the pace).
#include "santa_chunk.cuh"

namespace santa {

namespace {

constexpr int WD = 128, W_HALF = TROWS * 128;              // 128 rows of 128 bytes
constexpr int W_TILE = 2 * W_HALF;                         // Q, a block of K, of one value head
constexpr int W_K = W_TILE, W_V = W_K + 2 * W_TILE;        // offsets: Q, two of K, three of V
constexpr int W_BYTES = W_V + 3 * W_TILE, W_SMEM = W_BYTES + 1024;
constexpr int W_THREADS = 384;

enum { WQ_FULL, WK_FULL, WK_EMPTY = WK_FULL + 2, WV_FULL = WK_EMPTY + 2, WV_READY = WV_FULL + 3, WV_EMPTY = WV_READY + 3,
       WS_FULL = WV_EMPTY + 3, WP_FULL = WS_FULL + 2, WM_READY = WP_FULL + 2, WO_STEP = WM_READY + 2, WO_DONE = WO_STEP + 2, WO_FREE, WPIECE_SEEN, W_BARS };

// Stage and use of half h of V.
struct VStage {
  unsigned st, use;
  __device__ __forceinline__ explicit VStage(unsigned h) : st(h % 3), use(h / 3) {}
};

template <typename T>
__global__ void __launch_bounds__(W_THREADS, 1)
diff_wide_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, JoinArgs a) {
  constexpr float BIAS = fp16_bias<T>(CHUNK_BIAS);
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) unsigned long long s_bar[W_BARS];
  __shared__ Share sh;
  __shared__ long long s_sum[W_THREADS / 32];
  __shared__ int s_items[W_THREADS / 32], s_most[W_THREADS / 32];
  __shared__ float s_m[TROWS], s_ml[2][2][2][TROWS];   // the maximum handed on; [piece & 1][group][maximum, sum]
  __shared__ uint32_t s_tm;
  __shared__ int s_dead, s_bad[4], s_odd[4];   // of piece np: entry np & 3 holds np + 1
  __shared__ Walk s_walk[8];
  __shared__ Piece s_piece[8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  allow_dependents();

  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_addr(s_bar);
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  if (tid == 0) {
    s_dead = 0;
    for (int i = 0; i < 4; ++i) s_bad[i] = s_odd[i] = 0;
  }
  static_assert(W_BARS <= 64, "a lane of warps 10 and 11 each");
  if (tid >= 320 && tid < 320 + W_BARS) {
    const int i = tid - 320;
    const int count = i == WO_FREE || i == WPIECE_SEEN ? 8
                      : i >= WP_FULL && i < WM_READY + 2 ? 4
                      : i >= WV_READY && i < WV_READY + 3 ? 2 : 1;
    mbar_init(bar(i), (unsigned)count);
    mbar_fence_init();
  }
  if (warp == 8) tm_alloc(smem_addr(&s_tm), 512);
  if (tid == 288) {
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  take_share<W_THREADS>(a, sh, s_sum, s_items, s_most);
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tm = uniform(s_tm);
  volatile int* const dead = &s_dead;
  const uint32_t tmS = tm, tmO = tm + 256;           // group t: S (and P) at 128 t; O of value head f at 256 + 128 f
  const int per = TROWS / a.G;                       // tokens per tile

  if (warp >= 8) {
    Walk walk;
    Piece p;
    walk.start(a, sh);
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8) {
      // -------------------------------------------------------- the products
      constexpr uint32_t shape_s = mma_shape(std::is_same<T, bf16_t>::value, BKEYS, false);
      constexpr uint32_t shape_o = mma_shape(std::is_same<T, bf16_t>::value, WD, true);
      unsigned np = 0, kn = 0, vn = 0;                 // pieces, blocks of K and V so far
      unsigned done0 = 0, done1 = 0;                   // jobs of each group so far
      while (uniform(walk.next(a, sh, p))) {
        const int nblk = (int)uniform((unsigned)p.nblk);
        if (p.last && lane == 0) {   // the join of this item finds its pieces here
          PieceNote note = {0, 0, 0, 0};
          if (!p.whole) {
            const ChunkShare r = share_note(sh, p, (int)blockIdx.x);
            note.first = r.first;
            note.slot = r.slot;
            note.count = r.count;
          }
          a.notes[(p.s.q0 + p.i0) * item_heads(a) + p.kvh] = note;
        }
        if (nblk == 0) continue;
        wait_phase(bar(WQ_FULL), np & 1, a.err, dead);
        auto product_s = [&](auto group) {   // with block kn of all, for group t (one lane)
          constexpr int t = decltype(group)::value;
          const SmemOperand q(base, 16), kk(base + W_K + (kn & 1) * W_TILE, 16);
#pragma unroll
          for (int i = 0; i < WD / 16; ++i) {
            const uint32_t o = (uint32_t)((i >> 2) * W_HALF + (i & 3) * 32);
            mma_ss(tmS + 128 * t, q.at(o), kk.at(o), shape_s, i != 0);
          }
          mma_commit(bar(WS_FULL + t));
          mma_commit(bar(WK_EMPTY + (kn & 1)));
        };
        auto first_s = [&](auto group) {
          wait_phase(bar(WK_FULL + (kn & 1)), (kn >> 1) & 1, a.err, dead);
          tm_fence_after();
          if (elect_one()) product_s(group);
          __syncwarp();
          ++kn;
        };
        // O += P V of block k by group t, then S of block k + 2.  The second
        // half of V may come only when the first half of the block before is
        // done with, so the first half's products do not wait for it.
        auto job = [&](auto group, int k, unsigned& done) {
          constexpr int t = decltype(group)::value;
          const VStage v0(2 * vn), v1(2 * vn + 1);
          const bool more = k + 2 < nblk;
          wait_phase(bar(WV_READY + v0.st), v0.use & 1, a.err, dead);
          if (k == 0 && np > 0) wait_phase(bar(WO_FREE), (np - 1) & 1, a.err, dead);   // the previous piece's sums have been read
          wait_phase(bar(WP_FULL + t), done & 1, a.err, dead);
          ++done;
          tm_fence_after();
          const SmemOperand b0(base + W_V + v0.st * W_TILE, W_HALF), b1(base + W_V + v1.st * W_TILE, W_HALF);
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < BKEYS / 16; ++i) mma_ts(tmO, tmS + 128 * t + 8 * i, b0.at(i * 2048), shape_o, k > 0 || i != 0);
            mma_commit(bar(WV_EMPTY + v0.st));
          }
          __syncwarp();
          wait_phase(bar(WV_READY + v1.st), v1.use & 1, a.err, dead);
          if (more) wait_phase(bar(WK_FULL + (kn & 1)), (kn >> 1) & 1, a.err, dead);
          tm_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < BKEYS / 16; ++i) mma_ts(tmO + 128, tmS + 128 * t + 8 * i, b1.at(i * 2048), shape_o, k > 0 || i != 0);
            mma_commit(bar(WV_EMPTY + v1.st));
            mma_commit(bar(WO_STEP + t));
            if (more) product_s(group);
            if (k + 1 == nblk) mma_commit(bar(WO_DONE));
          }
          __syncwarp();
          ++vn;
          kn += more;
        };
        const std::integral_constant<int, 0> t0;
        const std::integral_constant<int, 1> t1;
        first_s(t0);
        if (nblk > 1) first_s(t1);
        for (int k = 0; k < nblk; k += 2) {
          job(t0, k, done0);
          if (k + 1 < nblk) job(t1, k + 1, done1);
        }
        ++np;
      }
      if (np > 0) wait_phase(bar(WO_DONE), (np - 1) & 1, a.err, dead);   // nothing is in flight when the CTA ends
      __syncwarp();
    } else if (warp == 9) {
      // ------------------------------------------------------------- the TMA
      const int rows = min(1 << a.page_shift, BKEYS);      // rows per box
      const int boxes = BKEYS / rows;
      unsigned np = 0, n = 0;
      while (walk.next(a, sh, p)) {
        if (p.nblk == 0) continue;
        const int pair = p.kvh >> 1, map = p.kvh & 1;
        const int32_t* const table = page_row(a, p.b);
        auto page_of = [&](int j) {   // lane l: page of box l of block j (INT32_MIN: no key of this pass there)
          const int key = (p.blk0 + j) * BKEYS + lane * rows;
          return j < p.nblk && lane < boxes && key < p.s.kv && key > p.s.from - rows ? max(table[key >> a.page_shift], -1) : INT32_MIN;
        };
        int pid = page_of(0), pid1 = page_of(1);
        for (int j = 0; j < p.nblk; ++j, ++n) {
          // a lane's box of block i, whose page is `page`
          auto there = [&](int page) { return page != INT32_MIN && (unsigned)page < (unsigned)a.n_pages; };
          auto row_of = [&](int page, int i) {
            return there(page) ? (page << a.page_shift) + (((p.blk0 + i) * BKEYS + lane * rows) & ((1 << a.page_shift) - 1)) : 0;
          };
          auto bytes_of = [&](int page) { return (unsigned)__popc(__ballot_sync(FULL, there(page))) * (unsigned)(rows * 2 * WD); };
          auto load_k = [&](int page, int i, unsigned at) {   // block i of the piece, block `at` of all
            const int st = at & 1, row = row_of(page, i);
            const unsigned bytes = bytes_of(page);
            if (at > 1) wait_phase(bar(WK_EMPTY + st), ((at >> 1) - 1) & 1, a.err, dead);
            if (lane == 0) mbar_expect_tx(bar(WK_FULL + st), bytes);
            __syncwarp();
            if (there(page)) {
#pragma unroll
              for (int h = 0; h < 2; ++h)
                tma_load(base + W_K + st * W_TILE + h * W_HALF + lane * rows * 128, &tmK, 64 * h, 2 * pair + map, row, bar(WK_FULL + st));
            }
          };
          const bool ok = there(pid);
          if (pid != INT32_MIN && !ok) {
            s_bad[np & 3] = np + 1;
            flag_error(a.err, ERR_PAGE);
          }
          const int row = row_of(pid, j);
          const unsigned bytes = bytes_of(pid);
          if (j == 0) {   // K, and Q once the previous piece's products are over
            load_k(pid, 0, n);
            if (np > 0) wait_phase(bar(WO_DONE), (np - 1) & 1, a.err, dead);
            if (lane == 0) {
              mbar_expect_tx(bar(WQ_FULL), (unsigned)(per * a.G * 2 * WD));
              for (int h = 0; h < 2; ++h)
                tma_load4(base + h * W_HALF, &tmQ, 64 * h, map, pair * a.G, (int)(p.s.q0 + p.i0), bar(WQ_FULL));
            }
            __syncwarp();
          }
          // the next K before this V, whose second half waits for the product
          // behind which that K's scores are issued
          if (j + 1 < p.nblk) load_k(pid1, j + 1, n + 1);
          // no sum of this piece before every softmax warp has seen that the previous one's were over
          if (j == 0 && np > 0) wait_phase(bar(WPIECE_SEEN), (np - 1) & 1, a.err, dead);
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const VStage v(2 * n + f);
            if (v.use > 0) wait_phase(bar(WV_EMPTY + v.st), (v.use - 1) & 1, a.err, dead);
            if (lane == 0) mbar_expect_tx(bar(WV_FULL + v.st), bytes);
            __syncwarp();
            if (ok) {
#pragma unroll
              for (int h = 0; h < 2; ++h)
                tma_load(base + W_V + v.st * W_TILE + h * W_HALF + lane * rows * 128, &tmV, 64 * h, 2 * pair + f, row, bar(WV_FULL + v.st));
            }
          }
          pid = pid1;   // looked up two blocks ahead
          pid1 = page_of(j + 2);
        }
        ++np;
      }
      // the copies are over before the CTA ends, also where a wait ran out
      for (unsigned i = n > 2 ? n - 2 : 0; i < n; ++i) wait_phase(bar(WK_FULL + (i & 1)), (i >> 1) & 1, a.err, dead);
      for (unsigned h = 2 * n > 3 ? 2 * n - 3 : 0; h < 2 * n; ++h) {
        const VStage v(h);
        wait_phase(bar(WV_FULL + v.st), v.use & 1, a.err, dead);
      }
      if (*dead)
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    } else {
      // -------------------- V: rows past the end or another pass's, odd values
      unsigned np = 0, n = 0;
      while (walk.next(a, sh, p)) {
        if (p.nblk == 0) continue;
        int lo0, hi0, lo1, hi1;
        visible_keys(a, p.s, p.s.kv - p.s.n + p.i0, lo0, hi0);
        visible_keys(a, p.s, p.s.kv - p.s.n + p.i1, lo1, hi1);
        for (int j = 0; j < p.nblk; ++j, ++n) {
          const int key0 = (p.blk0 + j) * BKEYS, live = min(BKEYS, p.s.kv - key0), first = p.s.from - key0;
          const bool partial = key0 < lo1 || key0 + BKEYS > hi0;
#pragma unroll 1
          for (int f = 0; f < 2; ++f) {
            const VStage v(2 * n + f);
            wait_phase(bar(WV_FULL + v.st), v.use & 1, a.err, dead);
            if (partial) {
              const uint32_t vd = base + W_V + v.st * W_TILE;
              bool found = false;
              for (int i = tid - 320; i < W_TILE / 16; i += 64) {
                const int r = (i >> 3) & (TROWS - 1);   // chunk i of the tile lies in row r of its half
                if (r >= live || r < first) {
                  sts128(vd + i * 16, make_uint4(0u, 0u, 0u, 0u));
                } else {
                  uint4 y = lds128(vd + i * 16);
                  if (odd16<T>(y)) {
                    y = make_uint4(without_odd16<T>(y.x), without_odd16<T>(y.y), without_odd16<T>(y.z), without_odd16<T>(y.w));
                    sts128(vd + i * 16, y);
                    found = true;
                  }
                }
              }
              if (found) s_odd[np & 3] = np + 1;
              fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(WV_READY + v.st));
          }
        }
        ++np;
      }
    }
  } else {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int t = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t mS = tmS + 128 * t + lanes, mO = tmO + lanes;
    unsigned np = 0, jobs = 0, others = 0;             // pieces, this group's and the other's jobs
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
      const int ta = pc.i0, tb = min(ta + per, pc.s.n) - 1;   // the tile's tokens
      int lo, hi, lo_last, hi_first;                   // keys that the row sees; that every row of the tile sees
      float m_first;                                   // infinite for rows past the tile's tokens, which never ask for a rescaling
      {
        const int first_pos = pc.s.kv - pc.s.n;
        int none;
        visible_keys(a, pc.s, first_pos + min(ta + row / a.G, tb), lo, hi);
        visible_keys(a, pc.s, first_pos + ta, none, hi_first);
        visible_keys(a, pc.s, first_pos + tb, lo_last, none);
        m_first = row < (tb - ta + 1) * a.G ? -INFINITY : INFINITY;
      }
      const float sl = a.sl2;
      const f2x sl_2 = pack2(sl, sl);
      float m = m_first;            // what the group's sum is relative to
      f2x l2[4] = {pack2(0.f, 0.f), pack2(0.f, 0.f), pack2(0.f, 0.f), pack2(0.f, 0.f)};
      for (int j = t; j < nblk; j += 2, ++jobs) {
        const int key0 = (blk0 + j) * BKEYS;
        wait_phase(bar(WS_FULL + t), jobs & 1, a.err, dead);
        tm_fence_after();
        uint32_t sr[32];
        const bool partial = key0 < lo_last || key0 + BKEYS > hi_first;
        auto mask32 = [&](int c0) {
          const int from = lo - key0 - c0, cn = hi - lo;
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if ((unsigned)(c - from) >= (unsigned)cn) sr[c] = 0xff800000u;
        };
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
        for (int c = 0; c < BKEYS; c += 32) {
          tm_ld32(mS + c, sr);
          tm_wait_ld();
          if (partial) mask32(c);
#pragma unroll
          for (int i = 0; i < 32; i += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mx[e] = fmaxf(fmaxf(mx[e], __uint_as_float(sr[i + 2 * e])), __uint_as_float(sr[i + 2 * e + 1]));
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl - BIAS;
        float mn = fmaxf(m_first, top);
        if (j > 0) {
          // the other group's maximum behind block j - 1: its ((j - 1) / 2)-th of this piece
          const unsigned seen = others + (unsigned)((j - 1) >> 1);
          wait_phase(bar(WM_READY + 1 - t), seen & 1, a.err, dead);
          const float old = *(volatile float*)&s_m[row];
          mn = fmaxf(old, top);
          if (__any_sync(FULL, mn > old + RESCALE)) {
            // The product of block j - 1, on the barrier of the other group's products, where no other phase can be
            // taken for it: the one before, of block j - 3, is over (the other group's scores of block j - 1, whose
            // maximum is here, were issued behind it), and the next, of block j + 1, waits for this group's P.
            wait_phase(bar(WO_STEP + 1 - t), seen & 1, a.err, dead);
            tm_fence_after();
            const float f = fast_exp2(old - (mn > -INFINITY ? mn : 0.f));
#pragma unroll 1
            for (int c = 0; c < 2 * WD; c += 16) {
              uint32_t o[16];
              tm_ld16(mO + c, o);
              tm_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tm_st16(mO + c, o);
            }
          } else {
            mn = old;
          }
        }
        s_m[row] = mn;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(WM_READY + t));
        if (mn != m) {   // grown, here or there, since this group's last block
          const float f = fast_exp2(m - mn);
#pragma unroll
          for (int e = 0; e < 4; ++e) l2[e] = mul2(l2[e], pack2(f, f));
          m = mn;
        }
        const float neg = m > -INFINITY ? -m : 0.f;
        const f2x neg2 = pack2(neg, neg);
#pragma unroll 1
        for (int c = 0; c < BKEYS; c += 32) {
          uint32_t pk[16];
          tm_ld32(mS + c, sr);
          tm_wait_ld();
          if (partial) mask32(c);
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float2 y0 = unpack2(ffma2(pack2(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])), sl_2, neg2));
            const float2 y1 = unpack2(ffma2(pack2(__uint_as_float(sr[e + 2]), __uint_as_float(sr[e + 3])), sl_2, neg2));
            const float p0 = fast_exp2(y0.x), p1 = fast_exp2(y0.y), p2 = fast_exp2(y1.x), p3 = fast_exp2(y1.y);
            l2[(e >> 1) & 3] = add2(l2[(e >> 1) & 3], pack2(p0, p1));
            l2[((e >> 1) + 1) & 3] = add2(l2[((e >> 1) + 1) & 3], pack2(p2, p3));
            pk[e / 2] = pack2h<T>(p0, p1);
            pk[e / 2 + 1] = pack2h<T>(p2, p3);
          }
          tm_st16(mS + c / 2, pk);
        }
        tm_wait_st();
        tm_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(WP_FULL + t));
      }
      // ------------------------------------------------------- the result
      float l = 0.f;
      {
        const float2 lp = unpack2(add2(add2(l2[0], l2[1]), add2(l2[2], l2[3])));
        l = lp.x + lp.y;
      }
      if (nblk > 0) {
        wait_phase(bar(WO_DONE), np & 1, a.err, dead);
        tm_fence_after();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(WPIECE_SEEN));
        float(&ml)[2][2][TROWS] = s_ml[np & 1];
        ml[t][0][row] = m;
        ml[t][1][row] = l;
        group_sync(2, 256);
        const float m0 = ml[0][0][row], m1 = ml[1][0][row];
        m = fmaxf(m0, m1);
        const float mu = m > -INFINITY ? m : 0.f;
        l = ml[0][1][row] * fast_exp2(m0 - mu) + ml[1][1][row] * fast_exp2(m1 - mu);
      }
      const bool bad = nblk > 0 && s_bad[np & 3] == (int)np + 1, odd = nblk > 0 && s_odd[np & 3] == (int)np + 1;
      const int tok = min(ta + row / a.G, tb), pair = pc.kvh >> 1, map = pc.kvh & 1;
      const bool live_row = row < per * a.G && ta + row / a.G <= tb;
      const long long at = (pc.s.q0 + tok) * a.H + 2 * (pair * a.G + row % a.G) + map;
      const long long part = ((long long)blockIdx.x * 2 + (pc.pos > sh.lo)) * a.rows + row;
      float* const to_o = (pc.whole ? a.row_o + at * (2 * WD) : a.part_o + part * (2 * WD)) + t * WD;
      float* const to_ml = pc.whole ? a.row_ml + at * 2 : a.part_ml + part * 2;
#pragma unroll 1
      for (int c = 0; c < WD; c += 32) {
        uint32_t o[32];
        if (nblk > 0) {
          tm_ld32(mO + t * WD + c, o);
          tm_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        if (nblk > 0 && c + 32 == WD) {
          tm_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(WO_FREE));
        }
        if (live_row) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) st_global8(to_o + c + e, o + e);
        }
      }
      if (live_row && t == 0) {
        to_ml[0] = m;
        to_ml[1] = bad ? -1.f : l;
      }
      if (odd) {   // what was taken out of V, to the rows that see its key (see santa_chunk.cuh)
        int clean_lo, clean_hi, none;
        visible_keys(a, pc.s, pc.s.kv - pc.s.n + pc.i0, none, clean_hi);
        visible_keys(a, pc.s, pc.s.kv - pc.s.n + pc.i1, clean_lo, none);
        const int32_t* const table = page_row(a, pc.b);
        const int end = min(pc.s.kv, (blk0 + nblk) * BKEYS);
#pragma unroll 1
        for (int key0 = blk0 * BKEYS; key0 < end; key0 += 32) {
          const int block = key0 & -BKEYS, key = key0 + lane;
          if (block >= clean_lo && block + BKEYS <= clean_hi) continue;
          const int pid = key < end && key >= pc.s.from ? table[key >> a.page_shift] : -1;
          long long at_v = 0;
          bool found = false;
          if ((unsigned)pid < (unsigned)a.n_pages) {
            at_v = ((((long long)pid << a.page_shift) + (key & ((1 << a.page_shift) - 1))) * a.Hkv + 2 * pair + t) * WD;
            const uint4* const v = reinterpret_cast<const uint4*>(static_cast<const T*>(a.V) + at_v);
#pragma unroll 4
            for (int q = 0; q < WD / 8; ++q) found |= odd16<T>(v[q]);
          }
          for (unsigned keys = __ballot_sync(FULL, found); keys; keys &= keys - 1) {
            const int u = __ffs(keys) - 1;
            const long long at_u = __shfl_sync(FULL, at_v, u);
            if (!live_row || key0 + u < lo || key0 + u >= hi) continue;
            const uint32_t* const v = reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.V) + at_u);
#pragma unroll 1
            for (int e = 0; e < WD / 2; ++e) {
              const float2 y = unpack2h<T>(v[e]);
              if (!(fabsf(y.x) <= 3.402823466e38f)) to_o[2 * e] += y.x;
              if (!(fabsf(y.y) <= 3.402823466e38f)) to_o[2 * e + 1] += y.y;
            }
          }
        }
      }
      if (nblk > 0) ++np;
      others += (unsigned)(t == 0 ? nblk >> 1 : (nblk + 1) >> 1);
    }
    tm_fence_before();
  }
  __syncthreads();
  if (warp == 8) {
    tm_fence_after();
    tm_free(tm, 512);
  }
  if (blockIdx.x == 0) wait_for_predecessor();   // not over before the pass that it may have started under
}

template <typename T>
cudaError_t inst(const JoinArgs& a, bool behind) {
  auto kern = diff_wide_kernel<T>;
  static std::atomic<unsigned long long> raised{0};
  const cudaError_t e = raise_smem((const void*)kern, W_SMEM, raised);
  if (e != cudaSuccess) return e;
  CUtensorMap tq, tk, tv;
  if (!encode_pairs(&tq, a.q, WD, a.H, a.total_q, a.G, TROWS / a.G) || !encode_cache<false, WD>(&tk, a, a.K) ||
      !encode_cache<false, WD>(&tv, a, a.V))
    return cudaErrorInvalidValue;
  return launch_pass(kern, (unsigned)a.splits, W_THREADS, W_SMEM, a.stream, behind, tq, tk, tv, a);
}

}  // namespace

cudaError_t launch_diff_wide(const JoinArgs& a, bool behind) {
  return a.dtype == 0 ? inst<bf16_t>(a, behind) : inst<fp16_t>(a, behind);
}

}  // namespace santa
