// Walks the shares of all CTAs of the chunk attention on the host, with the
// kernel's own arithmetic, and checks that every item is computed once.
//
// stdin: calls of "ctas q_heads kv_heads causal window nk max_q batch", then
// kv_lens and the numbers of new tokens.  stdout, for each: items, whether they
// are shared, then the number of items that were not computed exactly once and
// of those whose merge would not find exactly its pieces.
#include <cstdio>
#include <map>
#include <tuple>
#include <vector>

#include "santa_chunk_share.cuh"

using namespace santa;

struct Part {
  int cta, slot, blk0, nblk;
  bool whole;
};

int main() {
  int P0, H, Hkv, causal, window, nk, max_q, B;
  while (std::scanf("%d %d %d %d %d %d %d %d", &P0, &H, &Hkv, &causal, &window, &nk, &max_q, &B) == 8) {
    std::vector<int> kv(B), n(B);
    for (int& x : kv) if (std::scanf("%d", &x) != 1) return 1;
    for (int& x : n) if (std::scanf("%d", &x) != 1) return 1;
    std::vector<int64_t> off(B + 1, 0);
    for (int b = 0; b < B; ++b) off[b + 1] = off[b] + n[b];
    PagedArgs a = {};
    a.B = B, a.H = H, a.Hkv = Hkv, a.G = H / Hkv;
    a.kv_lens = kv.data(), a.q_offsets = off.data();
    a.nk = nk, a.max_q = max_q, a.total_q = off[B];
    a.causal = causal, a.window = window < nk ? window : 0;
    a.rows = 256, a.tokens = 2 * (128 / a.G);
    a.tiles = (max_q + a.tokens - 1) / a.tokens;

    long long total = 0, items = 0;
    int most = 0;
    for (long long i = 0; i < (long long)B * a.tiles; ++i) {
      const int w = item_weight(a, i, false);
      total += w, items += w > 0, most = std::max(most, w);
    }
    const long long T = total * Hkv;
    const long long places = std::min<long long>(P0, (long long)B * Hkv * a.tiles * chunk_blocks(a));
    const int P = (int)std::min(places, T);
    std::map<std::tuple<int, int, int>, std::vector<Part>> parts;
    std::map<std::tuple<int, int, int>, std::vector<ChunkShare>> notes;
    int split = 0;
    for (int c = 0; c < P; ++c) {
      Share sh = {};
      sh.T = T, sh.P = P, sh.b = B;
      sh.lo = share_begin(T, c, P), sh.hi = share_begin(T, c + 1, P);
      sh.split = share_split(T, P, items * Hkv, most);
      split |= sh.split;
      long long first = 0;
      for (long long i = 0; i < (long long)B * a.tiles; ++i) {
        const int w = item_weight(a, i, false);
        share_place(a, sh, sh.lo, i, first, w);
        first += w;
      }
      Walk walk;
      walk.start(a, sh);
      Piece p;
      for (int slot = 0; walk.next(a, sh, p); slot = 1) {
        const auto item = std::make_tuple(p.b, p.tile, p.kvh);
        parts[item].push_back({c, slot, p.blk0, p.nblk, p.whole});
        if (p.nblk > 0 && sh.split && !p.whole && p.last) notes[item].push_back(share_note(sh, p, c));
      }
    }
    int bad = 0, bad_merge = 0;
    for (int b = 0; b < B; ++b)
      for (int tile = 0; tile * a.tokens < n[b]; ++tile) {
        int i0, i1;
        tile_tokens(a, n[b], tile, i0, i1);
        const TileKeys tk = tile_keys(a, paged_seq(a, b, false), i0, i1, BKEYS);
        for (int kvh = 0; kvh < Hkv; ++kvh) {
          const auto item = std::make_tuple(b, tile, kvh);
          const std::vector<Part>& ps = parts[item];
          const std::vector<ChunkShare>& ns = notes[item];
          int at = tk.blk_lo, wholes = 0;
          bool fine = !ps.empty();
          for (const Part& p : ps) {
            fine &= p.nblk == 0 || p.blk0 == at;
            at += p.nblk;
            wholes += p.whole;
          }
          bad += !(fine && at == tk.blk_lo + tk.blk && wholes == (ps.size() == 1));
          bool merged = ns.size() == (ps.size() > 1 || wholes == 0);
          for (const ChunkShare& r : ns) {
            merged &= wholes == 0 && r.count == (int)ps.size();
            for (size_t k = 0; merged && k < ps.size(); ++k)
              merged = ps[k].cta == r.first + (int)k && ps[k].slot == (k == 0 ? r.slot : 0);
          }
          bad_merge += !merged;
        }
      }
    std::printf("%lld %d %d %d\n", items * Hkv, split, bad, bad_merge);
  }
  return 0;
}
