// Walks the shares of all CTAs of the joined passes of chunks on the host, with
// the kernels' own arithmetic: over the groups' prefixes (phase 1) and over what
// each sequence has of its own (phase 2).
//
// stdin: calls of "ctas q_heads kv_heads diff parts causal nk max_q max_prefix
// max_own max_group batch groups", then kv_lens, the numbers of new tokens, the
// groups' offsets (groups + 1) and prefixes.  stdout, for each call and phase:
// items, items not computed exactly once, notes that are missing or wrong,
// blocks outside the keys of the phase, and sequences refused.
#include <cstdio>
#include <map>
#include <tuple>
#include <vector>

#include "santa_join.cuh"

using namespace santa;

struct Part {
  int cta, slot, blk0, nblk;
  bool whole, last;
};

int main() {
  int P0, H, Hkv, diff, parts, causal, nk, max_q, max_prefix, max_own, max_group, B, groups;
  while (std::scanf("%d %d %d %d %d %d %d %d %d %d %d %d %d", &P0, &H, &Hkv, &diff, &parts, &causal, &nk, &max_q, &max_prefix,
                    &max_own, &max_group, &B, &groups) == 13) {
    std::vector<int> kv(B), n(B), first(groups + 1), prefix(groups);
    for (auto* v : {&kv, &n, &first, &prefix})
      for (int& x : *v) if (std::scanf("%d", &x) != 1) return 1;
    std::vector<int64_t> off(B + 1, 0);
    for (int b = 0; b < B; ++b) off[b + 1] = off[b] + n[b];
    for (int phase = 1; phase <= 2; ++phase) {
      JoinArgs a = {};
      a.H = H, a.Hkv = Hkv, a.G = H / Hkv, a.seqs = B, a.seq_q = max_q;
      a.kv_lens = kv.data(), a.q_offsets = off.data();
      a.nk = nk, a.total_q = off[B], a.causal = causal;
      a.phase = phase, a.diff = diff, a.n_groups = groups;
      a.group_offsets = first.data(), a.prefix_lens = prefix.data();
      a.max_prefix = max_prefix, a.max_own = max_own;
      a.group_q = (int)std::min<long long>((long long)max_group * max_q, a.total_q);
      a.B = phase == 1 ? groups : B, a.max_q = phase == 1 ? a.group_q : max_q;
      a.chunk = 1, a.heads = x_items(a) * parts;
      a.rows = 2 * CHUNK_ROWS, a.tokens = (diff ? 1 : 2) * (CHUNK_ROWS / a.G);
      a.tiles = (a.max_q + a.tokens - 1) / a.tokens;
      const int span = phase == 1 ? max_prefix : max_own;
      const long long blocks = (span + BKEYS - 1) / BKEYS + (phase == 2);
      const int places = (int)std::min<long long>(P0, (long long)a.B * a.heads * a.tiles * blocks);

      long long total = 0, items = 0;
      int most = 0, refused = 0;
      for (int b = 0; b < B; ++b) refused += phase == 2 && !paged_seq(a, b, false).ok;
      for (long long i = 0; i < (long long)a.B * a.tiles; ++i) {
        const int w = item_weight(a, i, false);
        total += w, items += w > 0, most = std::max(most, w);
      }
      const long long T = total * a.heads;
      const int P = share_ctas(a, T, (int)std::min<long long>(places, T), items * a.heads, most);
      std::map<std::tuple<int, int, int>, std::vector<Part>> got;
      std::map<std::tuple<int, int, int>, std::vector<PieceNote>> notes;
      int outside = 0;
      for (int c = 0; c < P; ++c) {
        Share sh = {};
        sh.T = T, sh.P = P, sh.b = a.B;
        sh.lo = share_begin(T, c, P), sh.hi = share_begin(T, c + 1, P);
        sh.split = item_split(a, T, P, items * a.heads, most);
        long long at = 0;
        for (long long i = 0; i < (long long)a.B * a.tiles; ++i) {
          const int w = item_weight(a, i, false);
          share_place(a, sh, sh.lo, i, at, w);
          at += w;
        }
        Walk walk;
        walk.start(a, sh);
        Piece p;
        for (int slot = 0; walk.next(a, sh, p); slot = 1) {
          const auto item = std::make_tuple(p.b, p.tile, p.kvh);
          got[item].push_back({c, slot, p.blk0, p.nblk, p.whole, p.last});
          outside += p.nblk > 0 && (p.blk0 * BKEYS + BKEYS <= p.s.from || (p.blk0 + p.nblk - 1) * BKEYS >= p.s.kv);
          if (p.last) {
            PieceNote note = {0, 0, 0, 0};
            if (!p.whole) {
              const ChunkShare r = share_note(sh, p, c);
              note.first = r.first, note.slot = r.slot, note.count = r.count;
            }
            notes[item].push_back(note);
          }
        }
      }
      int bad = 0, bad_note = 0;
      for (int b = 0; b < a.B; ++b) {
        const Seq s = paged_seq(a, b, false);
        for (int tile = 0; tile * a.tokens < s.n; ++tile) {
          int i0, i1;
          tile_tokens(a, s.n, tile, i0, i1);
          const TileKeys tk = tile_keys(a, s, i0, i1, BKEYS);
          bad += tile >= a.tiles;
          for (int x = 0; x < a.heads; ++x) {
            const std::vector<Part>& ps = got[std::make_tuple(b, tile, x)];
            const std::vector<PieceNote>& ns = notes[std::make_tuple(b, tile, x)];
            int at = tk.blk_lo, wholes = 0;
            bool fine = !ps.empty();
            for (const Part& p : ps) {
              fine &= p.nblk == 0 || p.blk0 == at;
              at += p.nblk;
              wholes += p.whole;
            }
            bad += !(fine && at == tk.blk_lo + tk.blk && wholes == (ps.size() == 1));
            bool found = ns.size() == 1 && ns[0].count == (wholes ? 0 : (int)ps.size());
            if (found && !wholes)
              for (size_t k = 0; k < ps.size(); ++k)
                found &= ps[k].cta == ns[0].first + (int)k && ps[k].slot == (k == 0 ? ns[0].slot : 0);
            bad_note += !found;
          }
        }
      }
      std::printf("%d %lld %d %d %d %d\n", phase, items * a.heads, bad, bad_note, outside, refused);
    }
  }
  return 0;
}
