// santa_chunk_share.cuh -- how the chunk attention's blocks of keys are divided
// over its CTAs: plain arithmetic on the lengths, the same in the kernel and on
// the host (where a test walks the shares of all CTAs).
#pragma once

#include <algorithm>

#include "santa_paged.cuh"

namespace santa {

constexpr int BKEYS = PG_CHUNK_KEYS;   // keys per block
constexpr int CHUNK_SHARE = 8;         // blocks of time that sharing an item costs
constexpr int CHUNK_LEAST = 16;        // items of no more blocks are never shared, and no merge is launched for them

// One CTA's share of the batch.  Items in the order (sequence, tile, KV head)
// weigh their blocks (at least one); CTA c of P takes the blocks
// [floor(T c / P), floor(T (c + 1) / P)) of the T, or (`split` false) the items
// that begin in that range.  Every role of the CTA walks the same pieces.
struct Share {
  long long lo, hi, T;
  int P, split;
  int b, kvh, tile;   // the item that holds block lo
  long long pos;      // its first block
  int known, i0, i1;  // whether its sequence, tokens and keys are here, too
  Seq s;
  TileKeys tk;
};
SANTA_HD long long share_begin(long long T, int c, int P) {
  if (T < (1ll << 24)) return (unsigned)T * (unsigned)c / (unsigned)P;   // c < 256
  return T * c / P;
}
struct Piece {
  int b, kvh, tile;
  Seq s;
  int i0, i1;         // first and last token
  int blk0, nblk;     // blocks of this piece (0: no key is visible)
  bool two;           // the second tile holds tokens
  bool whole, last;   // of the item: all its blocks, its last one
  long long pos;      // the item's first block
};
struct Walk {
  int b, kvh, tile, i0, i1;
  TileKeys tk;
  long long pos;
  Seq s;
  template <typename A>
  SANTA_HD void start(const A& a, const Share& sh) {
    b = sh.b;
    kvh = sh.kvh;
    tile = sh.tile;
    pos = sh.pos;
    if (sh.known) {   // looked up once for all roles
      s = sh.s;
      i0 = sh.i0;
      i1 = sh.i1;
      tk = sh.tk;
    } else if (b < a.B) {
      load(a);
    }
  }
  template <typename A>
  SANTA_HD void load(const A& a) {   // a sequence and its tile
    s = paged_seq(a, b, false);
    keys(a);
  }
  template <typename A>
  SANTA_HD void keys(const A& a) {
    tile_tokens(a, s.n, tile, i0, i1);
    tk = tile_keys(a, s, i0, i1, BKEYS);
  }
  template <typename A>
  SANTA_HD bool next(const A& a, const Share& sh, Piece& p) {
    for (;;) {
      if (b >= a.B || pos >= sh.hi) return false;
      if (kvh == item_heads(a) || tile * a.tokens >= s.n) {
        kvh = 0;
        if (++tile * a.tokens >= s.n) {
          tile = 0;
          if (++b < a.B) load(a);
        } else {
          keys(a);
        }
        continue;
      }
      const int w = max(tk.blk, 1);
      long long begin = max(sh.lo, pos) - pos, end = min(sh.hi, pos + w) - pos;
      if (!sh.split) {
        begin = pos >= sh.lo ? 0 : w;
        end = w;
      }
      p.pos = pos;
      p.kvh = kvh;
      ++kvh;
      pos += w;
      if (begin >= end) continue;
      p.b = b;
      p.tile = tile;
      p.s = s;
      p.i0 = i0;
      p.i1 = i1;
      p.blk0 = tk.blk_lo + (int)begin;
      p.nblk = tk.blk ? (int)(end - begin) : 0;
      p.two = i0 + a.tokens / 2 < s.n;
      p.whole = end - begin == w;
      p.last = end == w;
      return true;
    }
  }
};

// Item i = (sequence, tile): its blocks w, at least one, 0 where the tile has no token.
struct Item {
  int w, b, tile, i0, i1;
  Seq s;
  TileKeys tk;
};
template <typename A>
SANTA_HD Item item_at(const A& a, long long i, bool flag) {
  Item x;
  x.w = 0;
  if (i >= (long long)a.B * a.tiles) return x;
  x.b = i < (1ll << 31) ? (int)((unsigned)i / (unsigned)a.tiles) : (int)(i / a.tiles);   // 32-bit division takes a fifth of the time
  x.tile = (int)(i - (long long)x.b * a.tiles);
  x.s = paged_seq(a, x.b, flag && x.tile == 0);
  if (x.tile * a.tokens >= x.s.n) return x;
  tile_tokens(a, x.s.n, x.tile, x.i0, x.i1);
  x.tk = tile_keys(a, x.s, x.i0, x.i1, BKEYS);
  x.w = max(x.tk.blk, 1);
  return x;
}
template <typename A>
SANTA_HD int item_weight(const A& a, long long i, bool flag) {
  return item_at(a, i, flag).w;
}
SANTA_HD long long quotient(long long n, int d) {   // of numbers that are small as a rule
  return n < (1ll << 31) ? (long long)((unsigned)n / (unsigned)d) : n / d;
}

// Whether items are shared between CTAs, from their number, the blocks of the
// largest one and the total of T blocks over P CTAs.  A shared item costs about
// CHUNK_SHARE blocks of time (its sums out and in again); without sharing the
// longest CTA has about ceil(items / P) of the largest items.  Nothing here
// differs between CTAs (their shares do, by one block): an item that one CTA
// leaves to be shared and the next one does not take up would be lost.
SANTA_HD bool share_split(long long T, int P, long long items, int most) {
  const long long each = items <= P ? 1 : quotient(items + P - 1, P);
  return most > CHUNK_LEAST && each * most > quotient(T, P) + CHUNK_SHARE;
}
// Of P CTAs those that take part.
SANTA_HD int share_ctas(const PagedArgs&, long long, int P, long long, int) { return P; }
SANTA_HD bool item_split(const PagedArgs&, long long T, int P, long long items, int most) { return share_split(T, P, items, most); }
// The item that holds block lo, if it is item i = (sequence, tile), of w blocks
// per KV head, whose blocks of one head begin at `first`.
template <typename A>
SANTA_HD void share_place(const A& a, Share& sh, long long lo, long long i, long long first, int w) {
  const long long pos = first * item_heads(a);
  if (w == 0 || lo < pos || lo >= pos + (long long)w * item_heads(a)) return;
  sh.b = (int)(i / a.tiles);
  sh.tile = (int)(i - (long long)sh.b * a.tiles);
  sh.kvh = (int)(lo - pos) / w;
  sh.pos = pos + (long long)sh.kvh * w;
}
template <typename A>
SANTA_HD void share_place(const A& a, Share& sh, long long lo, long long first, const Item& x) {
  const long long pos = first * item_heads(a);
  if (x.w == 0 || lo < pos || lo >= pos + (long long)x.w * item_heads(a)) return;
  sh.b = x.b;
  sh.tile = x.tile;
  sh.kvh = (int)(lo - pos) / x.w;
  sh.pos = pos + (long long)sh.kvh * x.w;
  sh.s = x.s;
  sh.i0 = x.i0;
  sh.i1 = x.i1;
  sh.tk = x.tk;
  sh.known = 1;
}
// What CTA `cta`, which has the last piece of a shared item, leaves for the merge.
SANTA_HD ChunkShare share_note(const Share& sh, const Piece& p, int cta) {
  int c = (int)(p.pos * sh.P / sh.T);        // the CTA whose share holds the item's first block
  while (c + 1 < sh.P && share_begin(sh.T, c + 1, sh.P) <= p.pos) ++c;
  ChunkShare r;
  r.b = p.b;
  r.kvh = p.kvh;
  r.tile = p.tile;
  r.first = c;
  r.slot = share_begin(sh.T, c, sh.P) == p.pos ? 0 : 1;
  r.count = cta - c + 1;
  return r;
}

// Most blocks of keys of one item.
inline int chunk_blocks(const PagedArgs& a) {
  const int span = a.window ? (int)std::min<long long>(a.nk, (long long)a.window + a.tokens) : a.nk;
  return (span + BKEYS - 1) / BKEYS + (a.window ? 1 : 0);
}
inline bool chunk_may_share(const PagedArgs& a) { return chunk_blocks(a) > CHUNK_LEAST; }

}  // namespace santa
