// santa_join.cuh -- attention in passes whose sums a later kernel joins: what a
// group of sequences has in common (one pass, once for all of them), what each
// has of its own (another), and the two maps of differential heads.
//
// A pass is the paged attention's kernels over a batch of its own: phase 0 and 2
// over the batch's sequences (all keys, or those behind their group's prefix),
// phase 1 over the groups, whose "sequence" is the tokens of all their
// sequences and the keys of the prefix.  A row's sums are a maximum m, l = sum
// of 2^(s - m), o = sum of 2^(s - m) V; sums of disjoint sets of keys join as
// m* = max m_i, l = sum l_i 2^(m_i - m*), o alike.
#pragma once

#include "santa_chunk_share.cuh"
#include "santa_paged.cuh"

namespace santa {

constexpr int CHUNK_ROWS = 128;    // rows of a tile of the chunk attention
constexpr int ERR_PREFIX = 128;    // groups or prefixes that do not fit the batch

// Where the pieces of an item of the chunk attention are: slot `slot` of CTA
// `first` and slot 0 of the following ones, or (count 0) in the rows.
struct PieceNote {
  int first, slot, count, none;
};

struct JoinArgs : PagedArgs {
  int phase;
  int chunk;                       // the pass's kernel: 0 few rows, 1 chunks
  int heads;                       // items per tile
  int seqs, seq_q;                 // of the batch: sequences, most new tokens of one
  int n_groups, group_q;           // groups (0: none), most new tokens of one
  const int32_t* group_offsets;
  const int32_t* prefix_lens;
  int max_prefix, max_own;
  float* row_o;                    // chunks: sums of items that one CTA has whole, [total_q, H, width]
  float* row_ml;                   // [total_q, H, 2]; 2 x 2, one for each value head, in a differential e4m3 pass of chunks
  PieceNote* notes;                // chunks: [total_q, heads], at an item's first token
  int sources;                     // pieces of a row, about
  // differential heads: the weights of the second maps, the norm behind them
  int diff, one_map;               // one_map: an item is a map, over the columns of both value heads (santa_diff_wide.cu)
  const float* lambda;
  long long lambda_stride;         // from token to token (0: the same for all)
  const void* norm;                // [2 D] or null
  float eps, gain;
};

// A group's sequences [first, last), tokens and prefix.
struct Group {
  int first, last, n, prefix;
  long long q0;
  bool ok;
};
SANTA_HD Group group_at(const JoinArgs& a, int g) {
  Group r;
  r.first = a.group_offsets ? a.group_offsets[g] : 0;
  r.last = a.group_offsets ? a.group_offsets[g + 1] : a.seqs;
  r.prefix = a.prefix_lens[g];
  r.ok = r.first >= 0 && r.last >= r.first && r.last <= a.seqs && r.prefix >= 0 && r.prefix <= a.max_prefix;
  long long lo = 0, hi = 0;
  if (r.ok) {
    lo = a.q_offsets ? a.q_offsets[r.first] : (long long)r.first * a.seq_q;
    hi = a.q_offsets ? a.q_offsets[r.last] : (long long)r.last * a.seq_q;
    r.ok = lo >= 0 && hi >= lo && hi <= a.total_q && hi - lo <= a.group_q;
  }
  r.q0 = r.ok ? lo : 0;
  r.n = r.ok ? (int)(hi - lo) : 0;
  if (!r.ok) r.prefix = 0;
  return r;
}
// The last group that begins at or before sequence b.
SANTA_HD int group_of(const JoinArgs& a, int b) {
  if (!a.group_offsets) return 0;
  int lo = 0, hi = a.n_groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.group_offsets[mid] <= b) lo = mid;
    else hi = mid;
  }
  return lo;
}

// In phase 2 a sequence is refused whose group is, that no group holds, whose
// tokens are not among the group's (whose range two offsets give, those between
// them may be anything; the join finds a token's sums by its place there), whose
// new tokens begin inside the prefix, or with more keys of its own than stated.
SANTA_HD Seq paged_seq(const JoinArgs& a, int b, bool flag) {
  bool fine = true;
  Seq s;
  if (a.phase == 1) {
    const Group g = group_at(a, b);
    s.q0 = g.q0;
    s.n = g.n;
    s.kv = g.prefix;
    s.from = 0;
    s.ok = fine = g.ok;
  } else {
    s = paged_seq(static_cast<const PagedArgs&>(a), b, flag);
    if (a.phase == 2) {
      const Group g = group_at(a, group_of(a, b));
      fine = g.ok && g.first <= b && b < g.last;
      if (s.ok) fine = fine && s.n <= g.n && (unsigned)((int)s.q0 - (int)g.q0) <= (unsigned)(g.n - s.n) && g.prefix <= (a.causal ? max(s.kv - s.n, 0) : s.kv) && s.kv - g.prefix <= a.max_own;
      s.from = fine ? g.prefix : 0;
      if (!fine) s.kv = 0;
      s.ok = s.ok && fine;
    }
  }
#ifdef __CUDA_ARCH__
  if (!fine && flag) flag_error(a.err, ERR_PREFIX);
#endif
  return s;
}
SANTA_HD void visible_keys(const JoinArgs& a, const Seq& s, int pos, int& lo, int& hi) {
  if (a.phase == 1) {   // every token of a group stands behind its prefix
    lo = 0;
    hi = s.kv;
    return;
  }
  visible_keys(a, s.kv, pos, lo, hi);
  lo = min(max(lo, s.from), hi);
}
SANTA_HD int item_heads(const JoinArgs& a) { return a.heads; }
SANTA_HD int x_items(const JoinArgs& a) { return a.diff ? a.Hkv / 2 : a.Hkv; }   // KV heads, or pairs of them
// The sums of a pass are joined in any case, so that sharing an item costs little.
constexpr int JOIN_SHARE = 2;
SANTA_HD bool item_split(const JoinArgs&, long long T, int P, long long items, int most) {
  const long long each = items <= P ? 1 : quotient(items + P - 1, P);
  return most > 1 && each * most > quotient(T, P) + JOIN_SHARE;
}
// Items that are all as long (one group's) are divided into the same number of
// pieces each, so that no CTA has the end of one and the start of another: the
// second piece costs 8 us.  32 differential tokens behind 16384 keys, 8 items:
// 43.8 us with 96 CTAs, 49.0 with 95.
SANTA_HD int share_ctas(const JoinArgs&, long long T, int P, long long items, int most) {
  return items > 0 && items <= P && items * most == T ? P / (int)items * (int)items : P;   // 0: every group is refused or empty
}
// A group's prefix is looked up in the table's row of its first sequence.
SANTA_HD const int32_t* page_row(const JoinArgs& a, int b) {
  const int row = a.phase == 1 ? (a.group_offsets ? a.group_offsets[b] : 0) : b;
  return a.table + (long long)row * a.max_pages;
}

struct Passes {
  JoinArgs p[2];   // over the prefixes (n_groups 0: none), over what each sequence has of its own
};
// CTAs of a pass of few rows.
inline long long tokens_grid(const JoinArgs& a) { return (long long)a.B * a.tiles * a.heads * a.splits; }

// A launch that may start while the kernel before it in the stream still runs (`behind`; programmatic dependent launch).
template <typename... P, typename... X>
cudaError_t launch_pass(void (*kern)(P...), unsigned grid, int block, size_t smem, cudaStream_t stream, bool behind, const X&... x) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = behind ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, x...);
}

// Plans and launches of one pass, and of the kernel that joins two (prefixes.B = 0: none).
void plan_tokens(PagedArgs& a, int span, int more_blocks, int round = 0);   // sets rows, tiles, splits, split_blk
void plan_splits(PagedArgs& a, long long pieces, long long places, int blks, int fine_blks);
// `behind`: starts under the pass before it; `prefixes`: in the same launch, of few rows too
cudaError_t launch_join_tokens(const JoinArgs* prefixes, const JoinArgs& a, bool behind);
cudaError_t launch_join_chunk(const JoinArgs& a, bool behind);
void plan_diff_tokens(JoinArgs& a, int span, int more_blocks);
cudaError_t launch_diff_tokens(const JoinArgs* prefixes, const JoinArgs& a, bool behind);
cudaError_t launch_diff_chunk(const JoinArgs& a, bool behind);
cudaError_t launch_diff_wide(const JoinArgs& a, bool behind);
cudaError_t launch_join(const JoinArgs& prefixes, const JoinArgs& own);

}  // namespace santa
