// Where the tokens of a batch with prefixes stand in their groups, on the host with
// the kernels' own checks.
//
// stdin: calls of "total_q max_q max_group batch groups", then q_offsets (batch +
// 1) and the groups' offsets (groups + 1); every sequence has 100 keys, every
// group a prefix of 10.  stdout, for each: the sequences taken, and of their
// tokens those that are not among their group's.
#include <cstdio>
#include <vector>

#include "santa_join.cuh"

using namespace santa;

int main() {
  int max_q, max_group, B, groups;
  long long total_q;
  while (std::scanf("%lld %d %d %d %d", &total_q, &max_q, &max_group, &B, &groups) == 5) {
    std::vector<int64_t> off(B + 1);
    std::vector<int> first(groups + 1), prefix(groups, 10), kv(B, 100);
    for (int64_t& x : off) {
      long long v;
      if (std::scanf("%lld", &v) != 1) return 1;
      x = v;
    }
    for (int& x : first)
      if (std::scanf("%d", &x) != 1) return 1;
    JoinArgs own = {};
    own.H = own.Hkv = own.G = 1, own.B = own.seqs = B, own.max_q = own.seq_q = max_q, own.total_q = total_q;
    own.nk = 100, own.causal = 0, own.kv_lens = kv.data(), own.q_offsets = off.data();
    own.phase = 2, own.n_groups = groups, own.group_offsets = first.data(), own.prefix_lens = prefix.data();
    own.max_prefix = 10, own.max_own = 90;
    own.group_q = (int)std::min<long long>((long long)max_group * max_q, total_q);
    JoinArgs pre = own;
    pre.phase = 1, pre.B = groups, pre.max_q = own.group_q;
    int taken = 0, outside = 0;
    for (int b = 0; b < B; ++b) {
      const Seq s = paged_seq(own, b, false);
      if (!s.ok) continue;
      ++taken;
      const Seq g = paged_seq(pre, group_of(own, b), false);
      for (int i = 0; i < s.n; ++i) outside += s.q0 + i < g.q0 || s.q0 + i >= g.q0 + g.n;
    }
    std::printf("%d %d\n", taken, outside);
  }
  return 0;
}
