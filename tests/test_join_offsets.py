"""Offsets of tokens and of groups, good and bad, on the host with the kernels' own checks: whatever they hold, a token
that is computed is one of its group's (the join looks its sums up by its place there)."""
import random
import subprocess

import pytest

from stochastic_sparse_decode_split_gb300 import build as santa_build


@pytest.fixture(scope="module")
def places(tmp_path_factory):
    exe = tmp_path_factory.mktemp("offsets") / "join_offsets"
    subprocess.run([santa_build.nvcc(), "-std=c++17", "-O2", "--expt-relaxed-constexpr", "-I", santa_build.CSRC, "-o", str(exe),
                    __file__.replace("test_join_offsets.py", "join_offsets.cu")], check=True, capture_output=True)

    def run(calls):
        """(sequences taken, tokens outside their group) of each call (total_q, max_q, max_group, q_offsets, groups)."""
        text = [" ".join(str(x) for x in (total, max_q, most, len(off) - 1, len(first) - 1, *off, *first))
                for total, max_q, most, off, first in calls]
        out = subprocess.run([str(exe)], input="\n".join(text), capture_output=True, text=True, check=True).stdout
        rows = [tuple(int(x) for x in line.split()) for line in out.splitlines()]
        assert len(rows) == len(calls)
        return rows

    return run


def test_a_sequence_whose_tokens_are_not_among_its_groups_is_refused(places):
    # the offsets fall behind the third sequence: its tokens 100 .. 104 lie behind the group's, which end at 8
    assert places([(104, 4, 4, [0, 4, 100, 104, 8], [0, 4])]) == [(1, 0)]   # the second has too many, the last fewer than none
    # and before the group's
    assert places([(64, 64, 2, [40, 44, 4, 44, 48], [0, 1, 2, 4])])[0][1] == 0


def test_good_offsets_are_taken(places):
    rng = random.Random(1)
    calls = []
    for _ in range(200):
        B = rng.randint(1, 70)
        n = [rng.choice((0, 1, rng.randint(0, 50))) for _ in range(B)]
        off = [sum(n[:b]) + 3 for b in range(B + 1)]
        first = [0] + sorted(rng.randint(0, B) for _ in range(rng.randint(0, min(B, 5) - 1))) + [B]
        calls.append((off[-1] + 2, max(max(n), 1), B, off, first))
    for c, (taken, outside) in zip(calls, places(calls)):
        assert (taken, outside) == (len(c[3]) - 1, 0), c


def test_bad_offsets_of_any_kind(places):
    rng = random.Random(2)
    calls = []
    for _ in range(2000):
        B = rng.randint(1, 40)
        total = rng.randint(1, 300)
        off = sorted(rng.randint(0, total) for _ in range(B + 1))
        first = sorted(rng.randint(0, B) for _ in range(rng.randint(2, min(B, 6) + 1)))
        for v, hi in ((off, total), (first, B)):
            for _ in range(rng.randint(0, 3)):
                v[rng.randrange(len(v))] = rng.choice((rng.randint(0, hi), -1, hi + 5, 1 << 30))
        calls.append((total, rng.choice((1, 20, total)), rng.randint(1, B), off, first))
    assert all(outside == 0 for _, outside in places(calls))
