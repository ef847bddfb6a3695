"""How the passes over shared prefixes and over a sequence's own keys divide their blocks over the CTAs, walked on the
host with the kernels' own arithmetic: every item is computed once, its pieces are where its note says, and no block lies
outside the keys of the pass; groups and prefixes that do not fit are refused, and nothing else is."""
import random
import subprocess

import pytest

from stochastic_sparse_decode_split_gb300 import build as santa_build


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    exe = tmp_path_factory.mktemp("shares") / "join_shares"
    subprocess.run([santa_build.nvcc(), "-std=c++17", "-O2", "--expt-relaxed-constexpr", "-I", santa_build.CSRC, "-o", str(exe),
                    __file__.replace("test_join_shares.py", "join_shares.cu")], check=True, capture_output=True)

    def run(calls):
        """Of each call the lines of its two passes: (items, not once, wrong notes, outside, refused)."""
        text = []
        for c in calls:
            own = [k - p for k, p in zip(c["kv"], (c["prefix"][g] for g in range(len(c["prefix"]))
                                                   for _ in range(c["first"][g], c["first"][g + 1])))]
            sizes = [b - a for a, b in zip(c["first"], c["first"][1:])]
            head = [c.get("ctas", 152), c["H"], c["Hkv"], c.get("diff", 0), c.get("parts", 1), c.get("causal", 1),
                    c.get("nk", max(max(c["kv"]), 1)), max(max(c["n"]), 1), c.get("max_prefix", max(max(c["prefix"]), 1)),
                    c.get("max_own", max(max(own or [1]), 1)), c.get("max_group", max(sizes)), len(c["kv"]), len(c["prefix"])]
            text.append(" ".join(str(x) for x in (*head, *c["kv"], *c["n"], *c["first"], *c["prefix"])))
        out = subprocess.run([str(exe)], input="\n".join(text), capture_output=True, text=True, check=True).stdout
        rows = [tuple(int(x) for x in line.split()) for line in out.splitlines()]
        assert len(rows) == 2 * len(calls) and [r[0] for r in rows] == [1, 2] * len(calls)
        return [(rows[2 * i][1:], rows[2 * i + 1][1:]) for i in range(len(calls))]

    return run


def call(own, n, prefix, first=None, **kw):
    first = first or [0, len(own)]
    of = [prefix[g] for g in range(len(prefix)) for _ in range(first[g], first[g + 1])]
    return {"kv": [a + b for a, b in zip(own, of)], "n": n, "prefix": prefix, "first": first, "H": 32, "Hkv": 8, **kw}


def test_every_item_once_and_where_its_note_says(walk):
    rng = random.Random(4)
    calls = [call([1] * 4, [1] * 4, [600]), call([2000] * 64, [1] * 64, [32768]), call([5, 9], [5, 9], [1]),
             call([700, 1, 129], [600, 1, 129], [20000]), call([300, 4], [300, 4], [0]), call([1], [1], [1 << 20])]
    for _ in range(300):
        B = rng.randint(1, 40)
        groups = rng.randint(1, min(B, 5))
        first = [0] + sorted(rng.sample(range(1, B), groups - 1)) + [B]
        n = [rng.choice((1, rng.randint(0, 9), rng.randint(1, 400))) for _ in range(B)]
        own = [k + rng.choice((0, rng.randint(0, 20), rng.randint(0, 3000))) for k in n]
        H, Hkv = rng.choice(((32, 8), (28, 4), (16, 2), (6, 2), (16, 16), (8, 2)))
        diff = rng.randint(0, 1)
        calls.append(call(own, n, [rng.choice((0, rng.randint(1, 400), rng.randint(1, 30000))) for _ in range(groups)], first, H=H,
                          Hkv=Hkv, diff=diff, parts=rng.randint(1, 1 + diff), ctas=rng.choice((152, 152, 148, 7, 1))))
    for c, passes in zip(calls, walk(calls)):
        for items, once, notes, outside, refused in passes:
            assert (once, notes, outside, refused) == (0, 0, 0, 0), c
        tokens = [0] * len(c["prefix"])
        for g in range(len(tokens)):
            tokens[g] = sum(c["n"][c["first"][g]:c["first"][g + 1]])
        if max(tokens) > 0:
            assert passes[0][0] > 0


def test_what_does_not_fit_is_refused(walk):
    good = call([10, 20, 30], [1, 2, 3], [100, 50], [0, 2, 3])
    bad = [
        (dict(good, max_prefix=99, max_own=30), 2), (dict(good, max_own=29), 1), (dict(good, prefix=[-1, 50], max_prefix=50, max_own=200), 2),
        (dict(good, first=[0, 2, 4], max_group=2), 1), (dict(good, first=[1, 2, 3], max_group=2), 1), (dict(good, first=[0, 3, 2], max_group=3), 1),
        (dict(good, first=[0, 2, 2], max_group=2), 1), (dict(good, n=[11, 2, 3]), 1), (dict(good, n=[11, 2, 3], causal=0), 0),
        (dict(good, kv=[99, 120, 80], causal=0), 1), (dict(good, nk=115), 1),
    ]
    for (c, refused), (first, second) in zip(bad, walk([c for c, _ in bad])):
        assert second[4] == refused, (c, second)
        assert first[1:4] == second[1:4] == (0, 0, 0), c
