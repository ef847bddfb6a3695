"""How the chunk attention's blocks are divided over its CTAs, walked on the host with the kernel's own arithmetic: every
item is computed whole by one CTA, or by pieces that follow each other and that its merge finds, whatever the sizes."""
import random
import subprocess

import pytest

from stochastic_sparse_decode_split_gb300 import build as santa_build

CTAS = 152


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    exe = tmp_path_factory.mktemp("shares") / "chunk_shares"
    subprocess.run([santa_build.nvcc(), "-std=c++17", "-O2", "--expt-relaxed-constexpr", "-I", santa_build.CSRC, "-o", str(exe),
                    __file__.replace("test_chunk_shares.py", "chunk_shares.cu")], check=True, capture_output=True)

    def run(calls):
        text = []
        for kv, n, H, Hkv, causal, window, *ctas in calls:
            text.append(" ".join(str(x) for x in (*(ctas or [CTAS]), H, Hkv, int(causal), window, max(max(kv), 1), max(n), len(kv),
                                                  *kv, *n)))
        out = subprocess.run([str(exe)], input="\n".join(text), capture_output=True, text=True, check=True).stdout
        return [tuple(int(x) for x in line.split()) for line in out.splitlines()]

    return run


def check(walk, calls):
    got = walk(calls)
    assert len(got) == len(calls)
    wrong = [(c, g) for c, g in zip(calls, got) if g[2] or g[3]]
    assert not wrong, f"{len(wrong)} of {len(calls)} calls; the first: {wrong[0]} (items, shared, not computed once, wrong merges)"
    return got


# kv, new tokens, heads, KV heads, causal, window: calls in which one block more or less in a CTA's share is the
# difference between sharing and not sharing
BORDER = [
    ([4608], [1024], 32, 8, True, 0), ([5888] * 2, [512] * 2, 32, 8, True, 0), ([2176] * 9, [64] * 9, 32, 8, True, 0),
    ([2300] * 10, [64] * 10, 32, 8, True, 0), ([3000] * 3, [448] * 3, 16, 16, False, 0), ([2064], [656], 32, 8, True, 0),
    ([2400], [736], 32, 8, True, 0), ([2176], [2176], 16, 2, True, 0), ([2304], [768], 32, 8, True, 0),
]


def test_calls_at_the_border_of_sharing(walk):
    check(walk, BORDER)


def test_one_sequence_of_every_length(walk):
    got = check(walk, [([kv], [n], 32, 8, True, 0) for n in (17, 100, 256, 656, 1024, 2048) for kv in range(n, 9000, 16)])
    assert {g[1] for g in got} == {0, 1}
    got = check(walk, [([kv] * B, [n] * B, 16, 16, False, 0) for B in (1, 3, 8) for n in (60, 256, 448)
                       for kv in range(1500, 8000, 64)])
    assert {g[1] for g in got} == {0, 1}


def test_drawn_batches(walk):
    rng = random.Random(7)
    calls = []
    for _ in range(2500):
        B = rng.choice((1, 1, 2, 3, 5, 9, 30, 170))
        top = rng.choice((300, 2500, 6000, 40000) if B < 10 else (300, 4000))
        kv = [0 if rng.random() < 0.03 else rng.randint(1, top) for _ in range(B)]
        chunk = rng.choice((3, 20, 130, 700, 2100))
        n = [rng.randint(0 if rng.random() < 0.1 else 1, chunk) for _ in range(B)]
        n[0] = max(n[0], 1)
        H, Hkv = rng.choice(((32, 8), (28, 4), (16, 2), (8, 2), (6, 2), (10, 2), (5, 1), (16, 16), (8, 1), (3, 3)))
        causal = rng.random() < 0.8
        calls.append((kv, n, H, Hkv, causal, rng.choice((0, 0, rng.randint(1, top))) if causal else 0,
                      rng.choice((CTAS, CTAS, 148, 132, 7))))
    got = check(walk, calls)
    assert sum(g[1] for g in got) > 200 and sum(1 - g[1] for g in got) > 200
