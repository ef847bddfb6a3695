"""Joined attention at corners of what its documentation allows: batches of more tiles than a CTA has threads, many groups,
the largest head groups, nothing left to compute, two steps at once, weights of any stride."""
import random

import pytest
import torch

import stochastic_sparse_decode_split_gb300 as santa
from join_reference import Shared, check_diff
from join_routes import route
from paged_reference import Batch, check_attention

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    santa.library()


def weights(batch, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return (0.1 + 0.6 * torch.rand(batch.total_q, batch.H // 2, generator=gen)).to(batch.device)


def holds(batch, diff):
    step = batch.shared_step(diff=diff) if hasattr(batch, "full") else batch.step(diff=diff)
    if diff:
        w = weights(batch)
        out, lse = step.attend_diff(batch.q, w, return_lse=True)
        assert step.error() == 0
        check_diff(batch, out, lse, w)
    else:
        out, lse = step.attend(batch.q, return_lse=True)
        assert step.error() == 0
        check_attention(batch, out, lse)


def many(B, groups, most, seed):
    """Groups of any size, prefixes of any length, new tokens of any number up to `most` (and none)."""
    rng = random.Random(seed)
    first = [0] + sorted(rng.sample(range(1, B), groups - 1)) + [B]
    n = [rng.choice((0, 1, rng.randint(1, most))) for _ in range(B)]
    n[0] = most
    own = [k + rng.choice((0, rng.randint(0, 30))) for k in n]
    return [rng.choice((0, rng.randint(1, 40), rng.randint(1, 300))) for _ in range(groups)], first, own, n


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("diff,D,Hkv", [(False, 64, 2), (True, 64, 2), (True, 128, 2)])
def test_more_tiles_than_threads(diff, D, Hkv, e4m3):
    prefix, first, own, n = many(620, 5, 40, seed=D + diff)
    kernels = route(own, n, 8, Hkv, D, e4m3=e4m3, diff=diff, prefix=prefix, first=first)
    assert kernels[1] == ("own:wide" if diff and D == 128 and not e4m3 else "own:chunk") and "tokens" not in kernels[0]
    holds(Shared(prefix, first, own, n, 8, Hkv, D, BF16, e4m3, 16, seed=3, pairs=diff), diff)


@pytest.mark.parametrize("diff", [False, True])
@pytest.mark.parametrize("B,groups", [(70, 33), (80, 65), (150, 150)])
def test_many_groups(B, groups, diff):
    prefix, first, own, n = many(B, groups, 3, seed=B)
    holds(Shared(prefix, first, own, n, 8, 2, 64, FP16, False, 16, seed=1, pairs=diff), diff)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("diff", [False, True])
@pytest.mark.parametrize("n", [[1, 2, 1], [450, 390, 360]])
@pytest.mark.parametrize("G,D", [(8, 128), (7, 64), (5, 128), (3, 64), (1, 64), (1, 128)])
def test_head_groups_of_any_size(G, D, n, diff, e4m3):
    Hkv = 2 if G > 1 else 16
    holds(Shared([270], [0, 3], [k + 9 for k in n], n, G * Hkv, Hkv, D, BF16, e4m3, 32, seed=G, pairs=diff), diff)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("diff", [False, True])
@pytest.mark.parametrize("n", [[1, 2, 1], [350, 290, 260]])
def test_nothing_left_to_compute(n, diff, e4m3):
    """Every group refused (zeros), or no token at all (everything left as it was)."""
    batch = Shared([1270], [0, 3], [k + 9 for k in n], n, 16, 4, 128, BF16, e4m3, 32, seed=2, pairs=diff)
    step = batch.shared_step(diff=diff)
    w = weights(batch)
    call = (lambda **kw: step.attend_diff(batch.q, w, **kw)) if diff else (lambda **kw: step.attend(batch.q, **kw))
    batch.prefix_t.fill_(-1)
    out, lse = (x.clone() for x in call(return_lse=True))
    assert step.error() == santa.CACHE_DEVERR_PREFIX
    assert bool((out == 0).all()) and bool((lse == float("-inf")).all())
    batch.prefix_t.fill_(1270)
    batch.offsets.zero_()
    out.fill_(7.0)
    lse.fill_(7.0)
    call(out=out, lse=lse)
    assert step.error() == 0
    assert bool((out == 7).all()) and bool((lse == 7).all())


def test_two_steps_at_once():
    """Chunks and single tokens of two steps on two streams, again and again: each as it is alone."""
    one = Shared([1000], [0, 3], [700, 450, 651], [500, 450, 300], 28, 4, 128, FP16, False, 64, seed=1)
    two = Batch([2000, 1500], [700, 400], 8, 2, 128, BF16, False, 32, seed=2)
    few = Shared([4000], [0, 40], [1 + 9 * i % 90 for i in range(40)], [1] * 40, 8, 2, 128, BF16, True, 32, seed=3)
    steps = [one.shared_step(), two.step(diff=True), few.shared_step()]
    w = weights(two)
    calls = [lambda **kw: steps[0].attend(one.q, **kw), lambda **kw: steps[1].attend_diff(two.q, w, **kw), lambda **kw: steps[2].attend(few.q, **kw)]
    want = [c().clone() for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    outs = [[torch.empty_like(x) for _ in range(12)] for x in want]
    torch.cuda.synchronize()
    for i in range(12):
        for c, s, o in zip(calls, streams, outs):
            c(out=o[i], stream=s)
    torch.cuda.synchronize()
    for x, o in zip(want, outs):
        assert all(torch.equal(x, y) for y in o)
    assert all(s.error() == 0 for s in steps)


@pytest.mark.parametrize("n", [[2, 1], [700, 400]])
def test_weights_of_any_stride(n):
    """The same for all tokens, given once or as rows that lie on one another; rows of a wider tensor."""
    batch = Batch([2000, 1500], n, 8, 2, 128, BF16, False, 32, seed=2)
    step = batch.step(diff=True)
    w = weights(batch)
    one = step.attend_diff(batch.q, w[0].contiguous()).clone()
    assert torch.equal(one, step.attend_diff(batch.q, w[:1].expand(batch.total_q, 4)))
    rows = step.attend_diff(batch.q, w).clone()
    wide = torch.full((batch.total_q, 11), float("nan"), device="cuda")
    wide[:, 3:7] = w
    assert torch.equal(rows, step.attend_diff(batch.q, wide[:, 3:7])) and not torch.equal(rows, one)
    assert step.error() == 0
