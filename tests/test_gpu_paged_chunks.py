"""The chunk kernel of the paged attention at its edges, on calls large enough to reach it (two of many small items take
the kernel for few rows).  Masks, odd values, bad
pages, shared items and empty ones, against the definition in 64 bits."""
import pytest
import torch

import stochastic_sparse_decode_split_gb300 as santa
from paged_reference import Batch, check_attention

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    santa.library()


def attend(batch, window=0, nk=None, **kw):
    nk = max(max(batch.kv), 1) if nk is None else nk
    span = min(nk, window + max(batch.n)) if window else nk
    tiles = -(-max(batch.n) * (batch.H // batch.Hkv) // 16)
    assert max(batch.n) * (batch.H // batch.Hkv) > 16 and tiles * batch.B * batch.Hkv * span * 2 * batch.D > 1.2 * 2 ** 25
    step = batch.step(window=window, nk=nk, **kw)
    out, lse = (x.clone() for x in step.attend(batch.q, return_lse=True))   # the step's own outputs change with its next call
    return step, out, lse


def check(batch, window=0, nk=None, **kw):
    step, out, lse = attend(batch, window, nk, **kw)
    assert step.error() == 0
    check_attention(batch, out, lse, window=window, **kw)


CASES = [   # kv, new tokens, H, Hkv, D, type, page
    ([2000], [600], 8, 4, 128, BF16, 16),
    ([1500, 3, 700], [700, 3, 1], 8, 4, 128, BF16, 32),
    ([4100], [400], 14, 2, 128, FP16, 64),                    # groups of 7: tiles with unused rows
    ([1025, 1024, 1023], [513, 512, 511], 6, 2, 128, BF16, 128),
    ([3000, 40], [333, 40], 32, 8, 64, FP16, 256),
    ([900, 900, 900], [900, 900, 900], 5, 1, 64, BF16, 16),
    ([20000], [100], 8, 2, 128, BF16, 64),                    # few rows, long: every item is shared, one tile of two
    ([60000], [40], 4, 1, 128, BF16, 128),
    ([700] * 40, [20] * 40, 4, 2, 128, BF16, 16),             # many small items, the second tile empty
    ([300] * 300, [17] * 300, 2, 2, 64, FP16, 16),
    ([130] * 700, [9] * 700, 8, 4, 64, BF16, 16),             # more sequences than the CTA has threads
    ([1, 5000, 2, 17, 900], [1, 300, 2, 17, 129], 8, 2, 128, BF16, 16),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kv,n,H,Hkv,D,dtype,page", CASES)
def test_chunks(kv, n, H, Hkv, D, dtype, page, e4m3):
    check(Batch(kv, n, H, Hkv, D, dtype, e4m3, page, seed=len(kv) + kv[0]))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window", [1, 100, 128, 1000])
def test_chunks_in_a_window(window, e4m3):
    check(Batch([5000, 2500], [800, 777], 8, 4, 128, BF16, e4m3, 32, seed=window), window=window)


@pytest.mark.parametrize("e4m3", [False, True])
def test_chunks_without_a_mask(e4m3):
    check(Batch([1500, 700, 5], [448, 300, 200], 16, 16, 64, FP16, e4m3, 64, seed=3), causal=False)


@pytest.mark.parametrize("e4m3", [False, True])
def test_chunks_that_see_nothing(e4m3):
    """Empty sequences, sequences without new tokens, more new tokens than keys, padding behind the last."""
    batch = Batch([0, 2000, 0, 3000, 90], [300, 0, 2, 500, 400], 8, 4, 128, BF16, e4m3, 16, seed=1, pad=7)
    step = batch.step()
    out = torch.full((batch.total_q, 8, 128), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((batch.total_q, 8), 7.0, device="cuda")
    attend(batch)
    step.attend(batch.q, out=out, lse=lse)
    assert step.error() == 0
    check_attention(batch, out, lse)
    assert bool((out[batch.tokens:] == 7).all()) and bool((lse[batch.tokens:] == 7).all())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kv,n", [(1800, 700), (30000, 60)])
def test_chunks_with_odd_values_in_masked_places(kv, n, e4m3):
    """NaN and infinities reach the rows that see their key, and no other."""
    for window in (0, 1000):
        batch = Batch([kv], [n], 8, 4, 128, BF16, e4m3, 16, seed=n)
        if window and kv > 5000:
            continue
        for key, odd in ((kv - 2, float("nan")), (kv - 30, float("inf")), (kv - n // 2, float("-inf")), (5, float("nan"))):
            at, slot = int(batch.table[0, key // 16]), key % 16
            if e4m3:
                batch.vs[at, 0, slot] = float("nan")
            else:
                batch.V[at, slot, 0, 3:70] = odd
        at = int(batch.table[0, (kv - 1) // 16])
        if e4m3:
            batch.ks[at, 1, (kv - 1) % 16] = float("nan")
        else:
            batch.K[at, (kv - 1) % 16, 1] = float("nan")
        check(batch, window=window)


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_chunks_of_scales_far_apart(dtype):
    batch = Batch([2000], [700], 8, 4, 128, dtype, True, 16, seed=2)
    batch.vs *= torch.exp2(torch.randint(-40, 12, batch.vs.shape, device="cuda").float())
    check(batch)


def test_chunks_of_large_scores():
    """The maximum moves far from block to block: sums are rescaled, also those that two groups share."""
    for kv, n in ((2500, 700), (30000, 50)):
        batch = Batch([kv], [n], 8, 4, 64, BF16, False, 16, seed=8)
        batch.q *= 40
        check(batch)


@pytest.mark.parametrize("kv,n", [(2000, 600), (30000, 60)])
def test_device_refusals_of_chunks(kv, n):
    batch = Batch([kv, kv], [n, n], 8, 4, 64, BF16, False, 16, seed=3, shared_n=True)
    step, good, _ = attend(batch)
    assert step.error() == 0
    old = batch.table.clone()
    for bad in (batch.n_pages, -1, -2 ** 31):
        batch.table[1, 3] = bad
        out, lse = step.attend(batch.q, return_lse=True)
        assert step.error() == santa.CACHE_DEVERR_PAGE
        assert torch.equal(out[:n], good[:n]) and not bool(out[n:].any()) and bool((lse[n:] == float("-inf")).all())
    batch.table.copy_(old)
    batch.kv_t[0] = kv + 1
    out = step.attend(batch.q)
    assert step.error() == santa.DEVERR_NK_BOUND
    assert not bool(out[:n].any())
    torch.testing.assert_close(out[n:].float(), good[n:].float(), rtol=2 ** -6, atol=1e-3)   # other shares, other sums


def test_uneven_lengths_share_the_cards_ctas():
    """One long sequence among short ones: its items are cut over many CTAs, and the same call gives the same bits."""
    batch = Batch([40000, 100, 300, 50], [64, 100, 300, 50], 8, 2, 128, BF16, False, 64, seed=4)
    check(batch)
    a, b = attend(batch)[1:], attend(batch)[1:]
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_chunks_captured_and_replayed_over_other_lengths():
    batch = Batch([3000, 2000], [300, 300], 8, 4, 128, BF16, False, 16, seed=9, shared_n=True)
    step, out, lse = attend(batch)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step.attend(batch.q, out=out, lse=lse)
    for kv in ([3000, 2000], [301, 1999], [2500, 300]):
        batch.kv_t.copy_(torch.tensor(kv))
        batch.q.copy_(torch.randn_like(batch.q))
        g.replay()
        torch.cuda.synchronize()
        batch.kv, batch.used = kv, [-(-x // 16) for x in kv]
        check_attention(batch, out, lse)
    assert step.error() == 0


def test_an_output_that_is_16_but_not_32_bytes_aligned():
    batch = Batch([2000], [700], 8, 4, 64, BF16, False, 16, seed=9)
    step, good, _ = attend(batch)
    raw = torch.zeros(batch.q.numel() + 8, dtype=BF16, device="cuda")
    out = raw[8:].view(batch.q.shape)
    assert out.data_ptr() % 32 == 16
    step.attend(batch.q, out=out)
    assert torch.equal(out, good) and step.error() == 0


def test_what_lies_past_the_last_key_costs_nothing_in_e4m3():
    """Rows of the last block past the last key are NaN codes here: they must not be taken for odd values of the
    sequence, which are given back one by one (milliseconds where the call takes microseconds)."""
    batch = Batch([4000, 3001], [500, 300], 8, 4, 128, BF16, True, 16, seed=3)
    step, out, lse = attend(batch)
    assert step.error() == 0
    check_attention(batch, out, lse)
    clean = Batch([4000, 3001], [500, 300], 8, 4, 128, BF16, True, 16, seed=3)
    for pool in (clean.K, clean.V):
        raw = pool.view(torch.uint8)
        raw[(raw & 0x7F) == 0x7F] = 0
    times = []
    for b in (batch, clean):
        s = b.step()
        s.attend(b.q)
        marks = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        marks[0].record()
        for _ in range(5):
            s.attend(b.q)
        marks[1].record()
        marks[1].synchronize()
        times.append(marks[0].elapsed_time(marks[1]))
    assert times[0] < 10 * times[1]
