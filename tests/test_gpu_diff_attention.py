"""GPU parity of differential attention against its definition in 64 bits: single tokens and chunks, weights of heads and
of tokens, with and without the norm, masks, odd values, over a shared prefix."""
import pytest
import torch

import stochastic_sparse_decode_split_gb300 as santa
from join_reference import Shared, check_diff
from paged_reference import Batch

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    santa.library()


def learned(batch, per_token=False, norm=True, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    shape = (batch.total_q, batch.H // 2) if per_token else (batch.H // 2,)
    w = 0.1 + 0.6 * torch.rand(shape, generator=gen, device="cuda")
    n = (1 + 0.3 * torch.randn(2 * batch.D, generator=gen, device="cuda")).to(batch.dtype) if norm else None
    return w, n


def run(batch, shared=False, per_token=False, norm=True, gain=0.8, **kw):
    w, n = learned(batch, per_token, norm)
    step = batch.shared_step(diff=True, **kw) if shared else batch.step(diff=True, **kw)
    out, lse = step.attend_diff(batch.q, w, norm=n, eps=1e-5, gain=gain, return_lse=True)
    assert step.error() == 0
    check_diff(batch, out, lse, w, norm=n, eps=1e-5, gain=gain,
               **{k: v for k, v in kw.items() if k in ("causal", "window", "scale")})
    return step, w, n


TOKENS = [   # kv, new tokens, H, Hkv, D, type, page
    ([1], [1], 2, 2, 64, BF16, 16),
    ([1000], [1], 32, 8, 128, BF16, 16),
    ([15, 16, 17, 1, 300], [1] * 5, 8, 2, 128, BF16, 16),
    ([777, 1], [1, 1], 14, 2, 128, FP16, 32),
    ([2049, 64, 63, 65], [1] * 4, 6, 2, 64, FP16, 64),
    ([5000], [1], 8, 8, 64, BF16, 256),
    ([900, 33], [2, 5], 8, 2, 128, BF16, 16),
    ([257, 4, 100], [5, 4, 1], 6, 2, 64, FP16, 16),
    ([130], [16], 4, 4, 128, BF16, 32),
]
CHUNKS = [
    ([300], [100], 8, 2, 128, BF16, 16),
    ([129, 700, 31], [129, 64, 1], 8, 2, 64, FP16, 32),
    ([1111], [257], 14, 2, 128, FP16, 64),
    ([640, 90], [300, 70], 6, 2, 128, BF16, 128),
    ([2000], [130], 32, 8, 64, BF16, 256),
    ([515, 515], [515, 515], 10, 2, 64, BF16, 16),
    ([3500], [800], 4, 4, 128, BF16, 64),
]
# Contexts so long that the bound of the roundings reaches the size of the difference of two flat maps, whose norm then
# has no bound: compared before it.
LONG = [
    ([30000], [1], 16, 2, 128, BF16, 128),
    ([9000], [500], 16, 2, 64, FP16, 64),
    ([6000], [2000], 4, 2, 128, BF16, 64),
]


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kv,n,H,Hkv,D,dtype,page", TOKENS + CHUNKS)
def test_differential_attention(kv, n, H, Hkv, D, dtype, page, e4m3, norm):
    run(Batch(kv, n, H, Hkv, D, dtype, e4m3, page, seed=len(kv) + kv[0]), per_token=norm == e4m3, norm=norm)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kv,n,H,Hkv,D,dtype,page", LONG)
def test_long_contexts(kv, n, H, Hkv, D, dtype, page, e4m3):
    run(Batch(kv, n, H, Hkv, D, dtype, e4m3, page, seed=len(kv) + kv[0]), norm=False)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window", [1, 16, 100, 5000])
@pytest.mark.parametrize("n", [1, 200])
def test_in_a_window(n, window, e4m3):
    run(Batch([900, 333], [n, max(1, n // 3)], 8, 2, 128, BF16, e4m3, 32, seed=window), norm=False, window=window)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,kv", [([1, 1], [77, 1500]), ([448, 30], [1500, 5]), ([100, 9], [1, 64])])
def test_without_a_mask(n, kv, e4m3):
    run(Batch(kv, n, 8, 8, 64, FP16, e4m3, 64, seed=3), norm=False, causal=False)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("n", [1, 3, 150])
def test_rows_that_see_nothing(n, norm):
    batch = Batch([0, 40, 0, max(1, n - 2)], [n, n, 1, n], 8, 2, 128, BF16, False, 16, seed=n)
    run(batch, norm=False)
    w, nw = learned(batch, norm=norm)
    step = batch.step(diff=True)
    out = step.attend_diff(batch.q, w, norm=nw, eps=0.0)   # a row of zeros is not divided by its norm
    assert bool((out[:n] == 0).all()) and bool(torch.isfinite(out).all())


CASES = [   # prefixes, groups, own keys, new tokens, H, Hkv, D, type, page
    ([600], [0, 4], [5, 60, 1, 17], [1] * 4, 32, 8, 128, BF16, 16),
    ([1000], [0, 3], [33, 2, 700], [1] * 3, 28, 4, 128, FP16, 64),
    ([777, 5, 300], [0, 3, 4, 9], [9, 8, 7, 600, 5, 4, 3, 2, 1], [1] * 9, 6, 2, 64, BF16, 128),
    ([4000], [0, 70], [1 + 7 * i % 90 for i in range(70)], [1] * 70, 8, 2, 128, BF16, 16),
    ([2000], [0, 6], [10, 200, 7, 9, 40, 33], [5, 2, 7, 1, 3, 4], 16, 2, 64, FP16, 32),
    ([300, 0], [0, 2, 3], [600, 90, 7], [400, 70, 7], 8, 2, 128, BF16, 64),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("prefix,first,own,n,H,Hkv,D,dtype,page", CASES)
def test_over_a_shared_prefix(prefix, first, own, n, H, Hkv, D, dtype, page, e4m3):
    run(Shared(prefix, first, own, n, H, Hkv, D, dtype, e4m3, page, seed=len(own) + prefix[0], pairs=True), shared=True,
        per_token=True, norm=False)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [[1, 1], [150, 40]])
def test_odd_values_reach_the_rows_that_see_them(n, D, e4m3):
    batch = Batch([200, 60], n, 8, 2, D, BF16, e4m3, 16, seed=8)
    V = batch.V.view(torch.uint8) if e4m3 else batch.V
    V[int(batch.table[0, 11]), 5, 0, 17] = 0x7f if e4m3 else float("nan")
    V[int(batch.table[1, 2]), 3, 1, D - 1] = 0xff if e4m3 else float("inf")
    run(batch, norm=False)


def test_the_first_map_alone_is_the_plain_attention():
    """Weights of zero: the paged attention of the even heads, over both heads' values."""
    batch = Batch([500, 90], [3, 1], 8, 4, 128, BF16, False, 16, seed=1)
    step = batch.step(diff=True)
    out = step.attend_diff(batch.q, torch.zeros(4, device="cuda"))
    for f in range(2):
        V = batch.V.view(*batch.V.shape[:2], 2, 2, 128)[..., f:f + 1, :].expand(-1, -1, -1, 2, -1).reshape(batch.V.shape).contiguous()
        other = santa.PagedStep(santa.PagedCache.of(batch.K, V), batch.table, batch.kv_t, n_q_heads=8, nk=500, max_q=3,
                                total_q=4, q_offsets=batch.offsets)
        # query head 2h of pair h meets key head 2 (h / 2): heads 0, 2 and 4, 6 in pairs meet heads 0 and 2
        q = batch.q.view(4, 2, 2, 2, 128).transpose(2, 3).reshape(4, 8, 128).contiguous()
        want = other.attend(q).view(4, 2, 2, 2, 128)[:, :, 0]
        got = out.view(4, 2, 2, 2, 128)[..., f, :]
        assert float((got.float() - want.float()).abs().max()) <= 4 * 2.0 ** -8 * float(torch.nan_to_num(V.float()).abs().max())


def test_the_weights_from_their_vectors():
    v = torch.randn(4, 6, 64, device="cuda") * 0.1
    got = santa.diff_weights(*v, init=0.35)
    d = v.double()
    want = (d[0] * d[1]).sum(-1).exp() - (d[2] * d[3]).sum(-1).exp() + 0.35
    # 64 products and sums in 32 bits of values about 0.01, two exponentials near 1
    assert got.dtype == torch.float32 and float((got.double() - want).abs().max()) < 64 * 2.0 ** -23


def test_refusals_of_the_binding():
    batch = Batch([50], [2], 8, 2, 64, BF16, False, 16, seed=1)
    w = torch.ones(4, device="cuda")
    with pytest.raises(ValueError):
        batch.step().attend_diff(batch.q, w)
    step = batch.step(diff=True)
    for bad in (w.double(), w[:3], torch.ones(3, 4, device="cuda"), torch.ones(2, 8, device="cuda")[:, ::2], w.cpu(),
                torch.ones(4, 2, device="cuda").T):
        with pytest.raises(ValueError):
            step.attend_diff(batch.q, bad)
    with pytest.raises(ValueError):
        step.attend_diff(batch.q, w, norm=torch.ones(64, dtype=BF16, device="cuda"))
    with pytest.raises(ValueError):
        step.attend_diff(batch.q, w, out=torch.empty_like(batch.q))
    with pytest.raises(santa.SantaError):
        step.attend_diff(batch.q, w, norm=torch.ones(128, dtype=BF16, device="cuda"), eps=-1.0)
    with pytest.raises(santa.SantaError):
        step.attend_diff(batch.q, w, gain=float("nan"))
    odd = Batch([50], [2], 3, 1, 64, BF16, False, 16, seed=1)
    with pytest.raises(ValueError):
        odd.step(diff=True)
    wide = torch.rand(2, 9, device="cuda")[:, :4]   # rows of a wider tensor
    step.attend_diff(batch.q, wide)
    with pytest.raises(ValueError):
        batch.step(max_own=5)
    for kw in (dict(max_prefix=0), dict(max_own=-1), dict(max_group=0), dict(window=7), dict(group_offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            batch.step(prefix_lens=torch.zeros(1, dtype=torch.int32, device="cuda"), **kw)


def test_output_over_the_queries_and_other_streams():
    batch = Batch([300, 40], [1, 1], 8, 2, 128, BF16, False, 16, seed=2)
    w, n = learned(batch)
    step = batch.step(diff=True)
    want = step.attend_diff(batch.q, w, norm=n).clone()
    q = batch.q.clone()
    got = step.attend_diff(q, w, norm=n, out=q.view(2, 4, 256))
    assert torch.equal(got, want) and got.data_ptr() == q.data_ptr()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    other = step.attend_diff(batch.q, w, norm=n, stream=stream)
    stream.synchronize()
    assert torch.equal(other, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step.attend_diff(batch.q, w, norm=n)
    captured.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured, want) and step.error() == 0


def ramped(batch, every, factors):
    """The batch with the keys of every `every` positions of a sequence times the next of `factors` (powers of two)."""
    for b in range(batch.B):
        for i in range(batch.kv[b]):
            page, at, f = int(batch.table[b, i // batch.page]), i % batch.page, factors[i // every % len(factors)]
            if batch.e4m3:
                batch.ks[page, :, at] *= f
            else:
                batch.K[page, at] *= f
    return batch


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv,n", [([1400, 130], [1, 2]), ([1400, 700], [140, 300])])
@pytest.mark.parametrize("factors", [(0.25, 1, 2, 4, 8, 16), (16, 8, 1, 0.25), (0.5, 16, 0.25, 32, 1, 8)])
def test_maxima_that_grow_and_fall_along_the_keys(factors, kv, n, D, e4m3):
    """What a block's maximum is above the one before, a group's above the other's: nothing, a little, more than 2^8."""
    run(ramped(Batch(kv, n, 8, 2, D, BF16, e4m3, 32, seed=D), 97, factors), norm=False)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 150])
def test_a_bad_page_zeroes_the_rows_that_are_computed_with_it(n, D, e4m3):
    batch = Batch([700, 600], [n, n], 8, 2, D, FP16, e4m3, 32, seed=5)
    step, w, _ = run(batch, norm=False)
    want, want_lse = (x.clone() for x in step.attend_diff(batch.q, w, return_lse=True))
    batch.table[0, 1] = -1
    out, lse = step.attend_diff(batch.q, w, return_lse=True)
    assert step.error() == santa.CACHE_DEVERR_PAGE
    assert bool((out[:n] == 0).all()) and bool((lse[:n] == float("-inf")).all())
    assert torch.equal(out[n:], want[n:]) and torch.equal(lse[n:], want_lse[n:])


@pytest.mark.parametrize("n", [[1, 0, 2], [150, 0, 90]])
def test_padding_is_left_as_it_was(n):
    batch = Batch([200, 300, 150], n, 8, 2, 128, BF16, False, 16, seed=4, pad=9)
    w, _ = learned(batch, per_token=True)
    step = batch.step(diff=True)
    out = torch.full((batch.total_q, 4, 256), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((batch.total_q, 8), 7.0, device="cuda")
    step.attend_diff(batch.q, w, out=out, lse=lse)
    assert step.error() == 0
    check_diff(batch, out, lse, w)
    assert bool((out[batch.tokens:] == 7).all()) and bool((lse[batch.tokens:] == 7).all())


@pytest.mark.parametrize("D", [64, 128])
def test_captured_over_a_prefix_and_replayed_with_other_lengths(D):
    """One graph for every length within the bounds; the same bits from one replay to the next."""
    batch = Shared([4000], [0, 40], [1 + 9 * i % 90 for i in range(40)], [1] * 40, 16, 4, D, BF16, False, 32, seed=7, whole=True, pairs=True)
    w, _ = learned(batch)
    step = batch.shared_step(diff=True, max_own=100)
    step.attend_diff(batch.q, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step.attend_diff(batch.q, w, return_lse=True)
    longest = batch.kv
    for prefix in (4000, 3001, 128, 1, 0, 2500):
        batch.prefix[0] = prefix
        batch.kv = [min(k, prefix + 1 + 7 * b % 90) for b, k in enumerate(longest)]
        batch.prefix_t.fill_(prefix)
        batch.kv_t.copy_(torch.tensor(batch.kv, dtype=torch.int32))
        graph.replay()
        assert step.error() == 0
        check_diff(batch, out, lse, w)
        first, first_lse = out.clone(), lse.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, out) and torch.equal(first_lse, lse)
