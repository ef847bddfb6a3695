"""GPU parity of attention over shared prefixes against the plain definition in 64 bits: few and many rows, groups,
prefixes that end anywhere, what the kernels must not read, what they refuse."""
import pytest
import torch

import stochastic_sparse_decode_split_gb300 as santa
from join_reference import Shared
from paged_reference import check_attention

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    santa.library()


def attend(batch, **kw):
    step = batch.shared_step(**kw)
    out, lse = step.attend(batch.q, return_lse=True)
    assert step.error() == 0
    return out, lse


CASES = [   # prefixes, groups, own keys, new tokens, H, Hkv, D, type, page
    ([16], [0, 2], [1, 1], [1, 1], 1, 1, 64, BF16, 16),
    ([1], [0, 2], [1, 3], [1, 1], 8, 2, 128, BF16, 16),
    ([600], [0, 4], [5, 60, 1, 17], [1] * 4, 32, 8, 128, BF16, 16),
    ([1000], [0, 3], [33, 2, 700], [1] * 3, 28, 4, 128, FP16, 64),
    ([129], [0, 40], list(range(1, 41)), [1] * 40, 8, 2, 128, BF16, 32),
    ([4000], [0, 70], [1 + 7 * i % 90 for i in range(70)], [1] * 70, 8, 2, 64, FP16, 16),
    ([777, 5, 300], [0, 3, 4, 9], [9, 8, 7, 600, 5, 4, 3, 2, 1], [1] * 9, 6, 2, 128, BF16, 128),
    ([0, 64, 0], [0, 1, 3, 5], [30, 20, 10, 5, 400], [1] * 5, 16, 16, 64, FP16, 16),
    ([2000], [0, 6], [10, 200, 7, 9, 40, 33], [5, 2, 7, 1, 3, 4], 16, 2, 64, FP16, 32),
    ([300], [0, 2], [600, 90], [400, 70], 8, 2, 128, BF16, 64),
    ([5000, 90], [0, 2, 4], [130, 257, 30, 1], [129, 40, 30, 1], 14, 2, 128, FP16, 16),
    ([3001], [0, 3], [700, 300, 2], [300, 300, 2], 5, 1, 64, BF16, 256),
    ([40000], [0, 5], [100, 1, 2, 3, 4], [1] * 5, 8, 1, 128, BF16, 128),
    ([100], [0, 1], [50], [1], 8, 2, 128, BF16, 16),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("prefix,first,own,n,H,Hkv,D,dtype,page", CASES)
def test_shared_prefix(prefix, first, own, n, H, Hkv, D, dtype, page, e4m3):
    batch = Shared(prefix, first, own, n, H, Hkv, D, dtype, e4m3, page, seed=len(own) + prefix[0])
    check_attention(batch, *attend(batch))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [[1, 1, 1], [200, 3, 40]])
def test_without_a_mask_and_with_loose_bounds(n, e4m3):
    """Unmasked (more new tokens than keys of their own), bounds well above what there is."""
    batch = Shared([500], [0, 3], [3, 300, 70], n, 8, 4, 64, FP16, e4m3, 16, seed=2, shared_n=False)
    loose = dict(nk=3000, max_prefix=2500, max_own=900, max_group=3)
    batch.table = torch.nn.functional.pad(batch.table, (0, 200), value=-9)
    check_attention(batch, *attend(batch, causal=False, **loose), causal=False)


@pytest.mark.parametrize("n", [1, 30])
def test_uniform_steps_and_scale(n):
    batch = Shared([333], [0, 4], [n + 5] * 4, [n] * 4, 8, 2, 128, BF16, False, 16, seed=6, shared_n=True)
    check_attention(batch, *attend(batch, scale=0.2), scale=0.2)


def test_padding_left_as_it_was_and_sequences_without_tokens():
    batch = Shared([200], [0, 4], [20, 0, 35, 0], [1, 0, 3, 0], 8, 2, 64, FP16, False, 16, seed=1, pad=5)
    step = batch.shared_step()
    out = torch.full((batch.total_q, 8, 64), 7.0, dtype=FP16, device="cuda")
    lse = torch.full((batch.total_q, 8), 7.0, device="cuda")
    step.attend(batch.q, out=out, lse=lse)
    assert step.error() == 0
    check_attention(batch, out, lse)
    assert bool((out[batch.tokens:] == 7).all()) and bool((lse[batch.tokens:] == 7).all())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,own", [([1, 1, 1], [40, 1, 9]), ([200, 30, 1], [260, 30, 9])])
def test_odd_values_reach_the_rows_that_see_them(n, own, e4m3):
    """NaN and infinity among the values of the prefix and of a sequence's own keys."""
    batch = Shared([150], [0, 3], own, n, 8, 2, 128, BF16, e4m3, 16, seed=8)
    V = batch.V.view(torch.uint8) if e4m3 else batch.V
    spots = [(batch.full[0][3], 5, 0, 17), (batch.full[1][150 // 16], 7 if own[1] > 1 else 6, 1, 90)]
    for page, row, head, column in spots:
        V[page, row, head, column] = 0x7f if e4m3 else float("nan")
    if not e4m3:
        V[batch.full[0][150 // 16], 8, 1, 3] = float("inf")
    check_attention(batch, *attend(batch))


def test_what_does_not_fit_is_refused_and_the_rest_computed():
    """A bad group: zeros in its sequences' rows, the error bit, the other groups as they should be."""
    for n in ([1] * 6, [90, 1, 2, 3, 40, 1]):
        own = [k + 9 for k in n]
        batch = Shared([160, 70, 33], [0, 2, 4, 6], own, n, 8, 2, 128, BF16, False, 16, seed=4)
        good = batch.shared_step()
        want, want_lse = (x.clone() for x in good.attend(batch.q, return_lse=True))
        assert good.error() == 0
        for what, value, gone in (("prefix", [160, 71 + own[2], 33], (2, 3)), ("prefix", [160, -1, 33], (2, 3)),
                                  ("prefix", [160, 500, 33], (2, 3)), ("kv", [169, 0, 0, 0, 0, 0], None)):
            prefix, kv = list(batch.prefix), list(batch.kv)
            if what == "prefix":
                prefix = value
            else:
                kv[0], gone = 165 + n[0] - 9 - 2, (0,)   # its new tokens begin inside the prefix
            step = batch.shared_step()
            step.prefix_lens.copy_(torch.tensor(prefix, dtype=torch.int32))
            step.kv_lens.copy_(torch.tensor(kv, dtype=torch.int32))
            out, lse = step.attend(batch.q, return_lse=True)
            assert step.error() & santa.CACHE_DEVERR_PREFIX
            step.prefix_lens.copy_(torch.tensor(batch.prefix, dtype=torch.int32))
            step.kv_lens.copy_(torch.tensor(batch.kv, dtype=torch.int32))
            for b in range(6):
                rows = slice(int(batch.offsets[b]), int(batch.offsets[b + 1]))
                if b in gone:
                    assert bool((out[rows] == 0).all()) and bool((lse[rows] == float("-inf")).all())
                else:
                    torch.testing.assert_close(out[rows].float(), want[rows].float(), rtol=2.0 ** -6, atol=2.0 ** -6)


def test_a_bad_page_of_the_prefix_zeroes_its_group():
    batch = Shared([100, 64], [0, 2, 3], [5, 9, 4], [1] * 3, 8, 2, 64, BF16, False, 16, seed=3)
    batch.table[0, 2] = batch.n_pages
    step = batch.shared_step()
    out, lse = step.attend(batch.q, return_lse=True)
    assert step.error() == santa.CACHE_DEVERR_PAGE
    assert bool((out[:2] == 0).all()) and bool((lse[:2] == float("-inf")).all()) and bool(torch.isfinite(lse[2]).all())


@pytest.mark.parametrize("e4m3", [False, True])
def test_the_plain_attention_says_the_same(e4m3):
    """The same batch without its groups, tables filled in: both within their tolerance, so within the sum of both."""
    batch = Shared([700], [0, 5], [30, 2, 90, 17, 16], [1, 2, 1, 4, 1], 8, 2, 128, BF16, e4m3, 32, seed=9, whole=True)
    check_attention(batch, *attend(batch))
    step = batch.step()
    check_attention(batch, *step.attend(batch.q, return_lse=True))


def test_captured_and_replayed_with_other_lengths():
    """One graph, lengths and prefixes changed in place between its replays; another stream than the current one."""
    batch = Shared([320], [0, 4], [40, 30, 20, 10], [1] * 4, 8, 2, 128, BF16, False, 16, seed=5, whole=True)
    step = batch.shared_step(max_prefix=400, max_own=80, max_group=9)
    stream = torch.cuda.Stream()
    step.attend(batch.q, return_lse=True, stream=stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step.attend(batch.q, return_lse=True)
    for prefix, own in ((320, [40, 30, 20, 10]), (304, [50, 17, 18, 19]), (0, [60, 61, 62, 63])):
        kv = [prefix + k for k in own]
        short = [min(k, 320 + o) for k, o in zip(kv, batch.own)]
        step.prefix_lens.fill_(prefix)
        step.kv_lens.copy_(torch.tensor(short, dtype=torch.int32))
        graph.replay()
        assert step.error() == 0
        # the same keys seen as a batch of its own lengths
        keys = [batch.rows(b, "K")[:short[b]] for b in range(4)]
        for b in range(4):
            q = batch.q[b].double()
            s = torch.einsum("hd,khd->hk", q, keys[b].repeat_interleave(4, 1)) * 128 ** -0.5
            want = torch.logsumexp(s, 1)
            assert float((lse[b].double() - want).abs().max()) < 1e-4


def test_the_prefix_of_a_group_is_read_through_its_first_sequence_after_an_append():
    """A run as it is used: one sequence reads the prefix in, the others are made from it, all go on token by token."""
    H, Hkv, D, page, P = 8, 2, 128, 16, 75
    gen = torch.Generator(device="cuda").manual_seed(0)
    cache = santa.PagedCache(64, page, Hkv, D, dtype=BF16)
    rope = santa.rope_table(256, D)
    table = torch.full((3, 8), -1, dtype=torch.int32, device="cuda")
    table[0, :8] = torch.arange(8, dtype=torch.int32)
    make = lambda tokens, heads: torch.randn(tokens, heads, D, generator=gen, device="cuda").to(BF16)   # noqa: E731
    kp, vp = make(P, Hkv), make(P, Hkv)
    lens = torch.tensor([P], dtype=torch.int32, device="cuda")
    santa.PagedStep(cache, table[:1], lens, n_q_heads=H, nk=P, max_q=P).append(None, kp, vp, rope=rope)
    for b in (1, 2):   # a copy of the page that the prefix ends in, pages of their own behind it
        table[b, P // page:P // page + 3] = torch.arange(10 * b + 10, 10 * b + 13, dtype=torch.int32)
        for pool in (cache.K, cache.V):
            pool[10 * b + 10] = pool[P // page]
    plain = table.clone()
    plain[1:, :P // page] = table[0, :P // page]
    prefix = torch.tensor([P], dtype=torch.int32, device="cuda")
    kv = torch.full((3,), P, dtype=torch.int32, device="cuda")
    shared = santa.PagedStep(cache, table, kv, n_q_heads=H, nk=100, prefix_lens=prefix, max_prefix=80, max_own=20)
    alone = santa.PagedStep(cache, plain, kv, n_q_heads=H, nk=100)
    for _ in range(12):
        kv += 1
        q = shared.append(make(3, H), make(3, Hkv), make(3, Hkv), rope=rope)
        out, lse = shared.attend(q, return_lse=True)
        want, want_lse = alone.attend(q, return_lse=True)
        # both are within half a step of the result and of the probabilities (2^-8 each) of the same value
        assert float((out.float() - want.float()).abs().max()) <= 4 * 2.0 ** -8 * float(cache.V.float().abs().max())
        assert float((lse - want_lse).abs().max()) <= 1e-4
    assert shared.error() == 0 and alone.error() == 0


@pytest.mark.parametrize("own", [[5, 60, 1], [300, 400, 260]])
def test_output_over_the_queries_and_another_stream(own):
    batch = Shared([4000], [0, 3], own, [min(k, 250) if own[0] > 5 else 1 for k in own], 8, 2, 128, BF16, False, 16, seed=2)
    step = batch.shared_step()
    want = step.attend(batch.q).clone()
    q = batch.q.clone()
    got = step.attend(q, out=q)
    assert torch.equal(got, want) and got.data_ptr() == q.data_ptr()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    other = step.attend(batch.q, stream=stream)
    stream.synchronize()
    assert torch.equal(other, want) and step.error() == 0
