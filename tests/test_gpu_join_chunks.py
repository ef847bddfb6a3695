"""GPU parity of joined attention's chunk kernels at calls that are long enough for them: chunks of new tokens behind
prefixes, of plain and of differential heads, in windows, unmasked, with odd values, bad pages, padding, over other
streams and in graphs."""
import pytest
import torch

import join_cases
import stochastic_sparse_decode_split_gb300 as santa
from join_reference import Shared, diff_attention
from paged_reference import Batch, check_attention, half_step

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16
TYPES = [(False, BF16), (False, FP16), (True, BF16)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    santa.library()


def made(case, dtype, e4m3, seed=0, **kw):
    c = case[0]
    size = (c["n"], c["H"], c["Hkv"], c["D"], dtype, e4m3, c["page"], seed)
    if "prefix" in c:
        return Shared(c["prefix"], c["first"], c["kv"], *size, pairs=c.get("diff", False), **kw)
    return Batch(c["kv"], *size, **kw)


def weights(batch, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return (0.1 + 0.6 * torch.rand(batch.total_q, batch.H // 2, generator=gen)).to(batch.device)


def check_diff(batch, got, lse, w, **kw):
    """As ``join_reference.check_diff``, whose half step of the result is relative to it: below the smallest normal number
    steps are as large as there, so half of one is that number times the relative half step (2^-14 2^-11 in fp16, where a
    row that sees one key has results that small; without it 2^-25 of rounding has no place in the bound)."""
    want, want_lse, tol, tol_lse = diff_attention(batch, w, **kw)
    tol = tol + torch.finfo(batch.dtype).smallest_normal * half_step(batch.dtype)
    t = batch.tokens
    got, lse = got[:t].double(), lse[:t].double()
    fine = torch.isfinite(want[:t])
    assert torch.equal(torch.isfinite(got), fine), "finite where the definition is not, or the other way round"
    off = ((got - want[:t]).abs() - tol[:t])[fine]
    assert not off.numel() or float(off.max()) <= 0, f"out is {float(off.max()):.3g} over its tolerance"
    assert torch.equal(lse == float("-inf"), want_lse[:t] == float("-inf"))
    off = ((lse - want_lse[:t]).abs() - tol_lse[:t])[torch.isfinite(want_lse[:t])]
    assert not off.numel() or float(off.max()) <= 0, f"lse is {float(off.max()):.3g} over its tolerance"


def run(case, batch, norm=None, out=None, lse=None, **kw):
    """(step, out, lse, the check of them) of a case's call."""
    diff = case[0].get("diff", False)
    kw.update({k: case[0][k] for k in ("causal", "window") if k in case[0]})
    step = (batch.shared_step if "prefix" in case[0] else batch.step)(diff=diff, **kw)
    mask = {k: v for k, v in kw.items() if k in ("causal", "window", "scale")}
    if not diff:
        out, lse = step.attend(batch.q, out=out, lse=lse, return_lse=True)
        return step, out, lse, lambda: check_attention(batch, out, lse, **mask)
    w = weights(batch)
    out, lse = step.attend_diff(batch.q, w, norm=norm, eps=1e-5, gain=0.8, out=out, lse=lse, return_lse=True)
    return step, out, lse, lambda: check_diff(batch, out, lse, w, norm=norm, eps=1e-5, gain=0.8, **mask)


def holds(case, batch, **kw):
    step, _, _, check = run(case, batch, **kw)
    assert step.error() == 0
    check()


@pytest.mark.parametrize("e4m3,dtype", TYPES)
@pytest.mark.parametrize("case", range(len(join_cases.OWN_CHUNKS)))
def test_chunks_behind_prefixes(case, e4m3, dtype):
    """The rows of the other sequences name none of the pages that lie wholly inside the prefix."""
    holds(join_cases.OWN_CHUNKS[case], made(join_cases.OWN_CHUNKS[case], dtype, e4m3, seed=case))


@pytest.mark.parametrize("e4m3,dtype", TYPES)
@pytest.mark.parametrize("case", range(len(join_cases.WINDOWS)))
def test_differential_chunks_in_a_window(case, e4m3, dtype):
    holds(join_cases.WINDOWS[case], made(join_cases.WINDOWS[case], dtype, e4m3, seed=case))


@pytest.mark.parametrize("e4m3,dtype", TYPES)
@pytest.mark.parametrize("case", range(len(join_cases.UNMASKED)))
def test_without_a_mask(case, e4m3, dtype):
    holds(join_cases.UNMASKED[case], made(join_cases.UNMASKED[case], dtype, e4m3, seed=case))


@pytest.mark.parametrize("e4m3,dtype", TYPES)
@pytest.mark.parametrize("case", range(len(join_cases.NOTHING_SEEN)))
def test_rows_that_see_nothing(case, e4m3, dtype):
    """An empty sequence, more new tokens than keys by many and by two: zeros, and with a norm of eps 0 as well."""
    c = join_cases.NOTHING_SEEN[case]
    batch = made(c, dtype, e4m3, seed=case)
    holds(c, batch)
    step, out, lse, _ = run(c, batch)
    out = step.attend_diff(batch.q, weights(batch), norm=torch.ones(2 * batch.D, dtype=dtype, device="cuda"), eps=0.0)
    assert bool((out[:1360] == 0).all()) and bool((lse[:1360] == float("-inf")).all())   # 700, and 700 of which 40 see a key
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse[1360:1400]).all()) and bool((lse[1400:1402] == float("-inf")).all())


def place(batch, b, key):
    """(page, row in it) of a sequence's key; of a prefix its place in the first sequence's pages."""
    if hasattr(batch, "full"):
        g = batch.group[b]
        pages = batch.full[batch.first[g] if key < batch.prefix[g] else b]
    else:
        pages = batch.table[b].tolist()
    return pages[key // batch.page], key % batch.page


@pytest.mark.parametrize("e4m3,dtype", TYPES)
@pytest.mark.parametrize("case", range(len(join_cases.FORMS)))
def test_odd_values_reach_the_rows_that_see_them(case, e4m3, dtype):
    """NaN and infinities among the values: of keys that all rows see, that some see, that the last alone sees, of a prefix
    and of the keys next to its end; over e4m3 also a scale that is none."""
    c = join_cases.FORMS[case]
    batch = made(c, dtype, e4m3, seed=case)
    V = batch.V.view(torch.uint8) if e4m3 else batch.V
    odd = [0x7f, 0xff, 0x7f] if e4m3 else [float("nan"), float("inf"), float("-inf")]
    kv, n, D = batch.kv, batch.n, batch.D
    spots = [(0, 3, 0, 0), (0, kv[0] - 1, batch.Hkv - 1, D - 1), (0, kv[0] - n[0] // 2, 1, 17), (1, kv[1] - n[1], 0, D // 2),
             (1, kv[1] - 130, 1, 1), (1, kv[1] - n[1] - 1, batch.Hkv - 2, D - 2)]
    if "prefix" in c[0]:
        p = batch.prefix[-1]
        spots += [(batch.B - 1, p, 0, 5), (batch.B - 1, p - 1, 1, 33)]
    for i, (b, key, head, column) in enumerate(spots):
        page, at = place(batch, b, key)
        V[page, at, head, column] = odd[i % 3]
    if e4m3:
        page, at = place(batch, 1, kv[1] - n[1] // 3)
        batch.vs[page, 1, at] = float("nan")
    holds(c, batch)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("case", range(len(join_cases.FORMS)))
def test_a_bad_page_zeroes_the_rows_that_are_computed_with_it(case, e4m3):
    c = join_cases.FORMS[case]
    batch = made(c, BF16, e4m3, seed=case)
    step, out, lse, check = run(c, batch)
    assert step.error() == 0
    check()
    want, want_lse = out.clone(), lse.clone()
    own = batch.prefix[0] if "prefix" in c[0] else 0   # every token sees the first key behind the prefix
    bad = [((1, own // batch.page), {1})]
    if "prefix" in c[0]:
        bad.append(((0, 2), {b for b in range(batch.B) if batch.group[b] == 0}))
    for (b, i), gone in bad:
        for value in (-1, batch.n_pages):
            kept = int(batch.table[b, i])
            batch.table[b, i] = value
            step, out, lse, _ = run(c, batch)
            assert step.error() == santa.CACHE_DEVERR_PAGE
            batch.table[b, i] = kept
            for s in range(batch.B):
                rows = slice(int(batch.offsets[s]), int(batch.offsets[s + 1]))
                if s in gone:
                    assert bool((out[rows] == 0).all()) and bool((lse[rows] == float("-inf")).all())
                else:
                    assert torch.equal(out[rows], want[rows]) and torch.equal(lse[rows], want_lse[rows])


@pytest.mark.parametrize("case", range(len(join_cases.FORMS)))
def test_padding_and_sequences_without_tokens(case):
    """Rows behind the last token are left as they were; a sequence of the batch has no token."""
    c = dict(join_cases.FORMS[case][0])
    c["kv"], c["n"] = c["kv"] + [70], c["n"] + [0]
    if "prefix" in c:
        c["first"] = c["first"][:-1] + [len(c["n"])]
    c = (c,)
    batch = made(c, FP16, False, seed=case, pad=37)
    diff = c[0].get("diff", False)
    out = torch.full((batch.total_q, batch.H // 2, 2 * batch.D) if diff else batch.q.shape, 7.0, dtype=FP16, device="cuda")
    lse = torch.full((batch.total_q, batch.H), 7.0, device="cuda")
    step, _, _, check = run(c, batch, out=out, lse=lse)
    assert step.error() == 0
    check()
    assert bool((out[batch.tokens:] == 7).all()) and bool((lse[batch.tokens:] == 7).all())


NORM = [
    (dict(kv=[40, 30, 21, 18], n=[2, 1, 1, 3], H=16, Hkv=4, D=128, page=16, prefix=[150], first=[0, 4], diff=True),),
    (dict(kv=[40, 30, 21], n=[4, 1, 8], H=8, Hkv=4, D=64, page=32, prefix=[90, 7], first=[0, 2, 3], diff=True),),
    (dict(kv=[130, 100, 111], n=[90, 50, 70], H=16, Hkv=16, D=64, page=16, prefix=[100], first=[0, 3], diff=True),),
    (dict(kv=[300, 300], n=[256, 270], H=16, Hkv=8, D=128, page=64, prefix=[200], first=[0, 2], diff=True),),
    (dict(kv=[300, 300], n=[256, 270], H=16, Hkv=8, D=64, page=16, prefix=[200], first=[0, 2], diff=True),),
]


@pytest.mark.parametrize("e4m3,dtype", TYPES)
@pytest.mark.parametrize("case", range(len(NORM)))
def test_the_norm_over_a_shared_prefix(case, e4m3, dtype):
    batch = made(NORM[case], dtype, e4m3, seed=case)
    gen = torch.Generator().manual_seed(case)
    holds(NORM[case], batch, norm=(1 + 0.3 * torch.randn(2 * batch.D, generator=gen)).to(dtype).to(batch.device))


@pytest.mark.parametrize("case", range(len(join_cases.FORMS)))
def test_loose_bounds_and_a_scale(case):
    c = join_cases.FORMS[case]
    batch = made(c, BF16, False, seed=case + 9)
    loose = dict(nk=4096, scale=0.11)
    if "prefix" in c[0]:
        loose.update(max_prefix=3000, max_own=1100, max_group=batch.B)
    batch.table = torch.nn.functional.pad(batch.table, (0, 4096 // batch.page), value=-9)
    holds(c, batch, **loose)


@pytest.mark.parametrize("n", [300, 352])
@pytest.mark.parametrize("diff", [False, True])
def test_as_many_new_tokens_for_all(n, diff):
    c = (dict(kv=[n + 40] * 4, n=[n] * 4, H=16, Hkv=8, D=128, page=32, prefix=[1000], first=[0, 4], diff=diff),)
    batch = made(c, BF16, False, seed=n, shared_n=True)
    holds(c, batch)


@pytest.mark.parametrize("case", range(len(join_cases.FORMS)))
def test_output_over_the_queries_and_another_stream(case):
    c = join_cases.FORMS[case]
    batch = made(c, BF16, False, seed=case)
    step, out, lse, _ = run(c, batch)
    want, want_lse = out.clone(), lse.clone()
    q = batch.q.clone()
    if c[0].get("diff", False):
        w = weights(batch)
        got = step.attend_diff(q, w, gain=0.8, out=q.view(batch.total_q, batch.H // 2, 2 * batch.D))
        call = lambda **kw: step.attend_diff(batch.q, w, gain=0.8, return_lse=True, **kw)   # noqa: E731
    else:
        got = step.attend(q, out=q)
        call = lambda **kw: step.attend(batch.q, return_lse=True, **kw)   # noqa: E731
    assert torch.equal(got, want) and got.data_ptr() == q.data_ptr()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    out, lse = call(stream=stream)
    stream.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse) and step.error() == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("case", range(len(join_cases.FORMS)))
def test_captured_and_replayed_with_other_lengths(case, e4m3):
    """One graph for every length within the bounds; the same bits from one replay to the next."""
    c = join_cases.FORMS[case]
    shared, diff = "prefix" in c[0], c[0].get("diff", False)
    batch = made(c, BF16, e4m3, seed=case, **(dict(whole=True) if shared else {}))
    step = batch.shared_step(diff=diff) if shared else batch.step(diff=diff)
    w = weights(batch)
    call = (lambda: step.attend_diff(batch.q, w, return_lse=True)) if diff else (lambda: step.attend(batch.q, return_lse=True))
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = call()
    longest, prefixes = list(batch.kv), list(batch.prefix) if shared else []
    for part, less in ((1.0, 0), (0.5, 37), (0.0, 300), (1.0, 128)):
        own = [0] * batch.B
        if shared:
            batch.prefix = [int(p * part) for p in prefixes]
            batch.prefix_t.copy_(torch.tensor(batch.prefix, dtype=torch.int32))
            own = [batch.prefix[g] for g in batch.group]
        most = [prefixes[g] if shared else 0 for g in (batch.group if shared else [0] * batch.B)]
        batch.kv = [p + max(n, k - m - less) for p, n, k, m in zip(own, batch.n, longest, most)]
        batch.kv_t.copy_(torch.tensor(batch.kv, dtype=torch.int32))
        graph.replay()
        assert step.error() == 0
        if diff:
            check_diff(batch, out, lse, w)
        else:
            check_attention(batch, out, lse)
        first, first_lse = out.clone(), lse.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, out) and torch.equal(first_lse, lse)


FAR = [join_cases.FORMS[1], join_cases.FORMS[3], join_cases.FORMS[5],
       (dict(kv=[40, 30, 21, 18], n=[2, 1, 1, 3], H=16, Hkv=4, D=128, page=16, prefix=[150], first=[0, 4]),),
       (dict(kv=[400, 30], n=[2, 1], H=8, Hkv=2, D=128, page=16, diff=True),)]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("case", range(len(FAR)))
def test_pages_whose_offsets_pass_32_bits(case, e4m3):
    """The batch's pages at the end of a pool of more than 2^32 elements."""
    batch = made(FAR[case], BF16, e4m3, seed=case)
    row = batch.page * batch.Hkv * batch.D
    lead = 2 ** 32 // row + 5

    def behind(x):
        if x is None:
            return None
        raw = x.view(torch.uint8) if e4m3 and x.dtype != torch.float32 else x
        y = torch.zeros((lead + x.shape[0], *x.shape[1:]), dtype=raw.dtype, device="cuda")
        y[lead:] = raw
        return y.view(x.dtype)

    batch.K, batch.V, batch.ks, batch.vs = (behind(x) for x in (batch.K, batch.V, batch.ks, batch.vs))
    batch.n_pages += lead
    batch.table = torch.where(batch.table >= 0, batch.table + lead, batch.table)
    if hasattr(batch, "full"):
        batch.full = [[p + lead for p in pages] for pages in batch.full]
    holds(FAR[case], batch)
