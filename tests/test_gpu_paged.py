"""GPU parity of the paged cache's operators against their definitions in 64
bits: attention of tokens and chunks over pages, the write of new tokens (norm,
rotation, e4m3) and the way back to packed rows; and a run of them together."""
import pytest
import torch

import stochastic_sparse_decode_split_gb300 as santa
from paged_reference import F8, Batch, check_attention, half_step, quantised

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    santa.library()


def attend(batch, **kw):
    step = batch.step(**kw)
    out, lse = step.attend(batch.q, return_lse=True)
    assert step.error() == 0
    return out, lse


# ---------------------------------------------------------------- attention

TOKENS = [   # kv, new tokens, H, Hkv, D, type, page
    ([1], [1], 1, 1, 64, BF16, 16),
    ([1000], [1], 32, 8, 128, BF16, 16),
    ([15, 16, 17, 1, 300], [1] * 5, 8, 2, 128, BF16, 16),
    ([777, 1], [1, 1], 14, 2, 128, FP16, 32),
    ([2049, 64, 63, 65], [1] * 4, 6, 2, 64, FP16, 64),
    ([5000], [1], 8, 8, 64, BF16, 256),
    ([40000], [1], 8, 1, 128, BF16, 128),
    ([900, 33], [2, 5], 8, 2, 128, BF16, 16),
    ([257, 4, 100], [5, 4, 1], 6, 2, 64, FP16, 16),
    ([130], [16], 2, 2, 128, BF16, 32),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kv,n,H,Hkv,D,dtype,page", TOKENS)
def test_attention_of_few_tokens(kv, n, H, Hkv, D, dtype, page, e4m3):
    batch = Batch(kv, n, H, Hkv, D, dtype, e4m3, page, seed=len(kv) + kv[0])
    check_attention(batch, *attend(batch))


CHUNKS = [
    ([17], [17], 4, 1, 128, BF16, 16),
    ([300], [100], 8, 2, 128, BF16, 16),
    ([129, 700, 31], [129, 64, 1], 8, 2, 64, FP16, 32),
    ([1111], [257], 14, 2, 128, FP16, 64),
    ([640, 90], [300, 70], 6, 2, 128, BF16, 128),
    ([2000], [33], 32, 8, 128, BF16, 256),
    ([515, 515], [515, 515], 5, 1, 64, BF16, 16),
    ([400], [260], 2, 2, 128, BF16, 64),
    ([4100], [140], 10, 2, 64, BF16, 16),
    ([9000], [70], 8, 1, 128, BF16, 64),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kv,n,H,Hkv,D,dtype,page", CHUNKS)
def test_attention_of_a_chunk(kv, n, H, Hkv, D, dtype, page, e4m3):
    batch = Batch(kv, n, H, Hkv, D, dtype, e4m3, page, seed=len(kv) + kv[0])
    check_attention(batch, *attend(batch))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window", [1, 5, 16, 100, 129, 5000])
@pytest.mark.parametrize("n", [1, 40, 200])
def test_attention_in_a_window(n, window, e4m3):
    batch = Batch([900, 333], [n, max(1, n // 3)], 8, 2, 128, BF16, e4m3, 32, seed=window)
    check_attention(batch, *attend(batch, window=window), window=window)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,kv", [([1, 1], [77, 1500]), ([448, 30], [1500, 5]), ([100, 9], [1, 64])])
def test_attention_without_a_mask(n, kv, e4m3):
    """Cross attention: lengths of queries and keys have nothing to do with each other."""
    batch = Batch(kv, n, 8, 8, 64, FP16, e4m3, 64, seed=3)
    check_attention(batch, *attend(batch, causal=False), causal=False)


@pytest.mark.parametrize("n", [1, 3, 150])
def test_rows_that_see_nothing(n):
    """Empty sequences, and more new tokens than keys: zeros and -inf."""
    batch = Batch([0, 40, 0, max(1, n - 2)], [n, n, 1, n], 8, 2, 128, BF16, False, 16, seed=n)
    check_attention(batch, *attend(batch))
    check_attention(batch, *attend(batch, causal=False), causal=False)


def test_no_new_tokens_and_padding_left_as_it_was():
    for n in ([0, 1, 0], [0, 90, 3]):
        batch = Batch([50, 200, 7], n, 8, 2, 64, FP16, False, 16, seed=1, pad=5)
        step = batch.step()
        out = torch.full((batch.total_q, 8, 64), 7.0, dtype=FP16, device="cuda")
        lse = torch.full((batch.total_q, 8), 7.0, device="cuda")
        step.attend(batch.q, out=out, lse=lse)
        assert step.error() == 0
        check_attention(batch, out, lse)
        assert bool((out[batch.tokens:] == 7).all()) and bool((lse[batch.tokens:] == 7).all())


@pytest.mark.parametrize("n", [4, 120])
def test_scale_and_uniform_chunks(n):
    batch = Batch([200, 400, 300], [n] * 3, 8, 4, 64, BF16, False, 16, seed=5, shared_n=True)
    check_attention(batch, *attend(batch, scale=0.31), scale=0.31)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [3, 140])
def test_what_masked_keys_hold_does_not_matter(n, e4m3):
    """NaN and infinities in the keys and values of a chunk's later tokens reach the rows that see them, and no other;
    so do those that have left the window."""
    for window in (0, 60):
        batch = Batch([300], [n], 8, 2, 128, BF16, e4m3, 16, seed=n)
        for key, odd in ((298, float("nan")), (297, float("inf")), (5, float("-inf"))):
            at, slot = int(batch.table[0, key // 16]), key % 16
            if e4m3:   # an odd row comes as a scale that is not a number
                batch.vs[at, 0, slot] = float("nan")
            else:
                batch.V[at, slot, 0, 3:9] = odd
        at = int(batch.table[0, 299 // 16])
        (batch.ks if e4m3 else batch.K)[(at, 1, 299 % 16) if e4m3 else (at, 299 % 16, 1)] = float("nan")
        check_attention(batch, *attend(batch, window=window), window=window)


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_scales_far_apart(dtype):
    """e4m3 rows of magnitudes 2^-40 to 2^12 side by side: neither range nor order of the scales matters."""
    for n in (1, 50):
        batch = Batch([500], [n], 8, 2, 128, dtype, True, 16, seed=2)
        batch.vs *= torch.exp2(torch.randint(-40, 12, batch.vs.shape, device="cuda").float())
        check_attention(batch, *attend(batch))
        batch.vs.fill_(2.0 ** -66)
        if dtype == BF16:
            check_attention(batch, *attend(batch))


def test_large_scores_keep_to_the_definition():
    """Scores in the thousands: the running maximum moves far, the sums stay in range."""
    for n in (1, 64):
        batch = Batch([700], [n], 8, 2, 64, BF16, False, 16, seed=8)
        batch.q *= 40
        check_attention(batch, *attend(batch))


def test_device_refusals_of_the_attention():
    for n in (1, 60):
        batch = Batch([300, 200, 100], [n] * 3, 8, 2, 64, BF16, False, 16, seed=3, shared_n=True)
        good, lse = attend(batch)
        step = batch.step()
        batch.table[1, 2] = batch.n_pages            # one past the pool
        out, got = step.attend(batch.q, return_lse=True)
        assert step.error() == santa.CACHE_DEVERR_PAGE
        assert torch.equal(out[:n], good[:n]) and torch.equal(out[2 * n:], good[2 * n:])
        assert not bool(out[n:2 * n].any()) and bool((got[n:2 * n] == float("-inf")).all())
        batch.table[1, 2] = -1
        step.attend(batch.q)
        assert step.error() == santa.CACHE_DEVERR_PAGE
        batch.kv_t[1] = 301                          # above nk
        out = step.attend(batch.q)
        assert step.error() == santa.DEVERR_NK_BOUND
        assert torch.equal(out[:n], good[:n]) and not bool(out[n:2 * n].any())
        batch.kv_t[1] = -1
        step.attend(batch.q)
        assert step.error() == santa.DEVERR_NK_BOUND
        batch.kv_t[1] = 0
        assert torch.equal(step.attend(batch.q)[2 * n:], good[2 * n:]) and step.error() == 0


def test_bad_offsets_are_refused_and_the_rest_computed():
    for n in (2, 40):
        batch = Batch([300, 200, 100], [n] * 3, 8, 2, 64, BF16, False, 16, seed=3)
        good, _ = attend(batch)
        step = batch.step()
        for bad in ([0, n, n - 1, 3 * n], [0, n, 3 * n + 1, 3 * n], [-1, n, 2 * n, 3 * n], [0, 2 * n, 2 * n, 3 * n]):
            batch.offsets.copy_(torch.tensor(bad))
            out = torch.full_like(batch.q, 5.0)
            step.attend(batch.q, out=out)
            assert step.error() == santa.CACHE_DEVERR_CHUNK
            if bad[2:] == [2 * n, 3 * n]:
                assert torch.equal(out[2 * n:], good[2 * n:])


# ------------------------------------------------------------------- append

def reference_rows(x, weight, pos, rope, interleaved, eps):
    """float64 rows after norm and rotation, and the magnitudes that bound their 32-bit errors."""
    x = x.double()
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    size = x.abs()
    if rope is not None:
        r = 2 * rope.shape[1]
        c, s = rope[pos].double()[:, None].unbind(-1)
        a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
        new = (a * c - b * s, b * c + a * s)
        mag = (a.abs() * c.abs() + b.abs() * s.abs(), b.abs() * c.abs() + a.abs() * s.abs())
        join = lambda y: torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)  # noqa: E731
        x, size = torch.cat((join(new), x[..., r:]), -1), torch.cat((join(mag), size[..., r:]), -1)
    return x, size


APPENDS = [  # kv, n, H, Hkv, D, type, page, norm, rotated, interleaved
    ([1], [1], 1, 1, 64, BF16, 16, True, 64, False),
    ([100, 7, 64], [1, 1, 1], 32, 8, 128, BF16, 16, True, 128, False),
    ([300, 40], [129, 3], 14, 2, 128, FP16, 32, True, 64, True),
    ([2000], [1900], 32, 8, 128, BF16, 64, False, 128, False),
    ([33, 1000], [33, 500], 10, 2, 64, FP16, 16, True, 32, False),
    ([90], [90], 6, 2, 64, BF16, 128, False, 0, False),
    ([90, 5], [17, 5], 5, 1, 128, BF16, 256, True, 0, False),
    ([700], [600], 3, 3, 128, FP32, 16, True, 128, False),
    ([700, 9], [40, 9], 4, 2, 64, FP32, 16, True, 48, True),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("sliced", [False, True])
@pytest.mark.parametrize("kv,n,H,Hkv,D,dtype,page,norm,rotated,interleaved", APPENDS)
def test_append(kv, n, H, Hkv, D, dtype, page, norm, rotated, interleaved, sliced, e4m3):
    batch = Batch(kv, n, H, Hkv, D, dtype, e4m3, page, seed=kv[0], pad=3, planted=False)
    T = batch.total_q
    gen = torch.Generator(device="cuda").manual_seed(kv[0])
    wide = torch.randn(T, H + 2 * Hkv, D, generator=gen, device="cuda").to(dtype)
    q, k, v = wide[:, :H], wide[:, H:H + Hkv], wide[:, H + Hkv:]
    if not sliced:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=gen, device="cuda")).to(dtype) for _ in range(2))
    rope = santa.rope_table(max(kv), rotated) if rotated else None
    before = [batch.K.clone(), batch.V.clone()]
    step = batch.step()
    q_out = torch.full((T, H, D), 9.0, dtype=dtype, device="cuda")
    got = step.append(q, k, v, rope=rope, interleaved=interleaved, q_norm=qw if norm else None,
                      k_norm=kw if norm else None, eps=1e-5, q_out=q_out)
    assert step.error() == 0 and got is q_out
    t = batch.tokens
    pos = torch.cat([torch.arange(a - b, a) for a, b in zip(kv, n)]).cuda()
    seq = torch.repeat_interleave(torch.arange(batch.B), torch.tensor(n)).cuda()
    u, noise = half_step(dtype), 2.0 ** -20   # noise: a norm, a rotation and a quotient in 32 bits
    want, size = reference_rows(q[:t], qw if norm else None, pos, rope, interleaved, 1e-5)
    assert bool(((got[:t].double() - want).abs() <= u * want.abs() * (1 + noise) + noise * size + 2.0 ** -25).all())
    assert bool((got[t:] == 9).all())
    at, slot = batch.table[seq, pos // page].long(), pos % page
    want, size = reference_rows(k[:t], kw if norm else None, pos, rope, interleaved, 1e-5)
    if e4m3:
        code, scale = batch.K[at, slot].double(), batch.ks[at, :, slot].double()
        amax = want.abs().amax(-1)
        assert bool(((scale - amax / 448).abs() <= 2 * noise * size.amax(-1) / 448).all())
        step_ = 2.0 ** -4 * want.abs() + 2.0 ** -10 * scale[..., None]
        assert bool(((code * scale[..., None] - want).abs() <= step_ + 4 * noise * size.amax(-1, keepdim=True)).all())
        vc, vsc = quantised(v[:t].float())
        assert torch.equal(batch.V[at, slot].view(torch.uint8), vc.view(torch.uint8))
        assert torch.equal(batch.vs[at, :, slot], vsc)
    else:
        assert bool(((batch.K[at, slot].double() - want).abs() <= u * want.abs() * (1 + noise) + noise * size + 2.0 ** -25).all())
        assert torch.equal(batch.V[at, slot], v[:t])
    # nothing else of the pool was touched
    raw = torch.uint8 if e4m3 else {2: torch.int16, 4: torch.int32}[batch.K.element_size()]
    for pool, was in ((batch.K, before[0]), (batch.V, before[1])):
        same = pool.view(raw) == was.view(raw)
        same[at, slot] = True
        assert bool(same.all())


def test_append_in_place_and_without_queries():
    batch = Batch([60, 30], [20, 30], 8, 2, 128, BF16, False, 16, seed=4)
    rope = santa.rope_table(60, 128)
    k, v = (torch.randn(50, 2, 128, device="cuda").to(BF16) for _ in range(2))
    step = batch.step()
    apart = step.append(batch.q, k, v, rope=rope)
    K = batch.K.clone()
    again = step.append(batch.q, k, v, rope=rope, q_out=batch.q)
    assert again is batch.q and torch.equal(apart, again)
    batch.K.zero_()
    assert step.append(None, k, v, rope=rope) is None
    at = batch.table[[0] * 20 + [1] * 30, torch.cat([torch.arange(40, 60), torch.arange(30)]).cuda() // 16].long()
    slot = torch.cat([torch.arange(40, 60), torch.arange(30)]).cuda() % 16
    assert torch.equal(batch.K[at, slot], K[at, slot]) and step.error() == 0


def test_append_of_odd_values_and_zeros_in_e4m3():
    batch = Batch([4], [4], 2, 2, 64, BF16, True, 16, seed=4)
    k, v = (torch.randn(4, 2, 64, device="cuda").to(BF16) for _ in range(2))
    k[0, 0] = 0
    v[1, 1, 5] = float("nan")
    v[2, 0, 7] = float("-inf")
    v[3, 1] = 2.0 ** -80
    step = batch.step()
    step.append(batch.q, k, v)
    K, V = step.read(torch.tensor([0, 4], device="cuda"), 4)
    assert step.error() == 0
    assert not bool(K[0, 0].any()) and not bool(V[3, 1].any())
    assert bool(V[1, 1].isnan().all()) and bool(V[2, 0].isnan().all())
    assert bool(V[1, 0].isfinite().all()) and bool(V[2, 1].isfinite().all())


def test_device_refusals_of_the_append():
    batch = Batch([40, 30, 20], [2, 2, 2], 2, 2, 64, BF16, False, 16, seed=6)
    k = torch.randn(6, 2, 64, device="cuda").to(BF16)
    step = batch.step()

    def run(bits, rope=None):
        before = batch.K.clone()
        q_out = torch.full_like(batch.q, 3.0)
        step.append(batch.q, k, k, q_out=q_out, rope=rope)
        assert step.error() == bits
        changed = (batch.K.view(torch.int16) != before.view(torch.int16)).any(-1).any(-1)
        return q_out, changed

    table = batch.table.clone()
    batch.table[0, 2] = batch.n_pages
    q_out, changed = run(santa.CACHE_DEVERR_PAGE)
    assert int(changed.sum()) == 4
    batch.table.copy_(table)
    batch.K.zero_()
    batch.kv_t[0] = 1                                  # fewer keys than new tokens
    q_out, changed = run(santa.CACHE_DEVERR_CHUNK)
    assert int(changed.sum()) == 4 and bool((q_out[:2] == 3).all())
    batch.K.zero_()
    batch.kv_t[0] = 41                                 # above nk
    q_out, changed = run(santa.DEVERR_NK_BOUND)
    assert int(changed.sum()) == 4
    batch.K.zero_()
    batch.kv_t[0] = 40
    q_out, changed = run(santa.CACHE_DEVERR_POSITION, santa.rope_table(39, 64))
    assert int(changed.sum()) == 5 and bool((q_out[1] == 3).all())


# --------------------------------------------------------------------- read

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("kv,Hkv,D,page", [([1], 1, 64, 16), ([300, 0, 17, 64], 2, 128, 16), ([1000, 999], 8, 128, 64),
                                           ([257, 3], 3, 64, 256)])
def test_read(kv, Hkv, D, page, dtype, e4m3):
    batch = Batch(kv, [1] * len(kv), Hkv, Hkv, D, dtype, e4m3, page, seed=sum(kv))
    step = batch.step()
    off = torch.tensor([sum(kv[:b]) for b in range(len(kv) + 1)], device="cuda")

    def want(b, which):
        pool, scale = (batch.K, batch.ks) if which == "K" else (batch.V, batch.vs)
        at = batch.table[b, :batch.used[b]].long()
        x = pool[at]
        if e4m3:
            x = (x.float() * scale[at].transpose(1, 2)[..., None]).to(dtype)
        return x.reshape(-1, Hkv, D)[:kv[b]]

    K, V = step.read(off, sum(kv))
    assert step.error() == 0
    assert torch.equal(K, torch.cat([want(b, "K") for b in range(len(kv))]))
    assert torch.equal(V, torch.cat([want(b, "V") for b in range(len(kv))]))
    K, V = (torch.full((len(kv) * max(kv), Hkv, D), 5.0, dtype=dtype, device="cuda") for _ in range(2))
    step.read(K_out=K, V_out=V)
    for b in range(len(kv)):
        r = b * max(kv)
        assert torch.equal(V[r:r + kv[b]], want(b, "V")) and bool((V[r + kv[b]:r + max(kv)] == 5).all())
        assert torch.equal(K[r:r + kv[b]], want(b, "K")) and bool((K[r + kv[b]:r + max(kv)] == 5).all())


def test_device_refusals_of_the_read():
    batch = Batch([40, 30], [1, 1], 2, 2, 64, BF16, False, 16, seed=6)
    step = batch.step()
    K, V = (torch.full((70, 2, 64), 5.0, dtype=BF16, device="cuda") for _ in range(2))
    for off in ([0, 39, 70], [0, 40, 69], [-1, 40, 70], [0, 41, 71]):
        K.fill_(5.0)
        step.read(torch.tensor(off, device="cuda"), 70, K_out=K, V_out=V)
        assert step.error() == santa.CACHE_DEVERR_CHUNK
    batch.table[1, 1] = 99999
    K, V = step.read(torch.tensor([0, 40, 70], device="cuda"), 70)
    assert step.error() == santa.CACHE_DEVERR_PAGE
    assert not bool(K[56:70].any()) and bool(K[:56].any(-1).all())


# ----------------------------------------------------------------- together

@pytest.mark.parametrize("cache_dtype", [BF16, F8])
def test_prompt_then_tokens_then_samples(cache_dtype):
    """Prompts in two chunks, then single tokens, each step's attention against the definition on what the cache
    holds; then a sampled step over the same pages, with the draws of santa_decode on the packed rows."""
    H, Hkv, D, page, B = 8, 2, 128, 32, 3
    cache = santa.PagedCache(64, page, Hkv, D, cache_dtype)
    table = torch.randperm(64, device="cuda")[:B * 16].view(B, 16).to(torch.int32).contiguous()
    kv = torch.zeros(B, dtype=torch.int32, device="cuda")
    rope = santa.rope_table(512, D, by_parts=(4.0, 1.0, 4.0, 256))
    have = [0] * B
    view = Batch([1] * B, [1] * B, H, Hkv, D, BF16, cache_dtype == F8, page)
    for n in ([200, 45, 1], [77, 300, 130], [1, 1, 1], [1, 1, 1]):
        have = [a + b for a, b in zip(have, n)]
        kv.copy_(torch.tensor(have))
        T = sum(n)
        off = torch.tensor([sum(n[:b]) for b in range(B + 1)], device="cuda")
        step = santa.PagedStep(cache, table, kv, n_q_heads=H, dtype=BF16, nk=512, max_q=max(n), total_q=T, q_offsets=off)
        x = torch.randn(T, (H + 2 * Hkv) * D, device="cuda").to(BF16).view(T, H + 2 * Hkv, D)
        w = (1 + 0.1 * torch.randn(D, device="cuda")).to(BF16)
        q = step.append(x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], rope=rope, q_norm=w, k_norm=w)
        out, lse = step.attend(q, return_lse=True)
        assert step.error() == 0
        view.kv, view.n, view.tokens, view.total_q, view.q = have, n, T, T, q
        view.K, view.V, view.ks, view.vs, view.table = cache.K, cache.V, cache.k_scale, cache.v_scale, table
        view.used = [-(-k // page) for k in have]
        check_attention(view, out, lse)
    rows = sum(have)
    off = torch.tensor([sum(have[:b]) for b in range(B + 1)], device="cuda")
    idx, idx2 = (torch.full((B, H, 64), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    est = step.sample(q, 64, off, rows, seed=5, sample_idx=idx)
    K, V = step.read(off, rows)
    est2 = santa.santa_decode(q, K, V, 64, seed=5, nk=512, kv_offsets=off, sample_idx=idx2)
    assert torch.equal(idx, idx2)
    torch.testing.assert_close(est, est2, rtol=1e-5, atol=1e-6)
    dense = santa.santa_dense_decode(q, K, V, nk=512, kv_offsets=off)
    if cache_dtype == BF16:   # both exact attention: they differ by roundings to bf16
        assert float((dense - out.float()).abs().max()) <= 2 * half_step(BF16) * float(V.abs().max())


def test_captured_steps_and_another_stream():
    """A step captured into a graph and replayed over lengths and tokens changed in place; a call on a side stream."""
    for n in (1, 50):
        batch = Batch([300, 200], [n, n], 8, 2, 128, BF16, False, 16, seed=9, shared_n=True)
        step = batch.step()
        k, v = (torch.randn(2 * n, 2, 128, device="cuda").to(BF16) for _ in range(2))
        qo, out = torch.empty_like(batch.q), torch.empty_like(batch.q)
        lse = torch.empty(2 * n, 8, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step.append(batch.q, k, v, q_out=qo)
            step.attend(qo, out=out, lse=lse)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step.append(batch.q, k, v, q_out=qo)
            step.attend(qo, out=out, lse=lse)
        for kv in ([300, 200], [222, 60 + n]):
            batch.kv_t.copy_(torch.tensor(kv))
            batch.q.copy_(torch.randn_like(batch.q))
            g.replay()
            torch.cuda.synchronize()
            batch.kv = kv
            batch.used = [-(-x // 16) for x in kv]
            check_attention(batch, out, lse)
        side.wait_stream(torch.cuda.current_stream())
        got = step.attend(qo, stream=side)
        side.synchronize()
        assert torch.equal(got, out) and step.error() == 0


def test_the_same_call_gives_the_same_bits():
    for n in (1, 90):
        batch = Batch([3000, 500], [n, n], 32, 8, 128, BF16, False, 16, seed=9)
        a, b = attend(batch), attend(batch)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_a_cache_past_two_gigabytes_of_elements():
    """Row offsets past 2^31 elements and 2^32 bytes."""
    n_pages, page, Hkv, D = 17000, 128, 8, 128      # 2.2e9 elements
    K = torch.zeros((n_pages, page, Hkv, D), dtype=BF16, device="cuda")
    V = torch.zeros_like(K)
    batch = Batch([400], [1], 32, Hkv, D, BF16, False, page, seed=1)
    old = batch.table[0, :4].clone()
    new = torch.tensor([16999, 3, 16500, 9000], device="cuda")
    K[new], V[new] = batch.K[old.long()], batch.V[old.long()]
    for n in (1, 100):
        batch = Batch([400], [n], 32, Hkv, D, BF16, False, page, seed=1)
        K[new], V[new] = batch.K[batch.table[0, :4].long()], batch.V[batch.table[0, :4].long()]
        batch.table[0, :4] = new.to(torch.int32)
        batch.K, batch.V, batch.n_pages = K, V, n_pages
        check_attention(batch, *attend(batch))
    step = batch.step()
    x = torch.randn(100, Hkv, D, device="cuda").to(BF16)
    step.append(None, x, x)
    R, _ = step.read(torch.tensor([0, 400], device="cuda"), 400)
    assert step.error() == 0 and torch.equal(R[300:], x)


def test_a_steps_own_outputs_are_per_stream_and_kept():
    batch = Batch([300, 20], [1, 1], 8, 2, 64, BF16, False, 16, seed=2)
    step = batch.step()
    first, lse = step.attend(batch.q, return_lse=True)
    want, want_lse = first.clone(), lse.clone()
    assert step.attend(batch.q) is first
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = step.attend(batch.q, stream=side)
    side.synchronize()
    assert other is not first and torch.equal(other, want)
    mine = torch.empty_like(want)
    assert step.attend(batch.q, out=mine) is mine and torch.equal(mine, want) and torch.equal(lse, want_lse)
