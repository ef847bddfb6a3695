"""GPU parity of joined attention where a CTA has many blocks of one item, and maxima grow along them by more than the
2^8 that the chunk kernels let a sum's maximum fall behind."""
import pytest
import torch

import join_cases
import stochastic_sparse_decode_split_gb300 as santa
from join_reference import Shared, check_diff
from paged_reference import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    santa.library()


def made(case, dtype, e4m3, seed, **kw):
    c = case[0]
    if "prefix" in c:
        return Shared(c["prefix"], c["first"], c["kv"], c["n"], c["H"], c["Hkv"], c["D"], dtype, e4m3, c["page"], seed=seed,
                      pairs=c["diff"], **kw)
    return Batch(c["kv"], c["n"], c["H"], c["Hkv"], c["D"], dtype, e4m3, c["page"], seed=seed, **kw)


def grown(batch, factors, every=128):
    """The keys of every `every` positions times the next of `factors` (an e4m3 cache: their scales)."""
    for b in range(batch.B):
        shared = hasattr(batch, "full")
        pages = torch.tensor(batch.full[b] if shared else batch.table[b].tolist(), device=batch.K.device)
        from_ = batch.prefix[batch.group[b]] if shared and b != batch.first[batch.group[b]] else 0   # the first holds the prefix
        key = torch.arange(from_, batch.kv[b], device=batch.K.device)
        f = torch.tensor(factors, device=batch.K.device, dtype=torch.float32)[key // every % len(factors)]
        page, at = pages[key // batch.page].long(), key % batch.page
        if batch.e4m3:
            batch.ks[page, :, at] *= f[:, None]
        else:
            batch.K[page, at] = (batch.K[page, at].float() * f[:, None, None]).to(batch.K.dtype)
    return batch


# A row's largest score of 128 flat keys is about 2.6, 3.7 in powers of two, times the factor: steps of 3 are 11 powers.
STEPS = {
    "every block": [3 * (i + 1) for i in range(24)],
    "every other block": [3 * (i // 2 + 1) for i in range(48)],
    "every third block": [3 * (i // 3 + 1) for i in range(48)],
    "up and down": [1, 8, 2, 16, 4, 24, 8, 32],
}


@pytest.mark.parametrize("e4m3,dtype", [(False, torch.bfloat16), (False, torch.float16), (True, torch.bfloat16)])
@pytest.mark.parametrize("step", STEPS)
@pytest.mark.parametrize("case", range(len(join_cases.LONG_PIECES)))
def test_maxima_that_grow_from_block_to_block(case, step, e4m3, dtype):
    """Nearly every block asks for a rescaling of its rows' sums, in pieces of eight blocks and more."""
    batch = grown(made(join_cases.LONG_PIECES[case], dtype, e4m3, case + 3), STEPS[step])
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = 0.1 + 0.6 * torch.rand(batch.total_q, batch.H // 2, generator=gen, device="cuda")
    at = batch.shared_step(diff=True) if hasattr(batch, "full") else batch.step(diff=True)
    out, lse = at.attend_diff(batch.q, w, gain=0.8, return_lse=True)
    assert at.error() == 0
    check_diff(batch, out, lse, w, gain=0.8)
    again, lse_again = at.attend_diff(batch.q, w, gain=0.8, return_lse=True, out=torch.empty_like(out), lse=torch.empty_like(lse))
    assert torch.equal(out, again) and torch.equal(lse, lse_again)
