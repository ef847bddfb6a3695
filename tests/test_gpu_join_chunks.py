"""GPU parity of joined attention's chunk kernels at calls that are long enough for them: chunks of new tokens behind
prefixes, of plain and of differential heads."""
import pytest
import torch

import join_cases
import stochastic_sparse_decode_split_gb300 as santa
from join_reference import Shared, check_diff
from paged_reference import Batch, check_attention

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
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return 0.1 + 0.6 * torch.rand(batch.total_q, batch.H // 2, generator=gen, device="cuda")


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
