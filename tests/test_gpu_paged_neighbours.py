"""A token's output depends on its own query and keys only: to the last bit, whatever other tokens, padding, or memory that
belongs to nobody hold."""
import pytest
import torch

import stochastic_sparse_decode_split_gb300 as santa
from paged_reference import Batch

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    santa.library()


SHAPES = [   # kv, new tokens, H, Hkv, D, type: few rows, then chunks whose last tiles are not full
    ([3000, 40], [2, 1], 8, 2, 128, BF16), ([3000, 900], [500, 400], 8, 4, 128, BF16),
    ([2500, 2000, 77], [333, 270, 5], 14, 2, 128, FP16), ([4000, 4000], [700, 699], 6, 2, 64, BF16),
    ([30000, 2000], [40, 20], 10, 2, 64, FP16),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kv,n,H,Hkv,D,dtype", SHAPES)
def test_other_tokens_leave_every_bit(kv, n, H, Hkv, D, dtype, e4m3):
    batch = Batch(kv, n, H, Hkv, D, dtype, e4m3, 32, seed=5, pad=64)
    step = batch.step()
    good, good_lse = (x.clone() for x in step.attend(batch.q, return_lse=True))
    q = batch.q.clone()
    first = 0
    for b in range(batch.B + 1):      # one sequence's queries kept, all others and the padding grown, in turn
        last = first + n[b] if b < batch.B else batch.tokens
        if b < batch.B:
            for factor in (0.0, 30.0, 500.0):
                batch.q.copy_(q * factor)
                batch.q[first:last] = q[first:last]
                out, lse = step.attend(batch.q, return_lse=True)
                assert torch.equal(out[first:last], good[first:last]) and torch.equal(lse[first:last], good_lse[first:last])
        first = last
    assert step.error() == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_what_an_earlier_call_left_behind_leaves_every_bit(e4m3):
    """Groups of 7 heads leave rows of a tile that no query fills: they hold what the call before had there."""
    batch = Batch([2500, 2000], [333, 270], 14, 2, 128, FP16, e4m3, 32, seed=5)
    before = Batch([3000], [900], 8, 2, 128, FP16, e4m3, 32, seed=6)
    step, other = batch.step(), before.step()
    results = []
    for factor in (0.0, 1.0, 100.0, 1000.0):
        other.attend(before.q * factor)
        results.append([x.clone() for x in step.attend(batch.q, return_lse=True)])
    assert all(torch.equal(x, y) for r in results[1:] for x, y in zip(r, results[0]))
