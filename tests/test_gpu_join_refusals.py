"""What attention over shared prefixes refuses on the device, with both kernels of each pass: zeros in the rows that it
concerns, the error word, the other rows as they should be."""
import pytest
import torch

import stochastic_sparse_decode_split_gb300 as santa
from join_reference import Shared

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    santa.library()


def attend(step, batch, diff):
    w = torch.full((batch.H // 2,), 0.3, device="cuda")
    call = (lambda **kw: step.attend_diff(batch.q, w, **kw)) if diff else (lambda **kw: step.attend(batch.q, **kw))
    out, lse = (x.clone() for x in call(return_lse=True))
    return out, lse


def gone(x, lse):
    return bool((x == 0).all()) and bool((lse == float("-inf")).all())


# few rows and chunks over the prefix, over what the sequences have of their own
SHAPES = [([1] * 4, [64]), ([4] * 4, [4000]), ([60] * 4, [4000]), ([330] * 4, [1200])]


@pytest.mark.parametrize("diff", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,prefix", SHAPES)
def test_tokens_that_are_not_among_their_groups(n, prefix, e4m3, diff):
    """Offsets that decrease further on: a sequence whose tokens stand behind the end of its group's."""
    k = n[0]
    batch = Shared(prefix, [0, 4], [k + 5 + 3 * b for b in range(4)], n, 16, 4, 128, BF16, e4m3, 16, seed=k, pad=96 * k, pairs=diff)
    step = batch.shared_step(diff=diff)
    want, want_lse = attend(step, batch, diff)
    assert step.error() == 0
    # sequence 1 has too many tokens, sequence 3 fewer than none; 2 is sound by itself, but the group ends at 2 k
    batch.offsets.copy_(torch.tensor([0, k, 95 * k, 96 * k, 2 * k]))
    out, lse = attend(step, batch, diff)
    assert step.error() == santa.CACHE_DEVERR_CHUNK | santa.CACHE_DEVERR_PREFIX
    assert gone(out[95 * k:96 * k], lse[95 * k:96 * k])
    torch.testing.assert_close(out[:k].float(), want[:k].float(), rtol=2.0 ** -6, atol=2.0 ** -6)
    torch.testing.assert_close(lse[:k], want_lse[:k], rtol=2.0 ** -16, atol=2.0 ** -10)


@pytest.mark.parametrize("diff", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,prefix", SHAPES)
def test_groups_that_overlap(n, prefix, e4m3, diff):
    """Offsets that decrease: two groups have the third sequence, and neither's rows are to be had; the last is apart."""
    k, P = n[0], prefix[0]
    batch = Shared([P] * 4, [0, 2, 2, 4, 6], [k + 5 + 3 * b for b in range(6)], [k] * 6, 16, 4, 128, BF16, e4m3, 16, seed=k,
                   pairs=diff, whole=True)
    step = batch.shared_step(diff=diff, max_group=3)
    want, want_lse = attend(step, batch, diff)
    assert step.error() == 0
    batch.first_t.copy_(torch.tensor([0, 3, 2, 4, 6], dtype=torch.int32))
    out, lse = attend(step, batch, diff)
    assert step.error() == santa.CACHE_DEVERR_PREFIX
    assert gone(out[:4 * k], lse[:4 * k])
    torch.testing.assert_close(out[4 * k:].float(), want[4 * k:].float(), rtol=2.0 ** -6, atol=2.0 ** -6)
    torch.testing.assert_close(lse[4 * k:], want_lse[4 * k:], rtol=2.0 ** -16, atol=2.0 ** -10)
