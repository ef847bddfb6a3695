"""What the device refuses of a batch is reported also where no token comes by it."""
import pytest
import torch

import stochastic_sparse_decode_split_gb300 as santa
from paged_reference import Batch, check_attention

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    santa.library()


def append(batch, step):
    """The rows of the pool that a write changes, and the error bits."""
    batch.K.zero_()
    k = torch.ones(batch.total_q, batch.Hkv, batch.D, dtype=BF16, device="cuda")
    step.append(None, k, k)
    return int(batch.K.any(-1).any(-1).sum()), step.error()


def test_decreasing_offsets_that_no_token_finds():
    batch = Batch([40, 30, 20], [2, 0, 1], 2, 2, 64, BF16, False, 16, seed=1)
    step = batch.step()
    assert append(batch, step) == (3, 0)
    batch.offsets.copy_(torch.tensor([0, 2, 1, 3]))   # sequence 1 decreases; 0 and 2 are fine by themselves
    assert append(batch, step)[1] == santa.CACHE_DEVERR_CHUNK
    step.attend(batch.q)
    assert step.error() == santa.CACHE_DEVERR_CHUNK


@pytest.mark.parametrize("B,bad", [(3, 1), (300, 299), (300, 128)])
def test_a_length_out_of_bounds_of_a_sequence_without_tokens(B, bad):
    n = [1] * B
    n[bad] = 0
    batch = Batch([20] * B, n, 2, 2, 64, BF16, False, 16, seed=1)
    step = batch.step()
    assert append(batch, step) == (B - 1, 0)
    for length in (-1, 21):
        batch.kv_t[bad] = length
        assert append(batch, step) == (B - 1, santa.DEVERR_NK_BOUND)
        step.attend(batch.q)
        assert step.error() == santa.DEVERR_NK_BOUND


def test_more_tokens_than_keys_of_the_last_of_many():
    batch = Batch([20] * 200, [2] * 200, 2, 2, 64, BF16, False, 16, seed=1, pad=3)
    step = batch.step()
    assert append(batch, step) == (400, 0)
    batch.kv_t[199] = 1
    assert append(batch, step) == (398, santa.CACHE_DEVERR_CHUNK)


def test_sampling_refuses_what_it_would_answer_otherwise_than_the_attention():
    batch = Batch([40, 30], [1, 1], 2, 2, 64, BF16, False, 16, seed=1)
    offsets = torch.tensor([0, 40, 70], device="cuda")
    for window in (1, 39):
        with pytest.raises(ValueError, match="window"):
            batch.step(window=window).sample(batch.q, 8, offsets, 70)
    wide = batch.step(window=40).sample(batch.q, 8, offsets, 70, seed=3)   # no key is outside of it
    assert torch.equal(wide, batch.step().sample(batch.q, 8, offsets, 70, seed=3))
    two = Batch([40, 30], [2, 2], 2, 2, 64, BF16, False, 16, seed=1)
    with pytest.raises(ValueError, match="one token"):
        two.step().sample(two.q[:2], 8, offsets, 70)


@pytest.mark.parametrize("n", [3, 150])
def test_a_bound_above_the_number_of_tokens_is_none(n):
    batch = Batch([3000, 2000], [n, 0], 8, 4, 64, BF16, False, 16, seed=1)
    step = santa.PagedStep(batch.cache(), batch.table, batch.kv_t, n_q_heads=8, nk=3000, max_q=4096, total_q=n,
                           q_offsets=batch.offsets)
    out, lse = step.attend(batch.q, return_lse=True)
    assert step.error() == 0
    check_attention(batch, out, lse)
    k = torch.ones(n, 4, 64, dtype=BF16, device="cuda")
    step.append(None, k, k)
    K, _ = step.read(torch.tensor([0, 3000, 5000], device="cuda"), 5000)
    assert step.error() == 0 and bool((K[3000 - n:3000] == 1).all())
