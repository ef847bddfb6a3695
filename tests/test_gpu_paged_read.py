"""The way back to packed rows at its corners."""
import pytest
import torch

import stochastic_sparse_decode_split_gb300 as santa
from paged_reference import Batch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    santa.library()


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_batch_of_empty_sequences_has_no_rows(e4m3):
    batch = Batch([0, 0, 0], [1, 1, 1], 4, 2, 64, BF16, e4m3, 16, seed=1)
    step = batch.step(nk=32)
    offsets = torch.zeros(4, dtype=torch.int64, device="cuda")
    K, V = step.read(offsets, 0)
    assert K.shape == V.shape == (0, 2, 64) and K.dtype == V.dtype == BF16 and step.error() == 0
    K, V = step.read(offsets, 0, K_out=torch.empty_like(K), V_out=torch.empty_like(V))
    assert K.shape == (0, 2, 64) and step.error() == 0
    batch.kv_t[1] = 1                      # a key, and no row for it
    step.read(offsets, 0)
    assert step.error() == santa.CACHE_DEVERR_CHUNK
