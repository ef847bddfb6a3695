"""Attention in which one key outweighs each of very many others, and the others together still count."""
import math

import pytest
import torch

import stochastic_sparse_decode_split_gb300 as santa
from paged_reference import Batch, attention

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    santa.library()


@pytest.mark.parametrize("dtype,e4m3", [(FP16, False), (BF16, True), (FP16, True), (BF16, False)])
@pytest.mark.parametrize("gap", [12.0, 22.3, 25.5, 30.0])
@pytest.mark.parametrize("n,bits", [(1, 40), (4, 40), (6, 32), (64, 32)])
@pytest.mark.parametrize("every", [1 << 17, 48])
def test_many_small_weights_beside_a_large_one(every, n, bits, gap, dtype, e4m3):
    """Key 0, or every 48th, outweighs each of the others by 2^gap and has the value zero; the others have one value per
    column.

    Beside what the reference's tolerance counts, a probability in fp16 may be off by 2^-25 where the largest one is held
    as 2^15 (few rows) or at least 2^7 (chunks): by 2^-40 or 2^-32 of it for each key, over a sum that is at least the
    number of large ones.  Six tokens are chunks: 24 rows in 2 tiles of 16, for 2 KV heads of 2^17 keys, more than the
    3 * 2^17 up to which the other kernel has them."""
    kv, D = 1 << 17, 64
    batch = Batch([kv], [n], 8, 2, D, dtype, e4m3, 256, seed=1, planted=False)
    batch.q.fill_(1.0)
    key = torch.arange(0, kv, every, device="cuda")
    at, slot = batch.table[0, key // 256].long(), key % 256
    score = gap * math.log(2) / math.sqrt(D)   # of each element of a large key
    column = 1024.0 + 256 * (torch.arange(D, device="cuda") % 4)
    if e4m3:
        batch.K.view(torch.uint8).zero_()
        batch.K.view(torch.uint8)[at, slot] = 0x7E   # 448
        batch.ks[at, :, slot] = score / 448
        batch.V.copy_((column / 256).to(batch.V.dtype).expand(batch.V.shape))
        batch.vs.fill_(256.0)
        batch.V.view(torch.uint8)[at, slot] = 0
    else:
        batch.K.zero_()
        batch.K[at, slot] = score
        batch.V.copy_(column.to(dtype).expand(batch.V.shape))
        batch.V[at, slot] = 0
    step = batch.step()
    out, lse = step.attend(batch.q, return_lse=True)
    assert step.error() == 0
    want, want_lse, tol, tol_lse = attention(batch)
    rounding = 0.0 if dtype == BF16 and not e4m3 else kv * 2.0 ** -bits * float(column.max()) / len(key)
    assert bool(((out.double() - want).abs() <= tol + rounding).all())
    assert bool(((lse.double() - want_lse).abs() <= tol_lse).all())
