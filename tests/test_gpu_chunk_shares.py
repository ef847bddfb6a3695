"""The chunk attention where one block more or less per CTA decides whether items are shared: every row is written, and
from sums of this call."""
import pytest
import torch

import stochastic_sparse_decode_split_gb300 as santa
from paged_reference import Batch, check_attention
from test_chunk_shares import BORDER

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    santa.library()


def check(batch, **kw):
    """The call goes to the chunk kernel; outputs and the workspace's sums hold NaN beforehand."""
    tiles = -(-max(batch.n) * (batch.H // batch.Hkv) // 16)
    window = kw.get("window", 0)
    span = min(max(batch.kv), window + max(batch.n)) if window else max(batch.kv)
    assert tiles > 1 and tiles * batch.B * batch.Hkv * span > 3 * 2 ** 17
    step = batch.step(**kw)
    out = torch.full_like(batch.q, float("nan"))
    lse = torch.full(batch.q.shape[:2], float("nan"), device="cuda")
    step.workspace[256:].fill_(255)
    step.attend(batch.q, out=out, lse=lse)
    assert step.error() == 0
    check_attention(batch, out, lse, **kw)


@pytest.mark.parametrize("dtype,e4m3,D", [(torch.bfloat16, False, 128), (torch.bfloat16, True, 128), (torch.float16, False, 64)])
@pytest.mark.parametrize("kv,n,H,Hkv,causal,window", BORDER)
def test_calls_at_the_border_of_sharing(kv, n, H, Hkv, causal, window, dtype, e4m3, D):
    check(Batch(kv, n, H, Hkv, D, dtype, e4m3, 64, seed=kv[0]), causal=causal)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kv", range(1920, 2945, 128))
def test_across_the_border_of_sharing(kv, e4m3):
    check(Batch([kv], [700], 16, 4, 64, torch.bfloat16, e4m3, 128, seed=kv))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kv,n,H,Hkv,D,dtype,page", [
    ([700] * 100, [20] * 100, 4, 2, 128, torch.bfloat16, 16), ([300] * 330, [17] * 330, 4, 2, 64, torch.float16, 16),
    ([1300], [700], 8, 2, 128, torch.bfloat16, 16), ([1290, 700, 310], [300, 640, 300], 8, 4, 64, torch.float16, 32),
    ([1111], [640], 14, 2, 128, torch.float16, 64), ([640, 900], [640, 700], 6, 2, 128, torch.bfloat16, 128),
    ([2000], [200], 32, 8, 128, torch.bfloat16, 256), ([1600, 1600], [560, 515], 5, 1, 64, torch.bfloat16, 16),
    ([4100], [1200], 10, 2, 64, torch.bfloat16, 16), ([9000], [90], 8, 1, 128, torch.bfloat16, 64)])
def test_small_chunks(kv, n, H, Hkv, D, dtype, page, e4m3):
    check(Batch(kv, n, H, Hkv, D, dtype, e4m3, page, seed=len(kv) + kv[0]))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H,Hkv,D", [(16, 8, 128), (16, 16, 64)])
def test_pieces_of_every_kind_follow_each_other(H, Hkv, D, e4m3):
    """Items of two tiles, of one tile and several blocks (both softmax groups' sums are joined), of one tile and one block
    (the second group has no part), and of none, in every order on a CTA: no wait may take one piece's end for another's."""
    kinds = [(300, 90), (20, 20), (260, 30), (128, 128), (500, 200), (127, 3), (0, 2), (40, 40), (250, 250), (90, 1)]
    order = [kinds[i * j % 11 - 1] for j in range(1, 11) for i in range(1, 11)]
    batch = Batch([kv for kv, _ in order], [n for _, n in order], H, Hkv, D, torch.bfloat16, e4m3, 16, seed=H)
    check(batch)
    step = batch.step()
    good = [x.clone() for x in step.attend(batch.q, return_lse=True)]
    for _ in range(100):
        out, lse = step.attend(batch.q, return_lse=True)
    assert step.error() == 0
    assert torch.equal(out, good[0]) and torch.equal(lse, good[1])
