"""Steps made with as little as the binding asks for, and steps at work at the same time."""
import threading

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


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B,n", [(3, 1), (2, 4), (3, 500)])
def test_full_tables_need_no_lengths(B, n, e4m3):
    """Without kv_lens, nk, total_q and offsets: every sequence has as many keys as its table holds and max_q new tokens."""
    kv, page = 2048, 64
    batch = Batch([kv] * B, [n] * B, 8, 4, 128, BF16, e4m3, page, seed=n)
    table = batch.table[:, :kv // page].contiguous()
    step = santa.PagedStep(batch.cache(), table, n_q_heads=8, max_q=n)
    out, lse = step.attend(batch.q, return_lse=True)
    check_attention(batch, out, lse)
    K, V = (x.view(B, kv, 4, 128) for x in step.read())
    for b in range(B):
        assert torch.equal(K[b], batch.rows(b, "K").to(BF16)) and torch.equal(V[b], batch.rows(b, "V").to(BF16))
    new = torch.randn(B * n, 4, 128, device="cuda").to(BF16)
    assert step.append(None, new, new) is None
    if not e4m3:
        assert torch.equal(step.read()[1].view(B, kv, 4, 128)[:, kv - n:], new.view(B, n, 4, 128))
    assert step.error() == 0


def test_steps_at_the_same_time():
    """Steps over one cache, each in a host thread and on a stream of its own, tokens beside chunks."""
    shapes = [([3000, 900], [1, 1]), ([3000, 900], [500, 400]), ([3000, 900], [700, 1]), ([3000, 900], [4, 4])]
    batches = [Batch(*s, 8, 4, 128, BF16, False, 16, seed=6) for s in shapes]
    steps = [b.step() for b in batches]
    good = [[x.clone() for x in s.attend(b.q, return_lse=True)] for s, b in zip(steps, batches)]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(len(steps))

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            start.wait()
            for _ in range(50):
                got = steps[i].attend(batches[i].q, return_lse=True)
                if not all(torch.equal(x, y) for x, y in zip(got, good[i])):
                    wrong.append(i)
            wrong.extend([i] * (steps[i].error(stream) != 0))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(steps))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
