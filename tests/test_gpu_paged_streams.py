"""Calls of a step on streams other than the one that it was made on."""
import pytest
import torch

import stochastic_sparse_decode_split_gb300 as santa
from paged_reference import Batch

pytestmark = pytest.mark.gpu
BF16, F8 = torch.bfloat16, torch.float8_e4m3fn
BUSY = 200_000_000   # cycles: a tenth of a second


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    santa.library()


@pytest.mark.parametrize("explicit", [True, False])
@pytest.mark.parametrize("e4m3", [False, True])
def test_a_dropped_steps_memory_waits_for_its_calls(e4m3, explicit):
    """The step, its cache and its table are dropped while a busy side stream has yet to run their call: nobody else gets
    their memory before that."""
    batch = Batch([3000, 2000], [1, 1], 8, 2, 128, BF16, e4m3, 16, seed=1)
    good = batch.step().attend(batch.q).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step, q, out = batch.step(), batch.q, torch.zeros_like(good)
    torch.cuda.synchronize()
    held = [t for t in (step.workspace, step.page_table, step.kv_lens, step.q_offsets, *step._kept) if t is not None]
    sizes = [(t.untyped_storage().data_ptr(), t.untyped_storage().nbytes()) for t in held]
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
        if not explicit:
            step.attend(q, out=out)
    if explicit:
        step.attend(q, out=out, stream=side)
    del step, batch, held
    others = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in sizes for _ in range(4)]
    assert not side.query()   # the call has not run yet
    for x in others:
        assert all(x.data_ptr() + x.numel() <= at or at + n <= x.data_ptr() for at, n in sizes)
    side.synchronize()
    assert torch.equal(out, good)


def test_a_side_streams_first_call_comes_after_the_workspace_is_cleared():
    batch = Batch([3000, 2000], [1, 1], 8, 2, 128, BF16, False, 16, seed=1)
    step = batch.step()
    good = step.attend(batch.q).clone()
    side = torch.cuda.Stream()
    step.workspace.fill_(255)
    n = step.workspace.numel()
    torch.cuda.synchronize()
    del step
    torch.cuda._sleep(BUSY)
    step = batch.step()
    assert step.workspace.numel() == n
    out = step.attend(batch.q, stream=side)
    assert step.error(side) == 0
    assert torch.equal(out, good)


def test_a_captured_call_on_a_side_stream():
    batch = Batch([3000, 2000], [1, 1], 8, 2, 128, BF16, False, 16, seed=1)
    good = batch.step().attend(batch.q).clone()
    step, out = batch.step(), torch.zeros_like(good)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step.attend(batch.q, out=out)
    assert not bool(out.any())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, good) and step.error() == 0
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step.attend(batch.q, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, good)
