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


@pytest.mark.parametrize("sampled", [True, False])
def test_packed_copies_of_long_contexts_are_not_kept(sampled):
    batch = Batch([9000], [1], 8, 8, 128, BF16, False, 64, seed=2)
    step = batch.step()
    offsets = torch.tensor([0, 9000], device="cuda")

    def run():
        return step.sample(batch.q, 8, offsets, 9000) if sampled else step.read(offsets, 9000)

    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated()
    first = run()
    if not sampled:
        want = [batch.rows(0, "K"), batch.rows(0, "V")]
        second = run()
        assert not {x.data_ptr() for x in first} & {x.data_ptr() for x in second}
        assert all(torch.equal(x.double(), w) and torch.equal(y.double(), w) for x, y, w in zip(first, second, want))
        del second, want
    del first
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() - held < 1 << 20


def test_a_captured_read_of_a_long_context_keeps_its_outputs():
    batch = Batch([9000], [1], 8, 8, 128, BF16, False, 64, seed=2)
    step = batch.step()
    offsets = torch.tensor([0, 9000], device="cuda")
    step.read(offsets, 9000)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        K, V = step.read(offsets, 9000)
    at = (K.data_ptr(), V.data_ptr())
    del K, V
    others = [torch.full((9000, 8, 128), 3.0, dtype=BF16, device="cuda") for _ in range(6)]
    assert not any(x.data_ptr() in at for x in others)
    graph.replay()
    torch.cuda.synchronize()
    assert all(bool((x == 3.0).all()) for x in others) and step.error() == 0
    assert torch.equal(step._captured[0][0].double(), batch.rows(0, "K"))


def test_a_read_captured_on_a_stream_that_is_not_the_current_one():
    """As on the current one: the buffers that the graph writes to stay, though the step makes others."""
    batch = Batch([500, 300], [1, 1], 4, 2, 64, BF16, False, 16, seed=11)
    step = batch.step()
    offsets = torch.tensor([0, 500, 800], device="cuda")
    side, other, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    at = {x.data_ptr() for x in step.read(offsets, 800, stream=side)}
    with torch.cuda.graph(graph, stream=side):
        with torch.cuda.stream(other):
            assert {x.data_ptr() for x in step.read(offsets, 800, stream=side)} == at
    with torch.cuda.stream(side):
        step.read(offsets, 900)
        others = [torch.full((800, 2, 64), 3.0, dtype=BF16, device="cuda") for _ in range(8)]
        assert not {x.data_ptr() for x in others} & at
        graph.replay()
        side.synchronize()
    assert all(bool((x == 3.0).all()) for x in others) and step.error() == 0


def test_a_cache_in_fp32_is_sampled_from():
    batch = Batch([300, 90], [1, 1], 4, 2, 64, torch.float32, False, 16, seed=4)
    step = batch.step()
    offsets = torch.tensor([0, 300, 390], device="cuda")
    idx, idx2 = (torch.full((2, 4, 32), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    out = step.sample(batch.q, 32, offsets, 390, seed=7, sample_idx=idx)
    K, V = (torch.cat([batch.rows(b, x) for b in range(2)]).float() for x in "KV")
    want = santa.santa_decode(batch.q, K, V, 32, seed=7, nk=300, kv_offsets=offsets, sample_idx=idx2)
    assert step.error() == 0 and torch.equal(idx, idx2)
    torch.testing.assert_close(out, want, rtol=1e-5, atol=1e-6)
    with pytest.raises(santa.SantaError):
        step.attend(batch.q)


def test_captures_of_a_long_contexts_read_share_their_outputs():
    batch = Batch([9000], [1], 8, 8, 128, BF16, False, 64, seed=2)
    step = batch.step()
    offsets = torch.tensor([0, 9000], device="cuda")
    step.read(offsets, 9000)
    side, graphs, at = torch.cuda.Stream(), [], set()
    for _ in range(3):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            for _ in range(2):
                K, V = step.read(offsets, 9000)
                at.add((K.data_ptr(), V.data_ptr()))
    assert len(at) == 1 and len(step._captured) == 1
    for graph in graphs:
        K.zero_()
        graph.replay()
        assert torch.equal(K.double(), batch.rows(0, "K")) and torch.equal(V.double(), batch.rows(0, "V"))
