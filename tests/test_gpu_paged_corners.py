"""Calls at the corners of what the paged cache's documentation allows, on both attention kernels: scales of zero, the
output over the queries, a window that reaches past every key, odd values far apart in a long chunk, work that follows a
call whose merge has nothing to do, sizes that do not fit the C structure."""
import pytest
import torch

import stochastic_sparse_decode_split_gb300 as santa
from paged_reference import Batch, check_attention

pytestmark = pytest.mark.gpu
BF16, FP16, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
FEW, CHUNK = ([3000, 40], [2, 1], 8, 2, 128), ([3000, 900], [500, 400], 8, 4, 128)   # which kernel takes them


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    santa.library()


@pytest.mark.parametrize("shape", [FEW, CHUNK])
def test_values_under_a_scale_of_zero_count_in_the_softmax(shape):
    """Rows of zeros with a scale of zero, every third and then all: weights of a softmax whose values are zero."""
    for part in (3, 1):
        batch = Batch(*shape, BF16, True, 32, seed=4)
        batch.V.view(torch.uint8)[:, ::part] = 0
        batch.vs[:, :, ::part] = 0.0
        step = batch.step()
        out, lse = step.attend(batch.q, return_lse=True)
        assert step.error() == 0
        check_attention(batch, out, lse)
        assert part == 3 or not bool(out.any())


@pytest.mark.parametrize("odd", [-1.0, float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("shape", [FEW, CHUNK])
def test_a_v_scale_that_is_none_leaves_the_softmax_alone(shape, odd):
    batch = Batch(*shape, BF16, True, 32, seed=4)
    good, good_lse = (x.clone() for x in batch.step().attend(batch.q, return_lse=True))
    batch.vs[int(batch.table[0, 7 // 32]), 0, 7 % 32] = odd      # key 7 of sequence 0, KV head 0: all its tokens see it
    step = batch.step()
    out, lse = step.attend(batch.q, return_lse=True)
    n, G = shape[1][0], shape[2] // shape[3]
    assert bool(out[:n, :G].isnan().all())
    assert torch.equal(out[:n, G:], good[:n, G:]) and torch.equal(out[n:batch.tokens], good[n:batch.tokens])
    # the key's own weight enters the sum divided by another scale: rounding apart, the same
    assert float((lse[:batch.tokens] - good_lse[:batch.tokens]).abs().max()) <= 2.0 ** -16


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("shape", [FEW, CHUNK])
def test_the_output_may_be_the_queries(shape, e4m3):
    batch = Batch(*shape, BF16, e4m3, 16, seed=6)
    step = batch.step()
    good = step.attend(batch.q).clone()
    q = batch.q.clone()
    assert step.attend(q, out=q) is q and torch.equal(q, good) and step.error() == 0


@pytest.mark.parametrize("shape", [FEW, CHUNK])
def test_a_window_past_every_key_is_none(shape):
    batch = Batch(*shape, FP16, False, 16, seed=7)
    good = batch.step().attend(batch.q)
    for window in (3000, 3001, (1 << 31) - 1):
        assert torch.equal(batch.step(window=window).attend(batch.q), good)


@pytest.mark.parametrize("e4m3", [False, True])
def test_odd_values_all_over_a_long_chunk(e4m3):
    """A NaN and an infinity in many blocks, the first and the last key among them; rows see those up to their own."""
    batch = Batch([9000], [700], 4, 2, 64, BF16, e4m3, 64, seed=8)
    for i, key in enumerate([0, 31, 32, 4095, 8300, 8301, 8600, 8999]):
        at, slot = int(batch.table[0, key // 64]), key % 64
        if e4m3:
            batch.V.view(torch.uint8)[at, slot, 1, 5 + 7 * i] = 0x7F
        else:
            batch.V[at, slot, 1, 5 + 7 * i] = float("nan") if i % 2 else float("inf")
    step = batch.step()
    out, lse = step.attend(batch.q, return_lse=True)
    assert step.error() == 0
    check_attention(batch, out, lse)


def test_what_follows_a_call_without_anything_to_merge_sees_its_output():
    """Bounds that allow many splits, sequences too short for any: the merge ends at once, and nothing overtakes the call."""
    batch = Batch([90] * 256, [4] * 256, 8, 2, 128, BF16, False, 16, seed=9)
    table = torch.nn.functional.pad(batch.table, (0, 2048), value=-1).contiguous()
    step = santa.PagedStep(batch.cache(), table, batch.kv_t, n_q_heads=8, nk=32768, max_q=4, total_q=batch.total_q,
                           q_offsets=batch.offsets)
    good = step.attend(batch.q).clone()
    check = batch.step()
    torch.cuda.synchronize()
    assert torch.equal(check.attend(batch.q), good)
    out = torch.empty_like(good)
    for _ in range(50):
        out.zero_()
        step.attend(batch.q, out=out)
        assert torch.equal(out, good)


def test_an_e4m3_pool_is_made_in_place_and_reads_as_zeros():
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    cache = santa.PagedCache(4096, 64, 8, 128, F8)
    held = 2 * 4096 * 64 * 8 * (128 + 4)
    assert torch.cuda.max_memory_allocated() - before <= held + (1 << 20)
    assert cache.K.dtype == F8 and not bool(cache.K.view(torch.uint8).any()) and not bool(cache.V.view(torch.uint8).any())


def test_numbers_that_the_structure_cannot_hold_are_refused():
    cache = santa.PagedCache(8, 16, 2, 64)
    table = torch.zeros(1, 8, dtype=torch.int32, device="cuda")
    for kw in (dict(window=(1 << 32) + 5), dict(max_q=(1 << 32) + 1, total_q=1), dict(nk=(1 << 40) + 64), dict(n_q_heads=(1 << 32) + 4),
               dict(total_q=-1), dict(window=-1)):
        with pytest.raises(ValueError):
            santa.PagedStep(cache, table, **{"n_q_heads": 4, **kw})


def test_nothing_but_odd_values_in_a_long_chunk():
    """65536 keys of NaN codes per item and fewer CTAs than items: giving them back stays far below the bound of the
    kernel's waits, and the softmax's sums are those of the keys."""
    B, kv = 320, 65536
    batch = Batch([kv], [129], 1, 1, 64, BF16, True, 256, seed=10)
    batch.V.view(torch.uint8).fill_(0x7F)
    step = santa.PagedStep(batch.cache(), batch.table.expand(B, -1).contiguous(), batch.kv_t.expand(B).contiguous(), n_q_heads=1,
                           dtype=BF16, nk=kv, max_q=129)
    one, one_lse = (x.clone() for x in batch.step().attend(batch.q, return_lse=True))
    out, lse = step.attend(batch.q.repeat(B, 1, 1), return_lse=True)
    assert step.error() == 0 and bool(out.isnan().all()) and bool(one.isnan().all())
    # shared items and whole ones sum in another order
    assert float((lse.view(B, 129, 1) - one_lse).abs().max()) <= 2.0 ** -14


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kv,n,H,Hkv,D,dtype,page", [
    ([700] * 150, [20] * 150, 4, 2, 128, BF16, 16), ([300] * 500, [17] * 500, 2, 2, 64, FP16, 16),
    ([300] * 200, [5] * 199 + [17], 8, 2, 128, FP16, 32), ([2500] * 9, [3] * 8 + [70], 8, 1, 64, BF16, 64)])
def test_many_small_chunks(kv, n, H, Hkv, D, dtype, page, e4m3):
    """More items than CTAs, most of one tile of few rows: past the border between the kernels (3 * 2^13 blocks of 16 rows
    by 16 keys)."""
    batch = Batch(kv, n, H, Hkv, D, dtype, e4m3, page, seed=len(kv))
    assert -(-max(n) * (H // Hkv) // 16) * len(kv) * Hkv * max(kv) > 3 * 2 ** 17
    step = batch.step()
    out, lse = step.attend(batch.q, return_lse=True)
    assert step.error() == 0
    check_attention(batch, out, lse)


@pytest.mark.parametrize("nk", [4095, 4096, 4097])
@pytest.mark.parametrize("n", [12, 13])
def test_both_sides_of_the_border_between_the_kernels(n, nk):
    batch = Batch([nk, 4000, 900, 17, 4095, 33, 2048, 16], [n] * 8, 16, 2, 64, BF16, False, 32, seed=n)
    step = batch.step(nk=nk)
    out, lse = step.attend(batch.q, return_lse=True)
    assert step.error() == 0
    check_attention(batch, out, lse)


def test_a_captured_reads_outputs_outlive_a_read_of_other_sizes():
    """The graph writes to the buffers that the step had when it was captured: a read of more rows on that stream makes new
    ones, and the old ones must not go to anybody else."""
    batch = Batch([500, 300], [1, 1], 4, 2, 64, BF16, False, 16, seed=11)
    step = batch.step()
    offsets = torch.tensor([0, 500, 800], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step.read(offsets, 800)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            K, V = step.read(offsets, 800)
        at = (K.data_ptr(), V.data_ptr())
        del K, V
        good = [x.clone() for x in step.read(offsets, 900)]
        others = [torch.full((800, 2, 64), 3.0, dtype=BF16, device="cuda") for _ in range(8)]
        assert not any(x.data_ptr() in at for x in others)
        graph.replay()
        side.synchronize()
        assert all(bool((x == 3.0).all()) for x in others)
    assert torch.equal(good[0][:500].double(), batch.rows(0, "K")) and torch.equal(good[1][500:800].double(), batch.rows(1, "V"))
