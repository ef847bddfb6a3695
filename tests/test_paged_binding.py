"""What the paged cache's binding refuses by itself, without a GPU."""
import ctypes

import pytest

import stochastic_sparse_decode_split_gb300 as santa
from stochastic_sparse_decode_split_gb300 import build, paged


def bare(batch=2, total_q=2, nk=100, window=0):
    """A step without a device: what its checks read."""
    step = paged.PagedStep.__new__(paged.PagedStep)
    step.p, step.batch, step.total_q, step.nk = paged.PagedParams(), batch, total_q, nk
    step.p.window = window
    return step


@pytest.mark.parametrize("kw,what", [(dict(window=5), "window"), (dict(window=99), "window"), (dict(total_q=3), "one token"),
                                     (dict(batch=1, total_q=2), "one token")])
def test_sampling_refuses_windows_and_chunks(kw, what):
    with pytest.raises(ValueError, match=what):
        bare(**kw).sample(None, 8, None, 100)


def test_a_bound_above_the_number_of_tokens_needs_the_workspace_of_the_tokens():
    """max_q bounds the tokens of a sequence where q_offsets say how many there are: it may be above all of them."""
    build.build()
    lib = santa.library()

    def size(**kw):
        p = paged.PagedParams()
        p.batch, p.n_q_heads, p.n_kv_heads, p.head_dim, p.dtype, p.cache_dtype = 2, 32, 8, 128, 0, 0
        p.page_size, p.n_pages, p.page_table, p.max_pages, p.kv_lens, p.nk = 16, 4096, 4096, 2048, 4096, 30000
        p.q_offsets, p.max_q, p.total_q, p.causal = 4096, 300, 300, 1
        for k, v in kw.items():
            setattr(p, k, v)
        return lib.santa_paged_workspace_size(ctypes.byref(p))

    assert size() > 0
    assert {size(max_q=m) for m in (301, 2048, 2 ** 31 - 1)} == {size()}
    assert size(total_q=5, max_q=2048) == size(total_q=5, max_q=5) > 0
    assert size(q_offsets=None) == size(q_offsets=None, max_q=301) == 0 < size(q_offsets=None, max_q=150)


def test_the_largest_number_of_tokens():
    """A CTA per multiprocessor holds the sums of two shared items of 256 rows, whatever the number of tokens; where the
    number of the tile behind the last one would pass 2^31 the batch is refused."""
    build.build()
    p = paged.PagedParams()
    p.batch, p.n_q_heads, p.n_kv_heads, p.head_dim, p.dtype, p.cache_dtype = 1, 1, 1, 64, 0, 0
    p.page_size, p.n_pages, p.page_table, p.max_pages, p.kv_lens, p.nk = 16, 4096, 4096, 2048, 4096, 30000
    p.causal = 1
    sizes = []
    for p.total_q in (1 << 20, (1 << 31) - 257, (1 << 31) - 256, (1 << 31) - 1):
        p.max_q = p.total_q
        sizes.append(santa.library().santa_paged_workspace_size(ctypes.byref(p)))
    assert sizes[0] == sizes[1] and 0 < sizes[0] < 1 << 27 and sizes[2:] == [0, 0]
