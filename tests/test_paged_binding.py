"""What the paged cache's binding refuses by itself, without a GPU."""
import pytest

from stochastic_sparse_decode_split_gb300 import paged


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
