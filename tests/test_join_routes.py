"""Tests that are meant for one of the kernels of joined attention: the library's plans send their calls there, on the
host."""
import pytest

import join_cases
from join_routes import route


def check(cases):
    for case in cases:
        for e4m3 in (False, True):
            assert route(e4m3=e4m3, **case[0]) == join_cases.kernels(case, e4m3), (case, e4m3)
            if len(case) > 2:
                assert join_cases.blocks_per_cta(case, e4m3) >= case[2], (case, e4m3)


def test_calls_of_long_pieces():
    check(join_cases.LONG_PIECES)


def test_calls_of_chunks_behind_prefixes():
    check(join_cases.OWN_CHUNKS)


def test_calls_of_every_form_of_the_chunk_kernels():
    check(join_cases.FORMS + join_cases.WINDOWS + join_cases.UNMASKED + join_cases.NOTHING_SEEN)


@pytest.mark.parametrize("n,kernel", [(16, "tokens"), (1200, "chunk")])
def test_the_plain_attention_has_its_own(n, kernel):
    assert route([4000], [n], 8, 2, 128) == [kernel]
