"""Passes over shared prefixes in which nothing is left to divide: every group refused, or without tokens."""
from test_join_shares import call, walk   # noqa: F401 (a fixture)


def test_calls_whose_groups_are_all_refused(walk):   # noqa: F811
    good = call([10, 20, 30], [1, 2, 3], [100, 50], [0, 2, 3])
    for c in (dict(good, prefix=[-1, -1], max_prefix=100, max_own=200), dict(good, first=[3, 3, 3], max_group=1),
              dict(good, prefix=[200, 200], max_prefix=100, max_own=200)):
        first, second = walk([c])[0]
        assert first == (0, 0, 0, 0, 0), c
        assert second[1:] == (0, 0, 0, 3), c


def test_groups_without_tokens(walk):   # noqa: F811
    first, second = walk([call([10, 20, 30], [0, 0, 0], [100, 50], [0, 2, 3], max_group=1)])[0]
    assert first == second == (0, 0, 0, 0, 0)
