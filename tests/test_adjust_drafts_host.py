"""Refusals of an adjustment's number of drafts. Needs no GPU."""
import pytest

from tests.test_tree_host import L, _adjust  # noqa: F401


@pytest.mark.parametrize("bad", [
    dict(num_drafts=-1), dict(num_drafts=15), dict(num_drafts=21), dict(num_drafts=18, draft_tokens=None),
    dict(num_rows=3, num_drafts=4), dict(num_rows=3, num_drafts=2, draft_tokens=None),
    dict(num_rows=-5, num_drafts=-5),
])
def test_refusals(L, bad):  # noqa: F811
    assert _adjust(L, **bad) == 1


def test_nothing_to_do(L):  # noqa: F811
    assert _adjust(L, num_rows=0, num_drafts=5) == 0
