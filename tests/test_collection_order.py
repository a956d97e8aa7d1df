"""The order that conftest.py gives the tests."""
import types

from tests import conftest


def test_the_wait_that_runs_out_on_purpose_comes_last():
    names = ["test_a", "test_bounded_wait_gives_up", "test_calls_at_once[False]", "test_no_wait_ran_out", "test_b"]
    items = [types.SimpleNamespace(name=n, keywords=(), add_marker=lambda m: None) for n in names]
    conftest.pytest_collection_modifyitems(None, items)
    assert [i.name for i in items] == [n for n in names if n != names[1]] + [names[1]]
