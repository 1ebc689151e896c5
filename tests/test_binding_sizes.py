"""Workspace sizes that the binding keeps: an answer of 0 (no device state yet, for one because device
memory was full at that moment) is not kept, so that the same call works once the cause has gone."""
import pytest

import exact_long_sequence_gb300 as ela


class Library:
    def __init__(self, answers):
        self.answers = list(answers)

    def __getattr__(self, name):
        assert name.endswith("_bytes")
        return lambda *shape: self.answers.pop(0)


@pytest.mark.parametrize("query,args", [("_prefix_workspace_bytes", (0, 3, 8, 2, 1, 100, 20, 64)), ("_bwd_workspace_bytes", (0, 64))])
def test_a_size_is_kept_and_a_failure_is_not(monkeypatch, query, args):
    ask = getattr(ela, query)
    lib = Library([0, 0, 4096])
    monkeypatch.setattr(ela, "load_library", lambda path=None: lib)
    ask.cache_clear()
    assert [ela._size(ask, *args) for _ in range(5)] == [0, 0, 4096, 4096, 4096] and not lib.answers
    ask.cache_clear()
