"""tests/_threads.py tells a call that is stuck and one that raises from one that ends."""

from __future__ import annotations

import threading

import pytest

from tests._threads import run_together


def test_a_stuck_thread_is_told():
    free = threading.Event()
    with pytest.raises(TimeoutError, match="1 of 2"):
        run_together([free.wait, lambda: None], timeout=0.2)
    free.set()


def test_what_a_thread_raises_is_raised():
    def bad():
        assert False, "this one"

    with pytest.raises(AssertionError, match="this one"):
        run_together([bad, lambda: None], timeout=5)


def test_all_ran():
    ran = []
    run_together([lambda i=i: ran.append(i) for i in range(3)], timeout=5)
    assert sorted(ran) == [0, 1, 2]
