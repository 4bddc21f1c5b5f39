"""Host side of the layer front's Python binding: what it keeps, what it
hands to the library and what it needs to load.  No GPU."""

from __future__ import annotations

import ctypes
import sys
import threading

import combine_ep_plan_amd as ep


def test_norm_rules_are_one_object_whatever_thread_asks_first():
    """Threads that meet a norm's eps for the first time together all get the
    address of the one rule that is kept, and it holds that eps."""
    threads, n = 4, 20000
    eps = [1e-6 * (1 + i * 1e-7) for i in range(n)]
    got = [[0] * n for _ in range(threads)]
    start = threading.Barrier(threads)

    def ask(mine):
        start.wait()
        for i, e in enumerate(eps):
            mine[i] = ep._norm_rule(e, "int8")

    was = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        ts = [threading.Thread(target=ask, args=(g,)) for g in got]
        for t in ts:
            t.start()
        for t in ts:
            t.join()
    finally:
        sys.setswitchinterval(was)
    kept = [ctypes.addressof(ep._NORM_RULES[(e, "int8")]) for e in eps]
    for g in got:
        assert g == kept
    assert all(ep.ep_norm_rule_t.from_address(a).eps == e for a, e in zip(kept, eps))
