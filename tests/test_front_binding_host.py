"""Host side of the layer front's Python binding: what it keeps, what it
hands to the library and what it needs to load.  No GPU."""

from __future__ import annotations

import ctypes
import subprocess
import sys
import threading

import combine_ep_plan_amd as ep
from tests.test_abi_host import ROOT


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


NO_MARSHAL = """
import sys
import torch
sys.modules["combine_ep_plan_amd._marshal"] = None   # as where it is not built, or for another torch
import combine_ep_plan_amd as ep
ep.load_library()
assert ep.ep_status_string(0) == "EP_OK"
g = ep.Group(8, 1, 256, 2, 16, "ht")
assert g.recv_shape(16)[-1] == 256
x = torch.zeros(4, 64, dtype=torch.bfloat16)
try:
    ep.Buffer.quantize_int8(x)
except RuntimeError as e:
    print(e)
"""


def test_the_library_loads_without_the_marshalling_module():
    """Only the entry points that are marshalled in C++ need it, and they say so."""
    out = subprocess.run([sys.executable, "-c", NO_MARSHAL], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    assert "_marshal" in out.stdout and "python -m combine_ep_plan_amd.build" in out.stdout
