"""Host-side checks of the layer front's entry points at their edges: views
that are not what they say, and launches at the limit of 32-bit thread counts.
Every call is refused before anything would be enqueued, so no GPU is needed."""

from __future__ import annotations

import ctypes
import subprocess
import sys

import pytest

import combine_ep_plan_amd as ep
from tests.test_abi_front_host import (BF16, FP32, NW, OK, SHAPE, T_, TAG, UNSUPPORTED, WS, handle,  # noqa: F401
                                       lib, norm_rule, view)
from tests.test_abi_host import ROOT

# an ep_tensor_t whose four sizes end where readable memory ends
GUARDED = """
import ctypes, mmap, sys
import combine_ep_plan_amd as ep
lib, libc = ep.load_library(), ctypes.CDLL(None, use_errno=True)
m = mmap.mmap(-1, 2 * mmap.PAGESIZE)
base = ctypes.addressof(ctypes.c_char.from_buffer(m))
assert libc.mprotect(ctypes.c_void_p(base + mmap.PAGESIZE), mmap.PAGESIZE, 0) == 0
def view(dtype, tag, ndim, *sizes, at=None):
    t = ep.ep_tensor_t(0x7F0000000000, dtype, tag, ndim, 0, (ctypes.c_int64 * 4)(*sizes))
    if at is not None:
        ctypes.memmove(at, ctypes.byref(t), ctypes.sizeof(t))
        return ctypes.cast(at, ctypes.POINTER(ep.ep_tensor_t))
    return ctypes.pointer(t)
edge = base + mmap.PAGESIZE - ctypes.sizeof(ep.ep_tensor_t)
rule = ctypes.pointer(ep.ep_norm_rule_t(1e-6, 0, 0))
ok, w = view(0, ep.TAG_TOKENS, 2, 4, 256), view(0, ep.TAG_NORM_WEIGHT, 1, 256)
for ndim in (5, 64, -1, 0):
    bad = view(0, ep.TAG_TOKENS, ndim, 1, 1, 4, 256, at=edge)
    print(lib.ep_add_rmsnorm_bwd(rule, bad, w, ok, None, ok, None, None, None),
          lib.ep_add_rmsnorm(rule, bad, None, w, None, ok, None, None, None))
"""


def test_views_of_a_wrong_rank_are_refused_unread():
    """More sizes than a view has room for: refused by the rank alone."""
    out = subprocess.run([sys.executable, "-c", GUARDED], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, (out.returncode, out.stderr[-2000:])
    assert out.stdout.split() == [str(SHAPE)] * 8


def test_norm_bwd_checks_hidden_like_the_other_tensors(lib):  # noqa: F811
    """Tag before shape, as at every other entry point."""
    h, w = view(BF16, T_, 4, 256), view(BF16, NW, 256)
    f = lib.ep_add_rmsnorm_bwd
    assert f(norm_rule(), view(BF16, WS, 256), w, h, None, h, None, None, None) == TAG
    assert f(norm_rule(), view(BF16, T_, 256), w, h, None, h, None, None, None) == SHAPE
    assert f(norm_rule(), view(BF16, T_, 4, 252), w, h, None, h, None, None, None) == SHAPE
    assert f(norm_rule(), view(BF16, T_, -4, 256), w, h, None, h, None, None, None) == SHAPE


def _route_handle(lib, T, E):  # noqa: F811
    """A handle of T tokens on memory that is never touched."""
    from tests.test_abi_host import FAKE, create
    rc, g = create(lib, num_experts=E, num_ranks=1, hidden=64, max_tokens=T)
    assert rc == OK
    h = ctypes.c_void_p()
    assert lib.ep_handle_create(g, T, FAKE, 1 << 40, ctypes.byref(h)) == OK
    return h


@pytest.mark.parametrize("T", [(1 << 26) - 3, (1 << 26) - 1])
def test_route_counts_the_threads_it_launches(lib, T):  # noqa: F811
    """More than 256 experts: a wave a token, four to a workgroup; 2^24
    workgroups of 256 threads are past 32 bits."""
    E = 257
    h = _route_handle(lib, T, E)
    rule = ep.RouteRule().ptr
    lg, i, w = view(FP32, ep.TAG_ROUTER_LOGITS, T, E), view(3, ep.TAG_TOPK_IDX, T, 2), view(FP32, ep.TAG_TOPK_WEIGHTS, T, 2)
    assert lib.ep_route_scored(h, rule, lg, None, i, w, None, None) == UNSUPPORTED
    assert lib.ep_route_scored_bwd(h, rule, lg, i, w, None, lg, None) == UNSUPPORTED
