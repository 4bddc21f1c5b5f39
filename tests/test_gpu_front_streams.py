"""The layer front's calls on a stream given by its object or by its address."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import combine_ep_plan_amd as ep
from tests.gpu_util import dev_f32, dev_i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ep.load_library()


@pytest.mark.parametrize("raw", [False, True])
def test_dispatches_return_an_event_of_their_stream(raw):
    """The event of a dispatch on another stream is behind its rows."""
    T, H, E, k = 64, 256, 8, 2
    rng = np.random.default_rng(3)
    group = ep.Group(E, 1, H, k, T, "ht")
    b, h = ep.Buffer(group), ep.Handle(group, T)
    idx, w = dev_i32(rng.integers(0, E, (T, k))), dev_f32(rng.random((T, k)))
    h.plan(idx)
    x = torch.from_numpy(rng.normal(size=(T, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    codes, scales = b.quantize_int8(x)
    want8, want = b.dispatch_quantized(codes, scales, w, h)[0], b.dispatch(x, idx, w, handle=h)[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call, ref in ((lambda s: b.dispatch_quantized(codes, scales, w, h, stream=s), want8),
                      (lambda s: b.dispatch(x, idx, w, handle=h, stream=s), (want,))):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        out = call(side.cuda_stream if raw else side)
        got = out[0] if isinstance(out[0], tuple) else (out[0],)
        assert not out[-1].query()   # the stream still sleeps
        torch.cuda.current_stream().wait_event(out[-1])
        assert all(torch.equal(a, c) for a, c in zip(got, ref))
