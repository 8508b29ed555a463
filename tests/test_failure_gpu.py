"""Failure detection on the GPU without a fault: the time-bounded wait every
kernel uses runs out on an mbarrier nothing arrives on, reports
SR_DEVERR_TIMEOUT after about its bound, and the context stays usable (a decode
step afterwards still matches the oracle)."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

from kv_cache_routing_sr_b200 import inputs, native
from tests import gpu_helpers as H

pytestmark = pytest.mark.gpu


def test_bounded_wait_runs_out_and_reports():
    for limit_us in (20000, 200000):
        status, waited_ns = native.selftest_bounded_wait(limit_us)
        assert status == native.SR_DEVERR_TIMEOUT
        assert limit_us * 1000 <= waited_ns < limit_us * 1000 + 50_000_000  # the bound, plus at most 50 ms


def test_context_usable_after_a_timeout():
    native.selftest_bounded_wait(50000)
    x = inputs.make("tiny_4k", seed=61, device="cuda", max_ctx=2000)
    mask_g, act_g, out_g, dec = H.gpu_step(x)
    assert dec.workspace.device_error() == 0
    ref = H.oracle_full(x, x.tau)
    H.assert_route_equal(mask_g, act_g, ref.mask, ref.active_list)
    H.check_against_oracle(x, out_g, mask_g, what="after a bounded-wait timeout")


AFTER_AN_ERROR = """
import torch
from kv_cache_routing_sr_b200 import native
q = torch.randn(1, 32, 128, device="cuda").to(torch.bfloat16)
k0 = torch.randn(1, 8, 128, device="cuda").to(torch.bfloat16)
ws = native.Workspace(1, 32, 8, 64)
want, _ = native.route(q, k0, 0.6)
torch.cuda.synchronize()
seen = None
try:
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        try:
            ws.device_error()  # synchronises, which a capturing stream refuses
        except native.SinkRouterError as e:
            seen = e.status
except RuntimeError:
    pass  # the capture is void
assert seen == native.SR_ERR_CUDA
got, _ = native.route(q, k0, 0.6)
assert torch.equal(got, want)
assert b"capturing" in native.load().sr_last_cuda_error()
print("usable")
"""


def test_a_failed_call_is_not_reported_by_the_next_one():
    """A CUDA error that a call has returned is cleared: the next call succeeds. In a
    process of its own, since the voided capture is torch's affair too."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", AFTER_AN_ERROR], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "usable" in r.stdout, r.stderr[-2000:]
