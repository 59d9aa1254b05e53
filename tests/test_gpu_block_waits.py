"""The bounded waits of the kernels around a projection run out too: the self-test's
second kernel gives up after its own limit, and what it runs on stays usable."""
import time

import pytest
import torch

from gpu_common import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return require_cuda()


@pytest.mark.parametrize("timeout_us", [1000, 50_000])
def test_both_kernels_waits_run_out(nv, timeout_us):
    x = torch.randn(700, 512, device="cuda").to(torch.bfloat16)
    want = nv.residual_norm(x, x, pre=nv.Norm())
    torch.cuda.synchronize()
    assert nv.device_error() == (0, 0)
    t0 = time.perf_counter()
    nv.selftest_wait_timeout(timeout_us)
    torch.cuda.synchronize()
    seconds = time.perf_counter() - t0
    # One limit after the other (the clock that bounds them ticks every us or so).
    assert 2e-6 * timeout_us - 20e-6 <= seconds < 1.0
    assert nv.device_error() == (5, nv.SELFTEST_TAG)
    assert nv.device_error() == (0, 0)
    assert torch.equal(nv.residual_norm(x, x, pre=nv.Norm()).out, want.out)
