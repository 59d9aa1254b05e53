"""The shares of the expand's CTAs go by the work of the row tiles: tiles that are
left to the kernel of single rows weigh nothing, and a tile's adapters are counted
once each, whatever the order of its rows."""
import statistics

import pytest
import torch

from block_ops_ref import assert_close, lora64
from gpu_common import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return require_cuda()


def _timed(nv, x, y, ad, slot):
    """us of a call among others (median of several runs)."""
    out = torch.empty_like(y)
    got = []
    for _ in range(9):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        nv.lora(x, y, ad, slot, out=out)
        torch.cuda._sleep(2_000_000)             # the host is ahead
        a.record()
        for _ in range(20):
            nv.lora(x, y, ad, slot, out=out)
        b.record()
        b.synchronize()
        got.append(a.elapsed_time(b) * 1e3 / 20)
    assert nv.device_error() == (0, 0)
    return statistics.median(got)


def _inputs(nv, rows, k, n, rank, slots):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + n)

    def normal(*s, std=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)

    ad = nv.LoraAdapters(normal(slots, rank, k, std=k ** -0.5), normal(slots, n, rank, std=rank ** -0.5),
                         torch.rand(slots, generator=g, device="cuda") + 0.5)
    return normal(rows, k), normal(rows, n), ad


# Together, of the times apart: 1.25 and 0.94 (2.3 and 1.4 with the crowded tile weighed).
@pytest.mark.parametrize("rank,limit", [(16, 1.7), (64, 1.25)])
def test_a_crowded_tile_costs_the_others_nothing(nv, rank, limit):
    """A prefill (three tiles of one adapter each) beside a decoding batch of 64."""
    rows, k, n, slots = 512, 1024, 28672, 67
    x, y, ad = _inputs(nv, rows, k, n, rank, slots)
    at = torch.arange(rows, dtype=torch.int32, device="cuda")
    slot = torch.where(at < 384, at // 128, at - 381).clamp(max=slots - 1).to(torch.int32)
    want, err = lora64(x, y, ad, slot)
    assert_close(nv.lora(x, y, ad, slot), want, err)
    both = _timed(nv, x, y, ad, slot)
    prefill = _timed(nv, x[:384], y[:384], ad, slot[:384].contiguous())
    batch = _timed(nv, x[384:], y[384:], ad, slot[384:].contiguous())
    assert both < limit * (prefill + batch), (both, prefill, batch)


def test_order_inside_a_tile_does_not_matter(nv):
    rows, k, n, slots = 2048, 1024, 12288, 64
    x, y, ad = _inputs(nv, rows, k, n, 16, slots)
    at = torch.arange(rows, dtype=torch.int32, device="cuda")
    by_turns = torch.where(at < 128, at % 2 * 40, 5).to(torch.int32)
    one_by_one = torch.where(at < 128, at // 64 * 40, 5).to(torch.int32)
    times = []
    for slot in (by_turns, one_by_one):
        want, err = lora64(x, y, ad, slot)
        assert_close(nv.lora(x, y, ad, slot), want, err)
        times.append(_timed(nv, x, y, ad, slot))
    assert times[0] < 1.4 * times[1], times       # 1.02; 1.8 with turns counted as runs


@pytest.mark.parametrize("in_place", [False, True])
def test_every_tile_crowded(nv, in_place):
    """All shares are empty: every row goes by itself."""
    rows, k, n, slots = 384, 256, 28672, 128
    x, y, ad = _inputs(nv, rows, k, n, 16, slots)
    slot = torch.arange(rows, dtype=torch.int32, device="cuda").remainder(128)
    want, err = lora64(x, y, ad, slot)
    out = y.clone() if in_place else torch.full_like(y, float("nan"))
    nv.lora(x, out if in_place else y, ad, slot, out=out)
    torch.cuda.synchronize()
    assert nv.device_error() == (0, 0)
    assert_close(out, want, err)
