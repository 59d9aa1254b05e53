"""Padding rows of a batch of one request: a modulation tensor [1, 6 C] makes every
number but 0 padding, as one of several requests does for numbers past them."""
import pytest
import torch

from block_ops_ref import assert_close, residual_norm64
from gpu_common import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return require_cuda()


def _inputs(rows, cols):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    residual = torch.randn(rows, cols, generator=g, device="cuda").to(torch.bfloat16)
    y = torch.randn(rows, cols, generator=g, device="cuda").to(torch.bfloat16)
    mod = (torch.randn(3, 6 * cols, generator=g, device="cuda") * 0.3).to(torch.bfloat16)
    return residual, y, mod


@pytest.mark.parametrize("rows", [9, 4000])
@pytest.mark.parametrize("which", ["gate", "scale", "shift", "all"])
def test_one_request(nv, rows, which):
    cols = 1040
    residual, y, mod = _inputs(rows, cols)
    vectors = {n: mod[:1, i * cols:(i + 1) * cols] for i, n in enumerate(("gate", "scale", "shift"))
               if which in (n, "all")}
    live = torch.arange(rows, device="cuda") < rows - 3
    group = torch.where(live, 0, torch.arange(rows, device="cuda") - rows + 4).to(torch.int32)    # 1, 2, 3
    h = torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(h, 9.0)
    nv.residual_norm(residual, y, pre=nv.Norm("rms"), row_group=group, h=h, out=out, **vectors)
    want_h, e_h, want, e = residual_norm64(residual, y, pre=("rms", None, None, 1e-6),
                                           group=torch.zeros(rows, dtype=torch.int64, device="cuda"), **vectors)
    assert_close(h[live], want_h[live], e_h[live])
    assert_close(out[live], want[live], e[live])
    assert (h[~live] == 7.0).all() and (out[~live] == 9.0).all()


@pytest.mark.parametrize("rows", [9, 4000])
def test_one_vector_for_all(nv, rows):
    """[cols], and [1, cols] beside a vector of three requests, hold for every request."""
    cols = 1040
    residual, y, mod = _inputs(rows, cols)
    group = torch.arange(rows, device="cuda") % 3
    gate, scale, shift = (mod[:, i * cols:(i + 1) * cols] for i in range(3))
    for vectors, ref in ((dict(gate=gate[0], scale=scale[1]), dict(gate=gate[0], scale=scale[1])),
                         (dict(gate=gate[:1], shift=shift), dict(gate=gate[0], shift=shift))):
        r = nv.residual_norm(residual, y, pre=nv.Norm("rms"), row_group=group.to(torch.int32), **vectors)
        want_h, e_h, want, e = residual_norm64(residual, y, pre=("rms", None, None, 1e-6), group=group, **ref)
        assert_close(r.h, want_h, e_h)
        assert_close(r.out, want, e)
