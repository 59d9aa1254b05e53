"""residual_norm in place: row on row of one type and stride, else refused before any
device work (runs without a GPU)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def nv():
    from nvfp4_block_scaled_19_b200 import build
    build.build()
    import nvfp4_block_scaled_19_b200 as nv
    nv.lib()
    return nv


@pytest.fixture(scope="module")
def p():
    # Any aligned host address stands in for a device pointer.
    buf = ctypes.create_string_buffer(4096)
    p.keep = buf
    return (ctypes.addressof(buf) + 63) // 64 * 64


def _status(nv, p, **kw):
    a = nv.ResidualNormArgs()
    base = dict(rows=4, cols=64, residual=p, residual_stride=64, y=p + 512, y_stride=64, h=p + 1024, h_stride=64,
                out=p + 1536, out_stride=64, groups=1, residual_scale=1.0, branch_scale=1.0, pre_norm=1,
                pre_eps=1e-6)
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return nv.lib().nvfp4_residual_norm(ctypes.byref(a), None)


def test_rows_on_other_rows_are_refused(nv, p):
    for kw in (dict(h=p, h_stride=128), dict(h=p + 512, h_stride=72), dict(out=p + 512, out_stride=128),
               dict(out=p, out_stride=72), dict(h=p + 512, stream_dtype=1), dict(out=p, stream_dtype=1)):
        assert _status(nv, p, **kw) == 1, kw


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device answer")
def test_rows_on_themselves_reach_the_device_check(nv, p):
    for kw in (dict(), dict(h=p), dict(h=p + 512), dict(out=p), dict(out=p + 512), dict(h=p, out=p + 512),
               dict(h=p, stream_dtype=1), dict(out=p + 512, stream_dtype=1),
               dict(rows=1, h=p, h_stride=128, out=p + 512, out_stride=72)):
        assert _status(nv, p, **kw) == 3, kw


@pytest.mark.gpu
def test_one_tensor_for_both_results_is_refused():
    from gpu_common import require_cuda
    nv = require_cuda()
    r = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros_like(r)
    with pytest.raises(ValueError):
        nv.residual_norm(r, y, pre=nv.Norm(), h=r, out=r)
    with pytest.raises(nv.NVFP4Error) as e:
        wide = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
        nv.residual_norm(wide[:, :64], y, pre=nv.Norm(), h=wide.view(-1)[:256].view(4, 64))
    assert e.value.status == 1
    nv.residual_norm(r, y, pre=nv.Norm(), h=r, out=y)
