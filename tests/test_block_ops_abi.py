"""The entry points around a projection refuse bad arguments before any device
work (runs without a GPU)."""
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
    # Any aligned host address stands in for a device pointer: these calls fail
    # on their arguments before anything reaches a device.
    buf = ctypes.create_string_buffer(4096)
    p.keep = buf
    return (ctypes.addressof(buf) + 63) // 64 * 64


def _norm_args(nv, p, **kw):
    base = dict(rows=4, cols=64, residual=p, residual_stride=64, y=p, y_stride=64, h=p, h_stride=64,
                out=p, out_stride=64, groups=1, residual_scale=1.0, branch_scale=1.0,
                pre_norm=1, pre_eps=1e-6)
    base.update(kw)
    a = nv.ResidualNormArgs()
    for k, v in base.items():
        setattr(a, k, v)
    return a


NORM_REFUSED = [
    dict(rows=-1), dict(rows=1 << 31), dict(cols=0), dict(cols=24), dict(cols=32784, residual_stride=32784),
    dict(residual=None), dict(h=None, out=None), dict(y=None), dict(y=None, h=None, gate=None, post_norm=1),
    dict(pre_norm=0), dict(pre_norm=3), dict(post_norm=-1), dict(out=None), dict(out=None, pre_norm=0, scale=64),
    dict(pre_eps=float("nan")), dict(pre_eps=-1.0), dict(post_norm=2, post_eps=float("inf")),
    dict(post_weight=64), dict(residual_scale=float("nan")), dict(branch_scale=float("inf")),
    dict(groups=0), dict(groups=3), dict(stream_dtype=2), dict(vector_dtype=-1),
    dict(residual_stride=56), dict(residual_stride=68), dict(y_stride=63), dict(h_stride=0),
    dict(out_stride=1 << 60), dict(gate=64, gate_stride=32), dict(scale=64, scale_stride=65),
    dict(shift=64, shift_stride=-64), dict(q=64), dict(q=64, sf=64), dict(sf=64), dict(s_dec_rows=64),
    dict(amax_rows=64),
]


@pytest.mark.parametrize("kw", NORM_REFUSED, ids=str)
def test_residual_norm_invalid(nv, p, kw):
    a = _norm_args(nv, p, **kw)
    assert nv.lib().nvfp4_residual_norm(ctypes.byref(a), None) == 1


@pytest.mark.parametrize("kw", [dict(residual=8), dict(y=2), dict(h=4), dict(out=8), dict(gate=8),
                                dict(scale=24), dict(pre_weight=2), dict(row_group=2),
                                dict(q=16, sf=16, s_dec_rows=2), dict(q=8, sf=16, s_dec_rows=16),
                                dict(q=16, sf=16, s_dec_rows=16, amax_rows=3)], ids=str)
def test_residual_norm_misaligned(nv, p, kw):
    a = _norm_args(nv, p, **{k: p + v for k, v in kw.items()})
    assert nv.lib().nvfp4_residual_norm(ctypes.byref(a), None) == 2


def test_residual_norm_null(nv):
    assert nv.lib().nvfp4_residual_norm(None, None) == 1


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device answer")
def test_accepted_arguments_reach_the_device_check(nv, p):
    for kw in (dict(), dict(y=None, h=None), dict(h=None), dict(out=None, pre_norm=0),
               dict(rows=0, residual=None, y=None, h=None, out=None),
               dict(q=p, sf=p, s_dec_rows=p, out=None), dict(groups=2), dict(groups=3, row_group=p),
               dict(gate=p, gate_stride=0, scale=p, scale_stride=384, groups=2)):
        a = _norm_args(nv, p, **kw)
        assert nv.lib().nvfp4_residual_norm(ctypes.byref(a), None) == 3, kw


def _lora_args(nv, p, **kw):
    base = dict(rows=4, k=64, n=80, rank=16, slots=2, x=p, x_stride=64, y=p + 64, y_stride=80,
                out=p + 128, out_stride=80, a=p, b=p, scale=p, workspace=p)
    base.update(kw)
    a = nv.LoraArgs()
    for k, v in base.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(rows=(1 << 27) + 1), dict(k=0), dict(k=72), dict(k=(1 << 20) + 16), dict(n=8), dict(n=84),
    dict(n=(1 << 20) + 8), dict(rank=0), dict(rank=8), dict(rank=24), dict(rank=144), dict(slots=0),
    dict(slots=1 << 25), dict(x=None), dict(y=None), dict(out=None), dict(a=None), dict(b=None), dict(scale=None),
    dict(x_stride=56), dict(x_stride=68), dict(y_stride=72), dict(out_stride=0), dict(out_stride=1 << 39),
    dict(rows=1 << 16, workspace=None), dict(k=16, n=16, x_stride=16, rank=128, slots=1 << 25),
], ids=str)
def test_lora_invalid(nv, p, kw):
    assert nv.lib().nvfp4_lora(ctypes.byref(_lora_args(nv, p, **kw)), None) == 1


def test_lora_aliases_and_alignment(nv, p):
    f = nv.lib().nvfp4_lora
    assert f(None, None) == 1
    assert f(ctypes.byref(_lora_args(nv, p, out=p)), None) == 1                       # out over x
    assert f(ctypes.byref(_lora_args(nv, p, out=p + 64, out_stride=88)), None) == 1   # out over y, other rows
    for name in ("x", "y", "out", "a", "b", "workspace"):
        assert f(ctypes.byref(_lora_args(nv, p, **{name: p + 8})), None) == 2, name
    for name in ("scale", "row_slot"):
        assert f(ctypes.byref(_lora_args(nv, p, **{name: p + 2})), None) == 2, name


def test_lora_workspace_sizes(nv):
    f = nv.lib().nvfp4_lora_workspace_bytes
    assert f(-1, 64, 64, 16) == 0 and f(4096, 72, 64, 16) == 0 and f(4096, 64, 64, 144) == 0
    assert f(0, 4096, 4096, 64) == f(1, 4096, 4096, 128) == f(64, 4096, 4096, 64) == 0   # row by row
    for rows in (257, 5000, 1 << 27):
        # On tiles: the inner vectors as two bf16, a flag per tile, and fp32 sums of
        # the splits of K, of which there are at most as many as SMs.
        least = rows * 4 * 64 + (rows + 127) // 128 * 4
        assert least <= f(rows, 4096, 4096, 64) <= least + 148 * 128 * 64 * 4 + 16
        assert f(rows, 4096, 4096, 64) % 16 == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device answer")
def test_lora_accepted_arguments_reach_the_device_check(nv, p):
    for kw in (dict(), dict(rows=0, x=None, y=None, out=None), dict(row_slot=p), dict(out=p + 64),
               dict(rows=1 << 16)):
        assert nv.lib().nvfp4_lora(ctypes.byref(_lora_args(nv, p, **kw)), None) == 3, kw
