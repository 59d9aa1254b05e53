"""The norms before and after a block with its gate and residual scale, against
a plain implementation in 64 bits; their codes are bit for bit those of
quantize_rowwise on the bf16 result."""
import pytest
import torch

from block_ops_ref import assert_close, residual_norm64
from gpu_common import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return require_cuda()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _case(rows, cols, *, seed=0, stream=torch.bfloat16, vec=torch.bfloat16, post=None, pre="rms",
          gate=False, mod=False, groups=1, weights=True, pad=False):
    """Inputs of one call: (args of residual_norm, args of the 64-bit form)."""
    g = _gen(seed + 7 * rows + cols)

    def normal(*s, std=1.0, mean=0.0, dtype=vec):
        return (torch.randn(*s, generator=g, device="cuda") * std + mean).to(dtype)

    residual = normal(rows, cols, std=2.0, mean=0.3, dtype=stream)
    y = normal(rows, cols, std=1.5, mean=-0.5, dtype=torch.bfloat16)
    mods = normal(groups, 6 * cols, std=0.4)
    group = torch.sort(torch.randint(0, groups, (rows,), generator=g, device="cuda")).values
    row_group = group.to(torch.int32)
    if pad:
        lost = torch.rand(rows, generator=g, device="cuda") < 0.3
        row_group = torch.where(lost, torch.where(group % 2 == 0, -1, groups + 5).to(torch.int32), row_group)
    kw, ref = {}, {}
    for name, kind in (("post", post), ("pre", pre)):
        if kind is not None:
            w = normal(cols, std=0.3, mean=1.0) if weights else None
            b = normal(cols, std=0.2) if weights else None
            kw[name], ref[name] = (kind, w, b, 1e-5), (kind, w, b, 1e-5)
    if gate:
        kw["gate"] = ref["gate"] = mods[:, :cols]
    if mod:
        kw["scale"] = ref["scale"] = mods[:, 2 * cols:3 * cols]
        kw["shift"] = ref["shift"] = mods[:, cols:2 * cols]
    ref["group"] = group
    return residual, y, row_group, kw, ref


def _norms(nv, kw):
    return {k: nv.Norm(*v) if k in ("post", "pre") else v for k, v in kw.items()}


def _check(nv, case, **more):
    residual, y, row_group, kw, ref = case
    r = nv.residual_norm(residual, y, row_group=row_group, **_norms(nv, kw), **more)
    torch.cuda.synchronize()
    h, e_h, o, e_o = residual_norm64(residual, y, **ref, **{k: v for k, v in more.items() if k.endswith("_scale")})
    if r.h is not None:
        assert_close(r.h, h, e_h, "h")
    if r.out is not None:
        assert_close(r.out, o, e_o, "out")
    return r


def _same_codes(nv, r, rows=None):
    q = nv.quantize_rowwise(r.out.contiguous())
    assert torch.equal(r.quant.q, q.q) and torch.equal(r.quant.s_dec, q.s_dec)
    assert torch.equal(r.quant.sf, q.sf)


# Every width class, for a few rows and for many.
@pytest.mark.parametrize("rows", [1, 3, 130, 600])
@pytest.mark.parametrize("cols", [16, 48, 256, 272, 512, 784, 1024, 1040, 2048, 2064, 4096, 4112, 5120,
                                  8192, 8208, 12288, 16384, 16400, 32768])
def test_widths(nv, rows, cols):
    r = _check(nv, _case(rows, cols, post="rms", pre="layer", gate=True, mod=True,
                         groups=min(rows, 3)), want_quant=True)
    _same_codes(nv, r)


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vec", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("post", [None, "rms", "layer"])
@pytest.mark.parametrize("pre", [None, "rms", "layer"])
@pytest.mark.parametrize("rows,cols", [(37, 640), (1999, 1296), (700, 4112), (620, 5136)])
def test_types_and_norms(nv, stream, vec, post, pre, rows, cols):
    for gate, mod, weights in ((False, False, True), (True, pre is not None, False),
                               (True, pre is not None, True)):
        _check(nv, _case(rows, cols, stream=stream, vec=vec, post=post, pre=pre, gate=gate, mod=mod,
                         groups=5, weights=weights), residual_scale=0.75, branch_scale=-1.5)
    code, tag = nv.device_error()
    assert code == 0, f"device wait timed out (tag {tag})"


@pytest.mark.parametrize("rows", [65, 650])
def test_start_of_a_model(nv, rows):
    """No y: the norm of the (scaled) stream alone."""
    residual, _, row_group, kw, ref = _case(rows, 1536, pre="layer", mod=True, groups=2)
    r = nv.residual_norm(residual, row_group=row_group, residual_scale=3.0, **_norms(nv, kw))
    _, _, o, e_o = residual_norm64(residual, None, residual_scale=3.0, **ref)
    assert r.h is None
    assert_close(r.out, o, e_o)


def test_outputs_that_are_not_wanted(nv):
    case = _case(33, 512)
    full = _check(nv, case, want_quant=True)
    r = _check(nv, case, want_h=False, want_out=False, want_quant=True)
    assert r.h is None and r.out is None
    assert torch.equal(r.quant.q, full.quant.q) and torch.equal(r.quant.sf, full.quant.sf)


def test_consecutive_rows_without_row_group(nv):
    residual, y, _, kw, ref = _case(60, 256, gate=True, mod=True, groups=4)
    ref["group"] = torch.arange(60, device="cuda") // 15
    r = nv.residual_norm(residual, y, **_norms(nv, kw))
    h, e_h, o, e_o = residual_norm64(residual, y, **ref)
    assert_close(r.h, h, e_h)
    assert_close(r.out, o, e_o)
    with pytest.raises(nv.NVFP4Error):      # 59 rows are not 4 equal requests
        nv.residual_norm(residual[:59], y[:59], **_norms(nv, kw))


@pytest.mark.parametrize("rows", [90, 1700])
def test_unsorted_requests_and_one_vector_for_all(nv, rows):
    residual, y, _, kw, ref = _case(rows, 384, gate=True, mod=True, groups=6)
    g = torch.randint(0, 6, (rows,), generator=_gen(1), device="cuda")
    kw["gate"] = ref["gate"] = kw["gate"][2]     # [cols]
    ref["group"] = g
    r = nv.residual_norm(residual, y, row_group=g.to(torch.int32), **_norms(nv, kw))
    h, e_h, o, e_o = residual_norm64(residual, y, **ref)
    assert_close(r.h, h, e_h)
    assert_close(r.out, o, e_o)


@pytest.mark.parametrize("rows,cols", [(5, 512), (129, 1040), (400, 4096), (5000, 1040), (1000, 8192)])
def test_padding_rows_stay_as_they_were(nv, rows, cols):
    residual, y, row_group, kw, ref = _case(rows, cols, pad=True, gate=True, mod=True, groups=3)
    live = (row_group >= 0) & (row_group < 3)
    residual[~live], y[~live] = float("nan"), float("inf")     # never read into anything
    h = torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(h, 9.0)
    qt = nv.empty_nvfp4(rows, cols, row_scales=True)
    for t, v in ((qt.q, 0x5A), (qt.sf, 0x33), (qt.s_dec, 5.0)):
        t.fill_(v)
    amax = torch.full((rows,), -3.0, device="cuda")
    nv.residual_norm(residual, y, row_group=row_group, h=h, out=out, quant=qt, amax_rows=amax,
                     **_norms(nv, kw))
    torch.cuda.synchronize()
    want_h, e_h, want_o, e_o = residual_norm64(residual, y, **ref)
    assert_close(h[live], want_h[live], e_h[live])
    assert_close(out[live], want_o[live], e_o[live])
    assert (h[~live] == 7.0).all() and (out[~live] == 9.0).all()
    assert (qt.q[~live] == 0x5A).all() and (qt.s_dec[~live] == 5.0).all() and (amax[~live] == -3.0).all()
    ref_q = nv.quantize_rowwise(out)
    assert torch.equal(qt.q[live], ref_q.q[live]) and torch.equal(qt.s_dec[live], ref_q.s_dec[live])
    kb4 = (cols // 16 + 3) // 4
    def rows_of(sf):
        return sf.view(-1, kb4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, 4 * kb4)
    got, want = rows_of(qt.sf), rows_of(ref_q.sf)
    assert torch.equal(got[:rows][live], want[:rows][live])
    assert (got[:rows][~live] == 0x33).all() and (got[rows:] == 0).all()


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(70, 528), (3000, 528), (900, 6160)])
def test_strided_and_in_place(nv, stream, rows, cols):
    """Column slices of wider buffers, h over the residual, out over y."""
    residual, y, row_group, kw, ref = _case(rows, cols, stream=stream, post="layer", pre="rms", gate=True, mod=True)
    h, e_h, o, e_o = residual_norm64(residual, y, **ref)
    wide_r = torch.full((rows, cols + 64), 3.0, dtype=stream, device="cuda")
    wide_y = torch.full((rows, 2 * cols), 4.0, dtype=torch.bfloat16, device="cuda")
    wide_r[:, 32:32 + cols], wide_y[:, cols:] = residual, y
    rs, ys = wide_r[:, 32:32 + cols], wide_y[:, cols:]
    r = nv.residual_norm(rs, ys, row_group=row_group, h=rs, out=ys, **_norms(nv, kw))
    torch.cuda.synchronize()
    assert r.h is rs and r.out is ys
    assert_close(rs, h, e_h)
    assert_close(ys, o, e_o)
    assert (wide_r[:, :32] == 3.0).all() and (wide_r[:, 32 + cols:] == 3.0).all() and (wide_y[:, :cols] == 4.0).all()


@pytest.mark.parametrize("rows,cols", [(270, 256), (310, 512)])
def test_offsets_past_32_bits(nv, rows, cols):
    """Rows 2^23 elements apart: the last ones start beyond 2^31 elements."""
    stride = 1 << 23
    residual, y, row_group, kw, ref = _case(rows, cols)
    far = torch.empty(rows * stride, dtype=torch.bfloat16, device="cuda").view(rows, stride)[:, :cols]
    far.copy_(y)
    _, _, o, e_o = residual_norm64(residual, y, **ref)
    r = nv.residual_norm(residual, far, row_group=row_group, out=far, **_norms(nv, kw))
    assert_close(r.out, o, e_o)
    h, e_h, _, _ = residual_norm64(residual, y, **ref)
    assert_close(r.h, h, e_h)


@pytest.mark.parametrize("rows", [8, 400])
def test_rows_of_zeros_and_of_large_values(nv, rows):
    residual, y, row_group, kw, ref = _case(rows, 1024, pre="layer", weights=False)
    residual[0], y[0] = 0, 0                      # variance 0: out = 0
    residual[1], y[1] = 5.0, 0                    # constant row of a layer norm
    residual[2] *= 1e15
    residual[3] *= 1e-12
    y[3] *= 1e-12
    r = _check(nv, (residual, y, row_group, kw, ref), want_quant=True)
    assert (r.out[0] == 0).all() and (r.out[1] == 0).all()
    _same_codes(nv, r)


def test_empty(nv):
    z = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    r = nv.residual_norm(z, z, pre=nv.Norm(), want_quant=True)
    assert r.h.shape == r.out.shape == (0, 64) and r.quant.sf.numel() == 0


def test_oracle_codes(nv, orc):
    """The codes against the CPU oracle's, from the same bf16 values."""
    import numpy as np
    from workloads import bf16_bits
    r = _check(nv, _case(131, 336, post="rms", pre="rms"), want_quant=True)
    oq, osf, osd, _ = orc.quantize_rowwise(bf16_bits(r.out.cpu()), 131, 336)
    assert np.array_equal(r.quant.q.cpu().numpy(), oq) and np.array_equal(r.quant.sf.cpu().numpy(), osf)
    assert np.array_equal(r.quant.s_dec.cpu().numpy(), osd)


@pytest.mark.parametrize("rows", [200, 800])
def test_streams_and_graph(nv, rows):
    """Side stream with its inputs made there; a captured call replayed on new values."""
    case = _case(rows, 2048, post="rms", gate=True, mod=True, groups=2)
    residual, y, row_group, kw, ref = case
    norms = _norms(nv, kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = nv.residual_norm(residual, y, row_group=row_group, want_quant=True, **norms)
    with torch.cuda.stream(side):
        b = nv.residual_norm(residual, y, row_group=row_group, want_quant=True, **norms)
    torch.cuda.synchronize()
    for s, t in ((a.h, b.h), (a.out, b.out), (a.quant.q, b.quant.q), (a.quant.sf, b.quant.sf)):
        assert torch.equal(s, t)
    g = torch.cuda.CUDAGraph()
    x_in, y_in = residual.clone(), y.clone()
    with torch.cuda.graph(g):
        c = nv.residual_norm(x_in, y_in, row_group=row_group, want_quant=True, **norms)
    x_in.copy_(residual.flip(0))
    y_in.copy_(y.flip(0))
    g.replay()
    torch.cuda.synchronize()
    d = nv.residual_norm(residual.flip(0), y.flip(0), row_group=row_group, want_quant=True, **norms)
    for s, t in ((c.h, d.h), (c.out, d.out), (c.quant.q, d.quant.q), (c.quant.s_dec, d.quant.s_dec)):
        assert torch.equal(s, t)


def test_refusals(nv):
    r = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    norm = nv.Norm("rms", w)
    bad = [
        dict(residual=r.half(), y=r, pre=norm),                        # type of the stream
        dict(residual=r, y=r.float(), pre=norm),                       # type of y
        dict(residual=r, y=r[:3], pre=norm),                           # rows differ
        dict(residual=r.cpu(), y=r, pre=norm),                         # another device
        dict(residual=r, y=r, pre=nv.Norm("batch")),                   # no such norm
        dict(residual=r, y=r, pre=norm, scale=w.float()),              # vectors of two types
        dict(residual=r, y=r, pre=norm, scale=w[:32]),                 # a short vector
        dict(residual=r, y=r, pre=norm, scale=w.expand(2, 64), shift=w.expand(4, 64)),
        dict(residual=r, y=r, pre=nv.Norm("rms", w.expand(4, 64))),    # a weight per request
        dict(residual=r, gate=w, pre=norm),                            # a gate without a branch
        dict(residual=r, y=r, scale=w),                                # a scale without a norm
        dict(residual=r, y=r, pre=norm, row_group=torch.zeros(4, device="cuda", dtype=torch.int64)),
        dict(residual=r, y=r, pre=norm, row_group=torch.zeros(3, device="cuda", dtype=torch.int32)),
        dict(residual=r, y=r, pre=norm, out=r.t().contiguous().t()),   # rows that are not contiguous
        dict(residual=r, y=r, pre=norm, quant=nv.empty_nvfp4(4, 64)),  # one scale, not one per row
        dict(residual=r, y=r, pre=norm, amax_rows=torch.zeros(4, device="cuda")),  # amax without codes
    ]
    for kw in bad:
        with pytest.raises(ValueError):
            nv.residual_norm(kw.pop("residual"), kw.pop("y", None), **kw)
    wide = torch.zeros(4, 200, dtype=torch.bfloat16, device="cuda")
    for kw, status in [(dict(residual=r[:, :24], y=r[:, :24]), 1),     # cols % 16
                       (dict(residual=wide[:, 4:68], y=r), 2),         # not 16-byte aligned
                       (dict(residual=torch.zeros(4, 100, dtype=torch.bfloat16, device="cuda")[:, :64], y=r), 1),
                       (dict(residual=r, y=r, eps=float("nan")), 1),
                       (dict(residual=r, y=r, residual_scale=float("inf")), 1),
                       (dict(residual=r, y=r, want_out=False), 1)]:    # a norm nobody reads
        pre = nv.Norm(eps=kw.pop("eps", 1e-6))
        with pytest.raises(nv.NVFP4Error) as e:
            nv.residual_norm(kw.pop("residual"), kw.pop("y"), pre=pre, **kw)
        assert e.value.status == status


@pytest.mark.parametrize("field,make", [
    ("q", lambda t: t.cpu()), ("q", lambda t: t.float()), ("q", lambda t: t.t().contiguous().t()),
    ("sf", lambda t: t.cpu()), ("sf", lambda t: t[:-1]), ("sf", lambda t: t.repeat_interleave(2)[::2]),
    ("s_dec", lambda t: t.cpu()), ("s_dec", lambda t: t.half()), ("s_dec", lambda t: t.repeat_interleave(2)[::2]),
])
def test_refuses_codes_it_cannot_write(nv, field, make):
    r = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    q = nv.empty_nvfp4(4, 64, row_scales=True)
    setattr(q, field, make(getattr(q, field)))
    with pytest.raises(ValueError):
        nv.residual_norm(r, r, pre=nv.Norm(), quant=q)
