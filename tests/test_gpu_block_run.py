"""The operators around a projection in a run, as a block uses them: norm and
codes, projections with the requests' adapters, gate and residual, the next
norm.  Each step against the plain form of its own inputs, and the whole run
captured in a graph and replayed on other requests."""
import pytest
import torch

from block_ops_ref import assert_close, lora64, residual_norm64
from gpu_common import require_cuda

pytestmark = pytest.mark.gpu

C, H, REQUESTS = 512, 1152, 5


@pytest.fixture(scope="module")
def nv():
    return require_cuda()


def _model(nv):
    g = torch.Generator(device="cuda")
    g.manual_seed(3)

    def normal(*s, std=1.0, mean=0.0):
        return (torch.randn(*s, generator=g, device="cuda") * std + mean).to(torch.bfloat16)

    def adapters(k, n):
        return nv.pack_adapters([(normal(r, k, std=k ** -0.5), normal(n, r, std=0.5 * r ** -0.5), 1.0 / r)
                                 for r in (8, 24, 16)])

    return dict(up=nv.NVFP4Linear(normal(H, C, std=C ** -0.5)), down=nv.NVFP4Linear(normal(C, H, std=H ** -0.5)),
                up_ad=adapters(C, H), down_ad=adapters(H, C), norm=nv.Norm("layer"),
                post=nv.Norm("rms", normal(C, std=0.1, mean=1.0), eps=1e-5), normal=normal)


def _batch(m, rows, seed, stream):
    """Ragged requests, the last rows padding, an adapter (or none) per request."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    live = rows - rows // 7
    request = torch.randint(0, REQUESTS, (live,), generator=g, device="cuda").sort().values
    group = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    group[:live] = request
    of_request = torch.tensor([2, -1, 0, 1, 0], device="cuda")
    slot = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    slot[:live] = of_request[request]
    x = torch.randn(rows, C, generator=g, device="cuda") * 2
    mod = (torch.randn(REQUESTS, 6 * C, generator=g, device="cuda") * 0.3).to(torch.bfloat16)
    return x.to(stream), group, slot, mod


def _zeros(nv, rows):
    """Outputs of a norm whose padding rows are zero, as the tensors behind them then are."""
    q = nv.empty_nvfp4(rows, C, row_scales=True)
    for t in (q.q, q.sf, q.s_dec):
        t.zero_()
    return dict(out=torch.zeros(rows, C, dtype=torch.bfloat16, device="cuda"), quant=q)


def _block(nv, m, h, group, slot, mod):
    """One feed-forward block on the stream h (updated in place)."""
    chunk = [mod[:, i * C:(i + 1) * C] for i in range(6)]
    a = nv.residual_norm(h, pre=m["norm"], scale=chunk[0], shift=chunk[1], row_group=group,
                         **_zeros(nv, h.shape[0]))
    up = m["up"](a.out, xq=a.quant, adapters=m["up_ad"], row_slot=slot)
    act = torch.nn.functional.gelu(up)
    down = m["down"](act, adapters=m["down_ad"], row_slot=slot)
    b = nv.residual_norm(h, down, post=m["post"], gate=chunk[2], pre=m["norm"], scale=chunk[3], shift=chunk[4],
                         row_group=group, branch_scale=0.5, h=h, want_quant=True)
    return a, up, act, down, b


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [1, 37, 700])
def test_each_step_of_a_block(nv, rows, stream):
    m = _model(nv)
    h, group, slot, mod = _batch(m, rows, 5 + rows, stream)
    before = h.clone()
    a, up, act, down, b = _block(nv, m, h, group, slot, mod)
    torch.cuda.synchronize()
    code, tag = nv.device_error()
    assert code == 0, f"device wait timed out (tag {tag})"
    live = group >= 0
    n, kw = int(live.sum()), dict(group=group[live].long())
    layer, rms = ("layer", None, None, 1e-6), ("rms", m["post"].weight, None, 1e-5)
    chunk = [mod[:, i * C:(i + 1) * C] for i in range(6)]
    _, _, o, e = residual_norm64(before[live], None, pre=layer, scale=chunk[0], shift=chunk[1], **kw)
    assert_close(a.out[live], o, e, "first norm")
    q = nv.quantize_rowwise(a.out[:n].contiguous())          # live rows come first
    assert torch.equal(a.quant.q[:n], q.q) and torch.equal(a.quant.s_dec[:n], q.s_dec)
    base = nv.gemm(a.quant, m["up"].w)
    want, err = lora64(a.out, base, m["up_ad"], slot)
    assert_close(up[live], want[live], err[live], "up")
    base = m["down"](act)
    want, err = lora64(act, base, m["down_ad"], slot)
    assert_close(down[live], want[live], err[live], "down")
    hh, eh, o, e = residual_norm64(before[live], down[live], post=rms, gate=chunk[2], pre=layer, scale=chunk[3],
                                   shift=chunk[4], branch_scale=0.5, **kw)
    assert_close(h[live], hh, eh, "stream")
    assert_close(b.out[live], o, e, "second norm")
    assert torch.equal(h[~live], before[~live])              # padding stays as it was


def test_block_in_a_graph(nv):
    """Captured once, replayed on other values and other requests in the same buffers."""
    m = _model(nv)
    rows = 300
    bufs = [t.clone() for t in _batch(m, rows, 1, torch.float32)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        _block(nv, m, *bufs)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            a, up, act, down, b = _block(nv, m, *bufs)
    torch.cuda.current_stream().wait_stream(stream)
    for seed in (2, 3):
        new = _batch(m, rows, seed, torch.float32)
        for dst, src in zip(bufs, new):
            dst.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        live = new[1] >= 0
        h = new[0].clone()
        chunk = [new[3][:, i * C:(i + 1) * C] for i in range(6)]
        e = nv.residual_norm(h, pre=m["norm"], scale=chunk[0], shift=chunk[1], row_group=new[1], **_zeros(nv, rows))
        assert torch.equal(e.out, a.out) and torch.equal(e.quant.q, a.quant.q)
        y = m["up"](e.out, xq=e.quant, adapters=m["up_ad"], row_slot=new[2])
        assert torch.equal(y[live], up[live])
        z = m["down"](torch.nn.functional.gelu(y), adapters=m["down_ad"], row_slot=new[2])
        assert torch.equal(z[live], down[live])
        f = nv.residual_norm(h, z, post=m["post"], gate=chunk[2], pre=m["norm"], scale=chunk[3], shift=chunk[4],
                             row_group=new[1], branch_scale=0.5)
        assert torch.equal(f.h[live], bufs[0][live]) and torch.equal(f.out[live], b.out[live])
