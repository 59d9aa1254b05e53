"""Tensors that a call with stream= makes belong to that stream, so that neither
work queued on another one nor an early release can share their memory."""
import pytest
import torch

from gpu_common import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return require_cuda()


def _stream_of(t):
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not memory of the allocator")


ROWS, COLS = 640, 1024


def _made(nv, name, s):
    """The tensors that a call makes on stream s."""
    x = torch.randn(ROWS, COLS, device="cuda").to(torch.bfloat16)
    q, q8 = nv.quantize_dynamic(x), nv.quantize_fp8(x)
    one = torch.ones(1, device="cuda")
    ad = nv.LoraAdapters(x[:16].reshape(1, 16, COLS).contiguous(), torch.ones(1, COLS, 16, device="cuda").bfloat16(), one)
    s.wait_stream(torch.cuda.current_stream())
    if name == "residual_norm":
        r = nv.residual_norm(x, x, pre=nv.Norm(), want_quant=True, stream=s)
        made = [r.h, r.out, r.quant.q, r.quant.sf, r.quant.s_dec]
    elif name == "lora":
        made = [nv.lora(x, x, ad, stream=s)]
    elif name == "tensor_amax":
        made = [nv.tensor_amax(x, stream=s)]
    elif name == "gemm":
        made = [nv.gemm(q, q, stream=s)]
    elif name == "gemm_fp8":
        made = [nv.gemm_fp8(q8, q8, stream=s)]
    elif name == "quantize_fp8":
        t = nv.quantize_fp8(x, stream=s)
        made = [t.q, t.s_dec]
    else:
        call = {"quantize": lambda: nv.quantize(x, one, stream=s),
                "quantize_with_scale": lambda: nv.quantize_with_scale(x, one, stream=s),
                "quantize_one_pass": lambda: nv.quantize_one_pass(x, one, one.clone(), stream=s),
                "quantize_dynamic": lambda: nv.quantize_dynamic(x, stream=s),
                "quantize_rowwise": lambda: nv.quantize_rowwise(x, stream=s)}[name]
        t = call()
        made = [t.q, t.sf, t.s_dec]
    torch.cuda.synchronize()
    return made


@pytest.mark.parametrize("name", ["residual_norm", "lora", "tensor_amax", "quantize", "quantize_with_scale",
                                  "quantize_one_pass", "quantize_dynamic", "quantize_rowwise", "quantize_fp8",
                                  "gemm", "gemm_fp8"])
def test_results_belong_to_the_given_stream(nv, name):
    s = torch.cuda.Stream()
    for t in _made(nv, name, s):
        assert _stream_of(t) == s.cuda_stream


@pytest.mark.parametrize("name", ["residual_norm", "lora", "gemm"])
def test_memory_in_use_is_not_given_out(nv, name):
    """A result that the current stream still reads is dropped: the given stream
    gets other memory until that read is done."""
    s = torch.cuda.Stream()
    made = _made(nv, name, s)
    t = made[0]
    at, size = t.data_ptr(), t.numel() * t.element_size()
    torch.cuda._sleep(200_000_000)      # the current stream is busy, then reads t
    keep = t.clone()
    del made, t
    with torch.cuda.stream(s):
        others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert at not in [o.data_ptr() for o in others]
    torch.cuda.synchronize()
    assert keep.shape[0] == ROWS


def test_results_on_a_stream_equal_those_on_the_current_one(nv):
    x = torch.randn(ROWS, COLS, device="cuda").to(torch.bfloat16)
    y = torch.randn(ROWS, COLS, device="cuda").to(torch.bfloat16)
    want = nv.residual_norm(x, y, pre=nv.Norm("layer"), want_quant=True)
    w = nv.quantize_dynamic(x)
    want_y = nv.gemm(want.quant, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        r = nv.residual_norm(x, y, pre=nv.Norm("layer"), want_quant=True, stream=s)
        got = nv.gemm(r.quant, w, stream=s)
        h, out = r.h, r.out
        del r                                  # the codes, while the products may still run
        junk = [torch.full((ROWS, COLS), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(h, want.h) and torch.equal(out, want.out) and torch.equal(got, want_y)
        del junk


def test_the_sharded_amax_is_reduced_on_the_given_stream(nv, monkeypatch):
    from nvfp4_block_scaled_19_b200 import sharded
    x = torch.randn(ROWS, COLS, device="cuda").to(torch.bfloat16)
    want = sharded.quantize_sharded(x)
    seen = []
    reduce = sharded.all_reduce_max
    monkeypatch.setattr(sharded, "all_reduce_max",
                        lambda t, group=None: (seen.append(torch.cuda.current_stream()), reduce(t, group))[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sharded.quantize_sharded(x, stream=s)
    sharded.quantize_sharded(x)
    torch.cuda.synchronize()
    assert seen == [s, torch.cuda.current_stream()]
    assert torch.equal(got.q, want.q) and torch.equal(got.sf, want.sf) and torch.equal(got.s_dec, want.s_dec)


def test_a_stream_forked_inside_a_capture(nv):
    """Results made on a side stream of a captured region, some dropped at once."""
    x = torch.randn(ROWS, COLS, device="cuda").to(torch.bfloat16)
    y = torch.randn(ROWS, COLS, device="cuda").to(torch.bfloat16)
    w = nv.quantize_dynamic(x)
    ad = nv.LoraAdapters(torch.randn(2, 16, COLS, device="cuda").to(torch.bfloat16),
                         torch.randn(2, ROWS, 16, device="cuda").to(torch.bfloat16), torch.ones(2, device="cuda"))

    def chain(a, b, stream=None):
        r = nv.residual_norm(a, b, pre=nv.Norm("layer"), want_quant=True, stream=stream)
        p = nv.gemm(r.quant, w, stream=stream)
        return r.h, nv.lora(r.out, p, ad, stream=stream)

    x_in, y_in, side = torch.zeros_like(x), torch.zeros_like(y), torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        h, out = chain(x_in, y_in, side)
        torch.cuda.current_stream().wait_stream(side)
        h2 = h * 2
    for a, b in ((x, y), (y, x)):
        x_in.copy_(a)
        y_in.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        want_h, want = chain(a, b)
        assert torch.equal(h, want_h) and torch.equal(h2, want_h * 2) and torch.equal(out, want)
    assert nv.device_error() == (0, 0)
