"""The codes that residual_norm writes are quantize_rowwise's of its bf16 result,
bit for bit, for every block maximum and for results that are not finite, whichever
kernel the number of rows selects.  A row of zeros has out = shift, so that shift
puts any value there."""
import pytest
import torch

from gpu_common import require_cuda

pytestmark = pytest.mark.gpu

COLS = 8192


@pytest.fixture(scope="module")
def nv():
    return require_cuda()


def _check(nv, shift, rows):
    groups, cols = shift.shape
    zero = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    group = torch.arange(rows, device="cuda").remainder(groups).to(torch.int32)
    amax = torch.empty(rows, device="cuda")
    r = nv.residual_norm(zero, zero, pre=nv.Norm("rms"), shift=shift, row_group=group, want_quant=True,
                         amax_rows=amax)
    torch.cuda.synchronize()
    assert nv.device_error() == (0, 0)
    want = torch.where(shift == 0, torch.zeros_like(shift), shift)[group.long()]    # 0 + -0 = 0
    bits = torch.where(want.isnan(), 0x7FFF, want.view(torch.int16))    # arithmetic has one NaN
    assert torch.equal(r.out.view(torch.int16), bits.to(torch.int16))
    want_amax = torch.empty_like(amax)
    q = nv.quantize_rowwise(r.out, amax_rows=want_amax)
    for got, ref in ((r.quant.q, q.q), (r.quant.sf, q.sf), (r.quant.s_dec.view(torch.int32), q.s_dec.view(torch.int32)),
                     (amax.view(torch.int32), want_amax.view(torch.int32))):
        assert torch.equal(got, ref)


def _every_block_maximum():
    """One block of 16 per finite bf16 magnitude, in [64, 8192]: each row's largest
    value is within a factor of 16 of its smallest."""
    bits = torch.arange(0x7F80 // 510 * 510 + 510, device="cuda").clamp(max=0x7F7F).reshape(-1, 510)
    top = bits.to(torch.int16).view(torch.bfloat16)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rest = torch.rand(*top.shape, 16, generator=g, device="cuda") * 2 - 1
    v = (top.float().unsqueeze(-1) * rest).to(torch.bfloat16)
    v[:, :, 5] = top
    pad = torch.zeros(top.shape[0], 2, 16, dtype=torch.bfloat16, device="cuda")
    return torch.cat((v, pad), 1).reshape(top.shape[0], COLS)


@pytest.mark.parametrize("rows", [65, 260])     # a CTA per row; persistent CTAs
def test_every_block_maximum(nv, rows):
    shift = _every_block_maximum()
    assert shift.shape == (65, COLS)
    _check(nv, shift, rows)
    far = shift.clone()                          # the same blocks beside a much larger one
    far[:, -1] = 3.0e38
    _check(nv, far, rows)


@pytest.mark.parametrize("cols,few,many", [(256, 40, 40), (1040, 40, 5000), (4096, 40, 1000), (COLS, 40, 400),
                                           (8208, 40, 400)])
@pytest.mark.parametrize("bad", ["inf", "-inf", "nan", "both", "all", "overflow"])
def test_results_that_are_not_finite(nv, cols, few, many, bad):
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    shift = torch.randn(8, cols, generator=g, device="cuda").to(torch.bfloat16)
    inf, nan = float("inf"), float("nan")
    if bad == "both":
        shift[:, 3], shift[:, 18], shift[:, 20], shift[:, cols - 1] = inf, nan, inf, -inf
    elif bad == "all":
        shift[::2], shift[1::2] = inf, nan
    elif bad == "overflow":
        shift[:, ::37] = 3.3895e38               # the largest finite value
    else:
        for i in range(8):                       # every lane pair, both vectors of a thread
            shift[i, 16 * i + i] = shift[i, (cols // 2 + 24 * i) % cols] = float(bad)
    for rows in (few, many):
        _check(nv, shift, rows)
