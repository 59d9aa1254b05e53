"""Infinities in an adapter or in x: the row by itself and the tile kernels give the
infinities and NaN of the formula, and what is finite stays within its bounds."""
import pytest
import torch

from block_ops_ref import assert_close, lora64
from gpu_common import require_cuda

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module")
def nv():
    return require_cuda()


def _inputs(nv, rows, rank, k=512, n=256, slots=3):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + rank)

    def normal(*s, std=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)

    ad = nv.LoraAdapters(normal(slots, rank, k, std=k ** -0.5), normal(slots, n, rank, std=rank ** -0.5),
                         torch.tensor([1.0, -0.75, 0.5], device="cuda"))
    slot = torch.randint(-1, slots, (rows,), generator=g, device="cuda").to(torch.int32)
    return normal(rows, k), normal(rows, n), ad, slot


def _check(nv, x, y, ad, slot):
    got = nv.lora(x, y, ad, slot)
    torch.cuda.synchronize()
    assert nv.device_error() == (0, 0)
    want = y.double()
    for s in range(ad.scale.numel()):
        rows = torch.nonzero(slot == s).reshape(-1)
        # t as its fp32 sum: exact products, whatever the order 2^-17 of their magnitudes.
        xd, a = x[rows].double(), ad.a[s].double()
        t = ad.scale[s].double() * torch.einsum("mk,rk->mr", xd, a)
        want[rows] += (t.unsqueeze(1) * ad.b[s].double().unsqueeze(0)).sum(-1)
    fine = want.isfinite()
    clean = nv.LoraAdapters(*(torch.where(v.isfinite(), v, torch.zeros_like(v)) for v in (ad.a, ad.b, ad.scale)))
    _, err = lora64(torch.where(x.isfinite(), x, torch.zeros_like(x)), y, clean, slot)
    assert_close(got[fine], want[fine], err[fine])
    assert torch.equal(got[~fine].float().nan_to_num(nan=7.0, posinf=8.0, neginf=9.0),
                       want[~fine].float().nan_to_num(nan=7.0, posinf=8.0, neginf=9.0))
    return got, want


@pytest.mark.parametrize("rank", [16, 48, 64, 128])
@pytest.mark.parametrize("rows", [7, 300, 1500])       # row by row; tiles of several adapters
def test_infinite_entries_of_b(nv, rows, rank):
    x, y, ad, slot = _inputs(nv, rows, rank)
    for col, r in ((0, 0), (9, 3), (64, rank - 1), (255, rank // 2)):
        ad.b[0, col, r] = INF
        ad.b[1, col, r] = -INF
    got, want = _check(nv, x, y, ad, slot)
    hit = (slot == 0) | (slot == 1)
    assert want[hit][:, [0, 9, 64, 255]].isinf().all()     # an infinity, not a NaN


@pytest.mark.parametrize("rows", [7, 300, 1500])
def test_inner_vectors_of_few_bits(nv, rows):
    """t of one to eight bits, whose rest is zero, and t = 0 (times infinity: NaN)."""
    x, y, ad, _ = _inputs(nv, rows, 16)
    x.zero_()
    at = torch.arange(rows, device="cuda")
    x[at, at % 256] = 1.0
    value = torch.arange(256, device="cuda") - 128.0       # 0 among them
    ad.a[:] = 0
    ad.a[:, 0, :256] = value.to(torch.bfloat16)
    ad.a[:, 1, :] = 1.0
    ad.scale.fill_(1.0)
    ad.b[0, 5, 0] = INF
    ad.b[0, 6, 1] = -INF
    ad.b[0, 7, 2] = INF                                    # t is 0 there
    got, want = _check(nv, x, y, ad, torch.zeros(rows, dtype=torch.int32, device="cuda"))
    assert want[:, 7].isnan().all()


@pytest.mark.parametrize("rank", [16, 80])
@pytest.mark.parametrize("rows", [7, 300, 1500])
def test_infinite_inner_vectors(nv, rows, rank):
    """Infinite entries of A and of x: t is infinite, B finite, infinite or zero."""
    x, y, ad, slot = _inputs(nv, rows, rank)
    ad.a[0, 2, 7] = INF
    ad.b[0, 3], ad.b[0, 4, 2], ad.b[0, 5, 2] = 0.0, INF, -INF
    ad.a[1, 1:] = 0.0                                      # of rank 1, padded with zeros
    x[::5, 11] = -INF
    _check(nv, x, y, ad, slot)


@pytest.mark.parametrize("rows", [7, 300])
def test_the_largest_finite_inner_vectors(nv, rows):
    """t above the largest bf16 value, below fp32's: still finite."""
    x, y, ad, _ = _inputs(nv, rows, 16)
    x.zero_()
    x[:, 0], x[:, 1] = 2.0 ** 100, 2.0 ** 100
    ad.a[:] = 0
    ad.a[:, 0, 0], ad.a[:, 0, 1] = 255 * 2.0 ** 20, 7 * 2.0 ** 17         # t = 2^128 (1 - 2^-11)
    ad.scale.fill_(1.0)
    ad.b[:] = 0
    ad.b[:, :, 0] = 2.0 ** -120
    got, want = _check(nv, x, y, ad, torch.zeros(rows, dtype=torch.int32, device="cuda"))
    assert want.isfinite().all()
