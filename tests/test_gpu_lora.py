"""Low-rank adapters of many requests beside a projection, against a plain
implementation in 64 bits."""
import pytest
import torch

from block_ops_ref import assert_close, lora64
from gpu_common import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return require_cuda()


def _inputs(nv, rows, k, n, rank, slots, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 131 * rows + 7 * k + n + rank)

    def normal(*s, std=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)

    x, y = normal(rows, k), normal(rows, n)
    ad = nv.LoraAdapters(normal(slots, rank, k, std=k ** -0.5), normal(slots, n, rank, std=rank ** -0.5),
                         torch.rand(slots, generator=g, device="cuda") * 2 - 0.5)
    slot = torch.randint(-1, slots + 1, (rows,), generator=g, device="cuda").to(torch.int32)
    return x, y, ad, slot


def _check(nv, x, y, ad, slot, **kw):
    want, err = lora64(x, y, ad, slot)
    got = nv.lora(x, y, ad, slot, **kw)
    torch.cuda.synchronize()
    code, tag = nv.device_error()
    assert code == 0, f"device wait timed out (tag {tag})"
    assert_close(got, want, err)
    if slot is not None:  # rows without an adapter: y, bit for bit
        none = (slot < 0) | (slot >= ad.scale.numel())
        assert torch.equal(got[none], y[none])
    return got


ROWS = [1, 2, 7, 33, 64, 65, 128, 129, 200, 257, 513, 1000]


@pytest.mark.parametrize("k,n", [(1040, 1544), (5008, 6152)])   # by rows and on tiles
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("rank", [16, 32, 48, 64, 80, 96, 112, 128])
def test_rows_and_ranks(nv, rows, rank, k, n):
    x, y, ad, slot = _inputs(nv, rows, k, n, rank, 5)
    _check(nv, x, y, ad, slot)                              # any order
    _check(nv, x, y, ad, slot.sort().values.contiguous())   # requests in a row
    _check(nv, x, y, ad, None)                              # one adapter for all


@pytest.mark.parametrize("rows", [1, 100, 260, 300])
@pytest.mark.parametrize("k,n", [(16, 16), (16, 4096), (4096, 16), (48, 24), (64, 64), (80, 72), (112, 1000),
                                 (4112, 264), (12288, 4096), (2048, 12296)])
def test_shapes(nv, rows, k, n):
    _check(nv, *_inputs(nv, rows, k, n, 32, 3))


@pytest.mark.parametrize("rows,slots", [(70, 70), (256, 256), (300, 41), (500, 64)])
def test_an_adapter_for_every_row(nv, rows, slots):
    x, y, ad, _ = _inputs(nv, rows, 512, 640, 16, slots)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    slot = torch.randperm(max(rows, slots), generator=g, device="cuda")[:rows].remainder(slots).to(torch.int32)
    _check(nv, x, y, ad, slot)


@pytest.mark.parametrize("rank", [16, 80])
@pytest.mark.parametrize("in_place", [False, True])
def test_crowded_tiles_beside_others(nv, rank, in_place):
    """Tiles of many adapters, of one, of a few and of none in one call."""
    rows, slots = 640, 100
    x, y, ad, _ = _inputs(nv, rows, 1024, 2056, rank, slots)
    slot = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    slot[:100] = torch.arange(100, device="cuda", dtype=torch.int32)   # and 28 rows without
    slot[128:256] = 7
    slot[384:520] = torch.arange(136, device="cuda", dtype=torch.int32) // 40
    slot[520:] = torch.arange(120, device="cuda", dtype=torch.int32).flip(0) % slots
    _check(nv, x, y, ad, slot)
    if in_place:
        want, err = lora64(x, y, ad, slot)
        assert_close(nv.lora(x, y, ad, slot, out=y), want, err)


@pytest.mark.parametrize("rank", [16, 80])
@pytest.mark.parametrize("in_place", [False, True])
def test_tiles_of_unlike_cost(nv, rank, in_place):
    """Many columns and few row tiles, whose shares are weighed by their adapters:
    tiles of one, of several, of none, in any order, and a short last one."""
    rows, n, slots = 3000, 12296, 6
    x, y, ad, any_order = _inputs(nv, rows, 192, n, rank, slots)
    ragged = torch.full((rows,), 3, dtype=torch.int32, device="cuda")
    ragged[100:900] = -1                      # six whole tiles without an adapter
    ragged[900:1500] = torch.arange(600, device="cuda", dtype=torch.int32) // 50 % 6
    ragged[2500:] = 5
    none_at_ends = ragged.clone()
    none_at_ends[:1024], none_at_ends[-300:] = -1, slots
    for slot in (ragged, none_at_ends, any_order):
        want, err = lora64(x, y, ad, slot)
        out = y.clone() if in_place else torch.full_like(y, float("nan"))
        nv.lora(x, out if in_place else y, ad, slot, out=out)
        torch.cuda.synchronize()
        code, tag = nv.device_error()
        assert code == 0, f"device wait timed out (tag {tag})"
        assert_close(out, want, err)


@pytest.mark.parametrize("rank,slots,k", [(16, 40, 1040), (48, 21, 4112), (112, 7, 4096), (128, 13, 2048)])
@pytest.mark.parametrize("rows", [92, 252, 700])
def test_many_adapters_in_few_tiles(nv, rows, rank, slots, k):
    """Row tiles whose adapters are dealt out to several clusters: more and fewer
    adapters than clusters, tiles with one or none, contiguous and in any order."""
    n = 1032
    x, y, ad, any_order = _inputs(nv, rows, k, n, rank, slots)
    at = torch.arange(rows, device="cuda", dtype=torch.int32)
    runs = at * slots // rows
    one = torch.where(at < rows // 2, -1, slots - 1).to(torch.int32)
    for slot in (runs, one, any_order):
        want, err = lora64(x, y, ad, slot)
        out = torch.full_like(y, float("nan"))
        nv.lora(x, y, ad, slot, out=out)
        torch.cuda.synchronize()
        code, tag = nv.device_error()
        assert code == 0, f"device wait timed out (tag {tag})"
        assert_close(out, want, err)


@pytest.mark.parametrize("rows", [3, 300])
def test_no_row_has_an_adapter(nv, rows):
    x, y, ad, slot = _inputs(nv, rows, 256, 512, 16, 2)
    for v in (-1, 2, 2 ** 31 - 1, -2 ** 31):
        assert torch.equal(nv.lora(x, y, ad, torch.full_like(slot, v)), y)


@pytest.mark.parametrize("rows", [5, 150, 700])
def test_in_place_and_strided(nv, rows):
    k, n = 528, 392
    x, y, ad, slot = _inputs(nv, rows, k, n, 48, 4)
    want, err = lora64(x, y, ad, slot)
    wide_x = torch.full((rows, k + 40), 2.0, dtype=torch.bfloat16, device="cuda")
    wide_y = torch.full((rows, n + 96), 3.0, dtype=torch.bfloat16, device="cuda")
    wide_x[:, 16:16 + k], wide_y[:, 64:64 + n] = x, y
    ys = wide_y[:, 64:64 + n]
    got = nv.lora(wide_x[:, 16:16 + k], ys, ad, slot, out=ys)
    assert got is ys
    assert_close(ys, want, err)
    assert (wide_y[:, :64] == 3.0).all() and (wide_y[:, 64 + n:] == 3.0).all()


@pytest.mark.parametrize("rows", [6, 140, 600])
def test_non_finite_values_stay_in_their_rows(nv, rows):
    """An adapter of infinities and NaN, and rows of them, reach no other row."""
    x, y, ad, slot = _inputs(nv, rows, 320, 256, 32, 4)
    slot = torch.arange(rows, device="cuda").remainder(4).to(torch.int32)
    clean = nv.lora(x, y, ad, slot)
    ad.a[1, 3], ad.b[1, :, 5] = float("inf"), float("nan")
    x[2], y[3] = float("nan"), float("inf")
    got = nv.lora(x, y, ad, slot)
    fine = (slot != 1)
    fine[2] = fine[3] = False
    assert torch.equal(got[fine], clean[fine])
    assert got[slot == 1].isnan().all()


@pytest.mark.parametrize("rows", [1, 9, 300])
def test_same_bits_every_time(nv, rows):
    x, y, ad, slot = _inputs(nv, rows, 2048, 1024, 64, 3)
    first = nv.lora(x, y, ad, slot)
    for _ in range(3):
        assert torch.equal(nv.lora(x, y, ad, slot), first)


def test_offsets_past_32_bits(nv):
    rows, stride = 270, 1 << 23
    x, y, ad, slot = _inputs(nv, rows, 256, 512, 16, 2)
    want, err = lora64(x, y, ad, slot)
    far = torch.empty(rows * stride, dtype=torch.bfloat16, device="cuda").view(rows, stride)
    far[:, :256], far[:, 1024:1536] = x, y
    got = nv.lora(far[:, :256], far[:, 1024:1536], ad, slot, out=far[:, 1024:1536])
    assert_close(got, want, err)


@pytest.mark.parametrize("rows", [0, 4, 400])
def test_empty_streams_and_graph(nv, rows):
    x, y, ad, slot = _inputs(nv, rows, 512, 768, 32, 3)
    want = nv.lora(x, y, ad, slot)
    assert want.shape == (rows, 768)
    if rows == 0:
        return
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    a.wait_stream(torch.cuda.current_stream())
    b.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(8):      # two at a time, each with a workspace of its own
        for s in (a, b):
            with torch.cuda.stream(s):
                outs.append(nv.lora(x, y, ad, slot))
    outs.append(nv.lora(x, y, ad, slot, stream=a))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    x_in, y_in = torch.zeros_like(x), torch.zeros_like(y)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    res = []
    for g in graphs:
        with torch.cuda.graph(g):
            res.append(nv.lora(x_in, y_in, ad, slot))
    x_in.copy_(x)
    y_in.copy_(y)
    for g, s in zip(graphs, (a, b)):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g.replay()
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(res[0], want) and torch.equal(res[1], want)


def test_pack_adapters(nv):
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    parts = [(torch.randn(r, 64, generator=g, device="cuda").to(torch.bfloat16),
              torch.randn(80, r, generator=g, device="cuda").to(torch.bfloat16), 0.5 * r) for r in (4, 17, 1)]
    ad = nv.pack_adapters(parts)
    assert ad.a.shape == (3, 32, 64) and ad.b.shape == (3, 80, 32)
    x = torch.randn(9, 64, generator=g, device="cuda").to(torch.bfloat16)
    y = torch.zeros(9, 80, dtype=torch.bfloat16, device="cuda")
    slot = torch.tensor([0, 1, 2] * 3, dtype=torch.int32, device="cuda")
    got = _check(nv, x, y, ad, slot)
    for i, (a, b, s) in enumerate(parts):
        ref = s * (x[i::3].double() @ a.double().T @ b.double().T)
        assert float((got[i::3].double() - ref).norm() / ref.norm()) < 2.0 ** -8


def test_beside_the_layers(nv):
    """A request's adapters through NVFP4Linear, FP8Linear and the sharded
    layer: the layer's own output with lora added to it."""
    from nvfp4_block_scaled_19_b200.sharded import ShardedNVFP4Linear
    x, _, ad, slot = _inputs(nv, 300, 512, 768, 32, 3)
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    w = (torch.randn(768, 512, generator=g, device="cuda") * 512 ** -0.5).to(torch.bfloat16)
    for layer in (nv.NVFP4Linear(w), nv.FP8Linear(w), ShardedNVFP4Linear(w)):
        base = layer(x)
        got = layer(x, adapters=ad, row_slot=slot)
        assert torch.equal(got, nv.lora(x, base, ad, slot))
        assert not torch.equal(got, base)
    lin = nv.NVFP4Linear(w)
    fq = nv.FusedQuant(torch.ones(1, device="cuda"), nv.empty_nvfp4(300, 768), None)
    for kw in (dict(fused=fq), dict(want_y=False)):
        with pytest.raises(ValueError):
            lin(x, adapters=ad, row_slot=slot, **kw)
    with pytest.raises(ValueError):
        lin(x, row_slot=slot)
    with pytest.raises(ValueError):
        lin(None, xq=nv.quantize_rowwise(x), adapters=ad, row_slot=slot)


def test_refusals(nv):
    x, y, ad, slot = _inputs(nv, 4, 64, 80, 16, 2)
    L = nv.LoraAdapters
    bad = [
        (x.half(), y, ad, slot), (x, y.float(), ad, slot), (x[:3], y, ad, slot), (x[:, :48], y, ad, slot),
        (x, y[:, :64], ad, slot), (x, y.cpu(), ad, slot), (x, y, ad, slot.long()), (x, y, ad, slot[:3]),
        (x, y, ad, slot.cpu()), (x, y, L(ad.a[0], ad.b, ad.scale), slot),
        (x, y, L(ad.a, ad.b[:1], ad.scale), slot), (x, y, L(ad.a, ad.b, ad.scale[:1]), slot),
        (x, y, L(ad.a.float(), ad.b, ad.scale), slot), (x, y, L(ad.a, ad.b, ad.scale.double()), slot),
        (x, y, L(ad.a.transpose(1, 2), ad.b.transpose(1, 2), ad.scale), slot),
    ]
    for args in bad:
        with pytest.raises(ValueError):
            nv.lora(*args)
    with pytest.raises(ValueError):
        nv.lora(x, y, ad, slot, out=y.t().contiguous().t())

    def z(*s):
        return torch.zeros(*s, dtype=torch.bfloat16, device="cuda")

    one = torch.ones(1, device="cuda")
    for rank, k, n in ((8, 64, 80), (144, 64, 80), (24, 64, 80), (16, 72, 80), (16, 64, 84)):
        with pytest.raises(nv.NVFP4Error) as e:
            nv.lora(z(4, k), z(4, n), L(z(1, rank, k), z(1, n, rank), one))
        assert e.value.status == 1
    with pytest.raises(nv.NVFP4Error) as e:      # x and out are one tensor
        sq = z(4, 64)
        nv.lora(sq, z(4, 64), L(z(1, 16, 64), z(1, 64, 16), one), out=sq)
    assert e.value.status == 1
    with pytest.raises(nv.NVFP4Error) as e:      # not 16-byte aligned
        nv.lora(z(4, 128)[:, 4:68], y, ad, slot)
    assert e.value.status == 2
    for parts in ([], [(z(200, 64), z(80, 200), 1.0)], [(z(8, 64), z(80, 4), 1.0)],
                  [(z(8, 64), z(80, 8), 1.0), (z(8, 48), z(80, 8), 1.0)]):
        with pytest.raises(ValueError):
            nv.pack_adapters(parts)
