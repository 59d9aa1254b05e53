"""Workloads of the operators around an NVFP4 projection: the norms before and
after a block with its gate and residual scale (bf16 out, or NVFP4 codes that
feed a projection), and the low-rank adapters of many requests beside a
projection.

own = False runs each operator in its plain form, elementary torch operations
in 32 bits rounded once at the end; own = True makes the calls that a user of
the package makes.  exact() is the definition in 64 bits.

Definitions, per token row (g: the row's request, s: the row's adapter):
    norm         h = a r + c gate[g] * post(y),  out = pre(h) * (1 + scale[g]) + shift[g]
                 with post and pre none, RMS or layer norms
    norm_linear  the same out in bf16, quantized to NVFP4 with one scale per
                 row (2688 / amax), times a weight held in NVFP4
    lora         out = y + c[s] (x A[s]^T) B[s]^T, out = y for a row without adapter
"""
import math
import random

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    norm = dict(op="norm", post="none", gate=False, pre="rms", weight=True, modulate=False, groups=1,
                residual_scale=1.0, stream="bf16")
    dit = dict(norm, pre="layer", weight=False, gate=True, modulate=True, groups=2)
    lora = dict(op="lora")
    return [
        # One token of a language model: residual add and the next RMS norm.
        dict(norm, name="norm_decode_1", rows=1, cols=4096),
        # A decoding batch of several requests, norms on both sides of the
        # block, the residual stream kept in fp32.
        dict(norm, name="norm_batch_93", rows=93, cols=5120, post="rms", gate=True, modulate=True,
             groups=7, stream="f32"),
        # A diffusion transformer's adaptive layer norm, two images of odd sizes.
        dict(dit, name="norm_dit_4571", rows=4571, cols=2560),
        # The same at 2048^2 with a guidance batch of two.
        dict(dit, name="norm_dit_33792", rows=33792, cols=4096),
        # Prefill of a deep model: sandwich norms, scaled fp32 residual stream.
        dict(norm, name="norm_prefill_8192", rows=8192, cols=8192, post="rms", stream="f32",
             residual_scale=0.75),
        # Norm straight into the codes of an NVFP4 projection: a decoding batch,
        dict(norm, name="norm_linear_24", op="norm_linear", rows=24, cols=2048, n=6144),
        # and the 1024^2 diffusion step (4096 image + 512 text tokens).
        dict(dit, name="norm_linear_4608", op="norm_linear", rows=4608, cols=4096, n=12288, groups=1),
        # Adapters: one decoding token,
        dict(lora, name="lora_decode_1", rows=1, k=4096, n=4096, rank=16, slots=8, mix="each"),
        # a decoding batch in which every request brings its own adapter,
        dict(lora, name="lora_decode_61", rows=61, k=4096, n=12288, rank=32, slots=64, mix="each"),
        # the prefill of six requests of ragged lengths, one without adapter,
        dict(lora, name="lora_prefill_1337", rows=1337, k=5120, n=5120, rank=64, slots=6, mix="runs"),
        # an FFN up-projection at 2048^2 with the styles of two images,
        dict(lora, name="lora_up_16896", rows=16896, k=4096, n=12288, rank=16, slots=2, mix="runs"),
        # and a wide adapter beside a down-projection at 1024^2.
        dict(lora, name="lora_down_4608", rows=4608, k=12288, n=4096, rank=128, slots=3, mix="runs"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_linear", "lora", "lora"])
    if op == "lora":
        rank = 16 * rng.randint(1, 8)
        slots = rng.randint(1, min(64, 2048 // rank))
        k = 16 * _log_int(rng, 32, 768)
        n = 8 * _log_int(rng, 64, 1536)
        most = 16896 * (4096 + 2 * 12288) // (k + 2 * n)
        rows = _log_int(rng, 1, min(16896, most))
        return dict(op=op, rows=rows, k=k, n=n, rank=rank, slots=slots,
                    mix="each" if rows <= 128 and rng.random() < 0.7 else "runs")
    case = dict(op=op, post=rng.choice(["none", "rms", "layer"]), gate=rng.random() < 0.5,
                pre=rng.choice(["rms", "layer"]), weight=rng.random() < 0.5, modulate=rng.random() < 0.5,
                residual_scale=rng.choice([1.0, 0.5, 1.5]), stream=rng.choice(["bf16", "f32"]))
    if op == "norm":
        cols = 16 * _log_int(rng, 16, 512)
        most = 33792 * 4096 * 8 // (cols * (12 if case["stream"] == "f32" else 8))
        rows = _log_int(rng, 1, min(33792, most * 63 // 64))
    else:
        cols = 64 * _log_int(rng, 8, 64)
        rows = _log_int(rng, 1, 4608)
        case["n"] = 8 * _log_int(rng, 64, 1536)
    case.update(rows=rows, cols=cols, groups=rng.randint(1, min(8, rows)))
    return case


def _cuts(case, parts):
    """Ragged lengths of `parts` consecutive requests that fill the rows."""
    rows = case["rows"]
    rng = random.Random(str(sorted((k, str(v)) for k, v in case.items() if k != "name")))
    cuts = [0] + sorted(rng.randint(0, rows) for _ in range(parts - 1)) + [rows]
    return [b - a for a, b in zip(cuts, cuts[1:])], rng


def _slots(case):
    """The adapter of each row (-1: none): a slot of its own for each row, or
    one for each of `slots` consecutive requests, the last of several without."""
    if case["mix"] == "each":
        rng = _cuts(case, 1)[1]
        order = list(range(case["slots"]))
        rng.shuffle(order)
        return [order[i % len(order)] for i in range(case["rows"])]
    lengths, _ = _cuts(case, case["slots"])
    last = len(lengths) - 1
    return [-1 if last > 2 and i == last else i for i, n in enumerate(lengths) for _ in range(n)]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev).mul_(std).add_(mean).to(dtype)

    if case["op"] == "lora":
        m, k, n, r, s = (case[x] for x in ("rows", "k", "n", "rank", "slots"))
        channels = torch.exp(0.5 * torch.randn(k, generator=g, device=dev))
        x = torch.randn(m, k, generator=g, device=dev).mul_(channels).to(torch.bfloat16)
        return dict(case=case, x=x, y=normal(m, n), a=normal(s, r, k, std=k ** -0.5),
                    b=normal(s, n, r, std=0.3 * r ** -0.5),
                    scale=torch.rand(s, generator=g, device=dev) + 0.5,
                    row_slot=torch.tensor(_slots(case), dtype=torch.int32, device=dev),
                    out=torch.empty(m, n, dtype=torch.bfloat16, device=dev))

    m, c, groups = case["rows"], case["cols"], case["groups"]
    stream = torch.float32 if case["stream"] == "f32" else torch.bfloat16
    lengths, _ = _cuts(case, groups)
    # A block's six modulation vectors come from one projection, as its chunks.
    mod = normal(groups, 6 * c, std=0.3)
    s = dict(case=case, residual=normal(m, c, std=2.0, mean=0.1, dtype=stream),
             y=normal(m, c, std=1.5, mean=-0.2),
             gate=mod[:, 2 * c:3 * c] if case["gate"] else None,
             shift=mod[:, 3 * c:4 * c] if case["modulate"] else None,
             scale=mod[:, 4 * c:5 * c] if case["modulate"] else None,
             row_group=torch.tensor([i for i, n in enumerate(lengths) for _ in range(n)],
                                    dtype=torch.int32, device=dev),
             h=torch.empty(m, c, dtype=stream, device=dev))
    for name in ("post", "pre"):
        s[name + "_weight"] = normal(c, std=0.2, mean=1.0) if case["weight"] else None
        s[name + "_bias"] = normal(c, std=0.1) if case["weight"] and case[name] == "layer" else None
    if case["op"] == "norm":
        s["out"] = torch.empty(m, c, dtype=torch.bfloat16, device=dev)
    else:
        n = case["n"]
        w = normal(n, c, std=c ** -0.5).float()
        codes, sf, s_dec = _nvfp4(w, w.abs().max())
        s.update(w_q=codes[:, 0::2] | (codes[:, 1::2] << 4), w_sf=_tiled(sf), w_s_dec=s_dec.reshape(1))
    return s


# ------------------------------------------------------------------ plain form

def _norm(x, kind, weight, bias):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    if weight is not None:
        x = x * weight.float()
    return x if bias is None else x + bias.float()


def _stream_and_norm(s):
    case = s["case"]
    g = s["row_group"].long()
    z = s["y"].float()
    if case["post"] != "none":
        z = _norm(z, case["post"], s["post_weight"], s["post_bias"])
    if s["gate"] is not None:
        z = z * s["gate"].float()[g]
    h = case["residual_scale"] * s["residual"].float() + z
    n = _norm(h, case["pre"], s["pre_weight"], s["pre_bias"])
    if s["scale"] is not None:
        n = n * (1.0 + s["scale"].float()[g]) + s["shift"].float()[g]
    return h.to(s["residual"].dtype), n.to(torch.bfloat16)


def _nvfp4(x, amax):
    """E2M1 codes, E4M3 block scales (bytes) and the decode scale of fp32 x with
    the tensor (or row) scale 2688 / amax."""
    # Divisions of two tensors, or in 64 bits: one by a Python number is a product with its reciprocal.
    one = torch.ones_like(amax)
    s_enc = torch.where(amax == 0, one, (2688.0 * one) / amax).clamp(max=torch.finfo(torch.float32).max)
    blocks = x.reshape(x.shape[0], -1, 16)
    wide = s_enc.reshape(-1, 1)
    sixth = (blocks.abs().amax(-1).double() / 6.0).float()
    sf = (sixth * wide).clamp(max=448.0).to(torch.float8_e4m3fn)
    value = sf.float()
    inv = torch.where(value == 0, torch.zeros_like(value),
                      (wide / value).clamp(max=torch.finfo(torch.float32).max))
    t = blocks * inv.unsqueeze(-1)
    a = t.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return (code + 8 * torch.signbit(t)).to(torch.uint8).reshape(x.shape), sf.view(torch.uint8), one / s_enc


def _tiled(sf):
    """Row-major block scales in 128-row x 4-block tiles of 512 bytes, zero padded."""
    r, kb = sf.shape
    full = torch.zeros(-(-r // 128) * 128, -(-kb // 4) * 4, dtype=torch.uint8, device=sf.device)
    full[:r, :kb] = sf
    return full.reshape(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _untiled(sf, r, kb):
    kb4 = -(-kb // 4)
    return sf.reshape(-1, kb4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, 4 * kb4)[:r, :kb]


def _values(codes, sf):
    """fp32 values of E2M1 codes times their block scales."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    v = table[(codes & 7).long()] * (1.0 - 2.0 * (codes >> 3).float())
    return (v.reshape(codes.shape[0], -1, 16) * sf.view(torch.float8_e4m3fn).float().unsqueeze(-1)).reshape(codes.shape)


def _plain(s):
    case = s["case"]
    if case["op"] == "lora":
        m, (slots, r, k) = case["rows"], s["a"].shape
        slot = s["row_slot"].long()
        # Every adapter's product, of which each row keeps its own.
        mine = slot.unsqueeze(1) == torch.arange(slots, device=slot.device)
        t = (s["x"].float() @ s["a"].float().reshape(slots * r, k).T).reshape(m, slots, r)
        t = torch.where(mine.unsqueeze(-1), t * s["scale"].reshape(1, -1, 1), torch.zeros_like(t))
        d = t.reshape(m, slots * r) @ s["b"].float().permute(0, 2, 1).reshape(slots * r, -1)
        return (s["y"].float() + d).to(torch.bfloat16)
    h, x = _stream_and_norm(s)
    if case["op"] == "norm":
        return h, x
    x = x.float()
    codes, sf, s_dec = _nvfp4(x, x.abs().amax(-1))
    n, c = case["n"], case["cols"]
    w_codes = torch.stack((s["w_q"] & 15, s["w_q"] >> 4), -1).reshape(n, c)
    w = _values(w_codes, _untiled(s["w_sf"], n, c // 16))
    y = (_values(codes, sf) @ w.T) * (s_dec.unsqueeze(1) * s["w_s_dec"])
    return h, y.to(torch.bfloat16)


# ------------------------------------------------------------------ the calls

def _own(s):
    import nvfp4_block_scaled_19_b200 as nv

    case = s["case"]
    if case["op"] == "lora":
        adapters = nv.LoraAdapters(s["a"], s["b"], s["scale"])
        return nv.lora(s["x"], s["y"], adapters, s["row_slot"], out=s["out"])
    post = None if case["post"] == "none" else nv.Norm(case["post"], s["post_weight"], s["post_bias"], EPS)
    pre = nv.Norm(case["pre"], s["pre_weight"], s["pre_bias"], EPS)
    if case["op"] == "norm":
        r = nv.residual_norm(s["residual"], s["y"], post=post, gate=s["gate"], pre=pre, scale=s["scale"],
                             shift=s["shift"], row_group=s["row_group"],
                             residual_scale=case["residual_scale"], h=s["h"], out=s["out"])
        return r.h, r.out
    r = nv.residual_norm(s["residual"], s["y"], post=post, gate=s["gate"], pre=pre, scale=s["scale"],
                         shift=s["shift"], row_group=s["row_group"],
                         residual_scale=case["residual_scale"], h=s["h"], want_out=False, want_quant=True)
    w = nv.NVFP4Tensor(s["w_q"], s["w_sf"], s["w_s_dec"], case["n"], case["cols"])
    return r.h, nv.gemm(r.quant, w)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "lora":
        m, k, n, r = (case[x] for x in ("rows", "k", "n", "rank"))
        slots = [s for s in _slots(case) if s >= 0]
        return dict(bytes=2 * len(slots) * k + 4 * m * n + 2 * len(set(slots)) * r * (k + n) + 4 * m,
                    flops=2 * len(slots) * r * (k + n))
    m, c, groups = case["rows"], case["cols"], case["groups"]
    stream = 4 if case["stream"] == "f32" else 2
    vectors = groups * (case["gate"] + 2 * case["modulate"])
    if case["weight"]:
        vectors += sum(dict(none=0, rms=1, layer=2)[case[x]] for x in ("post", "pre"))
    size = m * c * (2 * stream + 2) + 2 * c * vectors + 4 * m
    if case["op"] == "norm":
        return dict(bytes=size + 2 * m * c, flops=20 * m * c)
    n = case["n"]
    return dict(bytes=size + n * c // 2 + n * c // 16 + 2 * m * n, flops=20 * m * c + 2 * m * n * c)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lora":
        out = s["y"].double()
        for slot in range(case["slots"]):
            rows = torch.nonzero(s["row_slot"] == slot).reshape(-1)
            low = torch.einsum("mk,rk->mr", s["x"][rows].double(), s["a"][slot].double())
            out.index_add_(0, rows, torch.einsum("mr,nr->mn", low * s["scale"][slot].double(), s["b"][slot].double()))
        return out

    def of_rows(v):
        return v.double().index_select(0, s["row_group"].to(torch.int64))

    def normed(v, name):
        if case[name] == "none":
            return v
        mean = v.sum(1, keepdim=True) / v.shape[1] if case[name] == "layer" else 0.0
        power = ((v - mean) ** 2).sum(1, keepdim=True) / v.shape[1]
        v = (v - mean) / torch.sqrt(power + EPS)
        if s[name + "_weight"] is not None:
            v = torch.mul(v, s[name + "_weight"].double())
        if s[name + "_bias"] is not None:
            v = torch.add(v, s[name + "_bias"].double())
        return v

    branch = normed(s["y"].double(), "post")
    if case["gate"]:
        branch = branch * of_rows(s["gate"])
    h = torch.add(branch, s["residual"].double(), alpha=case["residual_scale"])
    x = normed(h, "pre")
    if case["modulate"]:
        x = torch.addcmul(of_rows(s["shift"]), x, 1.0 + of_rows(s["scale"]))
    if case["op"] == "norm":
        return h, x
    # The quantization is defined on the bf16 value, each step of it one fp32
    # operation; the products of the codes are exact in 64 bits.
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    x = x.to(torch.bfloat16)
    amax = x.abs().amax(1).float()
    s_enc = torch.full_like(amax, 2688.0).div(amax)
    s_enc[amax == 0] = 1.0
    kb = case["cols"] // 16
    sf = x.abs().reshape(-1, kb, 16).amax(2).double().div(6.0).float().mul(s_enc.unsqueeze(1)).clamp(max=448.0)
    sf = sf.to(torch.float8_e4m3fn).float()
    inv = torch.where(sf > 0, s_enc.unsqueeze(1) / sf, torch.zeros_like(sf))
    t = (x.float().reshape(-1, kb, 16) * inv.unsqueeze(2)).double()
    # Nearest value of the grid, a tie to the one with the even code.
    up = torch.searchsorted(grid, t.abs().clamp(max=6.0)).clamp(min=1)
    below, above = grid[up - 1], grid[up]
    far = t.abs().clamp(max=6.0) - (below + above) / 2
    pick = torch.where((far > 0) | ((far == 0) & (up % 2 == 0)), up, up - 1)
    xv = (torch.copysign(grid[pick], t) * sf.double().unsqueeze(2)).reshape(x.shape)
    n, c = case["n"], case["cols"]
    nibbles = torch.empty(n, c, dtype=torch.int64, device=x.device)
    nibbles[:, 0::2] = s["w_q"] % 16
    nibbles[:, 1::2] = s["w_q"] // 16
    r = torch.arange(n, device=x.device).unsqueeze(1)
    b = torch.arange(kb, device=x.device).unsqueeze(0)
    at = ((r // 128) * -(-kb // 4) + b // 4) * 512 + (r % 32) * 16 + (r // 32) % 4 * 4 + b % 4
    w_sf = s["w_sf"][at].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
    wv = torch.cat((grid, -grid))[nibbles] * w_sf
    return h, xv @ wv.T * (s["w_s_dec"].double() / s_enc.double().unsqueeze(1))
