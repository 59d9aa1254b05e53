"""Plain implementations, in 64 bits, of the operators around a projection, with
the bounds that a kernel in fp32 arithmetic stays within."""
import torch

# A sum over a row adds at most 32 values in a chain per thread, then 5 by
# shuffles and 32 over the warps: under 128 roundings of 2^-24 with the handful
# of elementwise ones around it.
F32 = 128 * 2.0 ** -24
BF16 = 2.0 ** -8      # half a bf16 step, relative to the value
TINY = 2.0 ** -133    # half a step of the smallest bf16 values


def norm64(x, kind, weight, bias, eps):
    """(normed, normalised value before weight and bias, 1 / root)."""
    mean = x.mean(-1, keepdim=True) if kind == "layer" else 0.0
    inv = 1.0 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + eps)
    n = (x - mean) * inv
    v = n if weight is None else n * weight.double()
    return (v if bias is None else v + bias.double()), n, inv


def residual_norm64(residual, y, *, post=None, gate=None, pre=None, scale=None, shift=None,
                    group=None, residual_scale=1.0, branch_scale=1.0):
    """h, out in 64 bits and how far fp32 arithmetic may be from each (before
    any rounding to bf16).  post and pre are (kind, weight, bias, eps)."""
    r = residual.double()
    rows, cols = r.shape

    def per_row(v):
        if v is None:
            return None
        v = v.double()
        return v.expand(rows, cols) if v.dim() == 1 else v[group]

    def top(v):
        return v.abs().amax(-1, keepdim=True)

    def err_of_norm(x, err, kind, weight, bias, eps):
        # Values of a row are off by `err`; the mean and the differences add
        # roundings of the row's magnitude, the root a relative one.
        v, n, inv = norm64(x, kind, weight, bias, eps)
        w = 1.0 if weight is None else weight.double().abs()
        e = (2 * (err + (F32 * top(x) if kind == "layer" else 0.0)) * inv * (1 + top(n))
             + F32 * top(n)) * w + F32 * v.abs()
        return v, e if bias is None else e + F32 * bias.double().abs()

    h, e_h = residual_scale * r, F32 * (residual_scale * r).abs()
    if y is not None:
        z, e = y.double(), torch.zeros_like(r)
        if post is not None:
            z, e = err_of_norm(z, torch.zeros_like(r), *post)
        g = per_row(gate)
        g = 1.0 if g is None else g
        h = h + branch_scale * g * z
        e_h = e_h + F32 * (branch_scale * g * z).abs() + abs(branch_scale) * (e * g if gate is None else e * g.abs())
    if pre is None:
        return h, e_h, None, None
    o, e_o = err_of_norm(h, top(e_h), *pre)
    s, t = per_row(scale), per_row(shift)
    if s is not None:
        e_o = e_o * (1 + s).abs() + F32 * o.abs() * (1 + s.abs())
        o = o * (1 + s)
    if t is not None:
        e_o = e_o + F32 * (o.abs() + t.abs())
        o = o + t
    return h, e_h, o, e_o


def assert_close(got, ref, err, what=""):
    """|got - ref| within err, plus half a step where got is bf16."""
    bound = err + 1e-30
    if got.dtype == torch.bfloat16:
        bound = bound * (1 + BF16) + BF16 * ref.abs() + TINY
    off = (got.double() - ref).abs()
    worst = float((off / bound).max()) if off.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} times the bound"


def lora64(x, y, adapters, row_slot):
    """out and how far fp32 sums may be from it: a sum of K products, one of
    rank, whatever their order, in steps of at most 16 products that are each
    rounded (or cut off) to 24 bits, and an inner vector of at least 16 bits."""
    out = y.double().clone()
    err = torch.zeros_like(out)
    slots, rank, k = adapters.a.shape
    step = (k / 16 + rank / 16 + 64) * 2.0 ** -23 + 2.0 ** -16
    slot = torch.zeros(x.shape[0], dtype=torch.int64, device=x.device) if row_slot is None else row_slot.long()
    for s in range(slots):
        rows = torch.nonzero(slot == s).reshape(-1)
        if rows.numel() == 0:
            continue
        xd, a, b = x[rows].double(), adapters.a[s].double(), adapters.b[s].double()
        c = adapters.scale[s].double()
        out[rows] += c * (xd @ a.T) @ b.T
        err[rows] = step * c.abs() * ((xd.abs() @ a.abs().T) @ b.abs().T) + 2.0 ** -23 * y[rows].double().abs()
    return out, err
