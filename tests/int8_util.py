"""Inputs and 64-bit references for the products in 8-bit integers, their quantisation, and the rows of a
routing."""
import torch

HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}      # half a step, relative
LEAST = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}   # half the least step
TYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
I32 = dict(dtype=torch.int32, device="cuda")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def pitched(values, pitch, fill):
    """The same matrix with `pitch` values from row to row and `fill` between the rows."""
    room = torch.full((values.shape[0], pitch), fill, dtype=values.dtype, device=values.device)
    room[:, : values.shape[1]] = values
    return room[:, : values.shape[1]]


def codes(g, rows, cols, pitch=None):
    """Codes over the whole range, -128 among them; rows `pitch` bytes apart, other codes between."""
    q = torch.randint(-128, 128, (rows, cols), generator=g, device="cuda", dtype=torch.int8)
    return q if pitch is None else pitched(q, pitch, 77)


def scales(g, n):
    return torch.exp(torch.randn(n, generator=g, device="cuda")) * 2.0 ** -9


def activate(y, act):
    if act == "relu":
        return torch.where(torch.isnan(y), y, y.clamp(min=0))
    if act == "gelu":
        return 0.5 * y * (1 + torch.special.erf(y / 2 ** 0.5))
    if act == "silu":
        return y * torch.sigmoid(y)
    return y


def reference(a, sa, b, sb, out, alpha=1.0, beta=0.0, c=None, bias=None, act="none"):
    """(D, tolerance) in float64 of one product.

    The tolerance: the sum of integers is exact.  Its rounding to fp32 and the products with two
    scales and alpha are 4 roundings of the scaled sum t, beta C one of its own size, and the two
    additions one each of what they give: (4 |t| + |beta C| + 2 (|t| + |beta C| + |bias|)) 2^-24.  An
    activation's slope is below 1.13, its own evaluation good to 2^-20 of its argument.  D's rounding
    is half a step of its type."""
    t = torch.mm(a.double(), b.double().t().contiguous()) if a.shape[1] else torch.zeros(
        a.shape[0], b.shape[0], dtype=torch.float64, device=a.device)
    if a.shape[1]:
        t = t * sa.double()[:, None] * sb.double()[None, :]
    t = alpha * t
    y, size, own = t, t.abs(), 4 * t.abs()
    if c is not None and beta:
        y, size, own = y + beta * c.double(), size + (beta * c.double()).abs(), own + (beta * c.double()).abs()
    if bias is not None:
        y, size = y + bias.double(), size + bias.double().abs()
    tol = (own + 2 * size) * 2.0 ** -24
    if act != "none":
        tol = 1.13 * tol + 2.0 ** -20 * y.abs()
    y = activate(y, act)
    return y, tol + (y.abs() + tol) * HALF[out] + LEAST[out]


def close(got, want, tol):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), "NaN in other places"
    # what passes the type's range is infinite
    bad = ((got - want).abs() > tol) & ~(torch.isinf(got) & (got == torch.sign(want) * torch.inf) & (want.abs() + tol >= 65504))
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / tol)[bad].max()))


def quantised(x):
    """(codes, scale) of the rows of a float32 matrix, each operation rounded to float32 once."""
    top = x.abs().amax(1) if x.shape[1] else torch.zeros(x.shape[0], device=x.device)
    bad = ~torch.isfinite(top)
    t = top.masked_fill(bad, 0).clamp(min=127 * 2.0 ** -126)
    most = torch.full_like(t, 127.0)
    q = torch.round(x * (most / t)[:, None]).clamp(-127, 127).masked_fill(bad[:, None], 0).to(torch.int8)
    return q, (t / most).masked_fill(bad, float("nan"))


def routing(g, T, E, k, align=1, live=None):
    """order (rows) and slot (T, k) of a routing of T tokens to k of E experts, and its offsets, worked
    out assignment by assignment on the host; tokens where live is False go nowhere."""
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices.cpu() if T else torch.zeros(0, k).long()
    members = [[] for _ in range(E)]
    for i, e in enumerate(ids.flatten().tolist()):
        if live is None or live[i // k]:
            members[e].append(i)
    order = torch.full((T * k + E * (align - 1),), -1, dtype=torch.int32)
    slot, offsets = torch.full((T * k,), -1, dtype=torch.int32), [0]
    for m in members:
        for j, i in enumerate(m):
            order[offsets[-1] + j], slot[i] = i, offsets[-1] + j
        offsets.append(offsets[-1] + -(-len(m) // align) * align)
    return order.cuda(), slot.view(T, k).cuda(), torch.tensor(offsets, **I32)
