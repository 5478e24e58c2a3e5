"""Inputs and 64-bit references for the block-scaled products, the quantisation and the routing."""
import torch

BLOCK = 128


def up(n, m):
    return -(-n // m)


def codes(g, rows, cols, spread=0.0, device="cuda"):
    """Random e4m3 codes as bytes (no NaN): values of a normal draw scaled into the type's range;
    `spread` varies the size of the columns."""
    x = torch.randn(rows, cols, generator=g, device=device)
    if spread:
        x = x * torch.exp(spread * torch.randn(cols, generator=g, device=device))
    x = x * (448.0 / x.abs().amax().clamp(min=1e-30)) if x.numel() else x
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def values(q):
    """The float64 values of bytes that hold e4m3 codes."""
    return q.contiguous().view(torch.float8_e4m3fn).to(torch.float32).double()


def spread_scales(scale, rows, cols, row_block):
    """scale (row blocks, blocks of 128 columns) for each element of a rows x cols matrix."""
    r = torch.arange(rows, device=scale.device) // row_block
    c = torch.arange(cols, device=scale.device) // BLOCK
    return scale.double()[r][:, c]


def activate(y, act):
    if act == "relu":
        return torch.relu(y)
    if act == "gelu":
        return 0.5 * y * (1 + torch.special.erf(y / 2 ** 0.5))
    if act == "silu":
        return y * torch.sigmoid(y)
    return y


def reference(a, sa, b, sb, b_block, out, alpha=1.0, beta=0.0, c=None, bias=None, row_scale=None, act="none"):
    """(D, tolerance) in float64 of one product; a (M, K) and b (N, K) bytes, sa (M, blocks), sb
    (N / b_block, blocks).

    The tolerance, with T = |alpha rs| sum |a b| sa sb, the size of what is summed:
    * bf16 D: the 8-bit matrix instruction aligns a group of 8 products and drops what lies below
      2^-14 of the largest, at most 8 * 2^-14 of the group's T; the fp32 steps behind it, (blocks +
      8) * 2^-24 of T; the rounding to bf16, half a step, 2^-8 of the value.
    * f32 D: products of the codes are exact; 128 additions in the instruction, one multiply-add
      for each block, 8 further operations, each 2^-24 of T at most; the result 2^-24.
    * beta C and bias add 2 * 2^-24 of their own size.
    * an activation's slope is below 1.13; its own evaluation is good to 2^-20 of its argument
      (the GELU's erf to 1.5e-7)."""
    M, K = a.shape
    N = b.shape[0]
    va = values(a) * spread_scales(sa, M, K, 1) if K else torch.zeros(M, 0, dtype=torch.float64, device=a.device)
    vb = values(b) * spread_scales(sb, N, K, b_block) if K else torch.zeros(N, 0, dtype=torch.float64, device=a.device)
    y = alpha * torch.mm(va, vb.t().contiguous())
    size = abs(alpha) * torch.mm(va.abs(), vb.abs().t().contiguous())
    if row_scale is not None:
        y = y * row_scale.double()[:, None]
        size = size * row_scale.double().abs()[:, None]
    blocks = up(K, BLOCK)
    tol = size * ((2.0 ** -11 + (blocks + 8) * 2.0 ** -24) if out == "bf16" else (128 + blocks + 8) * 2.0 ** -24)
    for extra in (beta * c.double() if c is not None and beta else None,
                  bias.double()[None, :] if bias is not None else None):
        if extra is not None:
            y = y + extra
            tol = tol + 2 * 2.0 ** -24 * (extra.abs() + size)
    if act != "none":
        tol = 1.13 * tol + 2.0 ** -20 * y.abs()
    y = activate(y, act)
    return y, tol + y.abs() * (2.0 ** -8 if out == "bf16" else 2.0 ** -24) + 1e-30


def close(got, want, tol):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), "NaN in other places"
    bad = (got - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / tol)[bad].max()))
