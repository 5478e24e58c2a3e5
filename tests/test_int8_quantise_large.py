"""Quantisation of rows of inputs that no cache holds (128 MiB and more, which are read past the caches), by
every number of threads a row, with a gate, and gathered; bit for bit."""
import pytest
import torch

from hierarchical_tiling_amd import htint8 as Q
from int8_util import TYPE, gen, quantised
from test_int8_quantise import same

pytestmark = pytest.mark.gpu
MANY = 1 << 27      # bytes


def check(x, want_of, rows=None, **kw):
    rows = x.shape[0] if rows is None else rows
    room = torch.full((rows + 1, x.shape[1]), 99, dtype=torch.int8, device="cuda")
    q, scale = room[:rows], torch.empty(rows, device="cuda")
    Q.quantize(x, q, scale, **kw)
    for r in range(0, rows, max(1, rows // 4)):          # the reference piece by piece, for its memory
        at = slice(r, r + max(1, rows // 4))
        same((q[at], scale[at]), quantised(want_of(at)))
    assert (room[rows] == 99).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("cols", [300, 1000, 2047, 4000, 8192, 30000, 40001])
def test_rows(cols, dtype):
    g = gen(cols)
    size = 4 if dtype == "f32" else 2
    x = torch.randn(MANY // (cols * size) + 1, cols, generator=g, device="cuda").to(TYPE[dtype])
    check(x, lambda at: x[at].float())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("cols", [2048, 5001, 33000])
def test_gated(cols, dtype):
    """128 MiB with the gate, half of it without."""
    g = gen(cols)
    size = 4 if dtype == "f32" else 2
    both = torch.randn(MANY // (2 * cols * size) + 1, 2 * cols, generator=g, device="cuda").to(TYPE[dtype])
    gate, x = both[:, :cols], both[:, cols:]
    check(x, lambda at: gate[at].float().clamp(min=0) * x[at].float(), gate=gate, act="relu")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("div", [1, 2])
@pytest.mark.parametrize("gated", [False, True])
def test_gathered(div, gated, dtype):
    """Each row once, and twice; a few rows of zeros."""
    g = gen(div)
    n, cols = 17000, 4096
    x = torch.randn(n, cols, generator=g, device="cuda").to(TYPE[dtype])
    gate = torch.randn(n, cols, generator=g, device="cuda").to(TYPE[dtype]) if gated else None
    index = torch.randperm(n * div, generator=g, device="cuda").int()
    index[::1001] = -1

    def want(at):
        i = index[at].long()
        v = x[i.clamp(min=0) // div].float()
        if gated:
            v = v * gate[i.clamp(min=0) // div].float()
        return torch.where((i >= 0)[:, None], v, 0.0)

    check(x, want, rows=n * div, row_index=index, index_div=div, **(dict(gate=gate, act="none") if gated else {}))
