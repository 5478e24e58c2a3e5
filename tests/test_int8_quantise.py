"""Quantisation of rows to 8-bit integers, bit for bit."""
import pytest
import torch

from hierarchical_tiling_amd import htint8 as Q
from int8_util import I32, TYPE, activate, gen, pitched, quantised

pytestmark = pytest.mark.gpu


def quantize(x, rows=None, pitch=None, **kw):
    """(codes, scale), with the bytes around the codes watched."""
    rows, cols = x.shape[0] if rows is None else rows, x.shape[1]
    pitch = pitch or cols
    room = torch.full((rows + 2, max(pitch, 1)), 99, dtype=torch.int8, device="cuda")
    q, scale = room[1: rows + 1, :cols], torch.full((rows + 2,), -7.0, device="cuda")
    Q.quantize(x, q, scale[1: rows + 1], **kw)
    to = min(pitch, -(-cols // 16) * 16) if kw.get("pad") else cols
    assert (room[0] == 99).all() and (room[rows + 1] == 99).all() and (room[1: rows + 1, to:pitch] == 99).all()
    assert (room[1: rows + 1, cols:to] == 0).all() and scale[0] == -7.0 and scale[rows + 1] == -7.0
    return q, scale[1: rows + 1]


def same(got, want):
    assert torch.equal(got[0], want[0])
    assert torch.equal(got[1].view(torch.int32)[~torch.isnan(want[1])], want[1].view(torch.int32)[~torch.isnan(want[1])])
    assert torch.equal(torch.isnan(got[1]), torch.isnan(want[1]))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 8), (9, 511), (4, 513), (130, 2048), (7, 2049), (3, 4097), (2, 8192),
                                       (3, 8200), (2, 20011), (1, 32768), (2, 32775), (1, 100003)])
def test_rows(rows, cols, dtype):
    g = gen(rows + cols)
    x = (torch.randn(rows, cols, generator=g, device="cuda") * torch.exp(2 * torch.randn(rows, 1, generator=g, device="cuda"))).to(TYPE[dtype])
    same(quantize(x), quantised(x.float()))
    wide = pitched(x, cols + 5, 1000.0)          # rows at any alignment, other values between them
    same(quantize(wide, pitch=cols + 21, pad=True), quantised(x.float()))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_value_of_the_16_bit_types(dtype):
    """As rows of 256 values with the same upper bits, the infinities and NaN among them."""
    x = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16).view(TYPE[dtype]).view(256, 256)
    same(quantize(x), quantised(x.float()))
    x = x.t().contiguous()
    same(quantize(x), quantised(x.float()))


def test_ties_and_extremes():
    most, tiny = torch.finfo(torch.float32).max, 2.0 ** -149
    rows = [[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 126.5, -126.5], [0.0] * 8, [-0.0] * 8, [tiny] * 8, [tiny, -tiny] * 4,
            [most, -most, most / 254, 0, 1, 0, 0, 0], [2.0 ** -126] * 8, [127 * 2.0 ** -126, 0.5 * 2.0 ** -126, 0, 0, 0, 0, 0, 0],
            [float("inf")] + [1.0] * 7, [1.0] * 7 + [float("nan")], [float("-inf")] + [0.0] * 7]
    x = torch.tensor(rows, device="cuda")
    got = quantize(x)
    same(got, quantised(x))
    assert torch.isnan(got[1][8:]).all() and (got[0][8:] == 0).all()
    assert got[0][0].tolist() == [127, 0, 2, 2, 0, -2, 126, -126]


@pytest.mark.parametrize("cols", [1, 100, 3000, 40000])
@pytest.mark.parametrize("div", [1, 3])
def test_gathered_rows(cols, div):
    g = gen(cols)
    x = torch.randn(10, cols, generator=g, device="cuda").to(torch.bfloat16)
    index = torch.tensor([0, 10 * div - 1, -1, 10 * div, -(2 ** 31), 2 ** 31 - 1, 3, 3, 4, 7 * div], **I32)
    want = torch.zeros(10, cols, device="cuda")
    for r, i in enumerate(index.tolist()):
        if 0 <= i < 10 * div:
            want[r] = x[i // div].float()
    same(quantize(x, rows=10, row_index=index, index_div=div), quantised(want))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu", "none"])
@pytest.mark.parametrize("rows,cols", [(4, 37), (70, 600), (3, 5001), (2, 33000)])
def test_gated(rows, cols, act, dtype):
    """The gate's activation is good to 2^-20 of its argument (and relu and none are exact), the
    product rounds once: a code may be off by what that moves, plus half a step."""
    g = gen(rows + cols)
    both = (3 * torch.randn(rows, 2 * cols, generator=g, device="cuda")).to(TYPE[dtype])
    gate, x = both[:, :cols], both[:, cols:]
    q, scale = quantize(x, gate=gate, act=act)
    gd, xd = gate.double(), x.double()
    v = activate(gd, act) * xd
    err = ((2.0 ** -20 * gd.abs() if act in ("silu", "gelu") else 0) * xd.abs() + 2.0 ** -24 * v.abs())
    top = v.abs().amax(1)
    most = err.amax(1)
    assert ((scale.double() * 127 - top).abs() <= most + top * 2.0 ** -23).all()
    step = scale.double()[:, None]
    assert ((q.double() * step - v).abs() <= 0.5 * step * (1 + 2.0 ** -14) + err + v.abs() * 2.0 ** -22).all()
    if act in ("relu", "none"):
        same((q, scale), quantised(activate(gate.float(), act) * x.float()))


def test_gate_gathered_with_x():
    g = gen(3)
    both = torch.randn(6, 400, generator=g, device="cuda")
    index = torch.tensor([5, -1, 0, 0, 9], **I32)
    got = quantize(both[:, 200:], rows=5, gate=both[:, :200], act="none", row_index=index, index_div=2)
    want = torch.zeros(5, 200, device="cuda")
    for r, i in enumerate(index.tolist()):
        if i >= 0:
            want[r] = both[i // 2, :200] * both[i // 2, 200:]
    same(got, quantised(want))


def test_a_gate_that_is_not_finite():
    x, gate = torch.ones(4, 64, device="cuda"), torch.ones(4, 64, device="cuda")
    gate[1, 3], gate[2, 5] = float("nan"), float("inf")
    x[3, 7] = float("inf")
    q, scale = quantize(x, gate=gate)
    assert torch.isnan(scale[1:]).all() and (q[1:] == 0).all() and torch.isfinite(scale[0]) and (q[0] == 127).all()


def test_empty():
    x = torch.zeros(0, 8, device="cuda")
    quantize(x)
    q, scale = quantize(torch.zeros(3, 0, device="cuda"))
    assert (scale == 2.0 ** -126).all()
    q, scale = quantize(torch.zeros(0, 20, device="cuda"), rows=2, row_index=torch.tensor([0, 1], **I32))
    assert (q == 0).all() and (scale == 2.0 ** -126).all()
