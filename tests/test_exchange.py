"""Tokens to their experts' rows and back, with the gradients, against 64-bit references."""
import pytest
import torch

from hierarchical_tiling_amd import htroute as R
from int8_util import HALF, I32, LEAST, TYPE, gen, pitched, routing

pytestmark = pytest.mark.gpu

SIZES = [(1, 4, 1, 1, 1), (1, 8, 8, 8, 64), (5, 6, 3, 4, 7), (33, 5, 2, 16, 51), (40, 16, 7, 1, 512), (17, 12, 6, 3, 1000),
         (70, 9, 8, 8, 2051), (3, 64, 9, 2, 4096), (12, 70, 64, 1, 130), (9, 20, 15, 5, 5003), (257, 6, 5, 4, 16),
         (300, 5, 2, 1, 17), (270, 9, 7, 1, 515), (260, 4, 3, 8, 2056), (1100, 3, 1, 1, 40)]
DTYPES = ["bf16", "f16", "f32"]


def some(g, rows, cols, dtype, pitch=None):
    x = torch.randn(rows, cols, generator=g, device="cuda").to(TYPE[dtype])
    return x if pitch is None else pitched(x, pitch, 1000.0)


def watched(rows, cols, dtype, pitch):
    room = torch.full((rows + 2, pitch), -7.0, dtype=TYPE[dtype], device="cuda")
    return room, room[1: rows + 1, :cols]


def intact(room, cols):
    assert (room[0] == -7.0).all() and (room[-1] == -7.0).all() and (room[:, cols:] == -7.0).all()


def gathered(x, order, k):
    want = torch.zeros(order.numel(), x.shape[1], dtype=torch.float64, device="cuda")
    for p, a in enumerate(order.tolist()):
        if 0 <= a < x.shape[0] * k:
            want[p] = x[a // k].double()
    return want


def joined(y, slot, weights=None, add=None):
    """(out, tolerance): the k multiply-adds of fp32 one after the other lose 2^-24 each of what the
    sum's terms come to, out's rounding half a step."""
    T, k = slot.shape
    want = torch.zeros(T, y.shape[1], dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    if add is not None:
        want += add.double()
        size += add.double().abs()
    for t, row in enumerate(slot.tolist()):
        for j, s in enumerate(row):
            if 0 <= s < y.shape[0]:
                term = y[s].double() * (1.0 if weights is None else weights[t, j].double())
                want[t] += term
                size[t] += term.abs()
    return want, size * k * 2.0 ** -24


def near(got, want, tol, dtype):
    got = got.double()
    tol = tol + (want.abs() + tol) * HALF[dtype] + LEAST[dtype]
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / tol)[bad].max()))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,E,k,align,H", SIZES)
def test_gather(T, E, k, align, H, dtype):
    g = gen(T + H)
    live = [i % 4 != 3 for i in range(T)]
    order, slot, _ = routing(g, T, E, k, align, live)
    for px, py in ((H, H), (H + 3, H + 5)):
        x = some(g, T, H, dtype, px)
        room, y = watched(order.numel(), H, dtype, py)
        R.gather(x, order, slot, y)
        assert torch.equal(y.double(), gathered(x, order, k))
        intact(room, H)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("weight", [None, "f32", "same"])
@pytest.mark.parametrize("T,E,k,align,H", SIZES)
def test_combine(T, E, k, align, H, weight, dtype):
    g = gen(T + H)
    order, slot, _ = routing(g, T, E, k, align, [i % 4 != 3 for i in range(T)])
    w = None if weight is None else torch.randn(T, k, generator=g, device="cuda").to(TYPE[dtype if weight == "same" else "f32"])
    for p, add in ((H, None), (H + 3, some(g, T, H, dtype, H + 1))):
        y = some(g, order.numel(), H, dtype, p)
        room, out = watched(T, H, dtype, p)
        R.combine(y, slot, out, weights=w, add=add)
        near(out, *joined(y, slot, w, add), dtype)
        intact(room, H)


@pytest.mark.parametrize("H", [3, 130, 4099])
def test_combine_into_what_it_adds(H):
    g = gen(H)
    order, slot, _ = routing(g, 30, 8, 3)
    y, out = some(g, 90, H, "bf16"), some(g, 30, H, "bf16")
    want = joined(y, slot, None, out.clone())
    R.combine(y, slot, out, add=out)
    near(out, *want, "bf16")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("weight", ["f32", "same"])
@pytest.mark.parametrize("T,E,k,align,H", SIZES)
def test_combine_grad(T, E, k, align, H, weight, dtype):
    """A dot of H products: H fp32 steps at most in the order of the sums, far fewer in truth; each
    loses 2^-24 of what the terms come to."""
    g = gen(T + H)
    order, slot, _ = routing(g, T, E, k, align, [i % 4 != 3 for i in range(T)])
    wt = dtype if weight == "same" else "f32"
    w = torch.randn(T, k, generator=g, device="cuda").to(TYPE[wt])
    n = order.numel()
    flat = w.double().flatten()
    for p in (H, H + 3):
        d_out, y = some(g, T, H, dtype, p), some(g, n, H, dtype, p)
        want_dy = gathered(d_out, order, k)
        live = (order >= 0)
        want_dy[live] *= flat[order[live].long()][:, None]
        dots, size = torch.zeros(T, k, dtype=torch.float64, device="cuda"), torch.zeros(T, k, dtype=torch.float64, device="cuda")
        for t, row in enumerate(slot.tolist()):
            for j, s in enumerate(row):
                if s >= 0:
                    terms = d_out[t].double() * y[s].double()
                    dots[t, j], size[t, j] = terms.sum(), terms.abs().sum()
        for dy, dw in ((True, True), (True, False), (False, True)):
            room, d_y = watched(n, H, dtype, p)
            d_w = torch.full((T, k), -7.0, dtype=TYPE[wt], device="cuda")
            R.combine_grad(d_out, y if dw else None, order, slot, w, d_y if dy else None, d_w if dw else None)
            if dy:
                near(d_y, want_dy, 2.0 ** -24 * want_dy.abs(), dtype)
                intact(room, H)
            if dw:
                near(d_w, dots, size * H * 2.0 ** -24, wt)
                assert (d_w[slot < 0] == 0).all()


def test_order_and_slot_that_are_not_each_others():
    """Any values: rows go by order, sums by slot, every row is written, nothing else is."""
    g = gen(9)
    T, k, H, n = 20, 3, 77, 50
    x, y = some(g, T, H, "f32"), some(g, n, H, "f32")
    order = torch.randint(-5, T * k + 5, (n,), generator=g, device="cuda", dtype=torch.int32)
    slot = torch.randint(-5, n + 5, (T, k), generator=g, device="cuda", dtype=torch.int32)
    order[0], order[1], slot[0, 0], slot[0, 1] = 2 ** 31 - 1, -(2 ** 31), 2 ** 31 - 1, -(2 ** 31)
    w = torch.randn(T, k, generator=g, device="cuda")
    room, rows = watched(n, H, "f32", H)
    R.gather(x, order, slot, rows)
    assert torch.equal(rows.double(), gathered(x, order, k))
    intact(room, H)
    out = torch.empty(T, H, device="cuda")
    R.combine(y, slot, out, weights=w)
    near(out, *joined(y, slot, w), "f32")
    room, d_y = watched(n, H, "f32", H)
    d_w = torch.empty(T, k, device="cuda")
    R.combine_grad(x, y, order, slot, w, d_y, d_w)
    want = gathered(x, order, k)
    ok = (order >= 0) & (order < T * k)
    want[ok] *= w.double().flatten()[order[ok].long()][:, None]
    near(d_y, want, 2.0 ** -24 * want.abs(), "f32")
    intact(room, H)
    at = slot.clamp(0, n - 1).long()
    terms = y.double()[at] * x.double()[:, None, :]
    valid = (slot >= 0) & (slot < n)
    near(d_w, terms.sum(2) * valid, terms.abs().sum(2) * H * 2.0 ** -24, "f32")


def test_nan_where_nothing_goes():
    """Rows of no assignment, dropped tokens and their weights may hold anything."""
    g = gen(2)
    T, k, H = 12, 2, 100
    order, slot, _ = routing(g, T, 5, k, 8, [i >= 4 for i in range(T)])
    y = some(g, order.numel(), H, "bf16")
    y[order < 0] = float("nan")
    w, d_out = torch.randn(T, k, generator=g, device="cuda"), some(g, T, H, "bf16")
    w[:4], d_out[:4] = float("nan"), float("nan")
    out, d_y, d_w = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.empty_like(y), torch.empty_like(w)
    R.combine(y, slot, out, weights=w)
    R.combine_grad(d_out, y, order, slot, w, d_y, d_w)
    assert (out[:4] == 0).all() and (d_w[:4] == 0).all() and (d_y[order < 0] == 0).all()
    assert torch.isfinite(out).all() and torch.isfinite(d_y).all() and torch.isfinite(d_w).all()


def test_nothing_to_do():
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(*s, **I32)  # noqa: E731
    y = torch.full((3, 8), -7.0, device="cuda")
    R.gather(z(0, 8), i(3), i(0, 2), y)
    assert (y == 0).all()
    R.gather(z(4, 8), i(0), i(4, 2), z(0, 8))
    out = torch.full((4, 8), -7.0, device="cuda")
    R.combine(z(0, 8), i(4, 2), out)
    assert (out == 0).all()
    d_w = torch.full((4, 2), -7.0, device="cuda")
    R.combine_grad(z(4, 8), z(0, 8), i(0), i(4, 2), z(4, 2), z(0, 8), d_w)
    assert (d_w == 0).all()
    d_w.fill_(-7.0)
    R.combine_grad(z(4, 0), z(5, 0), i(5), i(4, 2), z(4, 2), z(5, 0), d_w)
    assert (d_w == 0).all()


def test_gradients_against_differences():
    """combine() is linear in y and in the weights: with values that are multiples of 1/8 all sums are
    exact in fp32, and so are differences."""
    g = gen(4)
    T, k, H = 6, 2, 24
    order, slot, _ = routing(g, T, 5, k, 4)
    n = order.numel()
    eighths = lambda *s: torch.randint(-16, 17, s, generator=g, device="cuda").float() / 8  # noqa: E731
    x, y, w, d_out = eighths(T, H), eighths(n, H), eighths(T, k), eighths(T, H)

    def loss(y, w):
        out = torch.empty(T, H, device="cuda")
        R.combine(y, slot, out, weights=w)
        return (out.double() * d_out.double()).sum()

    d_y, d_w, d_x = torch.empty(n, H, device="cuda"), torch.empty(T, k, device="cuda"), torch.empty(T, H, device="cuda")
    R.combine_grad(d_out, y, order, slot, w, d_y, d_w)
    base = loss(y, w)
    for p in range(n):
        for c in (0, 7, H - 1):
            moved = y.clone()
            moved[p, c] += 1
            assert loss(moved, w) - base == d_y[p, c].double()
    for t in range(T):
        for j in range(k):
            moved = w.clone()
            moved[t, j] += 1
            assert loss(y, moved) - base == d_w[t, j].double()
    R.combine(y, slot, d_x)       # the gradient of gather(), from y's place
    rows = torch.empty(n, H, device="cuda")
    for t in range(T):
        moved = x.clone()
        moved[t, 3] += 1
        R.gather(moved, order, slot, rows)
        after = (rows.double() * y.double()).sum()
        R.gather(x, order, slot, rows)
        assert after - (rows.double() * y.double()).sum() == d_x[t, 3].double()
