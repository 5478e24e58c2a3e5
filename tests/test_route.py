"""Expert routing and the balance loss on the GPU against plain references in integers and 64 bits."""
import pytest
import torch

from hierarchical_tiling_amd import htroute as R
from hierarchical_tiling_amd.htgemm import GemmError
from scaled_util import up

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


def plain_route(ids, mask, E, align, rows):
    T, k = ids.shape
    flat, groups = ids.flatten().tolist(), [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E and (mask is None or mask[i // k]):
            groups[e].append(i)
    order, slot, offsets = [-1] * rows, [-1] * (T * k), [0]
    for members in groups:
        for j, i in enumerate(members):
            order[offsets[-1] + j], slot[i] = i, offsets[-1] + j
        offsets.append(offsets[-1] + up(len(members), align) * align)
    return [len(m) for m in groups], offsets, order, slot


def routed(ids, E, align, mask=None, extra=0, order=True, slot=True):
    T, k = ids.shape
    rows = T * k + E * (align - 1) + extra
    out = [torch.full((n,), -9, **I32) for n in (E, E + 1, rows, T * k)]
    ws = torch.empty(R.workspace_size(T, k, E), dtype=torch.uint8, device="cuda")
    R.route(ids, out[0], out[1], out[2] if order else None, out[3] if slot else None, mask=mask, align=align, workspace=ws)
    return out


def ids_of(T, k, E, seed, skew=1.0):
    g = torch.Generator()
    g.manual_seed(seed)
    p = torch.rand(T, E, generator=g) + skew * torch.rand(E, generator=g)
    return p.topk(min(k, E), dim=1).indices.to(torch.int32)


@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (1, 3, 5), (7, 2, 1024), (37, 6, 64), (100, 1, 3), (1000, 2, 8),
                                   (1025, 2, 100), (3000, 8, 256), (5000, 4, 1024), (40000, 2, 60),
                                   (270000, 2, 70)])
@pytest.mark.parametrize("align", [1, 16, 128])
def test_route(T, k, E, align):
    ids = ids_of(T, k, E, T + E)
    got = routed(ids.cuda(), E, align, extra=5)
    for a, b in zip(got, plain_route(ids, None, E, align, got[2].numel())):
        assert a.tolist() == b


@pytest.mark.parametrize("T", [50, 3000])
def test_dropped_and_masked(T):
    """Ids outside the experts (the ends of the type among them), masked tokens, strided ids."""
    g = torch.Generator()
    g.manual_seed(T)
    wide = torch.randint(-3, 12, (T, 7), generator=g, dtype=torch.int32)
    wide[0, 0], wide[0, 1] = -2 ** 31, 2 ** 31 - 1
    mask = (torch.rand(T, generator=g) < 0.7).to(torch.uint8)
    ids = wide[:, :3]
    for m in (None, mask, torch.zeros_like(mask)):
        got = routed(wide.cuda()[:, :3], 9, 16, mask=None if m is None else m.cuda())
        for a, b in zip(got, plain_route(ids, m, 9, 16, got[2].numel())):
            assert a.tolist() == b
    only = routed(ids.cuda().contiguous(), 9, 1, order=False, slot=False)
    assert (only[2] == -9).all() and (only[3] == -9).all()


def test_tensors_elsewhere_are_refused():
    ids = ids_of(5, 2, 4, 1)
    good = [torch.empty(n, **I32) for n in (4, 5, 10, 10)]
    ws = torch.empty(R.workspace_size(5, 2, 4), dtype=torch.uint8, device="cuda")
    with pytest.raises(GemmError):
        R.route(ids, *good, workspace=ws)
    with pytest.raises(GemmError):
        R.route(ids.cuda(), *good[:3], good[3].cpu(), workspace=ws)
    one, live = torch.ones(1, device="cuda"), torch.empty(1, **I32)
    with pytest.raises(GemmError):
        R.balance_loss(torch.zeros(5, 4), good[0], 2, one, torch.zeros(4, device="cuda"), live, workspace=ws)
    with pytest.raises(GemmError):
        R.balance_grad(torch.zeros(5, 4, device="cuda"), good[0], 2, live, one.cpu(), torch.zeros(5, 4, device="cuda"))


def test_one_expert_takes_all():
    ids = torch.full((9000, 2), 3, **I32)     # the same expert twice for each token, several workgroups
    counts, offsets, order, slot = routed(ids, 4, 128)
    assert counts.tolist() == [0, 0, 0, 18000]
    assert offsets.tolist() == [0, 0, 0, 0, up(18000, 128) * 128]
    assert torch.equal(slot, torch.arange(18000, **I32)) and torch.equal(order[:18000], slot)


def reference(logits, counts, mask, topk, coef):
    """loss, prob and d loss / d logits in float64, a row of -infinity having no probabilities."""
    x = logits.double()
    E = x.shape[1]
    live = torch.ones(x.shape[0], dtype=torch.bool, device=x.device) if mask is None else mask.bool()
    x = torch.where(live[:, None], x, torch.zeros((), dtype=torch.float64, device=x.device))
    top = x.amax(1, keepdim=True) if x.numel() else x.new_zeros(x.shape[0], 1)
    p = torch.exp(x - torch.where(torch.isneginf(top), torch.zeros_like(top), top))
    total = p.sum(1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total) * live[:, None]
    n = int(live.sum())
    if n == 0:
        return x.new_zeros(()), x.new_zeros(E), torch.zeros_like(x), torch.zeros_like(x), 0
    prob = p.sum(0) / n
    f = counts.double() * E / (topk * n)
    g = coef * f / n
    grad = p * (g - (p * g).sum(1, keepdim=True))
    # what the gradient is formed from: the slopes relative to an even load
    h = (coef * (f - 1) / n).abs()
    size = p * (h + (p * h).sum(1, keepdim=True))
    return coef * (f * prob).sum(), prob, grad, size, n


EPS = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def run(logits, counts, topk, mask=None, coef=0.01, d_loss=1.0):
    T, E = logits.shape
    loss, prob, live = torch.full((1,), -9.0, device="cuda"), torch.full((E,), -9.0, device="cuda"), torch.full((1,), -9, **I32)
    ws = torch.empty(R.workspace_size(T, topk, E), dtype=torch.uint8, device="cuda")
    d = torch.full_like(logits, -9)
    R.balance_loss(logits, counts, topk, loss, prob, live, mask=mask, coef=coef, workspace=ws)
    R.balance_grad(logits, counts, topk, live, torch.tensor([d_loss], device="cuda"), d, mask=mask, coef=coef)
    return loss, prob, live, d


def check(logits, counts, topk, mask=None, coef=0.01, d_loss=1.0):
    """Tolerances: a probability is good to 2^-18 (exp within 2 ulp, a sum of up to 1024 terms in 16
    + 6 steps, a division, and room), the sums over the tokens of a wave (up to 2^5 rows at these
    sizes) and of 8 waves to 2^-18 more, the rest is double.  The gradient is p times a difference of slopes:
    2^-18 of p times their sizes, then the rounding to the logits' type, with the least step of fp16."""
    got = run(logits, counts, topk, mask, coef, d_loss)
    loss, prob, grad, size, n = reference(logits, counts, mask, topk, coef)
    assert got[2].item() == n
    assert ((got[1].double() - prob).abs() <= 2.0 ** -17 * prob).all()
    assert abs(got[0].item() - loss.item()) <= 2.0 ** -16 * abs(loss.item())
    tiny = 2.0 ** -25 if logits.dtype == torch.float16 else 1e-38
    tol = abs(d_loss) * (2.0 ** -18 * size + EPS[logits.dtype] * grad.abs()) + tiny
    assert ((got[3].double() - d_loss * grad).abs() <= tol).all()
    return got


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 4, 2), (37, 64, 6), (3, 65, 2), (64, 100, 4), (500, 256, 8),
                                   (257, 130, 2), (300, 512, 8), (70, 1000, 3), (8000, 16, 2),
                                   (70, 992, 3), (65, 1024, 8), (300, 204, 4), (9, 66, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_balance(T, E, k, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(T * E)
    wide = (2 * torch.randn(T, E + 3, generator=g, device="cuda")).to(dtype)
    logits = wide[:, :E]
    counts = routed(ids_of(T, k, E, E).cuda(), E, 1)[0]
    mask = (torch.rand(T, generator=g, device="cuda") < 0.6).to(torch.uint8)
    check(logits, counts, k)
    check(logits.contiguous(), counts, k, mask=mask, coef=0.5, d_loss=-3.0)


def test_even_load_is_coef():
    T, E, k = 128, 32, 4
    ids = (torch.arange(T * k, **I32) % E).view(T, k)
    counts = routed(ids, E, 1)[0]
    loss, _, _, d = run(torch.randn(T, E, device="cuda"), counts, k, coef=0.25)
    assert abs(loss.item() - 0.25) <= 0.25 * 2.0 ** -17
    assert (d == 0).all()      # the slopes are those of an even load: exactly zero


def test_all_masked_and_none():
    logits = torch.full((40, 20), float("nan"), device="cuda")
    counts = torch.zeros(20, **I32)
    loss, prob, live, d = run(logits, counts, 2, mask=torch.zeros(40, dtype=torch.uint8, device="cuda"))
    assert loss.item() == 0 and live.item() == 0 and (prob == 0).all() and (d == 0).all()
    loss, prob, live, _ = run(torch.empty(0, 20, device="cuda"), counts, 2)
    assert loss.item() == 0 and live.item() == 0 and (prob == 0).all()


def test_rows_without_a_choice_and_infinities():
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    logits = torch.randn(50, 70, generator=g, device="cuda")
    logits[3] = float("-inf")
    logits[4] = torch.finfo(torch.float32).min
    logits[5, ::2] = float("-inf")
    logits[6] = 3e38
    logits[7, 1:] = -3e38
    counts = routed(ids_of(50, 3, 70, 1).cuda(), 70, 1)[0]
    got = check(logits, counts, 3)
    assert (got[3][3] == 0).all()
    # NaN and infinity under the mask are not looked at; elsewhere they show
    mask = torch.ones(50, dtype=torch.uint8, device="cuda")
    mask[8:10] = 0
    logits[8, 5], logits[9] = float("nan"), float("inf")
    check(logits, counts, 3, mask=mask)
    loss, _, _, d = run(logits, counts, 3)
    assert loss.isnan().all() and d[8].isnan().all() and not d[7].isnan().any()


def test_gradient_against_differences():
    """Central differences of the loss itself along random directions, the step chosen so that the
    fp32 loss's own rounding (2^-24 of it, twice, over 2 h) stays below the 2^-7 asked for."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    T, E, k, h = 60, 40, 2, 2.0 ** -6
    logits = 1.5 * torch.randn(T, E, generator=g, device="cuda")
    counts = torch.zeros(E, **I32)
    counts[:4] = T * k // 4
    loss, _, _, d = run(logits, counts, k, coef=1.0)
    for _ in range(4):
        # along the gradient, with some noise: a slope that is not lost in the loss's last bits
        v = d / d.norm() + 0.3 * torch.randn(T, E, generator=g, device="cuda") / (T * E) ** 0.5
        up_, down = (run(logits + s * h * v, counts, k, coef=1.0)[0].double() for s in (1, -1))
        slope, want = ((up_ - down) / (2 * h)).item(), (d.double() * v.double()).sum().item()
        room = 2 * 2.0 ** -24 * abs(loss.item()) / h
        assert room < 2.0 ** -7 * abs(want)
        # the third-order term of the difference is h^2 / 6 of a third derivative below 8 slopes
        assert abs(slope - want) <= room + 2.0 ** -7 * abs(want)


def test_captured_and_replayed():
    """Route, loss and gradient in one graph, sharing a workspace, over several workgroups."""
    T, E, k = 3000, 96, 4
    ids, logits = torch.empty(T, k, **I32), torch.empty(T, E, device="cuda")
    ws = torch.empty(R.workspace_size(T, k, E), dtype=torch.uint8, device="cuda")
    rows = T * k + E * 15

    def buffers():
        return ([torch.empty(n, **I32) for n in (E, E + 1, rows, T * k)], torch.empty(1, device="cuda"),
                torch.empty(E, device="cuda"), torch.empty(1, **I32), torch.empty(T, E, device="cuda"))

    one = torch.ones(1, device="cuda")

    def step(b):
        R.route(ids, *b[0], align=16, workspace=ws)
        R.balance_loss(logits, b[0][0], k, b[1], b[2], b[3], workspace=ws)
        R.balance_grad(logits, b[0][0], k, b[3], one, b[4])

    ids.copy_(ids_of(T, k, E, 0))
    logits.normal_()
    captured, eager = buffers(), buffers()
    step(captured)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(captured)
    for seed in (1, 2, 3):
        ids.copy_(ids_of(T, k, E, seed, skew=seed))
        logits.normal_()
        step(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured[0] + list(captured[1:]), eager[0] + list(eager[1:])):
            assert torch.equal(a, b)
