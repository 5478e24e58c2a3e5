"""Rows of a routing and their quantisation at the largest sizes: 2^23 tokens, 2^26 rows, 2^24 columns."""
import pytest
import torch

from hierarchical_tiling_amd import htint8 as Q
from hierarchical_tiling_amd import htroute as R
from int8_util import I32, gen, quantised

pytestmark = pytest.mark.gpu


def test_most_tokens_and_rows():
    """Whole numbers up to 3: sums of 8 are exact in bf16 and dots of 3 in fp32."""
    T, k, H = 1 << 23, 8, 3
    n = T * k
    g = gen(1)
    order = torch.randperm(n, generator=g, device="cuda").int()
    slot = torch.empty(n, **I32)
    slot[order.long()] = torch.arange(n, **I32)
    slot = slot.view(T, k)
    x = torch.randint(-3, 4, (T, H), generator=g, device="cuda").to(torch.bfloat16)
    y = torch.full((n, H), 7.0, dtype=torch.bfloat16, device="cuda")
    R.gather(x, order, slot, y)
    token = (order // k).long()
    assert torch.equal(y, x[token])
    y.fill_(7.0)
    R.gather(x, order, None, y, topk=k)
    assert torch.equal(y, x[token])
    out, d_w = torch.empty_like(x), torch.empty(T, k, device="cuda")
    R.combine(y, slot, out)
    assert torch.equal(out, x * 8)
    w = torch.randint(-1, 2, (T, k), generator=g, device="cuda").float()
    d_y = torch.full_like(y, 7.0)
    R.combine_grad(x, y, order, slot, w, d_y, d_w)
    assert torch.equal(d_y, (x[token].float() * w.flatten()[order.long()][:, None]).to(torch.bfloat16))
    assert torch.equal(d_w, x.float().square().sum(1, keepdim=True).expand(T, k))


@pytest.mark.parametrize("pad", [0, 3])
def test_most_columns(pad):
    """Rows of 2^24 - pad values; d_weights sums whole numbers to less than 2^24, exact in fp32."""
    T, k, H = 3, 2, (1 << 24) - pad
    g = gen(pad)
    order = torch.tensor([5, 0, -1, 3, 1], **I32)
    slot = torch.tensor([[1, 4], [-1, 3], [-1, 0]], **I32)
    x = (torch.rand(T, H, generator=g, device="cuda") < 0.25).float()
    y = torch.full((5, H), 7.0, device="cuda")
    R.gather(x, order, slot, y)
    for p, a in enumerate(order.tolist()):
        assert torch.equal(y[p], x[a // k] if a >= 0 else torch.zeros_like(x[0]))
    w, out = torch.tensor([[2.0, 3.0], [1.0, -1.0], [4.0, 5.0]], device="cuda"), torch.empty_like(x)
    R.combine(y, slot, out, weights=w)
    for t in range(T):
        own = [(w[t, j], s) for j, s in enumerate(slot[t].tolist()) if s >= 0]
        assert torch.equal(out[t], sum(f * y[s] for f, s in own))
    d_y, d_w = torch.empty_like(y), torch.empty_like(w)
    R.combine_grad(x, y, order, slot, w, d_y, d_w)
    for p, a in enumerate(order.tolist()):
        assert torch.equal(d_y[p], w.flatten()[a] * x[a // k] if a >= 0 else torch.zeros_like(x[0]))
    want = torch.stack([torch.stack([(x[t].double() * y[s].double()).sum() if s >= 0 else x.new_zeros(()).double()
                                     for s in slot[t].tolist()]) for t in range(T)])
    assert want.max() < 2 ** 24 and torch.equal(d_w.double(), want)
    q, scale = torch.empty(T, H, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    z = torch.randn(T, H, generator=g, device="cuda")
    Q.quantize(z, q, scale)
    codes, steps = quantised(z)
    assert torch.equal(q, codes) and torch.equal(scale, steps)
