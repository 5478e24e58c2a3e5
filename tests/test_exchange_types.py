"""Rows of a routing joined by weights of every type, with the gradients; and products of the most groups."""
import pytest
import torch

from hierarchical_tiling_amd import htint8 as Q
from hierarchical_tiling_amd import htroute as R
from int8_util import TYPE, codes, gen, reference, routing, scales
from test_exchange import joined, near, some
from test_int8_epilogue import near as close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("weight", ["bf16", "f16", "f32"])
def test_weights(weight, dtype):
    g = gen(5)
    T, E, k, H = 70, 9, 5, 205
    order, slot, _ = routing(g, T, E, k, 4, [i % 4 != 3 for i in range(T)])
    n = order.numel()
    w = torch.randn(T, k, generator=g, device="cuda").to(TYPE[weight])
    y, add, d_out = some(g, n, H, dtype), some(g, T, H, dtype), some(g, T, H, dtype)
    out, d_y, d_w = torch.empty_like(d_out), torch.empty_like(y), torch.empty_like(w)
    R.combine(y, slot, out, weights=w, add=add)
    near(out, *joined(y, slot, w, add), dtype)
    R.combine_grad(d_out, y, order, slot, w, d_y, d_w)
    live = (order >= 0)[:, None]
    a = order.clamp(min=0).long()
    want = torch.where(live, d_out[a // k].double() * w.double().flatten()[a][:, None], 0.0)
    near(d_y, want, 2.0 ** -24 * want.abs(), dtype)
    terms = torch.where((slot >= 0)[..., None], y[slot.clamp(min=0).long()].double() * d_out[:, None, :].double(), 0.0)
    near(d_w, terms.sum(2), terms.abs().sum(2) * H * 2.0 ** -24, weight)       # H steps at most


@pytest.mark.parametrize("P", [48, 49])
def test_most_groups(P):
    """65535 groups, nearly all of them empty, the last ones not."""
    g = gen(P)
    E, N, K, M = 65535, 24, 48, 700
    sizes = torch.zeros(E, dtype=torch.int64)
    some_groups = [0, 1, 63, 64, 4095, 30000, 65533, 65534]
    sizes[some_groups] = torch.tensor([70, 1, 0, 200, 64, 33, 129, 100])
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)]).to(torch.int32).cuda()
    a, b, sa, sb = codes(g, M, K, P), codes(g, E * N, K, P), scales(g, M), scales(g, E * N).view(E, N)
    d = torch.full((M, N), -7.0, device="cuda")
    h = Q.Int8Gemm(Q.make_desc(M, N, K, "f32", lda=P, ldb=P, ldd=N, groups="rows", batch=E, b_stride_l=N * P, b_scale_l=N))
    h.run(a, sa, b, sb, d, offsets=offsets)
    at = offsets.tolist()
    for e in some_groups:
        r = slice(at[e], at[e + 1])
        if at[e + 1] > at[e]:
            close(d[r], *reference(a[r], sa[r], b[e * N: (e + 1) * N], sb[e], "f32"))
    assert (d[at[-1]:] == -7.0).all()
