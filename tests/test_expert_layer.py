"""The operators together, as an expert layer uses them: routing, quantised rows in expert order,
the grouped products with their activation and gates, and the layer's gradients."""
import pytest
import torch

from hierarchical_tiling_amd import htroute as R
from hierarchical_tiling_amd import htscaled as S
from scaled_util import BLOCK, close, reference, spread_scales, up, values

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


def quantised(x, both=False, block_rows=1, **kw):
    """(q, scale) of x, and (qt, scale_t) with both; rows padded to 16 bytes."""
    rows = x.shape[0] if kw.get("row_index") is None else kw["row_index"].numel()
    cols = x.shape[1]
    q = torch.zeros(rows, up(cols, 16) * 16, dtype=torch.uint8, device="cuda")
    qt = torch.zeros(cols, up(rows, 16) * 16, dtype=torch.uint8, device="cuda") if both else None
    if block_rows == 1:
        s = torch.empty(up(cols, BLOCK), rows, device="cuda").t()
        st = torch.empty(up(rows, BLOCK), cols, device="cuda").t() if both else None
    else:
        s, st = torch.empty(up(rows, BLOCK), up(cols, BLOCK), device="cuda"), None
    S.quantize(x, q[:, :cols], s, qt[:, :rows] if both else None, st, block_rows=block_rows, pad=True, **kw)
    return (q, s, qt, st) if both else (q, s)


def grouped(a, sa, b, sb, offsets, M, N, K, out="bf16", **kw):
    E = b.shape[0]
    h = S.ScaledGemm(S.make_desc(M, N, K, out, lda=a.stride(0), ldb=b.stride(1), ldd=N, a_scale_strides=sa.stride(),
                                 b_scale_strides=sb.stride()[1:], groups="rows", batch=E, b_stride_l=b.stride(0),
                                 b_scale_l=sb.stride(0), act=kw.get("act", "none"), row_scale="row_scale" in kw))
    d = torch.zeros(M, N, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
    h.run(a, sa, b, sb, d, offsets=offsets, row_scale=kw.get("row_scale"))
    return d


@pytest.mark.parametrize("T,E,k,H,F", [(1, 8, 2, 256, 384), (53, 8, 3, 256, 200), (700, 6, 2, 400, 512)])
def test_forward(T, E, k, H, F):
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn(T, E, generator=g, device="cuda")
    gate, ids = torch.softmax(logits, 1).topk(k, dim=1)
    ids = ids.to(torch.int32)
    w1, w2 = (torch.randn(E, n, m, generator=g, device="cuda") * m ** -0.5 for n, m in ((F, H), (H, F)))
    W1, W2 = ([torch.stack(t) for t in zip(*(quantised(w, block_rows=128) for w in ws))] for ws in (w1, w2))
    rows = T * k
    counts, offsets, order, slot = (torch.empty(n, **I32) for n in (E, E + 1, rows, T * k))
    ws = torch.empty(R.workspace_size(T, k, E), dtype=torch.uint8, device="cuda")
    R.route(ids, counts, offsets, order, slot, workspace=ws)
    a, sa = quantised(x, row_index=order, index_div=k)
    h = grouped(a, sa, *W1, offsets, rows, F, H, act="silu")
    b, sb = quantised(h)
    weight = gate.flatten()[order.long()].contiguous()
    y = grouped(b, sb, *W2, offsets, rows, H, F, row_scale=weight)
    out = torch.zeros(T, H, device="cuda").index_add_(0, order.long() // k, y.float())
    # step by step in 64 bits, each from the step's own inputs
    at = offsets.tolist()
    total = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        r = slice(at[e], at[e + 1])
        if at[e] == at[e + 1]:
            continue
        tokens = order[r].long() // k
        assert torch.equal(ids[tokens, order[r].long() % k], torch.full_like(tokens, e, dtype=torch.int32))
        back = values(a[r, :H]) * spread_scales(sa[r], at[e + 1] - at[e], H, 1)
        # half a step of e4m3: 2^-4 of the value, or 2^-10 of its scale among the least ones
        step = torch.maximum(x[tokens].double().abs() * 2.0 ** -4, spread_scales(sa[r], len(tokens), H, 1) * 2.0 ** -10)
        assert ((back - x[tokens].double()).abs() <= step * 1.001).all()
        close(h[r], *reference(a[r, :H], sa[r], W1[0][e, :, :H], W1[1][e], 128, "bf16", act="silu"))
        want, tol = reference(b[r, :F], sb[r], W2[0][e, :, :F], W2[1][e], 128, "bf16", row_scale=weight[r])
        close(y[r], want, tol)
        total.index_add_(0, tokens, want)
    assert (out.double() - total).norm() <= 2.0 ** -8 * total.norm() + 1e-30


@pytest.mark.parametrize("T,E,k,H,F", [(90, 5, 2, 256, 200), (600, 4, 3, 384, 256)])
def test_gradients(T, E, k, H, F):
    """d x = dy W and d W = dy^T x of the grouped product y = x W^T, from the transposed codes that
    one quantisation of each operand writes, against the formulas in 64 bits."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    w = torch.randn(E, F, H, generator=g, device="cuda") * H ** -0.5
    rows = T * k + E * 127
    counts, offsets, order, slot = (torch.empty(n, **I32) for n in (E, E + 1, rows, T * k))
    ws = torch.empty(R.workspace_size(T, k, E), dtype=torch.uint8, device="cuda")
    R.route(ids, counts, offsets, order, slot, align=128, workspace=ws)
    dy_flat = torch.randn(T * k, F, generator=g, device="cuda").to(torch.bfloat16)
    x_q, x_s, x_qt, x_st = quantised(x, both=True, row_index=order, index_div=k)
    d_q, d_s, d_qt, d_st = quantised(dy_flat, both=True, row_index=order)
    w_t, w_s = [], []
    for e in range(E):      # the transposed weight, with the blocks' scales transposed
        qt = torch.zeros(H, up(F, 16) * 16, dtype=torch.uint8, device="cuda")
        s = torch.empty(up(F, BLOCK), up(H, BLOCK), device="cuda")
        S.quantize(w[e], None, s, qt[:, :F], block_rows=128, pad=True)
        w_t.append(qt)
        w_s.append(s.t().contiguous())
    w_t, w_s = torch.stack(w_t), torch.stack(w_s)
    dx = grouped(d_q, d_s, w_t, w_s, offsets, rows, H, F)
    h = S.ScaledGemm(S.make_desc(F, H, rows, "f32", lda=d_qt.stride(0), ldb=x_qt.stride(0), ldd=H, b_block=1,
                                 a_scale_strides=d_st.stride(), b_scale_strides=x_st.stride(), groups="k", batch=E,
                                 d_stride_l=F * H))
    dw = torch.empty(E, F, H, device="cuda")
    h.run(d_qt, d_st, x_qt, x_st, dw, offsets=offsets)
    at = offsets.tolist()
    for e in range(E):
        r = slice(at[e], at[e + 1])
        n = at[e + 1] - at[e]
        if n:
            close(dx[r], *reference(d_q[r, :F], d_s[r], w_t[e][:, :F], w_s[e], 128, "bf16"))
        s = slice(at[e] // BLOCK, at[e + 1] // BLOCK)
        close(dw[e], *reference(d_qt[:, r], d_st[:, s], x_qt[:, r], x_st[:, s], 1, "f32"))
        # and the formula on the unquantised operands, off by the codes' rounding alone: a relative
        # 2^-4 for each factor at most, so (1 + 2^-4)^2 - 1 < 2^-2.9 of the sum of the sizes
        live = order[r][order[r] >= 0].long()
        dy, xs = dy_flat[live].double(), x[live // k].double()
        want, size = dy.t() @ xs, dy.t().abs() @ xs.abs()
        if live.numel():
            assert ((dw[e].double() - want).abs() <= 2.0 ** -2.9 * size + 1e-6).all()
        else:
            assert (dw[e] == 0).all()


def test_on_another_stream():
    """The layer's first half on a side stream gives what it gives on the default one."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    T, E, k, H, F = 300, 16, 2, 256, 256
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    w, ws_scale = [torch.stack(t) for t in zip(*(quantised(torch.randn(F, H, generator=g, device="cuda"), block_rows=128)
                                                 for _ in range(E)))]

    def layer():
        counts, offsets, order = (torch.empty(n, **I32) for n in (E, E + 1, T * k))
        R.route(ids, counts, offsets, order, workspace=torch.empty(R.workspace_size(T, k, E), dtype=torch.uint8, device="cuda"))
        a, sa = quantised(x, row_index=order, index_div=k)
        return grouped(a, sa, w, ws_scale, offsets, T * k, F, H, act="silu")

    want = layer()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = layer()
    side.synchronize()
    assert torch.equal(got, want)
