"""The operators together, as an expert layer uses them: in 8-bit integers (routing, rows quantised by
expert, products with the gated activation between them, rows joined by their gates), and in training
(tokens to their experts' rows, the library's grouped bf16 product, joined again, with gradients)."""
import pytest
import torch

from hierarchical_tiling_amd import htgemm as H
from hierarchical_tiling_amd import htint8 as Q
from hierarchical_tiling_amd import htroute as R
from int8_util import HALF, I32, close, gen, quantised, reference

pytestmark = pytest.mark.gpu


def routed(g, T, E, k, align, live=None):
    logits = torch.randn(T, E, generator=g, device="cuda")
    gates, ids = torch.softmax(logits, 1).topk(k, dim=1)
    rows = T * k + E * (align - 1)
    counts, offsets, order, slot = (torch.empty(n, **I32) for n in (E, E + 1, rows, T * k))
    R.route(ids.to(torch.int32).contiguous(), counts, offsets, order, slot, align=align, mask=live,
            workspace=torch.empty(R.workspace_size(T, k, E), dtype=torch.uint8, device="cuda"))
    return gates.contiguous(), offsets, order, slot.view(T, k)


def grouped(a, sa, w, sw, offsets, d):
    (M, K), (E, N, P) = a.shape, w.shape
    h = Q.Int8Gemm(Q.make_desc(M, N, K, "bf16", lda=a.stride(0), ldb=P, ldd=N, groups="rows", batch=E, b_stride_l=N * P,
                               b_scale_l=N))
    h.run(a, sa, w, sw, d, offsets=offsets)


@pytest.mark.parametrize("T,E,k,Hd,F", [(1, 8, 2, 256, 384), (53, 8, 3, 250, 200), (700, 6, 2, 400, 515), (40, 64, 8, 128, 64)])
@pytest.mark.parametrize("align,masked", [(1, False), (16, True)])
def test_forward(T, E, k, Hd, F, align, masked):
    g = gen(T + Hd)
    live = (torch.rand(T, generator=g, device="cuda") < 0.7).to(torch.uint8) if masked else None
    gates, offsets, order, slot = routed(g, T, E, k, align, live)
    n = order.numel()
    x = torch.randn(T, Hd, generator=g, device="cuda").to(torch.bfloat16)
    shared = torch.randn(T, Hd, generator=g, device="cuda").to(torch.bfloat16)
    weights = []
    for rows, cols in ((2 * F, Hd), (Hd, F)):
        w = (torch.randn(E * rows, cols, generator=g, device="cuda") * cols ** -0.5).to(torch.bfloat16)
        pitch = -(-cols // 16) * 16
        q, s = torch.empty(E * rows, pitch, dtype=torch.int8, device="cuda"), torch.empty(E * rows, device="cuda")
        Q.quantize(w, q[:, :cols], s, pad=True)
        want, scale = quantised(w.float())
        assert torch.equal(q[:, :cols], want) and torch.equal(s, scale) and (q[:, cols:] == 0).all()
        weights.append((q.view(E, rows, pitch), s.view(E, rows)))
    (w1, s1), (w2, s2) = weights

    def codes(cols):
        return torch.empty(n, -(-cols // 16) * 16, dtype=torch.int8, device="cuda")[:, :cols], torch.empty(n, device="cuda")

    a, sa = codes(Hd)
    Q.quantize(x, a, sa, row_index=order, index_div=k)
    h = torch.zeros(n, 2 * F, dtype=torch.bfloat16, device="cuda")
    grouped(a, sa, w1, s1, offsets, h)
    b, sb = codes(F)
    Q.quantize(h[:, F:], b, sb, gate=h[:, :F], act="silu")
    y = torch.zeros(n, Hd, dtype=torch.bfloat16, device="cuda")
    grouped(b, sb, w2, s2, offsets, y)
    out = torch.empty(T, Hd, dtype=torch.bfloat16, device="cuda")
    R.combine(y, slot, out, weights=gates, add=shared)
    # step by step in 64 bits, each from the step's own inputs
    at = offsets.tolist()
    total = shared.double()
    size = total.abs()
    for e in range(E):
        r = slice(at[e], at[e + 1])
        if at[e] == at[e + 1]:
            continue
        tokens = order[r].long()
        real = tokens >= 0
        source = torch.where(real[:, None], x[(tokens.clamp(min=0) // k)].float(), 0.0)
        want, scale = quantised(source)
        assert torch.equal(a[r], want) and torch.equal(sa[r], scale)
        close(h[r], *reference(a[r], sa[r], w1[e][:, :Hd], s1[e], "bf16"))
        up, gate = h[r][:, F:].double(), h[r][:, :F].double()
        v = gate * torch.sigmoid(gate) * up
        # a code is off by half a step and what the activation (2^-20 of its argument) moves
        step = sb[r].double()[:, None]
        assert ((b[r].double() * step - v).abs() <= 0.5 * step * (1 + 2.0 ** -14) + (2.0 ** -20 * gate * up).abs() + 2.0 ** -21 * v.abs()).all()
        close(y[r], *reference(b[r], sb[r], w2[e][:, :F], s2[e], "bf16"))
        term = y[r][real].double() * gates.flatten()[tokens[real]].double()[:, None]
        total.index_add_(0, tokens[real] // k, term)
        size.index_add_(0, tokens[real] // k, term.abs())
    tol = size * (k + 1) * 2.0 ** -24
    assert ((out.double() - total).abs() <= tol + (total.abs() + tol) * HALF["bf16"]).all()
    if masked:
        assert torch.equal(out[live == 0], shared[live == 0])


@pytest.mark.parametrize("T,E,k,Hd,N", [(60, 5, 2, 64, 72), (300, 8, 3, 128, 136)])
def test_training_step(T, E, k, Hd, N):
    """Whole numbers small enough that all sums are exact in fp32 and all values in bf16: forward and
    gradients equal autograd's in 64 bits."""
    g = gen(T)
    small = lambda *s: torch.randint(-1, 2, s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    live = (torch.rand(T, generator=g, device="cuda") < 0.8).to(torch.uint8)
    _, offsets, order, slot = routed(g, T, E, k, 16, live)
    n = order.numel()
    x, w, d_out = small(T, Hd), small(E, N, Hd), small(T, N)
    gates = torch.randint(1, 3, (T, k), generator=g, device="cuda").float()
    rows = torch.empty(n, Hd, dtype=torch.bfloat16, device="cuda")
    R.gather(x, order, slot, rows)
    y = torch.zeros(n, N, dtype=torch.bfloat16, device="cuda")
    out, d_y, d_gates = torch.empty_like(d_out), torch.empty_like(y), torch.empty_like(gates)

    def product(a, b, d, K, M):
        h = H.Gemm(H.make_desc(n, M, K, "bf16", (K, 1), (1, K), (M, 1), batch=E, batch_strides=(0, M * K, 0, 0), ragged_m=True))
        ws = torch.empty(h.workspace_bytes, dtype=torch.uint8, device="cuda")
        H.gemm_run_grouped(h.handle, a.data_ptr(), b.data_ptr(), None, d.data_ptr(), None, None, None, offsets.data_ptr(),
                           1.0, 0.0, stream=torch.cuda.current_stream().cuda_stream, workspace=ws.data_ptr())
        torch.cuda.synchronize()

    product(rows, w, y, Hd, N)
    R.combine(y, slot, out, weights=gates)
    R.combine_grad(d_out, y, order, slot, gates, d_y, d_gates)
    d_rows = torch.zeros_like(rows)
    product(d_y, w.transpose(1, 2).contiguous(), d_rows, N, Hd)
    d_x = torch.empty_like(x)
    R.combine(d_rows, slot, d_x)
    # on the host, in 64 bits
    xd, gd = x.double().cpu().requires_grad_(), gates.double().cpu().requires_grad_()
    wd, total = w.double().cpu(), 0
    expert = torch.searchsorted(offsets.cpu()[1:].contiguous(), slot.cpu().clamp(min=0), right=True)
    ok = (slot >= 0).cpu()
    for j in range(k):
        each = torch.stack([wd[e] @ xd[t] for t, e in enumerate(expert[:, j].tolist())])
        total = total + each * (gd[:, j] * ok[:, j])[:, None]
    assert torch.equal(out.double().cpu(), total.detach().to(torch.bfloat16).double())
    assert total.abs().max() <= 256          # a whole number that bf16 holds
    total.backward(d_out.double().cpu())
    assert torch.equal(d_gates.double().cpu(), gd.grad)
    assert torch.equal(d_x.double().cpu(), xd.grad.to(torch.bfloat16).double())
