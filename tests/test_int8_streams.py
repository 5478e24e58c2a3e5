"""The products in 8-bit integers, the quantisation and the rows of a routing in captured graphs, on other
streams, from two threads, and at sizes past 31 and 32 bits."""
import threading

import pytest
import torch

from hierarchical_tiling_amd import htint8 as Q
from hierarchical_tiling_amd import htroute as R
from int8_util import I32, close, codes, gen, quantised, reference, routing, scales

pytestmark = pytest.mark.gpu


class Work:
    """One call of each operator on buffers of its own; k in slices, so that the product has a
    workspace."""

    def __init__(self, seed, T=50, E=6, k=3, H=700, N=300, split=4):
        g = gen(seed)
        self.k = k
        self.order, self.slot, self.offsets = routing(g, T, E, k, 8, [i % 5 != 4 for i in range(T)])
        n = self.order.numel()
        self.x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
        self.w, self.d_out = torch.rand(T, k, generator=g, device="cuda"), torch.randn(T, N, generator=g, device="cuda")
        self.rows = torch.empty(n, H, dtype=torch.bfloat16, device="cuda")
        pitch = -(-H // 16) * 16
        self.a, self.sa = torch.empty(n, pitch, dtype=torch.int8, device="cuda")[:, :H], torch.empty(n, device="cuda")
        self.b, self.sb = codes(g, N, H, pitch), scales(g, N)
        self.y, self.out = torch.empty(n, N, device="cuda"), torch.empty(T, N, device="cuda")
        self.d_y, self.d_w, self.d_x = torch.empty(n, N, device="cuda"), torch.empty(T, k, device="cuda"), torch.empty_like(self.x)
        self.h = Q.Int8Gemm(Q.make_desc(n, N, H, "f32", lda=pitch, ldb=pitch, ldd=N, split_k=split))
        self.ws = torch.empty(self.h.workspace_bytes, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()

    def run(self, stream=None):
        R.gather(self.x, self.order, self.slot, self.rows, stream=stream)
        Q.quantize(self.rows, self.a, self.sa, stream=stream)
        self.h.run(self.a, self.sa, self.b, self.sb, self.y, workspace=self.ws, stream=stream)
        R.combine(self.y, self.slot, self.out, weights=self.w, stream=stream)
        R.combine_grad(self.d_out, self.y, self.order, self.slot, self.w, self.d_y, self.d_w, stream=stream)
        R.combine(self.rows, self.slot, self.d_x, stream=stream)

    def results(self):
        return [t.clone() for t in (self.rows, self.a, self.sa, self.y, self.out, self.d_y, self.d_w, self.d_x)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_and_replayed():
    w = Work(1)
    w.run()
    want = w.results()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        w.run()
    for i in range(4):
        for t in (w.rows, w.a, w.sa, w.y, w.out, w.d_y, w.d_w, w.d_x, w.ws):
            t.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(w.results(), want)
        w.x.mul_(-1)          # new inputs in the same places, and the program's own eager work between
        w.run()
        want = w.results()


def test_two_graphs_with_a_workspace_each():
    a, b = Work(2), Work(3)
    graphs, wants = [], []
    for w in (a, b):
        w.run()
        wants.append(w.results())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            w.run()
        graphs.append(graph)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        for st, graph in ((s, graphs[0]), (t, graphs[1])):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    assert same(a.results(), wants[0]) and same(b.results(), wants[1])


def test_streams_by_object_and_by_handle():
    w = Work(4)
    w.run()
    want = w.results()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        w.out.zero_()
        torch.cuda.synchronize()
        w.run(stream)
        side.synchronize()
        assert same(w.results(), want)


def test_two_threads():
    works = [Work(5), Work(6)]
    wants = []
    for w in works:
        w.run()
        wants.append(w.results())
    errors = []

    def many(w):
        try:
            stream = torch.cuda.Stream()
            for _ in range(50):
                w.run(stream)
            stream.synchronize()
        except Exception as e:      # shown by the assertion below
            errors.append(e)

    threads = [threading.Thread(target=many, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    assert all(same(w.results(), want) for w, want in zip(works, wants))


def test_one_handle_in_two_threads_with_a_workspace_each():
    g = gen(7)
    h = Q.Int8Gemm(Q.make_desc(70, 200, 2000, "f32", lda=2000, ldb=2000, ldd=200, split_k=5))
    sets = [(codes(g, 70, 2000), scales(g, 70), codes(g, 200, 2000), scales(g, 200), torch.empty(70, 200, device="cuda"),
             torch.empty(h.workspace_bytes, dtype=torch.uint8, device="cuda")) for _ in range(2)]
    torch.cuda.synchronize()

    def many(s):
        stream = torch.cuda.Stream()
        for _ in range(50):
            h.run(*s[:5], workspace=s[5], stream=stream)
        stream.synchronize()

    threads = [threading.Thread(target=many, args=(s,)) for s in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for s in sets:
        close(s[4], *reference(*s[:4], "f32"))


def test_runs_give_the_same_bits():
    w = Work(8, T=900, H=1000, N=1000, split=0)
    w.run()
    want = w.results()
    for _ in range(5):
        w.run()
        assert same(w.results(), want)


# ---- sizes past 31 and 32 bits ------------------------------------------------------------------
def test_quantisation_past_32_bits():
    """Rows whose first value lies past 2^31 and 2^32 values."""
    rows, cols = 70000, 65536
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    some = torch.tensor([0, 32767, 32768, 65535, 65536, 69999], device="cuda")
    g = gen(1)
    x[some] = torch.randn(6, cols, generator=g, device="cuda").to(torch.bfloat16)
    q, scale = torch.empty(rows, cols, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    Q.quantize(x, q, scale)
    want = quantised(x[some].float())
    assert torch.equal(q[some], want[0]) and torch.equal(scale[some], want[1])
    others = torch.ones(rows, dtype=torch.bool, device="cuda")
    others[some] = False
    assert (scale[others] == 2.0 ** -126).all() and not q.view(torch.int64).view(rows, -1)[others].any()


def test_rows_past_32_bits():
    """70000 rows of 65536 bf16 values, at both ends."""
    T, k, H = 35000, 2, 65536
    order = torch.arange(T * k, **I32).flip(0).contiguous()
    slot = torch.empty(T * k, **I32)
    slot[order.long()] = torch.arange(T * k, **I32)
    slot = slot.view(T, k)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    some = torch.tensor([0, 1, 16384, 16385, 32768, T - 1], device="cuda")
    x[some] = torch.randn(6, H, generator=gen(2), device="cuda").to(torch.bfloat16)
    y = torch.full((T * k, H), 7.0, dtype=torch.bfloat16, device="cuda")
    R.gather(x, order, slot, y)
    for j in range(k):
        assert torch.equal(y[slot[some, j].long()], x[some])
    assert torch.count_nonzero(y) == k * torch.count_nonzero(x)
    out = torch.empty_like(x)
    R.combine(y, slot, out)
    assert torch.equal(out, (x.float() * 2).to(torch.bfloat16))
    w, d_w = torch.full((T, k), 0.5, device="cuda"), torch.empty(T, k, device="cuda")
    d_y = torch.full_like(y, 7.0)
    R.combine_grad(x, y, order, slot, w, d_y, d_w)
    assert torch.equal(d_y, y * 0.5)
    dots = x[some].double().square().sum(1)
    assert ((d_w[some].double() - dots[:, None]).abs() <= H * 2.0 ** -24 * dots[:, None]).all()
    assert torch.count_nonzero(d_w) == 6 * k


@pytest.mark.parametrize("M,N,K", [(40000, 60000, 130), (300, 33000, 65536)])
def test_products_past_32_bits(M, N, K):
    """An output of 2.4 * 10^9 values; a B of 2.2 * 10^9 codes."""
    g = gen(M)
    P = -(-K // 16) * 16
    a, b, sa, sb = codes(g, M, K, P), codes(g, N, P)[:, :K], scales(g, M), scales(g, N)
    d = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    h = Q.Int8Gemm(Q.make_desc(M, N, K, lda=P, ldb=P, ldd=N))
    h.run(a, sa, b, sb, d, workspace=torch.empty(h.workspace_bytes, dtype=torch.uint8, device="cuda"))
    rows = torch.tensor([0, 1, M // 2, M - 1], device="cuda")
    close(d[rows], *reference(a[rows], sa[rows], b, sb, "bf16"))
    cols = torch.tensor([0, N // 2, N - 1], device="cuda")
    close(d[:, cols], *reference(a, sa, b[cols], sb[cols], "bf16"))


def test_rows_of_a_product_far_apart():
    """Leading dimensions of 2^24 bytes and more: past the 31 bits of a tile's offsets the kernels that load at
    any byte take the product."""
    g = gen(3)
    M, N, K, ld = 130, 140, 300, (1 << 24) + 16
    room_a, room_b = (torch.empty(n * ld, dtype=torch.int8, device="cuda") for n in (M, N))
    a, b = room_a.view(M, ld)[:, :K], room_b.view(N, ld)[:, :K]
    a.copy_(codes(g, M, K))
    b.copy_(codes(g, N, K))
    sa, sb, d = scales(g, M), scales(g, N), torch.empty(M, N, device="cuda")
    h = Q.Int8Gemm(Q.make_desc(M, N, K, "f32", lda=ld, ldb=ld, ldd=N))
    assert h.info.name.startswith(b"any")
    h.run(a, sa, b, sb, d, workspace=torch.empty(h.workspace_bytes, dtype=torch.uint8, device="cuda"))
    close(d, *reference(a, sa, b, sb, "f32"))
    for ld in ((1 << 23) - 48, 8355840 - 16):       # the largest that tile offsets allow, and near it
        a, b = (r[: n * ld].view(n, ld)[:, :K] for r, n in ((room_a, M), (room_b, N)))
        a.copy_(codes(g, M, K))
        b.copy_(codes(g, N, K))
        h = Q.Int8Gemm(Q.make_desc(M, N, K, "f32", lda=ld, ldb=ld, ldd=N))
        h.run(a, sa, b, sb, d, workspace=torch.empty(h.workspace_bytes, dtype=torch.uint8, device="cuda"))
        close(d, *reference(a, sa, b, sb, "f32"))
