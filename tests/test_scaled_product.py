"""Block-scaled e4m3 products on the GPU against a 64-bit reference."""
import pytest
import torch

from hierarchical_tiling_amd import htscaled as S
from hierarchical_tiling_amd.htgemm import GemmError
from scaled_util import BLOCK, close, codes, reference, up

pytestmark = pytest.mark.gpu

OUT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def scales(g, *shape):
    return torch.exp(torch.randn(*shape, generator=g, device="cuda")) * 1e-2


class Problem:
    """One product's operands, with a pitch, an offset of the bases and scale layouts of choice."""

    def __init__(self, M, N, K, out="bf16", b_block=128, seed=0, pad=0, off=0, k_major_scales=True, spread=0.0):
        g = gen(seed)
        self.M, self.N, self.K, self.out, self.b_block = M, N, K, out, b_block
        self.lda, self.ldb, self.ldd = K + pad, K + pad, N + (3 if pad else 0)

        def bytes_of(rows):
            full = torch.full((rows * (K + pad) + off + 16,), 0x7f, dtype=torch.uint8, device="cuda")
            view = full[off: off + rows * (K + pad)].view(rows, K + pad)
            view[:, :K] = codes(g, rows, K, spread)
            return full, view

        self.a_all, self.a_v = bytes_of(M)
        self.b_all, self.b_v = bytes_of(N)
        kb, nb = up(K, BLOCK), up(N, b_block)
        sa, sb = scales(g, M, kb), scales(g, nb, kb)
        self.sa = sa.t().contiguous().t() if k_major_scales else sa
        self.sb = sb.t().contiguous().t() if k_major_scales else sb
        self.a, self.b = self.a_v[:, :K], self.b_v[:, :K]
        self.bias = torch.randn(N, generator=g, device="cuda").to(OUT[out])
        self.c = torch.randn(M, self.ldd, generator=g, device="cuda").to(OUT[out])
        self.row_scale = torch.randn(M, generator=g, device="cuda")

    def desc(self, **kw):
        return S.make_desc(self.M, self.N, self.K, self.out, lda=self.lda, ldb=self.ldb, ldd=self.ldd,
                           b_block=self.b_block, a_scale_strides=self.sa.stride(), b_scale_strides=self.sb.stride(), **kw)

    def check(self, act="none", alpha=1.0, beta=0.0, bias=False, row_scale=False, in_place=False, **kw):
        h = S.ScaledGemm(self.desc(act=act, bias=bias, row_scale=row_scale, ldc=self.ldd if beta else 0, **kw))
        ws = torch.empty(max(h.workspace_bytes, 16), dtype=torch.uint8, device="cuda")
        d = self.c.clone() if in_place else torch.full((self.M, self.ldd), -7.0, dtype=OUT[self.out], device="cuda")
        h.run(self.a_v, self.sa, self.b_v, self.sb, d, C=(d if in_place else self.c) if beta else None,
              bias=self.bias if bias else None, row_scale=self.row_scale if row_scale else None, alpha=alpha,
              beta=beta, workspace=ws)
        want, tol = reference(self.a, self.sa, self.b, self.sb, self.b_block, self.out, alpha, beta,
                              self.c[:, :self.N], self.bias if bias else None,
                              self.row_scale if row_scale else None, act)
        close(d[:, :self.N], want, tol)
        if self.ldd > self.N:   # the columns past N stay as they were
            left = self.c if in_place else torch.full_like(d, -7.0)
            assert torch.equal(d[:, self.N:], left[:, self.N:])
        return h


SHAPES = [(1, 1, 16), (1, 16, 128), (3, 5, 144), (16, 33, 256), (17, 64, 272), (33, 130, 528), (64, 64, 1024),
          (65, 257, 400), (100, 128, 2064), (129, 140, 640), (200, 1000, 1040), (257, 300, 4096), (513, 1025, 384)]


@pytest.mark.parametrize("out,b_block", [("bf16", 128), ("bf16", 1), ("f32", 128), ("f32", 1)])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(shape, out, b_block):
    Problem(*shape, out=out, b_block=b_block, seed=sum(shape), spread=1.0).check()


@pytest.mark.parametrize("shape", [(1, 4096, 2048), (5, 8192, 512), (40, 4096, 1024), (64, 2048, 256),
                                   (300, 4096, 256), (4096, 4096, 256), (4000, 4100, 272), (4099, 4097, 1040)])
@pytest.mark.parametrize("out,b_block", [("bf16", 128), ("f32", 1), ("bf16", 1), ("f32", 128)])
def test_wide(shape, out, b_block):
    Problem(*shape, out=out, b_block=b_block, seed=1).check(act="silu", bias=True)


@pytest.mark.parametrize("shape,tile", [((333, 4096, 4224), 64), ((257, 5000, 3984), 64), ((130, 7168, 4112), 64),
                                        ((1000, 4096, 3984), 128), ((1000, 3900, 4112), 128),
                                        # near the sizes where another kernel is chosen
                                        ((130, 7168, 2064), 0), ((257, 8000, 1936), 0), ((2000, 2100, 2192), 0)])
@pytest.mark.parametrize("out,b_block", [("bf16", 128), ("f32", 1), ("bf16", 1), ("f32", 128)])
def test_two_halves_of_k(shape, tile, out, b_block):
    """Odd and even numbers of blocks, whole and partial last ones, between the two halves of the
    waves; with C, an activation and bias, and for whole and ragged columns."""
    p = Problem(*shape, out=out, b_block=b_block, seed=3, spread=1.0)
    h = p.check(act="gelu", bias=True, row_scale=True, alpha=0.5, beta=0.25)
    assert not tile or h.info.name.decode() == f"tile_{tile}x128_w2x2x2"


@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 3, 127), (7, 9, 129), (70, 65, 300), (16, 64, 1001)])
@pytest.mark.parametrize("off,pad", [(0, 0), (1, 0), (0, 5), (3, 16)])
def test_any_alignment(shape, off, pad):
    """Odd K, bases and leading dimensions; the bytes of the pitch are NaN codes."""
    for out, b_block in (("bf16", 128), ("f32", 1)):
        Problem(*shape, out=out, b_block=b_block, seed=5, off=off, pad=pad, k_major_scales=off == 0).check()


@pytest.mark.parametrize("shape", [(20, 96, 256), (150, 260, 512), (1, 500, 1024)])
def test_pitch_and_scale_layouts(shape):
    for pad in (16, 48):
        Problem(*shape, seed=6, pad=pad, k_major_scales=False).check()
        Problem(*shape, seed=6, pad=pad, b_block=1, out="f32", k_major_scales=False).check()


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_epilogue(act, out):
    for shape in ((9, 70, 256), (150, 384, 512), (320, 260, 256)):
        Problem(*shape, out=out, seed=7).check(act=act, alpha=0.75, beta=-1.5, bias=True, row_scale=True)
        Problem(*shape, out=out, seed=8, pad=16).check(act=act, beta=1.0, in_place=True)


@pytest.mark.parametrize("split", [2, 3, 7, 64])
def test_split_k(split):
    for shape in ((5, 40, 2064), (100, 200, 1040), (260, 130, 512)):
        h = Problem(*shape, seed=9, spread=1.0).check(bias=True, act="gelu", split_k=split)
        assert 1 < h.info.split_k <= split
        assert h.workspace_bytes == h.info.split_k * shape[0] * shape[1] * 4


def test_empty_and_no_k():
    Problem(4, 6, 0, seed=1).check(bias=True)
    Problem(4, 6, 0, seed=1, out="f32").check(beta=2.0, act="relu")
    for M, N in ((0, 5), (5, 0)):
        h = S.ScaledGemm(S.make_desc(M, N, 128, lda=128, ldb=128, ldd=N, a_scale_strides=(1, M), b_scale_strides=(1, 1)))
        h.run(None, None, None, None, None)


def test_beta_zero_reads_no_c():
    p = Problem(40, 50, 256, seed=2)
    p.c.fill_(float("nan"))
    h = S.ScaledGemm(p.desc(ldc=p.ldd))
    d = torch.empty(40, 50, dtype=torch.bfloat16, device="cuda")
    h.run(p.a_v, p.sa, p.b_v, p.sb, d, C=p.c, beta=0.0)
    assert not torch.isnan(d).any()


def test_nan_scale_and_code_reach_their_outputs_only():
    p = Problem(130, 260, 512, seed=3)
    p.sa[5, 2] = float("nan")
    p.b_v[17, 200] = 0x7f
    h = S.ScaledGemm(p.desc())
    d = torch.empty(130, 260, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(16, h.workspace_bytes), dtype=torch.uint8, device="cuda")
    h.run(p.a_v, p.sa, p.b_v, p.sb, d, workspace=ws)
    nan = torch.zeros(130, 260, dtype=torch.bool, device="cuda")
    nan[5] = True
    nan[:, 17] = True
    assert torch.equal(torch.isnan(d), nan)


@pytest.mark.parametrize("M,N,K", [(3, 50, 256), (70, 130, 144), (33, 40, 100)])
def test_batch(M, N, K):
    L = 3
    ps = [Problem(M, N, K, seed=20 + i) for i in range(L)]
    a, b = (torch.stack([getattr(p, n)[:, :K] for p in ps]).contiguous() for n in ("a_v", "b_v"))
    sa, sb = (torch.stack([getattr(p, n).contiguous() for p in ps]) for n in ("sa", "sb"))
    kb, nb = up(K, BLOCK), up(N, BLOCK)
    h = S.ScaledGemm(S.make_desc(M, N, K, lda=K, ldb=K, ldd=N, a_scale_strides=(kb, 1), b_scale_strides=(kb, 1), batch=L,
                                 a_stride_l=M * K, b_stride_l=N * K, d_stride_l=M * N, a_scale_l=M * kb, b_scale_l=nb * kb))
    d = torch.empty(L, M, N, dtype=torch.bfloat16, device="cuda")
    h.run(a, sa, b, sb, d)
    for i, p in enumerate(ps):
        close(d[i], *reference(p.a, p.sa, p.b, p.sb, 128, "bf16"))


def clamped(offsets, top):
    out, run = [], 0
    for o in offsets:
        run = max(run, min(max(o, 0), top))
        out.append(run)
    return out


ROWS = [([0, 3, 3, 20, 21, 40], 40), ([0, 0, 0, 130], 130), ([2, 5, 9], 12), ([0, 300, 310, 700], 700),
        ([0, 50, 20, 90, 200], 80), ([-5, 4, 4], 9), ([0] * 70 + [1, 2, 5], 6), ([0, 16, 32, 48, 64], 64), ([0, 0], 7)]


@pytest.mark.parametrize("case", range(len(ROWS)))
@pytest.mark.parametrize("N,K,out", [(130, 256, "bf16"), (64, 144, "f32"), (40, 100, "bf16"), (1030, 512, "bf16")])
def test_groups_of_rows(case, N, K, out):
    offsets, M = ROWS[case]
    G = len(offsets) - 1
    g = gen(case)
    p = Problem(M, N, K, out=out, seed=case)
    b = torch.stack([codes(g, N, K) for _ in range(G)])
    sb = scales(g, G, up(N, BLOCK), up(K, BLOCK))
    kb = up(K, BLOCK)
    h = S.ScaledGemm(S.make_desc(M, N, K, out, lda=p.lda, ldb=K, ldd=N, ldc=N, a_scale_strides=p.sa.stride(),
                                 b_scale_strides=(kb, 1), groups="rows", batch=G, b_stride_l=N * K,
                                 b_scale_l=sb.shape[1] * kb, bias=True, row_scale=True, act="silu"))
    c = p.c[:, :N].contiguous()
    d = torch.full((M, N), -7.0, dtype=OUT[out], device="cuda")
    h.run(p.a_v, p.sa, b, sb, d, C=c, beta=0.5, bias=p.bias, row_scale=p.row_scale,
          offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    lo = clamped(offsets, M)
    written = torch.zeros(M, dtype=torch.bool)
    for e in range(G):
        r = slice(lo[e], lo[e + 1])
        if lo[e + 1] > lo[e]:
            written[r] = True
            close(d[r], *reference(p.a[r], p.sa[r], b[e], sb[e], 128, out, 1.0, 0.5, c[r], p.bias, p.row_scale[r], "silu"))
    assert (d[~written.to(d.device)] == -7.0).all()


@pytest.mark.parametrize("offsets,K", [([0, 128, 128, 384, 512], 512), ([0, 256, 300], 300), ([0, 300, 300], 300),
                                       ([128, 130, 260, 400], 512), ([0, 1280, 1264], 1264), ([-3, 900, 128], 256)])
@pytest.mark.parametrize("M,N,b_block,out", [(70, 130, 1, "f32"), (20, 40, 128, "bf16"), (260, 300, 1, "f32")])
def test_groups_of_k(offsets, K, M, N, b_block, out):
    G = len(offsets) - 1
    p = Problem(M, N, K, out=out, b_block=b_block, seed=K)
    h = S.ScaledGemm(S.make_desc(M, N, K, out, lda=p.lda, ldb=p.ldb, ldd=N, ldc=N, b_block=b_block,
                                 a_scale_strides=p.sa.stride(), b_scale_strides=p.sb.stride(), groups="k", batch=G,
                                 c_stride_l=M * N, d_stride_l=M * N))
    d = torch.randn(G, M, N, device="cuda").to(OUT[out])
    c = d.clone()
    h.run(p.a_v, p.sa, p.b_v, p.sb, d, C=d, beta=1.0, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    lo = [o if o == K else o // BLOCK * BLOCK for o in clamped(offsets, K)]
    for e in range(G):
        k0, k1 = min(up(lo[e], BLOCK) * BLOCK, K), lo[e + 1]
        k1 = max(k0, k1)
        s = slice(k0 // BLOCK, up(k1, BLOCK))
        sa, sb = p.sa[:, s], p.sb[:, s]
        close(d[e], *reference(p.a[:, k0:k1], sa, p.b[:, k0:k1], sb, b_block, out, 1.0, 1.0, c[e]))


def test_captured_and_replayed():
    """A captured product (split along k) replays to the eager result with new operands in place."""
    p, q = Problem(100, 200, 1024, seed=1), Problem(100, 200, 1024, seed=2)
    h = S.ScaledGemm(p.desc(split_k=4))
    ws = torch.empty(h.workspace_bytes, dtype=torch.uint8, device="cuda")
    d, e = (torch.empty(100, 200, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    h.run(p.a_v, p.sa, p.b_v, p.sb, d, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.run(p.a_v, p.sa, p.b_v, p.sb, d, workspace=ws)
    for other in (p, q, p):
        a, b, sa, sb = other.a_v.clone(), other.b_v.clone(), other.sa.clone(), other.sb.clone()
        p.a_v.copy_(a), p.b_v.copy_(b), p.sa.copy_(sa), p.sb.copy_(sb)
        h.run(p.a_v, p.sa, p.b_v, p.sb, e, workspace=ws)
        d.fill_(-1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d, e)


def test_two_streams_at_once():
    p = Problem(300, 512, 2048, seed=4)
    h = S.ScaledGemm(p.desc(split_k=2))
    outs = []
    torch.cuda.synchronize()
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            ws = torch.empty(h.workspace_bytes, dtype=torch.uint8, device="cuda")
            d = torch.empty(300, 512, dtype=torch.bfloat16, device="cuda")
            for _ in range(3):
                h.run(p.a_v, p.sa, p.b_v, p.sb, d, workspace=ws)
            outs.append((d, ws))
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], outs[1][0])
    close(outs[0][0], *reference(p.a, p.sa, p.b, p.sb, 128, "bf16"))


def test_same_bits_every_time():
    p = Problem(520, 1100, 1040, seed=4, spread=1.0)
    h = S.ScaledGemm(p.desc())
    ws = torch.empty(max(16, h.workspace_bytes), dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(4):
        d = torch.empty(520, 1100, dtype=torch.bfloat16, device="cuda")
        h.run(p.a_v, p.sa, p.b_v, p.sb, d, workspace=ws)
        first = d if first is None else first
        assert torch.equal(d, first)


def test_every_code_is_converted_exactly():
    """All 256 codes through both matrix instructions, by a product with an identity."""
    a = torch.arange(256, dtype=torch.uint8, device="cuda").view(2, 128)
    b = torch.full((128, 128), 0, dtype=torch.uint8, device="cuda")
    b[torch.arange(128), torch.arange(128)] = 0x38    # 1.0
    one = torch.ones(2, 1, device="cuda")
    for out in ("bf16", "f32"):
        d = torch.empty(2, 128, dtype=OUT[out], device="cuda")
        for row in range(2):
            # one code at a time: a NaN code would reach every product of its row
            x = torch.zeros(128, 128, dtype=torch.uint8, device="cuda")
            x[torch.arange(128), torch.arange(128)] = a[row]
            full = torch.empty(128, 128, dtype=OUT[out], device="cuda")
            h = S.ScaledGemm(S.make_desc(128, 128, 128, out, lda=128, ldb=128, ldd=128, a_scale_strides=(0, 0),
                                         b_scale_strides=(0, 0), split_k=1))
            h.run(x, one, b, one, full)
            d[row] = full.diagonal()
        want = a.view(torch.float8_e4m3fn).float()
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(d), nan)
        assert torch.equal(d.float()[~nan], want[~nan])


def test_refusals_at_run():
    p = Problem(64, 64, 256, seed=1)
    h = S.ScaledGemm(p.desc(split_k=2))
    d = torch.empty(64, 64, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(h.workspace_bytes, dtype=torch.uint8, device="cuda")
    ok = dict(A=p.a_v, a_scale=p.sa, B=p.b_v, b_scale=p.sb, D=d, workspace=ws)
    for change, status in (({"workspace": None}, 1), ({"workspace": ws.data_ptr() + 8}, 1), ({"A": None}, 1),
                           ({"b_scale": None}, 1), ({"D": None}, 1), ({"bias": p.bias}, 1), ({"beta": 1.0}, 1),
                           ({"offsets": torch.zeros(2, dtype=torch.int32, device="cuda")}, 1),
                           ({"row_scale": p.row_scale}, 1), ({"A": p.a_v.cpu()}, 1), ({"D": d.data_ptr() + 1}, 4), ({"a_scale": p.sa.data_ptr() + 2}, 4)):
        with pytest.raises(GemmError) as err:
            h.run(**{**ok, **change})
        assert err.value.status == status, change
    h.close()
    h.close()


@pytest.mark.parametrize("rows,E,N,K,out", [
    (3000, 6, 640, 512, "bf16"), (700, 300, 96, 256, "bf16"), (2600, 3, 300, 400, "bf16"),
    (3000, 6, 640, 512, "f32"), (700, 300, 96, 256, "f32"), (2600, 3, 300, 400, "f32"),
    (8190, 32, 4096, 2048, "bf16")])
def test_many_groups_and_large_groups(rows, E, N, K, out):
    """Groups of more than a tile's rows, and more groups than lanes, against the product of each;
    the last through the ping-pong kernel."""
    g = gen(rows)
    p = Problem(rows, N, K, out=out, seed=rows, spread=1.0)
    to = torch.sort(torch.randint(0, E, (rows,), generator=g, device="cuda")).values
    counts = torch.bincount(to, minlength=E)
    offsets = torch.cat([torch.zeros_like(counts[:1]), counts.cumsum(0)]).to(torch.int32)
    b = torch.stack([codes(g, N, K) for _ in range(E)])
    kb = up(K, BLOCK)
    sb = scales(g, E, up(N, BLOCK), kb)
    h = S.ScaledGemm(S.make_desc(rows, N, K, out, lda=K, ldb=K, ldd=N, a_scale_strides=p.sa.stride(), b_scale_strides=(kb, 1),
                                 groups="rows", batch=E, b_stride_l=N * K, b_scale_l=sb.shape[1] * kb))
    assert (h.info.name == b"pingpong_256x256") == (rows == 8190)
    d = torch.empty(rows, N, dtype=OUT[out], device="cuda")
    h.run(p.a_v, p.sa, b, sb, d, offsets=offsets)
    at = offsets.tolist()
    for e in range(E):
        r = slice(at[e], at[e + 1])
        if at[e + 1] > at[e]:
            close(d[r], *reference(p.a[r], p.sa[r], b[e], sb[e], 128, out))


def test_every_kernel_is_chosen_somewhere():
    """The products of this file and the sizes of a decode, a prompt and a training step between
    them run every kernel."""
    names = set()
    for M, N, K, out in ((1, 4096, 4096, "bf16"), (17, 4096, 4096, "bf16"), (32, 8192, 8192, "bf16"), (64, 8192, 4096, "bf16"),
                         (333, 4096, 8192, "bf16"), (1000, 4096, 512, "bf16"), (1000, 4096, 4096, "bf16"),
                         (2000, 4096, 1024, "bf16"), (4096, 4096, 4096, "bf16"), (4096, 8192, 1024, "f32"), (5, 7, 9, "f32")):
        h = S.ScaledGemm(S.make_desc(M, N, K, out, lda=K, ldb=K, ldd=N, a_scale_strides=(1, M), b_scale_strides=(up(K, 128), 1)))
        names.add(h.info.name.decode())
    assert names == {"narrow_64x64", "stream_16x32_w4", "stream_16x16_w8", "stream_32x32_w4", "stream_64x32_w4",
                     "tile_64x128_w2x2", "tile_64x128_w2x2x2", "tile_128x128_w2x2", "tile_128x128_w2x2x2",
                     "pingpong_256x256"}
