"""Products in 8-bit integers against 64-bit references: every form, type and size where a kernel can
go wrong."""
import pytest
import torch

from hierarchical_tiling_amd import htint8 as Q
from int8_util import I32, TYPE, close, codes, gen, reference, scales

pytestmark = pytest.mark.gpu


def padded(K):
    return -(-K // 16) * 16


def run(M, N, K, out="bf16", lda=None, ldb=None, ldd=None, split_k=0, alpha=1.0, beta=0.0, bias=False, act="none",
        seed=0, offset=0):
    """One product into a D whose surroundings are watched; (D, info)."""
    g = gen(seed + M + 3 * N + 7 * K)
    lda, ldb, ldd = lda or max(padded(K), 16), ldb or max(padded(K), 16), ldd or N
    a, b = codes(g, M, K, lda), codes(g, N, K, ldb)
    if offset:      # bases off 16 bytes
        room = torch.full((M * lda + 64,), 77, dtype=torch.int8, device="cuda")
        moved = room[offset: offset + M * lda].view(M, lda)[:, :K]
        moved.copy_(a)
        a = moved
    sa, sb = scales(g, M), scales(g, N)
    c = torch.randn(M, ldd, generator=g, device="cuda").to(TYPE[out])[:, :N] if beta else None
    bv = torch.randn(N, generator=g, device="cuda").to(TYPE[out]) if bias else None
    room = torch.full((M + 2, ldd), -7.0, dtype=TYPE[out], device="cuda")
    d = room[1: M + 1, :N]
    h = Q.Int8Gemm(Q.make_desc(M, N, K, out, lda=lda, ldb=ldb, ldd=ldd, ldc=ldd if beta else 0, bias=bias, act=act,
                               split_k=split_k))
    ws = torch.full((h.workspace_bytes,), 0x5a, dtype=torch.uint8, device="cuda")
    h.run(a, sa, b, sb, d, C=c, bias=bv, alpha=alpha, beta=beta, workspace=ws)
    close(d, *reference(a, sa, b, sb, out, alpha, beta, c, bv, act))
    assert (room[0] == -7.0).all() and (room[M + 1] == -7.0).all() and (room[:, N:] == -7.0).all()
    return d, h.info


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 64, 16), (3, 5, 7), (16, 32, 128), (17, 33, 129), (64, 64, 130),
                                   (65, 127, 255), (100, 300, 1000), (129, 257, 513), (200, 70, 2050)])
def test_sizes(M, N, K, out):
    run(M, N, K, out)


@pytest.mark.parametrize("M,N,K,lda,ldb", [(5, 9, 3, 3, 3), (40, 72, 15, 15, 17), (33, 130, 16, 16, 19), (70, 140, 127, 127, 127),
                                           (130, 129, 145, 145, 151), (3, 200, 1029, 1030, 1029), (300, 260, 390, 391, 400)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_rows_at_any_byte(M, N, K, lda, ldb, out):
    assert run(M, N, K, out, lda=lda, ldb=ldb, bias=True, act="silu")[1].name.startswith(b"any")


@pytest.mark.parametrize("offset", [1, 4, 15])
@pytest.mark.parametrize("M", [2, 150])
def test_bases_at_any_byte(M, offset):
    run(M, 200, 500, offset=offset)
    run(M, 200, 5000, offset=offset)


@pytest.mark.parametrize("M", [1, 20, 60, 200, 700])
@pytest.mark.parametrize("out,act", [("bf16", "gelu"), ("f16", "relu"), ("f32", "silu"), ("f32", "none")])
def test_epilogue(M, out, act):
    run(M, 264, 272, out, ldd=280, alpha=-0.75, beta=1.5, bias=True, act=act)
    run(M, 203, 272, out, ldd=211, alpha=2.0, beta=-0.5, bias=True, act=act)


@pytest.mark.parametrize("M,N,K", [(1, 128, 4096), (16, 100, 2000), (50, 200, 1500), (130, 260, 1100)])
@pytest.mark.parametrize("split", [1, 2, 3, 64])
def test_slices_of_k_give_the_same_bits(M, N, K, split):
    whole = run(M, N, K, "f32", split_k=1)[0]
    part, info = run(M, N, K, "f32", split_k=split)
    assert torch.equal(whole, part) and info.split_k <= split


# shapes that every kernel is chosen for (test_int8_boundary.py looks that they are), with a ragged K
SHAPES = [(1, 4096, 4104), (16, 16384, 1000), (20, 512, 600), (24, 4096, 8000), (60, 300, 1000), (60, 4096, 8200), (64, 4096, 2100),
          (128, 4096, 1030), (300, 1024, 600), (333, 4096, 4100), (1000, 4096, 1050), (2048, 2100, 530), (2300, 4096, 270),
          (4096, 4096, 390), (5000, 300, 260), (2048, 2048, 2050), (64, 8190, 8180)]


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_shapes_of_every_kernel(M, N, K, out):
    run(M, N, K, out, bias=True)
    run(M, N, K, out, lda=K + 1, ldb=K + 1)


@pytest.mark.parametrize("name_of", ["stream", "tile", "pingpong", "any"])
def test_sums_of_the_largest_size(name_of):
    """All codes -128 at the longest K: sums of 2^31 - 2^14."""
    M, N = {"stream": (2, 32), "tile": (300, 200), "pingpong": (4096, 4096), "any": (3, 40)}[name_of]
    K = 131071
    lda = K if name_of == "any" else 131072
    a = torch.full((M, lda), -128, dtype=torch.int8, device="cuda")[:, :K]
    b = torch.full((N, lda), -128, dtype=torch.int8, device="cuda")[:, :K]
    one = torch.ones(max(M, N), device="cuda")
    d = torch.empty(M, N, device="cuda")
    h = Q.Int8Gemm(Q.make_desc(M, N, K, "f32", lda=lda, ldb=lda, ldd=N))
    assert h.info.name.startswith(name_of.encode())
    h.run(a, one, b, one, d, workspace=torch.empty(h.workspace_bytes, dtype=torch.uint8, device="cuda"))
    assert (d.double() == 2.0 ** 31 - 2.0 ** 14).all()


@pytest.mark.parametrize("M,N,K,batch", [(3, 70, 40, 5), (64, 128, 300, 3), (300, 300, 200, 2)])
@pytest.mark.parametrize("share_b", [False, True])
def test_batch(M, N, K, batch, share_b):
    g = gen(M + batch)
    P = padded(K)
    a, b = codes(g, batch * M, P).view(batch, M, P), codes(g, batch * N, P).view(batch, N, P)
    sa, sb = scales(g, batch * M).view(batch, M), scales(g, batch * N).view(batch, N)
    c = torch.randn(batch, M, N, generator=g, device="cuda")
    d = torch.empty(batch, M, N, device="cuda")
    h = Q.Int8Gemm(Q.make_desc(M, N, K, "f32", lda=P, ldb=P, ldd=N, ldc=N, batch=batch, a_stride_l=M * P,
                               b_stride_l=0 if share_b else N * P, c_stride_l=M * N, d_stride_l=M * N, a_scale_l=M,
                               b_scale_l=0 if share_b else N))
    h.run(a, sa, b, sb, d, C=c, beta=2.0)
    for i in range(batch):
        j = 0 if share_b else i
        close(d[i], *reference(a[i, :, :K], sa[i], b[j, :, :K], sb[j], "f32", beta=2.0, c=c[i]))


@pytest.mark.parametrize("sizes", [[0, 0, 0], [5], [1, 0, 300, 2, 64], [70] * 90, [0] * 70 + [200, 3] + [0] * 20])
@pytest.mark.parametrize("out,N,K,P", [("bf16", 200, 130, 144), ("f32", 256, 256, 256), ("bf16", 72, 33, 33)])
def test_groups_of_rows(sizes, out, N, K, P):
    g = gen(sum(sizes) + N)
    E, first, tail = len(sizes), 3, 11
    M = first + sum(sizes) + tail
    at = [first]
    for n in sizes:
        at.append(at[-1] + n)
    a, b = codes(g, M, P), codes(g, E * N, P).view(E, N, P)
    sa, sb = scales(g, M), scales(g, E * N).view(E, N)
    d = torch.full((M, N), -7.0, dtype=TYPE[out], device="cuda")
    h = Q.Int8Gemm(Q.make_desc(M, N, K, out, lda=P, ldb=P, ldd=N, groups="rows", batch=E, b_stride_l=N * P, b_scale_l=N,
                               act="silu"))
    h.run(a, sa, b, sb, d, offsets=torch.tensor(at, **I32))
    for e in range(E):
        r = slice(at[e], at[e + 1])
        if sizes[e]:
            close(d[r], *reference(a[r, :K], sa[r], b[e, :, :K], sb[e], out, act="silu"))
    assert (d[:first] == -7.0).all() and (d[M - tail:] == -7.0).all()


def test_offsets_out_of_range():
    """Clamped into [0, M] and made non-decreasing, as the header says."""
    g = gen(5)
    M, N, K = 100, 64, 64
    a, b, sa, sb = codes(g, M, K), codes(g, 4 * N, K).view(4, N, K), scales(g, M), scales(g, 4 * N).view(4, N)
    d = torch.full((M, N), -7.0, device="cuda")
    h = Q.Int8Gemm(Q.make_desc(M, N, K, "f32", lda=K, ldb=K, ldd=N, groups="rows", batch=4, b_stride_l=N * K, b_scale_l=N))
    h.run(a, sa, b, sb, d, offsets=torch.tensor([-50, 20, 10, 1000, 3], **I32))
    close(d[:20], *reference(a[:20], sa[:20], b[0], sb[0], "f32"))
    close(d[20:], *reference(a[20:], sa[20:], b[2], sb[2], "f32"))


def test_empty_and_without_k():
    g = gen(1)
    one = torch.ones(300, device="cuda")
    for M, N in ((0, 5), (5, 0)):
        h = Q.Int8Gemm(Q.make_desc(M, N, 16, "f32", lda=16, ldb=16, ldd=max(N, 1)))
        h.run(codes(g, M, 16), one, codes(g, N, 16), one, torch.empty(0, device="cuda"))
    for M, N in ((3, 40), (300, 300)):
        c = torch.randn(M, N, generator=g, device="cuda")
        bias, d = torch.randn(N, generator=g, device="cuda"), torch.empty(M, N, device="cuda")
        h = Q.Int8Gemm(Q.make_desc(M, N, 0, "f32", lda=0, ldb=0, ldd=N, ldc=N, bias=True, act="relu"))
        h.run(None, None, None, None, d, C=c, bias=bias, beta=0.5)
        close(d, *reference(codes(g, M, 0), one, codes(g, N, 0), one, "f32", beta=0.5, c=c, bias=bias, act="relu"))


@pytest.mark.parametrize("M", [2, 200])
def test_scales_that_are_not_finite(M):
    g = gen(M)
    N, K = 130, 128
    a, b, sa, sb = codes(g, M, K), codes(g, N, K), scales(g, M), scales(g, N)
    sa[1], sb[5] = float("nan"), float("nan")
    d = torch.empty(M, N, device="cuda")
    h = Q.Int8Gemm(Q.make_desc(M, N, K, "f32", lda=K, ldb=K, ldd=N))
    h.run(a, sa, b, sb, d, workspace=torch.empty(h.workspace_bytes, dtype=torch.uint8, device="cuda"))
    close(d, *reference(a, sa, b, sb, "f32"))
    assert torch.isnan(d[1]).all() and torch.isnan(d[:, 5]).all()


@pytest.mark.parametrize("M", [3, 400])
def test_d_may_be_c(M):
    g = gen(M)
    N, K = 200, 300
    a, b, sa, sb = codes(g, M, K, 304), codes(g, N, K, 304), scales(g, M), scales(g, N)
    c = torch.randn(M, N, generator=g, device="cuda")
    d = c.clone()
    h = Q.Int8Gemm(Q.make_desc(M, N, K, "f32", lda=304, ldb=304, ldd=N, ldc=N))
    h.run(a, sa, b, sb, d, C=d, beta=1.0, workspace=torch.empty(h.workspace_bytes, dtype=torch.uint8, device="cuda"))
    close(d, *reference(a, sa, b, sb, "f32", beta=1.0, c=c))
