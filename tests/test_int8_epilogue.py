"""What stands behind the sums of the products in 8-bit integers (alpha, C, D that is C, bias, every
activation, no k, scales that are not finite), in every kernel that has an epilogue of its own, in the
batch form and for groups of rows, against 64-bit references.  Each size names the kernel it is for, so
that a change of the choice shows here (test_int8_choice.py asks the same on the host)."""
import pytest
import torch

from hierarchical_tiling_amd import htint8 as Q
from int8_util import I32, TYPE, codes, gen, reference, scales

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "gelu", "silu"]

# (kernel, M, N, K, rows on 16 bytes): N on the tiles, whose rows of D can lie on lines of 128 bytes, and
# N that cuts a piece of 16 bytes
KERNELS = [("any_64x128", 333, 1024, 300, False), ("any_64x128", 333, 1003, 300, False),
           ("any_128x128", 2048, 2112, 530, False), ("any_128x128", 2048, 2101, 530, False),
           ("tile_64x128_w2x2", 333, 1024, 300, True), ("tile_64x128_w2x2", 333, 1003, 300, True),
           ("tile_64x128_w2x2x2", 333, 4096, 4100, True), ("tile_64x128_w2x2x2", 333, 4099, 4100, True),
           ("tile_128x128_w2x2", 2048, 2112, 530, True), ("tile_128x128_w2x2", 2048, 2101, 530, True),
           ("tile_128x128_w2x2x2", 2048, 2048, 2050, True), ("tile_128x128_w2x2x2", 2030, 2043, 2050, True),
           ("pingpong_256x256", 2300, 4096, 270, True), ("pingpong_256x256", 2300, 4099, 270, True)]
# (kernel, M, N, K, products)
BATCHES = [("tile_64x128_w2x2", 129, 131, 300, 64), ("tile_128x128_w2x2", 512, 1024, 300, 16),
           ("pingpong_256x256", 1024, 1024, 130, 16), ("pingpong_256x256", 1020, 1003, 130, 16)]
# (kernel, N, K, rows on 16 bytes, sizes of the groups): ping-pong tiles with both halves of their rows,
# with one and with a row of the second
GROUPS = [("pingpong_256x256", 2048, 300, True, [700, 0, 128, 129, 1, 1000, 256, 1772]),
          ("pingpong_256x256", 2043, 300, True, [700, 0, 128, 129, 1, 1000, 256, 1772]),
          ("tile_64x128_w2x2", 1000, 300, True, [900, 0, 1000, 1090]),
          ("tile_128x128_w2x2", 1024, 200, True, [1000, 128, 1, 0, 1500, 600, 1765]),
          ("any_128x128", 2048, 300, False, [700, 0, 128, 129, 1, 1000, 256, 1772])]


def pitch_of(K, on16):
    return max(-(-K // 16) * 16, 16) if on16 else K + 1


def made(kernel, M, N, K, out, **kw):
    h = Q.Int8Gemm(Q.make_desc(M, N, K, out, **kw))
    assert h.info.name.decode() == kernel
    return h, torch.empty(h.workspace_bytes, dtype=torch.uint8, device="cuda")


def near(got, want, tol):
    """Within the tolerance, and finite: no value here comes near its type's range."""
    assert float(want.abs().max()) < 60000
    off = (got.double() - want).abs()
    assert torch.isfinite(got).all() and (off <= tol).all(), float((off / tol).max())


def normal(g, out, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(TYPE[out])


def watched(M, N, ldd, out):
    """A D whose rows start on lines where ldd does, with rows above, below and columns behind."""
    room = torch.full((M + 2, ldd), -7.0, dtype=TYPE[out], device="cuda")
    return room, room[1: M + 1, :N]


def intact(room, N):
    assert (room[0] == -7.0).all() and (room[-1] == -7.0).all() and (room[:, N:] == -7.0).all()


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kernel,M,N,K,on16", KERNELS)
def test_alpha_c_bias_and_activations(kernel, M, N, K, on16, out):
    """Rows of D on lines of 128 bytes (64 values of 16 bits or 32 of 32 are one) and 8 and 3 values off
    them, with C and without."""
    g = gen(M + N)
    ld = pitch_of(K, on16)
    a, b, sa, sb = codes(g, M, K, ld), codes(g, N, K, ld), scales(g, M), scales(g, N)
    bias = normal(g, out, N)
    for step in (0, 8, 3):
        ldd = -(-N // 64) * 64 + step
        c = normal(g, out, M, ldd)[:, :N]
        for act in ACTS:
            for beta in (0.0, 1.5):
                h, ws = made(kernel, M, N, K, out, lda=ld, ldb=ld, ldd=ldd, ldc=ldd, bias=True, act=act, split_k=1)
                room, d = watched(M, N, ldd, out)
                h.run(a, sa, b, sb, d, C=c, bias=bias, alpha=-0.75, beta=beta, workspace=ws)
                near(d, *reference(a, sa, b, sb, out, -0.75, beta, c, bias, act))
                intact(room, N)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("kernel,M,N,K,on16", KERNELS)
def test_d_may_be_c(kernel, M, N, K, on16, out):
    g = gen(M + N + 1)
    ld = pitch_of(K, on16)
    a, b, sa, sb = codes(g, M, K, ld), codes(g, N, K, ld), scales(g, M), scales(g, N)
    for step in (0, 8, 3):
        ldd = -(-N // 64) * 64 + step
        for act in ("none", "gelu"):
            h, ws = made(kernel, M, N, K, out, lda=ld, ldb=ld, ldd=ldd, ldc=ldd, act=act, split_k=1)
            room, d = watched(M, N, ldd, out)
            d.copy_(normal(g, out, M, N))
            c = d.clone()
            h.run(a, sa, b, sb, d, C=d, beta=-1.25, workspace=ws)
            near(d, *reference(a, sa, b, sb, out, 1.0, -1.25, c, None, act))
            intact(room, N)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("kernel,M,N,K,on16", KERNELS)
def test_scales_that_are_not_finite(kernel, M, N, K, on16, out):
    """A NaN scale makes its row or column NaN and touches no other; C and bias do not hide it."""
    g = gen(M + N + 2)
    ld = pitch_of(K, on16)
    a, b, sa, sb = codes(g, M, K, ld), codes(g, N, K, ld), scales(g, M), scales(g, N)
    rows, cols = [1, M // 2, M - 1], [0, 5, N - 1]
    sa[rows], sb[cols] = float("nan"), float("nan")
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[rows], bad[:, cols] = True, True
    h, ws = made(kernel, M, N, K, out, lda=ld, ldb=ld, ldd=N, ldc=N, bias=True, act="silu", split_k=1)
    c, bias, d = normal(g, out, M, N), normal(g, out, N), torch.empty(M, N, dtype=TYPE[out], device="cuda")
    for beta in (0.0, 2.0):
        h.run(a, sa, b, sb, d, C=c, bias=bias, beta=beta, workspace=ws)
        want, tol = reference(a, sa, b, sb, out, 1.0, beta, c, bias, "silu")
        assert torch.equal(torch.isnan(d), bad)
        near(d[~bad], want[~bad], tol[~bad])


# without k the choice goes by the outputs alone: (kernel, M, N, leading dimension of A and B)
WITHOUT_K = [("stream_16x32_w4", 3, 40, 0), ("tile_64x128_w2x2", 1000, 2048, 0), ("tile_128x128_w2x2", 2300, 4096, 0),
             ("tile_128x128_w2x2", 2300, 4099, 0), ("any_64x128", 200, 300, 1), ("any_128x128", 2300, 4096, 1)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("kernel,M,N,ld", WITHOUT_K)
def test_without_k(kernel, M, N, ld, out):
    """D = act(beta C + bias): two roundings to fp32 at most, the activation's, and D's."""
    g = gen(M + N)
    c, bias, d = normal(g, out, M, N), normal(g, out, N), torch.empty(M, N, dtype=TYPE[out], device="cuda")
    none = torch.empty(0, device="cuda")
    for act in ACTS:
        h, _ = made(kernel, M, N, 0, out, lda=ld, ldb=ld, ldd=N, ldc=N, bias=True, act=act)
        h.run(None, None, None, None, d, C=c, bias=bias, beta=0.5)
        a, b = torch.empty(M, 0, dtype=torch.int8, device="cuda"), torch.empty(N, 0, dtype=torch.int8, device="cuda")
        near(d, *reference(a, none, b, none, out, 1.0, 0.5, c, bias, act))


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("kernel,M,N,K,batch", BATCHES)
def test_batch(kernel, M, N, K, batch, out):
    g = gen(M + N)
    P = pitch_of(K, True)
    a, b = codes(g, batch * M, K, P), codes(g, batch * N, K, P)
    sa, sb = scales(g, batch * M).view(batch, M), scales(g, batch * N).view(batch, N)
    c, bias = normal(g, out, batch, M, N), normal(g, out, N)
    for act, beta in (("none", 0.0), ("gelu", 2.0)):
        d = torch.full((batch * M + 2, N), -7.0, dtype=TYPE[out], device="cuda")
        h, ws = made(kernel, M, N, K, out, lda=P, ldb=P, ldd=N, ldc=N, bias=True, act=act, batch=batch, a_stride_l=M * P,
                     b_stride_l=N * P, c_stride_l=M * N, d_stride_l=M * N, a_scale_l=M, b_scale_l=N)
        inside = d[1: batch * M + 1]
        h.run(a, sa, b, sb, inside, C=c, bias=bias, beta=beta, workspace=ws)
        for i in range(batch):
            r = slice(i * M, (i + 1) * M)
            near(inside[r], *reference(a[r], sa[i], b[i * N: (i + 1) * N], sb[i], out, 1.0, beta, c[i], bias, act))
        assert (d[0] == -7.0).all() and (d[-1] == -7.0).all()


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("kernel,N,K,on16,sizes", GROUPS)
def test_groups_of_rows(kernel, N, K, on16, sizes, out):
    """With bias, activations, C and a C that is D; rows outside the groups are left as they were."""
    g = gen(N + K)
    E, P, first, tail = len(sizes), pitch_of(K, on16), 9, 5
    M = first + sum(sizes) + tail
    at = [first]
    for n in sizes:
        at.append(at[-1] + n)
    a, b, sa, sb = codes(g, M, K, P), codes(g, E * N, K, P), scales(g, M), scales(g, E * N).view(E, N)
    bias, offsets = normal(g, out, N), torch.tensor(at, **I32)
    for act, beta, in_place in (("none", 0.0, False), ("silu", 0.0, False), ("relu", 0.5, False), ("gelu", 0.5, True)):
        h, ws = made(kernel, M, N, K, out, lda=P, ldb=P, ldd=N, ldc=N, bias=True, act=act, groups="rows", batch=E,
                     b_stride_l=N * P, b_scale_l=N)
        c = normal(g, out, M, N)
        d = c.clone() if in_place else torch.full((M, N), -7.0, dtype=TYPE[out], device="cuda")
        was = d.clone()
        h.run(a, sa, b, sb, d, C=d if in_place else c, bias=bias, offsets=offsets, beta=beta, workspace=ws)
        for e in range(E):
            r = slice(at[e], at[e + 1])
            if sizes[e]:
                near(d[r], *reference(a[r], sa[r], b[e * N: (e + 1) * N], sb[e], out, 1.0, beta, c[r], bias, act))
        assert torch.equal(d[:first], was[:first]) and torch.equal(d[M - tail:], was[M - tail:])
