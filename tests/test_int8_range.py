"""Outputs past the ranges of the types: what bf16 and fp32 hold stays finite, what a type does not hold
is infinite, in every kernel with an epilogue of its own and in the streaming and joining ones."""
import pytest
import torch

from hierarchical_tiling_amd import htint8 as Q
from int8_util import TYPE, codes, gen, reference
from test_int8_epilogue import KERNELS, pitch_of

pytestmark = pytest.mark.gpu
# the last two: a streaming kernel, and k in slices
CASES = [(M, N, K, on16, 1) for _, M, N, K, on16 in KERNELS[::2]] + [(9, 300, 200, True, 1), (70, 300, 600, True, 3)]


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K,on16,split", CASES)
def test_range(M, N, K, on16, split, out):
    g = gen(M + N)
    ld = pitch_of(K, on16)
    a, b = codes(g, M, K, ld), codes(g, N, K, ld)
    # scales whose products spread the outputs from nothing to past fp32's range
    sa = 2.0 ** (torch.arange(M, device="cuda") % 61).float()
    sb = 2.0 ** (torch.arange(N, device="cuda") % 61).float()
    d = torch.empty(M, N, dtype=TYPE[out], device="cuda")
    h = Q.Int8Gemm(Q.make_desc(M, N, K, out, lda=ld, ldb=ld, ldd=N, split_k=split))
    assert h.info.split_k == split
    h.run(a, sa, b, sb, d, workspace=torch.empty(h.workspace_bytes, dtype=torch.uint8, device="cuda"))
    want, tol = reference(a, sa, b, sb, out)
    most = torch.finfo(TYPE[out]).max
    # half a step above the largest value rounds to infinity; the four roundings to fp32 move a value
    # by 2^-22 of it
    edge = most * (1 + torch.finfo(TYPE[out]).eps / 4)
    low, high = want.abs() < edge * (1 - 2.0 ** -22), want.abs() > edge * (1 + 2.0 ** -22)
    got = d.double()
    assert torch.isfinite(got[low]).all() and ((got - want).abs() <= tol)[low & (want.abs() <= most)].all()
    assert torch.equal(got[high], torch.copysign(torch.tensor(torch.inf, device="cuda").double(), want[high]))
    # with 61 rows and more outputs go up to 2^60 * 2^60 * 2^14 and more, past 2^128 and so past every
    # type's range; with 9 they stay below 2^8 * 2^60 * 200 * 2^14, within bf16's and fp32's
    assert high.any() == (M > 60 or out == "f16") and (want[low].abs() > 65519).any() == (out != "f16")


@pytest.mark.parametrize("M", [9, 333, 2300])
def test_past_fp32(M):
    N, K = 4096, 270
    g = gen(M)
    a, b = codes(g, M, K, 272), codes(g, N, K, 272)
    sa, sb = torch.full((M,), 2.0 ** 100, device="cuda"), torch.full((N,), 2.0 ** 100, device="cuda")
    for out in ("bf16", "f32"):
        d = torch.empty(M, N, dtype=TYPE[out], device="cuda")
        h = Q.Int8Gemm(Q.make_desc(M, N, K, out, lda=272, ldb=272, ldd=N))
        h.run(a, sa, b, sb, d, workspace=torch.empty(h.workspace_bytes, dtype=torch.uint8, device="cuda"))
        s = torch.mm(a.double(), b.double().t().contiguous())
        want = torch.where(s == 0, 0.0, torch.copysign(torch.tensor(torch.inf, device="cuda").double(), s))
        assert torch.equal(d.double(), want)
