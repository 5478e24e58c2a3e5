"""The binding of the block-scaled product refuses tensors that the kernels would read or write past:
on host tensors, before anything reaches the library."""
import pytest
import torch

from hierarchical_tiling_amd import htscaled as S
from hierarchical_tiling_amd.htgemm import GEMM_ERR_INVALID_ARG, GemmError

M, N, K, L = 40, 72, 512, 3
KB = K // 128
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def fake_gfx950(monkeypatch):
    monkeypatch.setenv("HTGEMM_FAKE_ARCH", "gfx950")


@pytest.fixture
def reached(monkeypatch):
    """Ends a call where it would reach the library: every check of the binding has passed."""
    class Reached(Exception):
        pass

    class Library:
        def gemm_scaled_run(self, handle, args, stream):
            raise Reached
    monkeypatch.setattr(S, "_here", lambda stream: (-1, 0))     # the "device" of host tensors
    S.lib()
    real = S._lib
    monkeypatch.setattr(Library, "__getattr__", lambda self, name: getattr(real, name), raising=False)
    monkeypatch.setattr(S, "_lib", Library())
    return Reached


def codes(n):
    return torch.zeros(n, dtype=torch.uint8)


def single(out="bf16", **kw):
    h = S.ScaledGemm(S.make_desc(M, N, K, out, lda=K + 16, ldb=K, ldd=N + 3, ldc=N, a_scale_strides=(1, M),
                                 b_scale_strides=(KB, 1), bias=True, row_scale=True, **kw))
    t = torch.float32 if out == "f32" else BF16
    args = dict(A=codes((M - 1) * (K + 16) + K), a_scale=torch.zeros(KB, M), B=codes(N * K), b_scale=torch.zeros(1, KB),
                D=torch.zeros((M - 1) * (N + 3) + N, dtype=t), C=torch.zeros(M * N, dtype=t), bias=torch.zeros(N, dtype=t),
                row_scale=torch.zeros(M), workspace=torch.zeros(max(1, h.workspace_bytes), dtype=torch.uint8))
    return h, args


def shorter(t, by=1):
    """The same tensor without its last values, in memory of its own."""
    return t.flatten()[:t.numel() - by].clone()


def refused(h, args, beta=1.0):
    with pytest.raises(GemmError) as err:
        h.run(**args, beta=beta)
    assert err.value.status == GEMM_ERR_INVALID_ARG


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_workspace_of_another_handle(out, reached):
    h, args = single(out, split_k=4)
    assert h.workspace_bytes == 4 * M * N * 4
    with pytest.raises(reached):
        h.run(**args, beta=1.0)
    refused(h, {**args, "workspace": shorter(args["workspace"])})
    # the bytes count, not the values
    as_floats = torch.zeros(4 * M * N)
    with pytest.raises(reached):
        h.run(**{**args, "workspace": as_floats}, beta=1.0)
    refused(h, {**args, "workspace": shorter(as_floats)})


@pytest.mark.parametrize("name", ["A", "a_scale", "B", "b_scale", "D", "C", "bias", "row_scale"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_one_value_too_few(name, out, reached):
    h, args = single(out)
    with pytest.raises(reached):
        h.run(**args, beta=1.0)
    refused(h, {**args, name: shorter(args[name])})


def test_memory_counts_not_the_shape(reached):
    """A view is taken by what lies behind its first value; an expanded one has no more than that."""
    h, args = single()
    wide = torch.zeros(M, K + 16, dtype=torch.uint8)
    with pytest.raises(reached):
        h.run(**{**args, "A": wide[:, :K]}, beta=1.0)
    with pytest.raises(reached):
        h.run(**{**args, "A": wide[:1]}, beta=1.0)
    refused(h, {**args, "A": wide[1:]})
    refused(h, {**args, "a_scale": torch.zeros(1).expand(KB, M)})
    with pytest.raises(reached):      # C is not looked at without beta
        h.run(**{**args, "C": None})


@pytest.mark.parametrize("name,other", [("A", torch.float8_e5m2), ("B", BF16), ("a_scale", torch.float64), ("b_scale", BF16),
                                        ("D", torch.float32), ("C", torch.float32), ("bias", torch.float16), ("row_scale", BF16)])
def test_another_type(name, other, reached):
    h, args = single()
    refused(h, {**args, name: args[name].to(other)})
    for codes_of in (torch.int8, torch.float8_e4m3fn):
        with pytest.raises(reached):
            h.run(**{**args, "A": args["A"].to(codes_of)}, beta=1.0)


def test_groups_and_batches(reached):
    def check(h, args):
        with pytest.raises(reached):
            h.run(**args)
        for name in args:
            refused(h, {**args, name: shorter(args[name])}, beta=0.0)

    i32 = dict(dtype=torch.int32)
    common = dict(lda=K, ldb=K, ldd=N, b_scale_strides=(KB, 1))
    a, sa = codes(M * K), torch.zeros(KB, M)
    h = S.ScaledGemm(S.make_desc(M, N, K, **common, a_scale_strides=(1, M), groups="rows", batch=L, b_stride_l=N * K, b_scale_l=KB))
    check(h, dict(A=a, a_scale=sa, B=codes(L * N * K), b_scale=torch.zeros(L, KB), D=torch.zeros(M, N, dtype=BF16),
                  offsets=torch.zeros(L + 1, **i32)))
    h = S.ScaledGemm(S.make_desc(M, N, K, **common, a_scale_strides=(1, M), groups="k", batch=L, d_stride_l=M * N))
    check(h, dict(A=a, a_scale=sa, B=codes(N * K), b_scale=torch.zeros(1, KB), D=torch.zeros(L, M, N, dtype=BF16),
                  offsets=torch.zeros(L + 1, **i32)))
    h = S.ScaledGemm(S.make_desc(M, N, K, **common, a_scale_strides=(1, M), batch=L, a_stride_l=M * K, b_stride_l=N * K,
                                 d_stride_l=M * N, a_scale_l=M * KB, b_scale_l=KB))
    check(h, dict(A=codes(L * M * K), a_scale=torch.zeros(L, KB, M), B=codes(L * N * K), b_scale=torch.zeros(L, KB),
                  D=torch.zeros(L, M, N, dtype=BF16)))
    # operands that all products share
    h = S.ScaledGemm(S.make_desc(M, N, K, **common, a_scale_strides=(1, M), batch=L, d_stride_l=M * N))
    check(h, dict(A=a, a_scale=sa, B=codes(N * K), b_scale=torch.zeros(1, KB), D=torch.zeros(L, M, N, dtype=BF16)))


def test_empty_products_need_nothing(reached):
    for m, n, k in ((0, N, K), (M, 0, K)):
        h = S.ScaledGemm(S.make_desc(m, n, k, lda=k, ldb=k, ldd=n, a_scale_strides=(1, 1), b_scale_strides=(1, 1)))
        with pytest.raises(reached):
            h.run(codes(0), torch.zeros(0), codes(0), torch.zeros(0), torch.zeros(0, dtype=BF16))
    h = S.ScaledGemm(S.make_desc(M, N, 0, lda=0, ldb=0, ldd=N, a_scale_strides=(1, 1), b_scale_strides=(1, 1)))
    with pytest.raises(reached):
        h.run(codes(0), torch.zeros(0), codes(0), torch.zeros(0), torch.zeros(M, N, dtype=BF16))
    refused(h, dict(A=codes(0), a_scale=torch.zeros(0), B=codes(0), b_scale=torch.zeros(0), D=torch.zeros(M * N - 1, dtype=BF16)), 0.0)
