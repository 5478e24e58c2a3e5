"""Products in 8-bit integers without k: D is act(beta C + bias), whatever alpha and the scales are."""
import pytest
import torch

from hierarchical_tiling_amd import htint8 as Q

pytestmark = pytest.mark.gpu


# every kernel that is chosen without k (rows on 16 bytes and off them)
@pytest.mark.parametrize("M,N,ld", [(3, 40, 0), (1000, 2048, 0), (2300, 4096, 0), (200, 300, 1), (2300, 4096, 1)])
@pytest.mark.parametrize("alpha", [float("inf"), float("nan"), 3.0])
def test_alpha_and_scales_do_not_matter(M, N, ld, alpha):
    c = torch.arange(M * N, device="cuda").view(M, N) % 1001 - 500.0
    bias, d = torch.arange(N, device="cuda") % 77 - 30.0, torch.empty(M, N, device="cuda")
    nan = torch.full((max(M, N),), float("nan"), device="cuda")
    h = Q.Int8Gemm(Q.make_desc(M, N, 0, "f32", lda=ld, ldb=ld, ldd=N, ldc=N, bias=True, act="relu"))
    for scale in (None, nan):
        h.run(None, scale, None, scale, d, C=c, bias=bias, alpha=alpha, beta=0.5)
        assert torch.equal(d, (0.5 * c + bias).clamp(min=0))       # whole and half numbers: exact
