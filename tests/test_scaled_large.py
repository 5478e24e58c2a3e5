"""Sizes whose launch would have 2^32 threads or more, which the runtime would run as what is left
modulo 2^32."""
import pytest
import torch

from hierarchical_tiling_amd import htscaled as S


@pytest.mark.gpu
def test_quantise_more_rows_than_a_launch_has_waves():
    """2^26 rows are 2^26 waves of 64; the halves by themselves give the same bits."""
    rows, half = 2 ** 26 + 3, 2 ** 25
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(rows, 1, generator=g, device="cuda").to(torch.float16)
    q, s = torch.full((rows, 1), 0xee, dtype=torch.uint8, device="cuda"), torch.full((rows, 1), -1.0, device="cuda")
    S.quantize(x, q, s)
    for part in (slice(0, half), slice(half, rows)):
        q1, s1 = torch.empty_like(q[part]), torch.empty_like(s[part])
        S.quantize(x[part], q1, s1)
        assert torch.equal(q[part], q1) and torch.equal(s[part], s1)
    live = x != 0
    assert ((q & 0x7f == 0x7e) == live).all()    # the largest code, each row's only value
    # scale = t / 448 and 448 * scale, an ulp at most each
    assert ((s * 448 - x.float().abs()).abs()[live] <= 2.0 ** -22 * x.float().abs()[live]).all()
