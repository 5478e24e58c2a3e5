"""Quantisation of every value of the 16-bit types, bit for bit the documented fp32 steps."""
import numpy as np
import pytest
import torch

from hierarchical_tiling_amd import htscaled as S
from scaled_util import BLOCK
from test_quantise import outputs, same, steps

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("pow2", [False, True])
def test_every_value(dtype, pow2):
    """In order of the bits (blocks of neighbours), shuffled (a block's largest beside all others), and
    with each as the largest of its block; infinities and NaN among them."""
    bits = np.arange(65536, dtype=np.uint16)
    rng = np.random.default_rng(1)
    own = np.tile(bits[:, None], (1, 4))
    own[:, 1] = bits >> 1 & 0x3fff           # smaller ones beside it
    own[:, 2] = bits & 0x7f80
    own[:, 3] = rng.integers(0, 0x2000, 65536)
    for pattern in (bits.reshape(256, 256), rng.permutation(bits).reshape(128, 512), own[:4096], own[31744 - 2048: 31744 + 100], own[32768 - 200: 32768 + 4000]):
        x = torch.from_numpy(pattern.copy().view(np.int16)).view(dtype)
        host = x.float().numpy()
        rows, cols = pattern.shape
        q, qt, s, st = outputs(rows, cols)
        S.quantize(x.cuda(), q, s, qt, st, pow2=pow2)
        with np.errstate(invalid="ignore"):
            w, ws = steps(host, 1, BLOCK, pow2)
            same(q, w), same(s, ws)
            w, ws = steps(np.ascontiguousarray(host.T), 1, BLOCK, pow2)
            same(qt, w), same(st, ws)
        q2, _, s2, _ = outputs(rows, cols)
        S.quantize(x.cuda(), q2, s2, pow2=pow2)
        assert torch.equal(q, q2) and torch.equal(s.isnan(), s2.isnan()) and torch.equal(s.nan_to_num(-1), s2.nan_to_num(-1))
