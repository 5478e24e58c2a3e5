"""Scale layouts of the quantisation: those whose scales have places of their own, and no others."""
import ctypes

import pytest
import torch

from hierarchical_tiling_amd import htscaled as S
from hierarchical_tiling_amd.htgemm import GemmError

P = 1 << 20   # an aligned number in place of an address: the calls here end before they use it
LAYOUT, ARCH = 3, 5


def status(monkeypatch, rows, cols, **kw):
    """The call's status with a device that no check of the layout has refused before: GEMM_ERR_ARCH."""
    monkeypatch.setenv("HTGEMM_FAKE_ARCH", "gfx942")
    a = S.quant_args(x=P, x_type=2, block_rows=1, index_div=1, rows=rows, cols=cols, ldx=cols, q=P, ldq=cols, scale=P)
    for k, v in kw.items():
        setattr(a, k, v)
    return S.lib().quant_blocks(ctypes.byref(a), None)


@pytest.mark.parametrize("rows,cols,r,c,ok", [
    (4, 256, 0, 1, False), (4, 256, 1, 0, False), (4, 256, 0, 0, False), (4, 128, 1, 0, True), (4, 128, 0, 1, False),
    (1, 256, 0, 1, True), (1, 256, 1, 0, False), (1, 128, 0, 0, True), (4, 256, 2, 1, True), (4, 256, 1, 4, True),
    (4, 256, 1, 3, False), (4, 384, 2, 1, False), (4, 384, 3, 1, True), (4, 384, 5, 2, True), (4, 384, 4, 2, False),
    (4, 256, 1, 1, False), (0, 256, 0, 0, True), (4, 0, 0, 0, True),
    (1 << 29, 256, 2 ** 62, 1, True), (1 << 29, 256, 1, 2 ** 62, True), (4, 256, -1, 8, False)])
def test_scale_of_rows(rows, cols, r, c, ok, monkeypatch):
    assert status(monkeypatch, rows, cols, scale_r=r, scale_c=c) == (ARCH if ok else LAYOUT)
    # the transpose's: cols lines of the rows' blocks
    t = dict(q=None, scale=None, qt=P, ldqt=cols, scale_t=P, scale_t_c=r, scale_t_r=c)
    assert status(monkeypatch, cols, rows, **t) == (ARCH if ok else LAYOUT)


@pytest.mark.parametrize("rows,cols,r,c,ok", [(128, 256, 0, 1, True), (129, 256, 0, 1, False), (129, 256, 2, 1, True),
                                              (256, 128, 1, 0, True), (256, 129, 1, 0, False), (256, 129, 1, 2, True)])
def test_scale_of_square_blocks(rows, cols, r, c, ok, monkeypatch):
    assert status(monkeypatch, rows, cols, block_rows=128, scale_r=r, scale_c=c) == (ARCH if ok else LAYOUT)


@pytest.mark.parametrize("rows,cols,pitch,extra", [(4, 100, 112, 12), (4, 100, 200, 12), (3, 5, 16, 11), (1, 5, 9, 4), (2, 33, 40, 7),
                                                   (4, 96, 112, 0), (4, 100, 100, 0)])
@pytest.mark.parametrize("turned", [False, True])
def test_padding_behind_the_last_row(rows, cols, pitch, extra, turned, monkeypatch):
    """On host tensors: memory that ends with the padding is taken, a byte less is refused."""
    class Reached(Exception):
        pass

    def here(stream):
        raise Reached
    monkeypatch.setattr(S, "_here", here)
    x = torch.zeros((cols, rows) if turned else (rows, cols))
    for missing in (0, 1):
        flat = torch.zeros(3 + (rows - 1) * pitch + cols + extra - missing, dtype=torch.uint8)
        codes = flat[3:].as_strided((rows, cols), (pitch, 1)) if extra or not missing else None
        if codes is None:
            continue
        blocks = torch.zeros(x.shape[0], -(-x.shape[1] // 128)), torch.zeros(x.shape[1], -(-x.shape[0] // 128))
        out = dict(qt=codes, scale_t=blocks[1]) if turned else dict(q=codes, scale=blocks[0])
        with pytest.raises(GemmError if missing else Reached):
            S.quantize(x, pad=True, **out)
        with pytest.raises(Reached):
            S.quantize(x, pad=False, **out)


@pytest.mark.gpu
def test_expanded_scales_are_refused():
    x = torch.randn(5, 300, device="cuda")
    q, qt = torch.empty(5, 300, dtype=torch.uint8, device="cuda"), torch.empty(300, 5, dtype=torch.uint8, device="cuda")
    s, st = torch.empty(5, 3, device="cuda"), torch.empty(300, 1, device="cuda")
    S.quantize(x, q, s, qt, st)
    for kw in (dict(scale=torch.empty(1, 3, device="cuda").expand(5, 3), scale_t=st),
               dict(scale=torch.empty(5, 1, device="cuda").expand(5, 3), scale_t=st),
               dict(scale=s, scale_t=torch.empty(1, 1, device="cuda").expand(300, 1))):
        with pytest.raises(GemmError) as err:
            S.quantize(x, q, qt=qt, **kw)
        assert err.value.status == LAYOUT
