"""Streams of another device than the current one are refused, as its tensors are."""
import pytest
import torch

from hierarchical_tiling_amd import htroute as R
from hierarchical_tiling_amd import htscaled as S
from hierarchical_tiling_amd.htgemm import GEMM_ERR_INVALID_ARG, GemmError


class Elsewhere:
    """What a call reads of a torch stream on device 1."""
    device_index, cuda_stream = 1, 0


def calls(device):
    i32 = dict(dtype=torch.int32, device=device)
    x, one = torch.zeros(4, 128, device=device), torch.zeros(1, device=device)
    ids, counts, live = torch.zeros(4, 2, **i32), torch.zeros(128, **i32), torch.zeros(1, **i32)
    ws = torch.zeros(R.workspace_size(4, 2, 128), dtype=torch.uint8, device=device)
    codes, scale = torch.zeros(4, 128, dtype=torch.uint8, device=device), torch.zeros(4, 1, device=device)
    h = S.ScaledGemm(S.make_desc(4, 4, 128, "f32", lda=128, ldb=128, ldd=4, a_scale_strides=(1, 1), b_scale_strides=(1, 1)))
    return {
        "product": lambda s: h.run(codes, scale, codes, scale, torch.zeros(4, 4, device=device), stream=s),
        "quantise": lambda s: S.quantize(x, codes, scale, stream=s),
        "route": lambda s: R.route(ids, counts, torch.zeros(129, **i32), workspace=ws, stream=s),
        "loss": lambda s: R.balance_loss(x, counts, 2, one, torch.zeros(128, device=device), live, workspace=ws, stream=s),
        "gradient": lambda s: R.balance_grad(x, counts, 2, live, one, torch.zeros_like(x), stream=s)}


NAMES = ["product", "quantise", "route", "loss", "gradient"]


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device(name, monkeypatch):
    """On the host: the current device is 0 by what the binding asks; nothing reaches the library."""
    monkeypatch.setenv("HTGEMM_FAKE_ARCH", "gfx950")
    call = calls("cpu")[name]
    monkeypatch.setattr(S, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(S, "_device", lambda: 0)
    monkeypatch.setattr(S, "_elsewhere", lambda *a: pytest.fail("the stream was not looked at"))
    with pytest.raises(GemmError) as err:
        call(Elsewhere())
    assert err.value.status == GEMM_ERR_INVALID_ARG and "stream" in str(err.value)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_this_device(name):
    stream = torch.cuda.Stream()
    call = calls("cuda")[name]
    torch.cuda.synchronize()
    call(stream)
    call(stream.cuda_stream)
    stream.synchronize()
