"""The binding's quantisation refuses an index_div that no 32-bit number holds, as one below 1."""
import pytest
import torch

from hierarchical_tiling_amd import htgemm as H
from hierarchical_tiling_amd import htint8 as Q
from hierarchical_tiling_amd import htscaled as S


@pytest.mark.parametrize("div", [0, -1, 1 << 31, 1 << 40, -(1 << 40)])
def test_refused(div, monkeypatch):
    monkeypatch.setenv("HTGEMM_FAKE_ARCH", "gfx950")
    monkeypatch.setattr(S, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(S, "_device", lambda: -1)
    for index in (None, torch.zeros(4, dtype=torch.int32)):
        with pytest.raises(H.GemmError) as e:
            Q.quantize(torch.zeros(4, 8), torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4), row_index=index, index_div=div)
        assert e.value.status == H.GEMM_ERR_INVALID_ARG
