"""Tokens to their experts' rows by order alone (no slot)."""
import pytest
import torch

from hierarchical_tiling_amd import htgemm as H
from hierarchical_tiling_amd import htroute as R
from hierarchical_tiling_amd import htscaled as S
from int8_util import I32, TYPE, gen, pitched, routing


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,E,k,align,H", [(1, 4, 1, 1, 1), (33, 5, 2, 16, 51), (17, 12, 6, 3, 1000), (70, 9, 8, 8, 2051),
                                           (9, 20, 15, 5, 5003), (1100, 3, 1, 1, 40), (900, 16, 8, 16, 264)])
def test_same_rows_as_with_slot(T, E, k, align, H, dtype):
    g = gen(T + H)
    order, slot, _ = routing(g, T, E, k, align, [i % 4 != 3 for i in range(T)])
    n = order.numel()
    order[::7] = torch.randint(-9, T * k + 9, (len(order[::7]),), generator=g, **I32)     # any values
    for px, py in ((H, H), (H + 3, H + 5)):
        x = pitched(torch.randn(T, H, generator=g, device="cuda").to(TYPE[dtype]), px, 1000.0)
        room = torch.full((n + 2, py), -7.0, dtype=TYPE[dtype], device="cuda")
        y, with_slot = room[1: n + 1, :H], torch.empty(n, H, dtype=TYPE[dtype], device="cuda")
        R.gather(x, order, None, y, topk=k)
        R.gather(x, order, slot, with_slot)
        live = ((order >= 0) & (order < T * k))[:, None]
        want = torch.where(live, x[(order.clamp(0, T * k - 1) // k).long()], torch.zeros((), dtype=TYPE[dtype], device="cuda"))
        assert torch.equal(y, want) and torch.equal(with_slot, want)
        assert (room[0] == -7.0).all() and (room[-1] == -7.0).all() and (room[:, H:] == -7.0).all()


@pytest.mark.gpu
def test_no_tokens():
    y = torch.full((5, 8), -7.0, device="cuda")
    R.gather(torch.empty(0, 8, device="cuda"), torch.zeros(5, **I32), None, y, topk=2)
    assert (y == 0).all()


@pytest.mark.parametrize("slot,topk", [(None, None), (None, 0), (None, 65), (None, 2.0), ("given", 3)])
def test_refused(slot, topk, monkeypatch):
    monkeypatch.setenv("HTGEMM_FAKE_ARCH", "gfx950")
    monkeypatch.setattr(S, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(S, "_device", lambda: -1)
    i32 = dict(dtype=torch.int32)
    with pytest.raises(H.GemmError) as e:
        R.gather(torch.zeros(4, 8), torch.zeros(9, **i32), torch.zeros(4, 2, **i32) if slot else None, torch.zeros(9, 8), topk=topk)
    assert e.value.status == H.GEMM_ERR_INVALID_ARG
