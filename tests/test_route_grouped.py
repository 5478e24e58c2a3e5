"""The routing's order and offsets as the library's grouped product takes them: each expert's rows of
a bf16 matrix, gathered by the order, through gemm_run_grouped and back to their tokens by the slots."""
import pytest
import torch

from hierarchical_tiling_amd import htgemm as H
from hierarchical_tiling_amd import htroute as R

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("T,E,k,align,masked", [(1, 8, 2, 1, False), (150, 12, 3, 1, True), (150, 12, 3, 16, True),
                                                (700, 5, 2, 128, False), (40, 64, 1, 1, True)])
def test_tokens_through_their_experts(T, E, k, align, masked):
    """Whole numbers: the products are exact and rounded to bf16 once."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T + E)
    K, N = 128, 136
    x = torch.randint(-3, 4, (T, K), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randint(-3, 4, (E, N, K), generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    mask = (torch.rand(T, generator=g, device="cuda") < 0.8).to(torch.uint8) if masked else None
    rows = T * k + E * (align - 1)
    counts, offsets, order, slot = (torch.empty(n, **I32) for n in (E, E + 1, rows, T * k))
    R.route(ids, counts, offsets, order, slot, mask=mask, align=align,
            workspace=torch.empty(R.workspace_size(T, k, E), dtype=torch.uint8, device="cuda"))
    gathered = torch.where((order >= 0)[:, None], x[(order.clamp(min=0) // k).long()], torch.zeros((), dtype=torch.bfloat16, device="cuda"))
    h = H.Gemm(H.make_desc(rows, N, K, "bf16", (K, 1), (1, K), (N, 1), batch=E, batch_strides=(0, N * K, 0, 0), ragged_m=True))
    ws = torch.empty(h.workspace_bytes, dtype=torch.uint8, device="cuda")
    d = torch.full((rows, N), -7.0, dtype=torch.bfloat16, device="cuda")
    H.gemm_run_grouped(h.handle, gathered.data_ptr(), w.data_ptr(), None, d.data_ptr(), None, None, None, offsets.data_ptr(),
                       1.0, 0.0, stream=torch.cuda.current_stream().cuda_stream, workspace=ws.data_ptr())
    per_token = torch.matmul(x.float().cpu(), w.float().cpu().transpose(1, 2).contiguous()).transpose(0, 1)    # (T, E, N)
    want = per_token[torch.arange(T)[:, None], ids.cpu().long()].to(torch.bfloat16).view(T * k, N)
    live = torch.ones(T * k, dtype=torch.bool) if mask is None else mask.cpu().bool().repeat_interleave(k)
    at = slot.cpu().long()
    assert ((at >= 0) == live).all()
    assert torch.equal(d.cpu()[at[live]], want[live])
    # rows up to `align` of a group are its own, of zeros; those behind the last group stay as they were
    fill = torch.ones(rows, dtype=torch.bool)
    fill[at[live]] = False
    last = int(offsets[-1])
    assert (d.cpu()[:last][fill[:last]] == 0).all() and (d[last:] == -7.0).all()
