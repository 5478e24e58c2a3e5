"""The balance loss of millions of tokens: the sums over tokens keep what the probabilities have."""
import pytest
import torch

from hierarchical_tiling_amd import htroute as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,lean,dtype", [
    (1 << 18, [2.0, 0.1, -1.3], torch.float32), (1 << 22, [2.0, 0.1, -1.3], torch.float32), (1 << 23, [2.0, 0.1, -1.3, 0.4], torch.bfloat16),
    (3_000_001, [0.0, 5.0], torch.float16), (1 << 20, [0.3] * 30 + [3.0], torch.float32), (300_000, [0.007 * i for i in range(1000)], torch.float16),
    (1 << 17, [0.01 * i for i in range(600)], torch.bfloat16)])
def test_equal_rows(T, lean, dtype):
    """Rows that are all alike, so that every rounding of a chain of additions goes the same way.

    Tolerance, in units of 2^-24 of a probability: arguments below 8 are off by 2^-22 and exp by 2
    ulp, 4 + 4 in the value and as much in the sum it is divided by; 15 + 6 additions of that sum;
    division and product 2; 3 additions of the rows that a wave has in hand; 3 roundings of the sums
    to fp32.  That is 45, below 64; what joins in double adds nothing."""
    E = len(lean)
    row = torch.tensor(lean, device="cuda").to(dtype)
    logits = row.repeat(T, 1)
    counts = torch.arange(E, dtype=torch.int32, device="cuda") + 1
    loss, prob, live = torch.empty(1, device="cuda"), torch.empty(E, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(R.workspace_size(T, 1, E), dtype=torch.uint8, device="cuda")
    R.balance_loss(logits, counts, 1, loss, prob, live, coef=1.0, workspace=ws)
    want = torch.softmax(row.double(), 0)
    assert live.item() == T
    assert ((prob.double() - want).abs() <= 2.0 ** -18 * want).all(), float(((prob.double() - want) / want).abs().max() * 2 ** 24)
    f = counts.double() * E / T
    assert abs(loss.item() - (f * want).sum().item()) <= 2.0 ** -17 * (f * want).sum().item()
