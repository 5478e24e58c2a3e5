"""Block quantisation on the GPU: bit for bit the documented fp32 steps, done here with numpy, and
within the rounding's bound of the source."""
import numpy as np
import pytest
import torch

from hierarchical_tiling_amd import htscaled as S
from hierarchical_tiling_amd.htgemm import GemmError
from scaled_util import BLOCK, up

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
MIN = np.float32(2.0 ** -126)


def steps(x, rb, cb, pow2):
    """(codes, scales) of a float32 array, a scale for each rb x cb block."""
    R, C = x.shape
    q = np.zeros((R, C), np.uint8)
    scale = np.zeros((up(R, rb), up(C, cb)), np.float32)
    for i in range(scale.shape[0]):
        for j in range(scale.shape[1]):
            block = x[i * rb:(i + 1) * rb, j * cb:(j + 1) * cb]
            top = np.float32(np.abs(block).max())
            if not np.isfinite(block).all():
                scale[i, j], codes = np.nan, np.full(block.shape, 0x7f, np.uint8)
            else:
                if pow2:
                    e = max(int(np.ceil(np.log2(np.float64(top) / 448))) if top > 0 else -126, -126)
                    s, inv = np.float32(2.0 ** e), np.float32(2.0 ** -e)
                else:
                    t = max(top, np.float32(448) * MIN)
                    s, inv = t / np.float32(448), np.float32(448) / t
                v = np.clip(block * inv, np.float32(-448), np.float32(448))
                assert v.dtype == np.float32
                scale[i, j] = s
                codes = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            q[i * rb:(i + 1) * rb, j * cb:(j + 1) * cb] = codes
    return q, scale


def source(rows, cols, dtype, seed, ld=None):
    g = torch.Generator()
    g.manual_seed(seed)
    full = torch.randn(rows, ld or cols, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))
    return full.to(TYPES[dtype]).cuda()[:, :cols]


def outputs(rows, cols, pitch=0):
    """q, scale, qt, scale_t with the pitch's bytes set to 0xee."""
    q = torch.full((rows, cols + pitch), 0xee, dtype=torch.uint8, device="cuda")
    qt = torch.full((cols, rows + pitch), 0xee, dtype=torch.uint8, device="cuda")
    return q, qt, torch.full((up(cols, BLOCK), rows), -1.0, device="cuda").t(), torch.full((cols, up(rows, BLOCK)), -1.0, device="cuda")


def same(got, want):
    got = got.cpu().numpy()
    assert np.array_equal(got, want, equal_nan=got.dtype == np.float32), (np.argwhere(got != want)[:5], got[got != want][:5], want[got != want][:5])


SIZES = [(1, 1), (1, 8), (3, 127), (2, 128), (5, 300), (127, 129), (128, 128), (129, 257), (130, 1000), (300, 513), (16, 2048)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pow2", [False, True])
def test_rows_and_turned(rows, cols, dtype, pow2):
    x = source(rows, cols, dtype, rows + cols)
    host = x.float().cpu().numpy()
    q, qt, s, st = outputs(rows, cols)
    S.quantize(x, q, s, pow2=pow2)
    w, ws = steps(host, 1, BLOCK, pow2)
    same(q, w), same(s, ws)
    q2, qt, s2, st = outputs(rows, cols)
    S.quantize(x, q2, s2, qt, st, pow2=pow2)
    same(q2, w), same(s2, ws)
    w, ws = steps(np.ascontiguousarray(host.T), 1, BLOCK, pow2)
    same(qt, w), same(st, ws)
    _, qt2, _, st2 = outputs(rows, cols)
    S.quantize(x, qt=qt2, scale_t=st2, pow2=pow2)
    assert torch.equal(qt, qt2) and torch.equal(st, st2)


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_square_blocks(rows, cols, dtype):
    x = source(rows, cols, dtype, 3 * rows + cols)
    for pow2 in (False, True):
        w, ws = steps(x.float().cpu().numpy(), BLOCK, BLOCK, pow2)
        for both in (False, True):
            q, qt, _, _ = outputs(rows, cols)
            s = torch.empty(up(rows, BLOCK), up(cols, BLOCK), device="cuda")
            S.quantize(x, q, s, qt if both else None, block_rows=128, pow2=pow2)
            same(q, w), same(s, ws)
            if both:
                same(qt, w.T)
        _, qt, _, _ = outputs(rows, cols)
        S.quantize(x, None, s, qt, block_rows=128, pow2=pow2)
        same(qt, w.T)


@pytest.mark.parametrize("rows,cols", [(5, 300), (129, 257), (40, 16)])
def test_error_bound(rows, cols):
    """Each value is within half a step, 2^-4 of it, or half the least step (2^-10 scales) of the
    source, and a little of fp32's own rounding."""
    x = source(rows, cols, "f32", 9)
    q, _, s, _ = outputs(rows, cols)
    S.quantize(x, q, s)
    sc = s.double().repeat_interleave(BLOCK, 1)[:, :cols]
    back = q.view(torch.float8_e4m3fn).float().double() * sc
    tol = torch.maximum(x.double().abs() * 2.0 ** -4, sc * 2.0 ** -10) * (1 + 2.0 ** -18)
    assert ((back - x.double()).abs() <= tol).all()


@pytest.mark.parametrize("pad", [False, True])
@pytest.mark.parametrize("rows,cols,pitch", [(3, 100, 40), (130, 260, 3), (20, 512, 16), (17, 5, 0)])
def test_pitch(rows, cols, pitch, pad):
    """pad continues rows with zeros to 16 or the pitch; nothing else between the rows is touched."""
    x = source(rows, cols, "bf16", 1, ld=cols + 5)
    for both in (False, True):
        q, qt, s, st = outputs(rows, cols, pitch)
        S.quantize(x, q[:, :cols], s, qt[:, :rows] if both else None, st if both else None, pad=pad)
        w, ws = steps(x.float().cpu().numpy(), 1, BLOCK, False)
        same(q[:, :cols], w), same(s, ws)
        for t, n in ((q, cols),) + (((qt, rows),) if both else ()):
            end = min(t.shape[1], up(n, 16) * 16) if pad else n
            assert (t[:, n:end] == 0).all()
            assert (t[:, end:] == 0xee).all()


@pytest.mark.parametrize("div", [1, 3])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_gathered_rows(div, block_rows):
    """Rows by index, some of them none (below zero, or past the source)."""
    n, cols, rows = 37, 260, 150
    x = source(n, cols, "bf16", 2)
    g = torch.Generator()
    g.manual_seed(1)
    index = torch.randint(-5, n * div + 6, (rows,), generator=g, dtype=torch.int32)
    index[0], index[1], index[2] = -2 ** 31, 2 ** 31 - 1, n * div - 1
    src = torch.div(index.long(), div, rounding_mode="floor")
    live = (index >= 0) & (src < n)
    gathered = torch.where(live[:, None], x.float().cpu()[src.clamp(0, n - 1)], torch.zeros(1)).numpy()
    q, qt, s, st = outputs(rows, cols)
    if block_rows == 128:
        s, st = torch.empty(up(rows, BLOCK), up(cols, BLOCK), device="cuda"), None
    S.quantize(x, q, s, qt, st, block_rows=block_rows, row_index=index.cuda(), index_div=div)
    w, ws = steps(gathered, block_rows, BLOCK, False)
    same(q, w), same(s, ws)
    if block_rows == 1:
        q2, _, s2, _ = outputs(rows, cols)
        S.quantize(x, q2, s2, row_index=index.cuda(), index_div=div)
        assert torch.equal(q, q2) and torch.equal(s, s2)
        w, ws = steps(np.ascontiguousarray(gathered.T), 1, BLOCK, False)
        same(qt, w), same(st, ws)
    else:
        same(qt, w.T)


def test_gather_from_no_rows():
    x = torch.empty(0, 200, dtype=torch.bfloat16, device="cuda")
    q, _, s, _ = outputs(4, 200)
    S.quantize(x, q, s, row_index=torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert (q == 0).all() and (s == float(MIN)).all()


@pytest.mark.parametrize("pow2", [False, True])
def test_special_values(pow2):
    """NaN and infinities mark their own block alone; zeros, the least and the largest numbers."""
    x = torch.randn(140, 400)
    x[0, 3], x[1, 130], x[2, 399] = float("nan"), float("inf"), float("-inf")
    x[3], x[4], x[5, :128], x[6, :128] = 0, 1e-45, 3.4e38, 2.0 ** -120
    x[7, :128], x[8, :128], x[9, :128] = 448 * 2.0 ** -126, 449 * 2.0 ** -126, -0.0
    x[10, :128], x[11, :128] = 1.75, 1.7500001
    host = x.numpy()
    q, qt, s, st = outputs(140, 400)
    S.quantize(x.cuda(), q, s, qt, st, pow2=pow2)
    w, ws = steps(host, 1, BLOCK, pow2)
    same(q, w), same(s, ws)
    w, ws = steps(np.ascontiguousarray(host.T), 1, BLOCK, pow2)
    same(qt, w), same(st, ws)
    sq = torch.empty(2, 4, device="cuda")
    S.quantize(x.cuda(), q, sq, qt, block_rows=128, pow2=pow2)
    w, ws = steps(host, BLOCK, BLOCK, pow2)
    same(q, w), same(sq, ws), same(qt, w.T)


def test_empty_and_misaligned_source():
    for r, c in ((0, 5), (5, 0)):
        q, _, s, _ = outputs(r, c)
        S.quantize(torch.empty(r, c, device="cuda"), q, s)
    flat = torch.randn(1 + 9 * 263, device="cuda").to(torch.bfloat16)
    x = flat[1:].view(9, 263)[:, :257]
    q, qt, s, st = outputs(9, 257)
    S.quantize(x, q, s, qt, st)
    w, ws = steps(x.float().cpu().numpy(), 1, BLOCK, False)
    same(q, w), same(s, ws)


def test_tensors_elsewhere_are_refused():
    x = source(4, 256, "bf16", 1)
    q, _, s, _ = outputs(4, 256)
    for args in ((x.cpu(), q, s), (x, q.cpu(), s), (x, q, s.cpu())):
        with pytest.raises(GemmError):
            S.quantize(*args)


def test_captured_and_replayed():
    x = source(200, 300, "bf16", 1)
    q, qt, s, st = outputs(200, 300)
    e = outputs(200, 300)
    S.quantize(x, q, s, qt, st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.quantize(x, q, s, qt, st)
    for seed in (2, 3, 4):
        x.copy_(source(200, 300, "bf16", seed))
        S.quantize(x, e[0], e[2], e[1], e[3])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q, e[0]) and torch.equal(qt, e[1]) and torch.equal(s, e[2]) and torch.equal(st, e[3])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_an_empty_matrix(dtype):
    """Every index points outside a matrix without rows: zeros, with the least scale."""
    x = torch.empty(0, 200, dtype=dtype, device="cuda")
    at = torch.tensor([-1, 0, 5, 2 ** 31 - 1, -2 ** 31] * 30, dtype=torch.int32, device="cuda")
    q = torch.full((150, 200), 9, dtype=torch.uint8, device="cuda")
    qt = torch.full((200, 150), 9, dtype=torch.uint8, device="cuda")
    s, st = torch.full((150, 2), -1.0, device="cuda"), torch.full((200, 2), -1.0, device="cuda")
    for both in (False, True):
        S.quantize(x, q, s, qt if both else None, st if both else None, row_index=at)
        assert (q == 0).all() and (s == 2.0 ** -126).all()
    assert (qt == 0).all() and (st == 2.0 ** -126).all()
