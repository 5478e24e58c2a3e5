"""Products whose launch would have 2^32 threads along x are refused: the runtime would run such a
launch as what is left modulo 2^32, without an error.  On the host; pointers are numbers that nothing
reads, and without a GPU a launch that is let through ends as GEMM_ERR_LAUNCH."""
import ctypes

import pytest

from hierarchical_tiling_amd import htgemm as H

P, MOST, LAUNCH = 1 << 20, 2 ** 30 - 1, 6


@pytest.fixture(autouse=True)
def on_the_host(monkeypatch):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the sizes that fit would run")
    monkeypatch.setenv("HTGEMM_FAKE_ARCH", "gfx950")


def configs():
    name = ctypes.create_string_buffer(128)
    out = []
    for i in range(H.lib().gemm_num_configs()):
        H.lib().gemm_config_name(i, name, 128)
        out.append(name.value.decode())
    return out


def status(run):
    try:
        run()
    except H.GemmError as e:
        return e.status
    return H.GEMM_OK


@pytest.mark.parametrize("M,N", [(MOST, 64), (MOST, 520), (64, MOST), (1 << 25, 64)])
def test_one_product_by_every_kernel(M, N):
    K = 64
    for index, name in enumerate(configs()):
        if name.split("_")[1:3] != ["ak", "bk"] or "skinny" in name:
            continue
        h = H.Gemm(H.make_desc(M, N, K, name.split("_")[0], (K, 1), (1, K), (N, 1), force_config=index, split_k=1))
        i = h.info
        assert i.name.decode() == name
        got = status(lambda: H.gemm_run(h.handle, P, P, None, P, None, 1.0, 0.0, workspace=P if h.workspace_bytes else None, stream=0))
        threads = i.grid * i.waves * 64
        assert got == (H.GEMM_ERR_INVALID_ARG if threads >= 2 ** 32 else LAUNCH), (name, threads)


def test_groups():
    name = "bf16_ak_bk_64x64x64_w2x2_m16_vec"
    K, N, G = 64, 64, 4
    for M, refused in ((MOST, True), (MOST - (8 << 6), False), (1 << 20, False)):
        h = H.Gemm(H.make_desc(M, N, K, "bf16", (K, 1), (1, K), (N, 1), force_config=configs().index(name), batch=G,
                               batch_strides=(0, N * K, 0, 0), ragged_m=True))
        got = status(lambda: H.gemm_run_grouped(h.handle, P, P, None, P, None, None, None, P, 1.0, 0.0, stream=0, workspace=P))
        assert (got == H.GEMM_ERR_INVALID_ARG) == refused and got != H.GEMM_OK
