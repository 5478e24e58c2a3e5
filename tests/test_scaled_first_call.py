"""First calls of two threads at once: what a first call fills in is whole when another can see it."""
import sys

import pytest
import torch

from hierarchical_tiling_amd import htroute as R
from hierarchical_tiling_amd import htscaled as S


def every_step(f, code, look):
    """Runs f() and, before each instruction of the function with this code, what another thread that
    came there would find: look()."""
    def trace(frame, event, arg):
        if frame.f_code is not code:
            return None
        frame.f_trace_opcodes = True
        look()
        return trace

    before = sys.gettrace()
    sys.settrace(trace)
    try:
        return f()
    finally:
        sys.settrace(before)


def test_the_way_to_the_stream(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: None)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 77, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    for name in ("_raw_stream", "_device"):
        monkeypatch.setattr(S, name, None)
    steps = []

    def look():
        steps.append(S._raw_stream is None or S._device() == 3)

    assert every_step(lambda: S._here(None), S._here.__code__, look) == (3, 77)
    assert len(steps) > 5 and all(steps)


def test_the_types_of_the_routing(monkeypatch):
    for name in ("_i32t", "_f32t"):
        monkeypatch.setattr(R, name, None)
    steps = []

    def look():
        steps.append(R._i32t is None or (R._i32t is torch.int32 and R._f32t is torch.float32))

    every_step(R._types, R._types.__code__, look)
    assert len(steps) > 5 and all(steps) and R._f32t is torch.float32


@pytest.mark.parametrize("fill,table", [(lambda: S._kinds(S.DTYPES["bf16"]), "_KINDS"), (lambda: S.type_code(torch.zeros(1)), "_TYPE_CODES")])
def test_tables(fill, table, monkeypatch):
    monkeypatch.setattr(S, table, {})
    whole = {"_KINDS": 2, "_TYPE_CODES": 3}[table]
    sizes = []
    code = (S._kinds if table == "_KINDS" else S.type_code).__code__
    every_step(fill, code, lambda: sizes.append(len(getattr(S, table))))
    assert set(sizes) <= {0, whole} and len(getattr(S, table)) == whole
