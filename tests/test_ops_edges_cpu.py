"""The operators around the layer on the CPU: limits at their edges, what the
binding makes for a call, and which kernel form a call takes."""
import ast
import inspect

import pytest
import torch

import combine_router_gemm_softmax_b200 as M
from combine_router_gemm_softmax_b200 import _lib


@pytest.fixture(scope="module")
def L():
    from combine_router_gemm_softmax_b200 import build
    build.build()
    return M.lib()


def test_calls_with_a_stream_make_their_tensors_for_it():
    """Every function that takes a stream makes outputs and workspaces by _empty (or workspace), and hands it the
    stream: memory of the current stream may still be written by earlier work there."""
    tree = ast.parse(inspect.getsource(_lib))
    made = 0
    for f in tree.body:
        if not isinstance(f, ast.FunctionDef) or f.name == "_empty" or "stream" not in [a.arg for a in f.args.args]:
            continue
        for call in ast.walk(f):
            if not isinstance(call, ast.Call):
                continue
            name = ast.unparse(call.func)
            assert name not in ("torch.empty", "torch.zeros", "torch.full", "torch.empty_like"), f.name
            if name in ("_empty", "_matrix", "workspace"):
                made += 1
                assert ast.unparse(call.args[-1]) == "stream", f.name
    assert made > 30


class Other:
    """A stream that is not the current one, and the tensors' record of it."""

    def __init__(self, log):
        self.log = log

    def __enter__(self):
        self.log.append("enter")

    def __exit__(self, *exc):
        self.log.append("exit")


def test_memory_for_another_stream(monkeypatch):
    log = []
    empty = torch.empty

    class Recorded:
        def record_stream(self, s):
            log.append(("record", s))

    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "current")
    monkeypatch.setattr(torch, "empty", lambda *a, **k: log.append("empty") or Recorded())
    _lib._empty((2, 3), torch.float32, "cpu", Other(log))
    assert log == ["enter", "empty", "exit", ("record", "current")]
    monkeypatch.setattr(torch, "empty", empty)
    assert _lib._empty((2, 3), torch.float32, "cpu", None).shape == (2, 3)


PTR = 1 << 20  # an aligned address that no refused call reads


def test_products_of_too_many_tiles_are_refused(L):
    """bf16 tiles are counted in 32 bits; the documented answer comes before any CUDA call."""
    most = (1 << 31) - 1025
    wide = M.MoeGemmConfig(rows=most, n=1 << 26, k=8, groups=1, dtype=M.MOE_DTYPE_BF16)
    deep = M.MoeGemmConfig(rows=most, n=8, k=1 << 26, groups=1, dtype=M.MOE_DTYPE_BF16)
    both = M.MoeGemmConfig(rows=128, n=1 << 26, k=1 << 26, groups=1, dtype=M.MOE_DTYPE_BF16)
    U = M.MOE_ERR_UNSUPPORTED
    assert L.moe_linear(wide, PTR, PTR, None, None, None, PTR, None, None) == U
    assert L.moe_linear_dgrad(deep, PTR, PTR, None, None, PTR, None, None) == U
    assert L.moe_linear_wgrad(both, PTR, PTR, PTR, None, None, None) == U


@pytest.mark.parametrize("kw", [dict(ldw=1 << 36, n=1 << 29), dict(ldw=1 << 36, n=(1 << 30) - 1),
                                dict(ldw=1 << 36, n=1 << 28, w_stride=1 << 36), dict(ldw=(1 << 62) + 8, n=5),
                                dict(ldw=1 << 37, n=8), dict(n=8, w_stride=1 << 37)])
def test_weight_strides_are_checked_without_overflow(L, kw):
    """Strides whose product with n leaves 64 bits once looked like short ones."""
    cfg = M.MoeGemmConfig(rows=8, k=32, groups=2, dtype=M.MOE_DTYPE_F32, **kw)
    assert L.moe_grouped_gemm(cfg, PTR, PTR, PTR, None, None, None, PTR, None, None) == M.MOE_ERR_UNSUPPORTED
    assert L.moe_grouped_gemm_dgrad(cfg, PTR, PTR, PTR, None, None, PTR, None, None) == M.MOE_ERR_UNSUPPORTED
