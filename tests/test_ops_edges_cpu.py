"""The operators around the layer on the CPU: limits at their edges, what the
binding makes for a call, and which kernel form a call takes."""
import ast
import ctypes
import inspect

import pytest
import torch

import combine_router_gemm_softmax_b200 as M
from combine_router_gemm_softmax_b200 import _lib
from ops_forms import FORMS, LONG, form_of, name_of


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


# ------------------------------------------------------------------ forms

@pytest.mark.parametrize("case", FORMS, ids=name_of)
def test_cases_take_their_form(L, case):
    """On a B200's 148 SMs. A change of the rule that moves a case has to bring another one for its form."""
    assert form_of(case, 148)[:2] == case[6:]


def test_long_cases_take_every_form(L):
    have = set()
    for sizes, length, width, forward, dgrad in LONG:
        assert M.moe_product_form_used("forward", sum(sizes), width, length, len(sizes))[0] == forward
        assert M.moe_product_form_used("dgrad", sum(sizes), length, width, len(sizes))[0] == dgrad
        have |= {("forward", forward), ("dgrad", dgrad)}
    tiles = {M.MOE_FORM_SINGLE, M.MOE_FORM_PAIR, M.MOE_FORM_SPLIT}
    assert have == {(p, f) for p in ("forward", "dgrad") for f in tiles} | {("forward", M.MOE_FORM_FEW_ROWS)}


def test_cases_cover_every_form(L):
    have = {(c[0], c[1], isinstance(c[2], int), c[6]) for c in FORMS}
    for dense in (True, False):
        for product in ("forward", "dgrad", "wgrad"):
            for dt in (torch.bfloat16, torch.float32):
                forms = {M.MOE_FORM_SINGLE, M.MOE_FORM_SPLIT}
                if dt == torch.bfloat16:
                    forms.add(M.MOE_FORM_PAIR)
                # few rows in fp32 over groups: tests/test_gpu_ops.py ("one_row_each", "few")
                if product == "forward" and (dense or dt == torch.bfloat16):
                    forms.add(M.MOE_FORM_FEW_ROWS)
                assert {(product, dt, dense, f) for f in forms} <= have


def test_form_query_refuses(L):
    I, U = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED
    form = (ctypes.c_int32 * 3)(7, 7, 7)
    cfg = M.MoeGemmConfig(rows=8, n=16, k=32, groups=2, dtype=M.MOE_DTYPE_BF16)
    for args in ((None, 0, 148, form), (cfg, 3, 148, form), (cfg, -1, 148, form), (cfg, 0, 0, form), (cfg, 0, 148, None)):
        assert L.moe_product_form_used(*args) == I
    assert L.moe_product_form_used(M.MoeGemmConfig(rows=8, n=16, k=31, groups=2), 0, 148, form) == U
    assert L.moe_product_form_used(M.MoeGemmConfig(rows=(1 << 31) - 1025, n=1 << 26, k=8, groups=1), 0, 148, form) == U
    assert list(form) == [7, 7, 7]
    assert L.moe_product_form_used(cfg, 0, 148, form) == M.MOE_OK and list(form) == [M.MOE_FORM_FEW_ROWS, 0, 1]
    with pytest.raises(ValueError, match="product"):
        M.moe_product_form_used("backward", 8, 16, 32)


def test_stalled_cases_take_every_tiled_form(L):
    from test_gpu_ops_edges import STALLS
    assert {(c[0], c[6]) for c in STALLS} >= {(p, f) for p, f in (
        ("forward", M.MOE_FORM_SINGLE), ("forward", M.MOE_FORM_PAIR), ("forward", M.MOE_FORM_SPLIT),
        ("dgrad", M.MOE_FORM_PAIR), ("dgrad", M.MOE_FORM_SPLIT), ("wgrad", M.MOE_FORM_PAIR), ("wgrad", M.MOE_FORM_SPLIT))}


def test_what_is_no_tensor_is_a_type_error():
    for check in (lambda t: _lib._strided(t, (2, 2), torch.float32, -1, "t"), lambda t: _lib._plain(t, (2, 2), torch.float32, -1, "t"),
                  lambda t: _lib._axes(t, 2, "t"), lambda t: _lib._first(t, 2, "t")):
        for t in ([[1.0, 2.0], [3.0, 4.0]], 3, torch.zeros(2, 2).numpy()):
            with pytest.raises(TypeError, match="t: expected a torch.Tensor"):
                check(t)
    with pytest.raises(TypeError, match="z: "):
        _lib._required(None, "z")
    with pytest.raises(ValueError, match="offsets"):
        M.moe_grouped_gemm_wgrad(torch.zeros(4, 8), torch.zeros(0, dtype=torch.int32), torch.zeros(4, 8))


def test_act_backward_needs_no_product_sizes(L):
    cfg = M.MoeGemmConfig(rows=0, n=8, dtype=M.MOE_DTYPE_F32, act=M.MOE_ACT_SILU)  # k and groups left at zero
    assert L.moe_act_backward(cfg, None, None, None, None) == M.MOE_OK
    assert L.moe_act_backward(M.MoeGemmConfig(rows=4, n=8, act=9), PTR, PTR, PTR, None) == M.MOE_ERR_INVALID_ARG
    assert L.moe_act_backward(M.MoeGemmConfig(rows=4, n=0), PTR, PTR, PTR, None) == M.MOE_ERR_INVALID_ARG
