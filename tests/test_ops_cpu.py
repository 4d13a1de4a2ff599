"""The operators around the layer on the CPU: what their entry points refuse
(every check fails before the library touches CUDA) and the 64-bit oracle that
the GPU tests compare them with."""
import ctypes
import math

import numpy as np
import pytest
import torch

import combine_router_gemm_softmax_b200 as M
from oracle import ops as R


@pytest.fixture(scope="module")
def L():
    from combine_router_gemm_softmax_b200 import build
    build.build()
    return M.lib()


# ------------------------------------------------------------------ oracle

@pytest.mark.parametrize("counter,key,want", [  # the generator's published test vectors
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_generator_vectors(counter, key, want):
    got = R.philox4x32([np.array([c]) for c in counter], key)
    assert tuple(int(g[0]) for g in got) == want


def test_dropout_words_are_laid_out_by_place():
    w = R.dropout_words(5, 11, seed=0x0123456789ABCDEF, at=(3 << 32) | 9)
    for r, c in ((0, 0), (2, 7), (4, 10)):
        one = R.philox4x32([np.array([v]) for v in (c // 4, r, 9, 3)], (0x89ABCDEF, 0x01234567))
        assert int(w[r, c]) == int(one[c % 4][0])
    # a row of a taller matrix is the same row; the offset wraps at 2^64
    assert np.array_equal(R.dropout_words([2], 11, 5, 7), R.dropout_words(3, 11, 5, 7)[2:])
    assert np.array_equal(R.dropout_words(2, 8, 5, 2 ** 64 + 1), R.dropout_words(2, 8, 5, 1))


@pytest.mark.parametrize("name", R.ACTS)
def test_slopes_are_differences(name):
    # central differences of step 1e-5 in 64 bits: truncation below f''' h^2 / 6 ~ 1e-10, rounding below 1e-10
    u = torch.linspace(-6.0, 6.0, 241, dtype=torch.float64) + 0.0125  # off relu's kink
    h = 1e-5
    diff = (R.act(u + h, name) - R.act(u - h, name)) / (2 * h)
    assert float((diff - R.act_slope(u, name)).abs().max()) < 1e-8


@pytest.mark.parametrize("name", R.ACTS)
def test_product_gradients_are_differences(name):
    g = torch.Generator().manual_seed(3)
    off = [0, 3, 3, 7]
    x = torch.randn(8, 5, generator=g, dtype=torch.float64)
    w = torch.randn(3, 4, 5, generator=g, dtype=torch.float64)
    b = torch.randn(3, 4, generator=g, dtype=torch.float64)
    dy = torch.randn(8, 4, generator=g, dtype=torch.float64)

    def loss(x, w, b):
        return float((R.act(R.product(x, off, w, b)[0], name) * dy)[:7].sum())

    u, _ = R.product(x, off, w, b)
    du = torch.zeros_like(dy)
    du[:7] = (dy * R.act_slope(u, name))[:7]
    dx, _ = R.input_gradient(du, off, w)
    dw, db, _, _ = R.weight_gradient(du, off, x)
    h = 1e-6
    for t, grad, at in ((x, dx, (1, 2)), (x, dx, (6, 4)), (w, dw, (0, 1, 3)), (w, dw, (1, 0, 0)), (w, dw, (2, 3, 1)),
                        (b, db, (0, 2)), (b, db, (2, 0))):
        keep = t[at].item()
        t[at] = keep + h
        up = loss(x, w, b)
        t[at] = keep - h
        down = loss(x, w, b)
        t[at] = keep
        assert abs((up - down) / (2 * h) - grad[at].item()) < 1e-7  # rounding of the sums over 2 h: about 1e-9


# ------------------------------------------------------------------ refusals of the C entry points

def gcfg(**kw):
    base = dict(rows=8, n=16, k=32, groups=2, dtype=M.MOE_DTYPE_BF16, act=M.MOE_ACT_NONE)
    base.update(kw)
    return M.MoeGemmConfig(**base)


PTR = 1 << 20  # an aligned address that no refused call reads


def forward(L, cfg, **kw):
    a = dict(x=PTR, offsets=PTR, w=PTR, bias=None, residual=None, preact=None, y=PTR)
    a.update(kw)
    return L.moe_grouped_gemm(cfg, a["x"], a["offsets"], a["w"], a["bias"], a["residual"], a["preact"], a["y"], None, None)


BAD_CONFIGS = [
    (dict(rows=-1), M.MOE_ERR_INVALID_ARG),
    (dict(n=0), M.MOE_ERR_INVALID_ARG),
    (dict(k=0), M.MOE_ERR_INVALID_ARG),
    (dict(groups=0), M.MOE_ERR_INVALID_ARG),
    (dict(groups=257), M.MOE_ERR_UNSUPPORTED),
    (dict(groups=256, n=1 << 23), M.MOE_ERR_UNSUPPORTED),
    (dict(rows=(1 << 31) - 1024), M.MOE_ERR_UNSUPPORTED),
    (dict(k=(1 << 31) - 8), M.MOE_ERR_UNSUPPORTED),
    (dict(k=(1 << 26) + 8), M.MOE_ERR_UNSUPPORTED),
    (dict(n=(1 << 26) + 8, groups=1), M.MOE_ERR_UNSUPPORTED),
    (dict(dtype=2), M.MOE_ERR_INVALID_ARG),
    (dict(ldx=24), M.MOE_ERR_INVALID_ARG),
    (dict(ldx=36), M.MOE_ERR_UNSUPPORTED),
    (dict(k=31), M.MOE_ERR_UNSUPPORTED),
    (dict(ldy=8), M.MOE_ERR_INVALID_ARG),
    (dict(ldy=20), M.MOE_ERR_UNSUPPORTED),
    (dict(ldx=1 << 37), M.MOE_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD_CONFIGS + [
    (dict(act=5), M.MOE_ERR_INVALID_ARG),
    (dict(act=-1), M.MOE_ERR_INVALID_ARG),
    (dict(ldw=16), M.MOE_ERR_INVALID_ARG),
    (dict(ldw=34), M.MOE_ERR_UNSUPPORTED),
    (dict(w_stride=256), M.MOE_ERR_INVALID_ARG),
    (dict(w_stride=516), M.MOE_ERR_UNSUPPORTED),
])
def test_products_refuse_configs(L, kw, code):
    cfg = gcfg(**kw)
    assert forward(L, cfg) == code
    assert L.moe_grouped_gemm_dgrad(cfg, PTR, PTR, PTR, None, None, PTR, None, None) == code


@pytest.mark.parametrize("kw,code", BAD_CONFIGS)
def test_weight_gradient_refuses_configs(L, kw, code):
    assert L.moe_grouped_gemm_wgrad(gcfg(**kw), PTR, PTR, PTR, PTR, None, None, None) == code


def test_products_refuse_pointers(L):
    I, U = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED
    cfg = gcfg()
    assert forward(L, None) == I
    for name in ("x", "offsets", "w", "y"):
        assert forward(L, cfg, **{name: None}) == I
    for name in ("x", "w", "residual", "preact", "y"):
        assert forward(L, cfg, **{name: PTR + 8}) == U
    assert forward(L, cfg, bias=PTR + 2) == U
    assert forward(L, cfg, offsets=PTR + 2) == U
    assert forward(L, gcfg(ldr=8), residual=PTR) == I
    assert forward(L, gcfg(ldr=20), residual=PTR) == U
    assert forward(L, gcfg(ldz=8), preact=PTR) == I
    for z, r in ((PTR, None), (None, PTR)):
        assert L.moe_grouped_gemm_dgrad(gcfg(ldz=24, ldr=24), PTR, PTR, PTR, z, r, PTR, None, None) == I
    assert L.moe_grouped_gemm_dgrad(cfg, None, PTR, PTR, None, None, PTR, None, None) == I
    assert L.moe_grouped_gemm_dgrad(cfg, PTR, PTR, PTR, PTR + 4, None, PTR, None, None) == U
    assert L.moe_grouped_gemm_wgrad(cfg, PTR, None, PTR, PTR, None, None, None) == I
    assert L.moe_grouped_gemm_wgrad(cfg, PTR, PTR, None, PTR, None, None, None) == I
    assert L.moe_grouped_gemm_wgrad(cfg, PTR, PTR, PTR, PTR + 2, None, None, None) == U
    # the dense forms have one group
    assert L.moe_linear(cfg, PTR, PTR, None, None, None, PTR, None, None) == I
    assert L.moe_linear_dgrad(cfg, PTR, PTR, None, None, PTR, None, None) == I
    assert L.moe_linear_wgrad(cfg, PTR, PTR, PTR, None, None, None) == I


def test_no_rows_is_no_work(L):
    empty = gcfg(rows=0)
    assert forward(L, empty, x=None, y=None) == M.MOE_OK
    assert L.moe_grouped_gemm_dgrad(empty, None, PTR, PTR, None, None, None, None, None) == M.MOE_OK
    assert L.moe_act_backward(gcfg(rows=0, groups=1), None, None, None, None) == M.MOE_OK
    assert L.moe_dropout(0, 4, 0, None, 0, None, 0, None, 0, 0.5, PTR, 0, None) == M.MOE_OK


def test_act_backward_refuses(L):
    one = gcfg(groups=1)
    assert L.moe_act_backward(None, PTR, PTR, PTR, None) == M.MOE_ERR_INVALID_ARG
    assert L.moe_act_backward(one, PTR, None, PTR, None) == M.MOE_ERR_INVALID_ARG
    assert L.moe_act_backward(gcfg(groups=1, ldz=8), PTR, PTR, PTR, None) == M.MOE_ERR_INVALID_ARG
    assert L.moe_act_backward(one, PTR, PTR + 8, PTR, None) == M.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), M.MOE_ERR_INVALID_ARG),
    (dict(cols=0), M.MOE_ERR_INVALID_ARG),
    (dict(dtype=7), M.MOE_ERR_INVALID_ARG),
    (dict(p=1.0), M.MOE_ERR_INVALID_ARG),
    (dict(p=-0.1), M.MOE_ERR_INVALID_ARG),
    (dict(p=math.nan), M.MOE_ERR_INVALID_ARG),
    (dict(rng=None), M.MOE_ERR_INVALID_ARG),
    (dict(x=None), M.MOE_ERR_INVALID_ARG),
    (dict(y=None), M.MOE_ERR_INVALID_ARG),
    (dict(ldx=4), M.MOE_ERR_INVALID_ARG),
    (dict(residual=PTR, ldr=4), M.MOE_ERR_INVALID_ARG),
    (dict(x=PTR + 2), M.MOE_ERR_UNSUPPORTED),
    (dict(rng=PTR + 4), M.MOE_ERR_UNSUPPORTED),
])
def test_dropout_refuses(L, kw, code):
    a = dict(rows=4, cols=8, dtype=0, x=PTR, ldx=0, residual=None, ldr=0, y=PTR, ldy=0, p=0.5, rng=PTR, offset=0)
    a.update(kw)
    assert L.moe_dropout(*a.values(), None) == code


def test_combine_dropout_refuses(L):
    cfg = M.config(8, 128, 4, 2, 128)
    I, U = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED

    def call(cfg=cfg, y_perm=PTR, dest=PTR, gate=PTR, residual=None, p=0.5, rng=PTR, y=PTR):
        ref = None if cfg is None else ctypes.byref(cfg)
        return L.moe_unpermute_combine_dropout(ref, y_perm, dest, gate, residual, p, rng, 0, y, None)

    assert call(cfg=None) == I
    assert call(cfg=M.config(8, 96, 4, 2, 128)) == U
    assert call(cfg=M.config(8, 128, 4, 5, 128)) == U
    assert call(cfg=M.config(0, 96, 4, 2, 128)) == U
    for name in ("y_perm", "dest", "gate", "y"):
        assert call(**{name: None}) == I
    assert call(p=1.0) == I and call(p=1.5) == I and call(rng=None) == I
    assert call(residual=PTR + 8) == U and call(y=PTR + 8) == U
    assert call(cfg=M.config(0, 128, 4, 2, 128), y_perm=None, dest=None, gate=None, y=None) == M.MOE_OK


# ------------------------------------------------------------------ refusals of the binding

def test_binding_refuses_cpu_tensors_and_wrong_types():
    x, w = torch.zeros(4, 8), torch.zeros(16, 8)
    with pytest.raises(ValueError, match="CUDA"):
        M.moe_linear(x, w)
    with pytest.raises(TypeError):
        M.moe_linear(None, w)
    with pytest.raises(TypeError):
        M.moe_grouped_gemm(x, None, w)
    with pytest.raises(ValueError, match="CUDA"):
        M.moe_dropout(x, 0.5)


def test_binding_refuses_strides_and_shapes():
    from combine_router_gemm_softmax_b200 import _lib
    cpu = -1  # the device index of CPU tensors
    t = torch.zeros(6, 8)
    assert _lib._strided(t, (6, 8), torch.float32, cpu, "t")[1] == 8
    assert _lib._strided(torch.zeros(6, 12)[:, :8], (6, 8), torch.float32, cpu, "t")[1] == 12
    for bad in (t.T, torch.zeros(1, 8).expand(6, 8), torch.zeros(6, 16)[:, ::2]):
        with pytest.raises(ValueError, match="t: "):
            _lib._strided(bad, tuple(bad.shape), torch.float32, cpu, "t")
    with pytest.raises(ValueError, match="shape"):
        _lib._strided(t, (6, 7), torch.float32, cpu, "t")
    with pytest.raises(ValueError, match="dtype"):
        _lib._strided(t, (6, 8), torch.bfloat16, cpu, "t")
    with pytest.raises(ValueError, match="contiguous"):
        _lib._plain(t.T, (8, 6), torch.float32, cpu, "t")
    with pytest.raises(ValueError, match="act"):
        _lib._act("tanh")
    # groups of a weight may lie apart, not on one another
    w = torch.zeros(3, 10, 8)[:, :6]
    assert _lib._weights(w, 3, 6, 8, torch.float32, cpu)[2] == 80
    with pytest.raises(ValueError, match="overlap"):
        _lib._weights(torch.zeros(6, 8).expand(3, 6, 8), 3, 6, 8, torch.float32, cpu)
