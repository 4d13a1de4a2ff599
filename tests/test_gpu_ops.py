"""The operators around the layer on the GPU against the 64-bit oracle.

Tolerances, element by element:
  - a sum of K products in 32 bits is off by at most (K + 4) roundings of 2^-23
    (truncation counted, twice the half step) of S = sum |a b|;
  - an activation carries an error of its argument on times 1.13 (the largest
    slope of all of them, GELU's), and its own evaluation adds, for fp32
    outputs, 8 ulp, for bf16 outputs (fast exponential and reciprocal, Phi to
    1.5e-7) 1e-5 of the value and 1e-6 of the argument;
  - a slope is good to 1e-5 (bf16) or 2e-6 (fp32) absolutely;
  - every rounding of the result adds half a step of its type, eps / 2.
"""
import math

import pytest
import torch

import combine_router_gemm_softmax_b200 as M
from oracle import ops as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def eps2(dt):
    return torch.finfo(dt).eps / 2


def sum_error(k, scale):
    return (k + 4) * 2.0 ** -23 * scale


def close(got, want, tol, what=""):
    """|got - want| <= tol; NaN and infinities nowhere."""
    got = got.detach().cpu().double()
    off = (got - want).abs() - tol
    assert torch.isfinite(got).all(), what
    assert bool((off <= 0).all()), f"{what}: {float(off.max()):.3e} over the bound at {int(off.argmax())}"


def rounded(tol, want, dt):
    """tol, and the rounding of a value at most tol away to dt (and below dt's normal range, its smallest step)."""
    return tol + eps2(dt) * (want.abs() + tol) + 1e-38


def matrix(shape, dt, g, pad=0, scale=1.0, poison=False):
    """Device matrix; with pad, a view of rows `pad` elements wider than the
    width rounded up to 8, whose other columns hold NaN (if poison) or zeros."""
    t = (torch.randn(shape, generator=g) * scale).to(dt)
    if not pad:
        return t.to(DEV)
    wide = torch.full((*shape[:-1], (shape[-1] + 7) // 8 * 8 + pad), math.nan if poison else 0.0, dtype=dt)
    wide[..., :shape[-1]] = t
    return wide.to(DEV)[..., :shape[-1]]


def offsets_of(sizes, first=0):
    off = [first]
    for s in sizes:
        off.append(off[-1] + s)
    return off


# row counts a group: empty ones, single rows, around the row tiles of every kernel, a long one
GROUPS = {
    "one_row_each": [1, 0, 1, 1, 0, 0, 1, 1, 1, 1],
    "few": [3, 0, 9, 1],
    "tiles": [64, 128, 65, 0, 127, 129, 1],
    "ragged": [0, 300, 7, 0, 511, 33, 0],
    "single_group": [333],
    "none": [0, 0, 0],
}
SHAPES = [  # (groups, k, n, pad): widths off every tile, odd ones inside padded rows
    ("one_row_each", 256, 136, 0), ("one_row_each", 37, 51, 8), ("few", 8, 8, 0), ("few", 200, 264, 0),
    ("few", 1, 1, 8), ("tiles", 64, 256, 0), ("tiles", 72, 520, 0), ("tiles", 131, 77, 16), ("ragged", 384, 200, 0),
    ("ragged", 515, 1027, 8), ("single_group", 1024, 312, 0), ("none", 64, 64, 0),
]


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("name,k,n,pad", SHAPES)
@pytest.mark.parametrize("act,extras", [("none", ""), ("gelu", "bp"), ("silu", "br"), ("gelu_tanh", "rp"),
                                        ("relu", "brp")])
def test_forward(dt, name, k, n, pad, act, extras):
    g = torch.Generator().manual_seed(1)
    off = offsets_of(GROUPS[name], first=2)
    rows, E = off[-1] + 3, len(off) - 1
    x = matrix((rows, k), dt, g, pad, poison=True)
    w = matrix((E, n, k), dt, g, pad, 1 / math.sqrt(k), poison=True)
    bias = torch.randn((E, n), generator=g).to(DEV) if "b" in extras else None
    res = matrix((rows, n), dt, g, pad) if "r" in extras else None
    pre = matrix((rows, n), dt, g, pad) if "p" in extras else None
    y = matrix((rows, n), dt, g, pad)
    before, pre_before = y.clone(), None if pre is None else pre.clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = M.moe_grouped_gemm(x, torch.tensor(off, dtype=torch.int32, device=DEV), w, bias=bias, act=act, residual=res,
                             preact=pre, y=y, status=status)
    assert out is y and int(status.item()) == 0
    u, scale = R.product(x.cpu(), off, w.cpu(), None if bias is None else bias.cpu())
    a, b = off[0], off[-1]
    u, scale = u[a:b], scale[a:b]
    err = sum_error(k, scale)
    if pre is not None:
        close(pre[a:b], u, rounded(err, u, dt), "preact")
        assert torch.equal(pre[:a], pre_before[:a]) and torch.equal(pre[b:], pre_before[b:])
    v = R.act(u, act)
    err = 1.13 * err + (0 if act in ("none", "relu") else
                        1e-5 * v.abs() + 1e-6 * u.abs() if dt == BF16 else 8 * 2.0 ** -23 * (v.abs() + 0.1 * u.abs()))
    if res is not None:
        r = res[a:b].cpu().double()
        v, err = v + r, err + 2.0 ** -24 * (v.abs() + r.abs())
    close(y[a:b], v, rounded(err, v, dt), "y")
    # rows outside every group stay as they were, and columns beyond the width too
    assert torch.equal(y[:a], before[:a]) and torch.equal(y[b:], before[b:])
    if pad and rows:
        base = torch.as_strided(y, (rows, y.stride(0) - n), (y.stride(0), 1), n)
        assert torch.equal(base[:rows - 1], torch.zeros_like(base[:rows - 1]))


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("name,k,n,pad", SHAPES)
@pytest.mark.parametrize("act,residual", [(None, False), ("gelu", False), ("silu", True), ("gelu_tanh", True),
                                          ("relu", False), (None, True)])
def test_dgrad(dt, name, k, n, pad, act, residual):
    g = torch.Generator().manual_seed(2)
    off = offsets_of(GROUPS[name], first=1)
    rows, E = off[-1] + 2, len(off) - 1
    dy = matrix((rows, n), dt, g, pad, poison=True)
    w = matrix((E, n, k), dt, g, pad, 1 / math.sqrt(n), poison=True)
    z = matrix((rows, k), dt, g, pad, 1.5, poison=True) if act else None
    res = matrix((rows, k), dt, g, pad) if residual else None
    dx = matrix((rows, k), dt, g, pad)
    before = dx.clone()
    M.moe_grouped_gemm_dgrad(dy, torch.tensor(off, dtype=torch.int32, device=DEV), w, z=z, act=act or "none",
                             residual=res, dx=dx)
    u, scale = R.input_gradient(dy.cpu(), off, w.cpu())
    a, b = off[0], off[-1]
    v, err = u[a:b], sum_error(n, scale[a:b])
    if z is not None:
        slope = R.act_slope(z[a:b].cpu(), act)
        v, err = v * slope, 1.13 * err + v.abs() * (1e-5 if dt == BF16 else 2e-6)
    if res is not None:
        r = res[a:b].cpu().double()
        v, err = v + r, err + 2.0 ** -24 * (v.abs() + r.abs())
    close(dx[a:b], v, rounded(err, v, dt), "dx")
    assert torch.equal(dx[:a], before[:a]) and torch.equal(dx[b:], before[b:])


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("name,k,n,pad", SHAPES)
def test_wgrad(dt, name, k, n, pad):
    g = torch.Generator().manual_seed(3)
    off = offsets_of(GROUPS[name], first=1)
    rows, E = off[-1] + 2, len(off) - 1
    dy = matrix((rows, n), dt, g, pad, poison=True)
    x = matrix((rows, k), dt, g, pad, poison=True)
    # rows of no group hold NaN: no group's sums may see them
    dy[:off[0]], dy[off[-1]:], x[:off[0]], x[off[-1]:] = (math.nan,) * 4
    dw = torch.full((E, n, k), math.nan, device=DEV)
    db = torch.full((E, n), math.nan, device=DEV)
    M.moe_grouped_gemm_wgrad(dy, torch.tensor(off, dtype=torch.int32, device=DEV), x, dw=dw, dbias=db)
    want, want_b, scale, scale_b = R.weight_gradient(dy.cpu(), off, x.cpu())
    most = max(b - a for _, (a, b) in R.groups(off))
    close(dw, want, rounded(sum_error(most, scale), want, F32), "dw")
    close(db, want_b, rounded(sum_error(most, scale_b), want_b, F32), "dbias")
    # without a dbias the same weight gradient
    assert torch.equal(M.moe_grouped_gemm_wgrad(dy, torch.tensor(off, dtype=torch.int32, device=DEV), x), dw)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("m,k,n", [(1, 512, 768), (2, 24, 40), (5, 2048, 96), (17, 640, 264), (33, 128, 128),
                                   (77, 1408, 512), (200, 64, 2056), (777, 264, 392)])
def test_dense(dt, m, k, n):
    """The dense forms equal the grouped ones with one group of all rows, bit for bit, and the oracle."""
    g = torch.Generator().manual_seed(4)
    x, w, dy = matrix((m, k), dt, g), matrix((n, k), dt, g, scale=1 / math.sqrt(k)), matrix((m, n), dt, g)
    bias, res = torch.randn(n, generator=g).to(DEV), matrix((m, n), dt, g)
    all_rows = torch.tensor([0, m], dtype=torch.int32, device=DEV)
    y = M.moe_linear(x, w, bias=bias, act="silu", residual=res)
    assert torch.equal(y, M.moe_grouped_gemm(x, all_rows, w[None], bias=bias[None], act="silu", residual=res))
    u, scale = R.product(x.cpu(), [0, m], w.cpu()[None], bias.cpu()[None])
    v, r = R.act(u, "silu"), res.cpu().double()
    err = 1.13 * sum_error(k, scale) + 1e-5 * v.abs() + 1e-6 * u.abs() + 2.0 ** -24 * (v.abs() + r.abs())
    close(y, v + r, rounded(err, v + r, dt), "y")
    dx = M.moe_linear_dgrad(dy, w)
    assert torch.equal(dx, M.moe_grouped_gemm_dgrad(dy, all_rows, w[None]))
    v, scale = R.input_gradient(dy.cpu(), [0, m], w.cpu()[None])
    close(dx, v, rounded(sum_error(n, scale), v, dt), "dx")
    db = torch.empty(n, device=DEV)
    dw = M.moe_linear_wgrad(dy, x, dbias=db)
    assert torch.equal(dw, M.moe_grouped_gemm_wgrad(dy, all_rows, x)[0])
    want, want_b, scale, scale_b = R.weight_gradient(dy.cpu(), [0, m], x.cpu())
    close(dw, want[0], rounded(sum_error(m, scale[0]), want[0], F32), "dw")
    close(db, want_b[0], rounded(sum_error(m, scale_b[0]), want_b[0], F32), "db")


LARGE = [  # (rows of each group, k, n, pad): enough tiles for every way the bf16 kernel cuts a product up
    ([4099], 1032, 1408, 0), ([2500], 2048, 2048, 0), ([640], 4096, 264, 0), ([150], 6000, 640, 0), ([20000], 72, 160, 0),
    ([600, 0, 1, 257, 1500, 63, 1030, 255], 520, 1400, 0), ([2048, 2047, 2049, 0, 300], 640, 1288, 0),
    ([700, 900, 1200, 0, 31, 2000], 1001, 1111, 8), ([130] * 40, 264, 776, 0),
    ([9, 70, 200, 0, 1, 3, 64, 65] * 24, 200, 328, 0),
]


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("sizes,k,n,pad", LARGE)
def test_large(dt, sizes, k, n, pad):
    """Products of many tiles (the oracle's formulas evaluated in 64 bits on the GPU)."""
    g = torch.Generator().manual_seed(14)
    off = offsets_of(sizes, first=3)
    rows, E = off[-1] + 5, len(sizes)
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    x, dy = matrix((rows, k), dt, g, pad, poison=True), matrix((rows, n), dt, g, pad, poison=True)
    w = matrix((E, n, k), dt, g, pad, 1 / math.sqrt(k), poison=True)
    bias, res, z = torch.randn((E, n), generator=g).to(DEV), matrix((rows, n), dt, g, pad), matrix((rows, k), dt, g, pad)
    for t in (x, dy):
        t[:3], t[off[-1]:] = math.nan, math.nan
    pre, y = matrix((rows, n), dt, g, pad), matrix((rows, n), dt, g, pad)
    dx, before = matrix((rows, k), dt, g, pad), y.clone()
    db = torch.full((E, n), math.nan, device=DEV)
    dw = torch.full((E, n, k), math.nan, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    M.moe_grouped_gemm(x, o, w, bias=bias, act="gelu", residual=res, preact=pre, y=y, status=status)
    M.moe_grouped_gemm_dgrad(dy, o, w, z=z, act="silu", dx=dx, status=status)
    M.moe_grouped_gemm_wgrad(dy, o, x, dw=dw, dbias=db, status=status)
    assert int(status.item()) == 0
    assert torch.equal(y[:3], before[:3]) and torch.equal(y[off[-1]:], before[off[-1]:])

    def near(got, want, tol, t, what):
        off_by = (got.double() - want).abs() - rounded(tol, want, t)
        assert torch.isfinite(got).all() and bool((off_by <= 0).all()), (what, float(off_by.max()))

    for e in range(E):
        a, b = off[e], off[e + 1]
        xd, dd, wd, rd = x[a:b].double(), dy[a:b].double(), w[e].double(), res[a:b].double()
        u, err = xd @ wd.T + bias[e].double(), sum_error(k, xd.abs() @ wd.abs().T + bias[e].double().abs())
        near(pre[a:b], u, err, dt, "preact")
        v = R.act(u, "gelu")
        err = 1.13 * err + 1e-5 * v.abs() + 1e-6 * u.abs() + 2.0 ** -24 * (v.abs() + rd.abs())
        near(y[a:b], v + rd, err, dt, "y")
        s = R.act_slope(z[a:b], "silu")
        v, err = (dd @ wd) * s, sum_error(n, dd.abs() @ wd.abs())
        near(dx[a:b], v, 1.13 * err + 1e-5 * (dd @ wd).abs(), dt, "dx")
        # bf16: 16 rows a step of the tensor cores, 768 an accumulator, and a rounding for each accumulator
        steps = min(b - a, 768) / 16 + (b - a) / 768 + 1 if dt == BF16 else b - a
        near(dw[e], dd.T @ xd, sum_error(steps, dd.abs().T @ xd.abs()), F32, "dw")
        near(db[e], dd.sum(0), sum_error(b - a, dd.abs().sum(0)), F32, "db")


def test_other_groups_infinities_stay_theirs():
    """Infinities in one group's rows and weights reach no other group's outputs."""
    for dt in (F32, BF16):
        g = torch.Generator().manual_seed(5)
        off = offsets_of([70, 5, 130])
        o = torch.tensor(off, dtype=torch.int32, device=DEV)
        x, dy = matrix((off[-1], 200), dt, g), matrix((off[-1], 136), dt, g)
        w = matrix((3, 136, 200), dt, g)
        clean = [M.moe_grouped_gemm(x, o, w), M.moe_grouped_gemm_dgrad(dy, o, w), M.moe_grouped_gemm_wgrad(dy, o, x)]
        x[70:75], dy[70:75], w[1] = math.inf, math.inf, math.inf
        got = [M.moe_grouped_gemm(x, o, w), M.moe_grouped_gemm_dgrad(dy, o, w), M.moe_grouped_gemm_wgrad(dy, o, x)]
        for c, d in zip(clean[:2], got[:2]):
            assert torch.equal(c[:70], d[:70]) and torch.equal(c[75:], d[75:])
        assert torch.equal(clean[2][0], got[2][0]) and torch.equal(clean[2][2], got[2][2])


def test_bad_offsets_stay_in_bounds_and_are_reported():
    g = torch.Generator().manual_seed(6)
    for dt in (F32, BF16):
        for off in ([0, 40, 9000, 50], [-5, 10, 20, 64], [0, 50, 20, 64], [70, 80, 90, 100], [5, 1 << 30, -(1 << 30), 3]):
            o = torch.tensor(off, dtype=torch.int32, device=DEV)
            x, dy, w = matrix((64, 40), dt, g), matrix((64, 48), dt, g), matrix((3, 48, 40), dt, g)
            guard = torch.zeros((192, 48), dtype=dt, device=DEV)
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
            M.moe_grouped_gemm(x, o, w, y=guard[64:128], status=status)
            assert int(status.item()) == M.MOE_STATUS_BAD_OFFSETS
            assert not guard[:64].any() and not guard[128:].any()
            M.moe_grouped_gemm_dgrad(dy, o, w, status=status)
            M.moe_grouped_gemm_wgrad(dy, o, x, status=status)
            assert int(status.item()) == M.MOE_STATUS_BAD_OFFSETS


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_same_call_gives_the_same_bits_in_place_and_under_capture(dt):
    """Two runs, a residual that is the output itself, another stream, and a captured call replayed on new inputs."""
    g = torch.Generator().manual_seed(7)
    off = offsets_of([130, 0, 7, 90])
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    x, w, res = matrix((off[-1], 264), dt, g), matrix((4, 136, 264), dt, g), matrix((off[-1], 136), dt, g)
    dy = matrix((off[-1], 136), dt, g)

    def run():
        y = res.clone()
        return (M.moe_grouped_gemm(x, o, w, act="gelu", residual=y, y=y), M.moe_grouped_gemm_dgrad(dy, o, w),
                M.moe_grouped_gemm_wgrad(dy, o, x))

    first = run()
    assert torch.equal(first[0], M.moe_grouped_gemm(x, o, w, act="gelu", residual=res))
    for a, b in zip(first, run()):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = torch.empty_like(res)
    M.moe_grouped_gemm(x, o, w, act="gelu", residual=res, y=y, stream=side)
    side.synchronize()
    assert torch.equal(first[0], y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    keep = (x.clone(), o.clone())
    x.copy_(torch.randn(x.shape, generator=g).to(dt))
    o.copy_(torch.tensor(offsets_of([1, 100, 0, 126]), dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(captured, run()):
        assert torch.equal(a, b)
    x.copy_(keep[0])
    o.copy_(keep[1])
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(captured, first):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_many_short_rows(dt):
    """Far more row blocks than a grid's second axis holds, at the smallest widths."""
    g = torch.Generator().manual_seed(15)
    for sizes in ([700001], [300000, 0, 1, 400000]):
        off = offsets_of(sizes)
        o = torch.tensor(off, dtype=torch.int32, device=DEV)
        x, w = matrix((off[-1], 8), dt, g), matrix((len(sizes), 8, 8), dt, g)
        y = M.moe_grouped_gemm(x, o, w)
        for e, (a, b) in R.groups(off):
            u, s = x[a:b].double() @ w[e].double().T, x[a:b].double().abs() @ w[e].double().abs().T
            assert bool(((y[a:b].double() - u).abs() <= rounded(sum_error(8, s), u, dt)).all())
        dw = M.moe_grouped_gemm_wgrad(y, o, x)
        for e, (a, b) in R.groups(off):
            u, s = y[a:b].double().T @ x[a:b].double(), y[a:b].double().abs().T @ x[a:b].double().abs()
            assert bool(((dw[e].double() - u).abs() <= rounded(sum_error(b - a, s), u, F32)).all())


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_operands_apart_and_off_their_usual_alignment(dt):
    """Groups of W further apart than their rows are, fp32 operands on 4 bytes, outputs on 16 bytes but not 32."""
    g = torch.Generator().manual_seed(16)
    off = offsets_of([100, 3, 180])
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    rows, k, n = off[-1], 72, 88
    x, dy, res = matrix((rows, k), dt, g), matrix((rows, n), dt, g), matrix((rows, n), dt, g)
    w = matrix((3, n, k), dt, g)
    bias = torch.randn((3, n), generator=g).to(DEV)
    ref = M.moe_grouped_gemm(x, o, w, bias=bias, act="silu", residual=res)
    dref, wref = M.moe_grouped_gemm_dgrad(dy, o, w), M.moe_grouped_gemm_wgrad(dy, o, x)
    space = torch.full((3 * (n * 80 + 24),), math.nan, dtype=dt, device=DEV)
    apart = torch.as_strided(space, (3, n, k), (n * 80 + 24, 80, 1))
    apart.copy_(w)
    odd = torch.empty(3 * n + 1, device=DEV)[1:].view(3, n)
    odd.copy_(bias)
    y = torch.empty(rows * n + 8, dtype=dt, device=DEV)[16 // x.element_size():][:rows * n].view(rows, n)
    assert y.data_ptr() % 32 == 16
    assert torch.equal(M.moe_grouped_gemm(x, o, apart, bias=odd, act="silu", residual=res, y=y), ref)
    assert torch.equal(M.moe_grouped_gemm_dgrad(dy, o, apart), dref)
    dw = torch.empty(3 * n * k + 1, device=DEV)[1:].view(3, n, k)
    db = torch.empty(3 * n + 1, device=DEV)[1:].view(3, n)
    assert torch.equal(M.moe_grouped_gemm_wgrad(dy, o, x, dw=dw, dbias=db), wref)
    # a residual whose rows lie apart from the output's
    wide = torch.zeros((rows, n + 8), dtype=dt, device=DEV)[:, :n]
    wide.copy_(res)
    assert torch.equal(M.moe_grouped_gemm(x, o, w, bias=bias, act="silu", residual=wide), ref)


@pytest.mark.parametrize("rows,k,n,tiles", [(200, 640, 128, False), (1100, 640, 128, False), (640, 4096, 264, True),
                                            (4099, 1032, 1408, True)])
def test_a_wait_that_runs_out_is_reported(rows, k, n, tiles):
    """The tensor-core tiles' timeout path on every way a product is cut up:
    the MMA warp waits on a barrier that nothing signals until its limit, the
    call ends with the status bit, and the next one is right. (The forward of
    few rows, tiles = False, has no wait that could run out.)"""
    g = torch.Generator().manual_seed(17)
    x, w, dy = matrix((rows, k), BF16, g), matrix((n, k), BF16, g), matrix((rows, n), BF16, g)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    calls = (lambda: M.moe_linear(x, w, status=status), lambda: M.moe_linear_dgrad(dy, w, status=status),
             lambda: M.moe_linear_wgrad(dy, x, status=status))
    for i, call in enumerate(calls):
        ref = call().clone()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        assert M.lib().moe_debug_stall_next_gemms(1) == M.MOE_OK
        try:
            call()
            torch.cuda.synchronize()
        finally:
            M.lib().moe_debug_stall_next_gemms(0)
        assert int(status.item()) == (M.MOE_STATUS_TIMEOUT if tiles or i > 0 else 0)
        status.zero_()
        assert torch.equal(call(), ref)
        assert int(status.item()) == 0


def test_calls_side_by_side_do_not_disturb_one_another():
    """The same products on two streams at once, many times over, and dropout between them."""
    g = torch.Generator().manual_seed(18)
    off = offsets_of([70, 0, 400, 33])
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    x, w, dy = matrix((off[-1], 520), BF16, g), matrix((4, 264, 520), BF16, g), matrix((off[-1], 264), BF16, g)
    few, rng = matrix((4, 520), BF16, g), torch.tensor([1, 2], device=DEV)

    def run(s=None):
        return [M.moe_grouped_gemm(x, o, w, act="gelu", stream=s), M.moe_grouped_gemm_dgrad(dy, o, w, stream=s),
                M.moe_grouped_gemm_wgrad(dy, o, x, stream=s), M.moe_linear(few, w[0], stream=s),
                M.moe_dropout(x, 0.4, rng, residual=x, stream=s)]

    ref = run()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(run(s))
    torch.cuda.synchronize()
    for r in got:
        for a, b in zip(r, ref):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_rows_beyond_31_bits(dt):
    """Elements past 2^31 from the start of x and y: a few rows 2^24 elements apart."""
    g = torch.Generator().manual_seed(8)
    rows, k, n, ld = 140, 40, 24, 1 << 24
    space = torch.zeros(rows * ld, dtype=dt, device=DEV)
    x = space.view(rows, ld)[:, :k]
    y = space.view(rows, ld)[:, 64:64 + n]
    x.copy_(torch.randn((rows, k), generator=g).to(dt))
    w = matrix((n, k), dt, g)
    M.moe_linear(x, w, y=y)
    v, scale = R.product(x.cpu(), [0, rows], w.cpu()[None])
    close(y, v, rounded(sum_error(k, scale), v, dt), "y")
    assert torch.equal(M.moe_linear_wgrad(y, x), M.moe_linear_wgrad(y.contiguous(), x.contiguous()))
    rng = torch.tensor([3, 4], device=DEV)
    out = space.view(rows, ld)[:, 128:128 + k]
    M.moe_dropout(x, 0.5, rng, y=out)
    assert torch.equal(out, M.moe_dropout(x.contiguous(), 0.5, rng))


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("act", R.ACTS)
def test_act_backward(dt, act):
    g = torch.Generator().manual_seed(9)
    for rows, n, pad in ((1, 1, 8), (3, 8, 0), (65, 131, 8), (257, 520, 0)):
        dy, z = matrix((rows, n), dt, g, pad, poison=True), matrix((rows, n), dt, g, pad, 3.0, poison=True)
        dz = M.moe_act_backward(dy, z, act)
        v = dy.cpu().double()
        err = v.abs() * (0 if act in ("none", "relu") else 1e-5 if dt == BF16 else 2e-6)
        want = v * R.act_slope(z.cpu(), act)
        close(dz, want, rounded(err, want, dt), act)
        assert torch.equal(M.moe_act_backward(dy, z, act, dz=dy), dz)  # in place


def test_gradients_are_differences():
    """Kernel gradients against central differences of the kernels' own fp32
    forward: the loss <dy, y> is a sum of N ~ 400 fp32 outputs of size ~1,
    whose errors of 2^-20 each make the difference over 2 h = 0.02 uncertain by
    about 2^-20 * sqrt(400) * 2 / 0.02 ~ 2e-3; the third derivatives of the
    activations add h^2 / 6 * |f'''| ~ 2e-5 for weights of size 1."""
    g = torch.Generator().manual_seed(10)
    off = offsets_of([6, 0, 9])
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    x, w = matrix((15, 12), F32, g), matrix((3, 20, 12), F32, g, scale=0.3)
    b, dy = torch.randn((3, 20), generator=g).to(DEV), matrix((15, 20), F32, g)
    for act in ("none", "gelu", "gelu_tanh", "silu"):
        pre = torch.empty((15, 20), device=DEV)

        def loss():
            return float((M.moe_grouped_gemm(x, o, w, bias=b, act=act, preact=pre).double() * dy.double()).sum())

        loss()
        du = M.moe_act_backward(dy, pre.clone(), act)
        dx = M.moe_grouped_gemm_dgrad(du, o, w)
        db = torch.empty_like(b)
        dw = M.moe_grouped_gemm_wgrad(du, o, x, dbias=db)
        for t, grad, at in ((x, dx, (0, 3)), (x, dx, (14, 11)), (w, dw, (0, 19, 2)), (w, dw, (2, 0, 7)),
                            (w, dw, (1, 3, 3)), (b, db, (2, 5)), (b, db, (1, 1))):
            keep = t[at].item()
            t[at] = keep + 0.01
            up = loss()
            t[at] = keep - 0.01
            down = loss()
            t[at] = keep
            assert abs((up - down) / 0.02 - grad[at].item()) < 5e-3, (act, at)


# ------------------------------------------------------------------ dropout

DROPOUT = [(1, 1, 8), (3, 5, 8), (1, 64, 0), (7, 1000, 0), (64, 36, 0), (33, 2047, 8), (130, 4096, 0), (2000, 24, 0)]


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,pad", DROPOUT)
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout(dt, rows, cols, pad, p, residual):
    g = torch.Generator().manual_seed(11)
    x = matrix((rows, cols), dt, g, pad)
    res = matrix((rows, cols), dt, g, pad) if residual else None
    seed, at, offset = -7, (1 << 62) + 12345, (1 << 63) + 5
    rng = None if p == 0 else torch.tensor([seed, at], device=DEV)
    y = matrix((rows, cols), dt, g, pad)
    assert M.moe_dropout(x, p, rng, offset, residual=res, y=y) is y
    want = R.dropout(x.cpu(), p, seed, at + offset)
    err = 2.0 ** -23 * want.abs()
    if residual:
        r = res.cpu().double()
        want, err = want + r, err + 2.0 ** -24 * (want.abs() + r.abs())
    close(y, want, rounded(err, want, dt), "y")
    # in place on x and on the residual, and backward: the same mask on dy
    if residual:
        assert torch.equal(M.moe_dropout(x, p, rng, offset, residual=res, y=res), y)
    else:
        dy = matrix((rows, cols), dt, g)
        dx = M.moe_dropout(dy, p, rng, offset)
        back = R.dropout(dy.cpu(), p, seed, at + offset)
        close(dx, back, rounded(2.0 ** -23 * back.abs(), back, dt), "dx")
        assert torch.equal(M.moe_dropout(x, p, rng, offset, y=x), y)


def test_dropped_places_are_zero_whatever_they_hold():
    for dt in (F32, BF16):
        rng = torch.tensor([1, 2], device=DEV)
        ones = M.moe_dropout(torch.ones((40, 72), dtype=dt, device=DEV), 0.5, rng)
        for bad in (math.nan, math.inf, -math.inf):
            x = torch.where(ones == 0, torch.full_like(ones, bad), torch.ones_like(ones))
            assert torch.equal(M.moe_dropout(x, 0.5, rng), ones)


def test_dropout_keeps_its_share():
    """The kept share of n draws deviates from 1 - p by more than 5 sqrt(p (1 - p) / n) once in 1.7 million."""
    n = 4096 * 1024
    for i, p in enumerate((0.05, 0.3, 0.9)):
        y = M.moe_dropout(torch.ones((4096, 1024), device=DEV), p, torch.tensor([i, 99], device=DEV))
        share = float((y != 0).double().mean())
        assert abs(share - (1 - p)) < 5 * math.sqrt(p * (1 - p) / n)
        # neighbouring offsets, rows and columns draw independently: the agreement of two masks is (1-p)^2 + p^2
        z = M.moe_dropout(torch.ones((4096, 1024), device=DEV), p, torch.tensor([i, 99], device=DEV), 1)
        agree = (1 - p) ** 2 + p ** 2
        for a, b in ((y, z), (y[1:], y[:-1]), (y[:, 1:], y[:, :-1])):
            got = float(((a != 0) == (b != 0)).double().mean())
            assert abs(got - agree) < 6 * math.sqrt(agree * (1 - agree) / (n - 4096))


def test_captured_dropout_draws_anew_when_the_counter_moves():
    rng = torch.tensor([5, 0], device=DEV)
    x = torch.ones((64, 128), device=DEV)
    M.moe_dropout(x, 0.5, rng)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = M.moe_dropout(x, 0.5, rng, 3)
        rng[1] += 1
    rng.copy_(torch.tensor([5, 0]))
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.cpu().double(), R.dropout(torch.ones(64, 128), 0.5, 5, step + 3))


@pytest.mark.parametrize("dt,d", [(F32, 36), (F32, 260), (BF16, 128), (BF16, 640)])
@pytest.mark.parametrize("k", [1, 2, 5, 8])
@pytest.mark.parametrize("p,residual", [(0.0, False), (0.3, True), (0.3, False), (0.0, True)])
def test_combine_dropout(dt, d, k, p, residual):
    g = torch.Generator().manual_seed(12)
    T, E = 203, 8
    cfg = M.config(T, d, E, k, 128, dt, "identity")
    y_perm = matrix((T * k, d), dt, g)
    dest = torch.randperm(T * k, generator=g).reshape(T, k).to(torch.int32)
    dest[torch.rand((T, k), generator=g) < 0.3] = -1
    dest[5] = -1  # a token that kept nothing
    far = dest.clone()  # destinations outside y_perm count as dropped
    far[dest < 0] = torch.tensor([T * k, 1 << 30, -7], dtype=torch.int32)[torch.randint(0, 3, (int((dest < 0).sum()),), generator=g)]
    gate = torch.rand((T, k), generator=g)
    res = matrix((T, d), dt, g) if residual else None
    rng = torch.tensor([77, 13], device=DEV) if p else None
    y = M.moe_unpermute_combine_dropout(cfg, y_perm, dest.to(DEV), gate.to(DEV), p, rng, 21, residual=res)
    rows = torch.cat([y_perm.cpu().double(), torch.zeros((1, d), dtype=torch.float64)])[dest.long()]
    parts = gate.double()[..., None] * rows
    want = R.dropout(parts.sum(1), p, 77, 13 + 21)
    err = (k + 2) * 2.0 ** -24 / (1 - p) * parts.abs().sum(1) + 2.0 ** -23 * want.abs()
    if residual:
        r = res.cpu().double()
        want, err = want + r, err + 2.0 ** -24 * (want.abs() + r.abs())
    close(y, want, rounded(err, want, dt), "y")
    assert torch.equal(M.moe_unpermute_combine_dropout(cfg, y_perm, far.to(DEV), gate.to(DEV), p, rng, 21, residual=res), y)
    if residual:
        assert torch.equal(M.moe_unpermute_combine_dropout(cfg, y_perm, dest.to(DEV), gate.to(DEV), p, rng, 21, residual=res, y=res), y)
    if not p and not residual:
        assert torch.equal(y, M.moe_unpermute_combine(cfg, y_perm, dest.to(DEV), gate.to(DEV)))


# ------------------------------------------------------------------ as a block

@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_block_forward_and_backward(dt):
    """A block of GELU experts with biases beside a shared expert, with residual
    dropout, forward and backward. Each stage is checked on the GPU's own
    inputs to it, so that the tolerances are those of one stage."""
    g = torch.Generator().manual_seed(13)
    T, d, E, k, F, Fs, p = 301, 256, 8, 2, 384, 200, 0.1
    cfg = M.config(T, d, E, k, 128, dt, "identity")
    h = matrix((T, d), dt, g)
    wr = matrix((E, d), dt, g, scale=1 / math.sqrt(d))
    w1, w2 = matrix((E, F, d), dt, g, scale=1 / math.sqrt(d)), matrix((E, d, F), dt, g, scale=1 / math.sqrt(F))
    b1, b2 = torch.randn((E, F), generator=g).to(DEV), torch.randn((E, d), generator=g).to(DEV)
    s1, s2 = matrix((Fs, d), dt, g, scale=1 / math.sqrt(d)), matrix((d, Fs), dt, g, scale=1 / math.sqrt(Fs))
    rng = torch.tensor([41, 42], device=DEV)
    idx, gate = M.moe_route(cfg, h, wr)
    pm = M.moe_permute(cfg, h, idx)
    off_d, xp = pm["offsets"], pm["x_perm"]
    off = off_d.tolist()
    z1 = torch.empty((T * k, F), dtype=dt, device=DEV)
    a1 = M.moe_grouped_gemm(xp, off_d, w1, bias=b1, act="gelu", preact=z1)
    yp = M.moe_grouped_gemm(a1, off_d, w2, bias=b2)
    zs = torch.empty((T, Fs), dtype=dt, device=DEV)
    hs = M.moe_linear(h, s1, act="silu", preact=zs)
    shared = M.moe_linear(hs, s2, residual=h)  # h + shared expert
    out = M.moe_unpermute_combine_dropout(cfg, yp, pm["dest_row"], gate, p, rng, 1, residual=shared)

    def product(x, o, w, b=None):
        return R.product(x.cpu(), o, w.cpu(), None if b is None else b.cpu())

    def check(got, want, err, what):
        close(got, want, rounded(err, want, dt), what)

    u, s = product(xp, off, w1, b1)
    check(z1, u, sum_error(d, s), "z1")
    v = R.act(u, "gelu")
    check(a1, v, 1.13 * sum_error(d, s) + 1e-5 * v.abs() + 1e-6 * u.abs(), "a1")
    u, s = product(a1, off, w2, b2)
    check(yp, u, sum_error(F, s), "yp")
    u, s = product(h, [0, T], s1[None])
    v = R.act(u, "silu")
    check(hs, v, 1.13 * sum_error(d, s) + 1e-5 * v.abs() + 1e-6 * u.abs(), "hs")
    u, s = product(hs, [0, T], s2[None])
    check(shared, u + h.cpu().double(), sum_error(Fs, s) + 2.0 ** -22 * (u.abs() + h.cpu().double().abs()), "shared")
    dest, gates = pm["dest_row"].cpu().long(), gate.cpu().double()
    parts = gates[..., None] * yp.cpu().double()[dest]
    v = R.dropout(parts.sum(1), p, 41, 43) + shared.cpu().double()
    check(out, v, 2.0 ** -20 * (parts.abs().sum(1) + shared.cpu().double().abs()), "out")

    # backward from dout: the residual's path, the routed experts', the shared expert's
    dout = matrix((T, d), dt, g)
    dcomb = M.moe_dropout(dout, p, rng, 1)
    dyp = torch.zeros((T * k, d), dtype=dt, device=DEV)
    flat = pm["dest_row"].reshape(-1).long()
    dyp[flat] = (gate.reshape(-1, 1) * dcomb.float().repeat_interleave(k, 0)).to(dt)
    dz1 = M.moe_grouped_gemm_dgrad(dyp, off_d, w2, z=z1, act="gelu")
    db2 = torch.empty((E, d), device=DEV)
    dw2 = M.moe_grouped_gemm_wgrad(dyp, off_d, a1, dbias=db2)
    dxp = M.moe_grouped_gemm_dgrad(dz1, off_d, w1)
    dw1 = M.moe_grouped_gemm_wgrad(dz1, off_d, xp)
    dzs = M.moe_linear_dgrad(dout, s2, z=zs, act="silu")
    dh = M.moe_linear_dgrad(dzs, s1, residual=dout)
    ds2, ds1 = M.moe_linear_wgrad(dout, hs), M.moe_linear_wgrad(dzs, h)

    v = R.dropout(dout.cpu(), p, 41, 43)
    check(dcomb, v, 2.0 ** -23 * v.abs(), "dcomb")
    u, s = R.input_gradient(dyp.cpu(), off, w2.cpu())
    check(dz1, u * R.act_slope(z1.cpu(), "gelu"), 1.13 * sum_error(d, s) + 1e-5 * u.abs(), "dz1")
    u, s = R.input_gradient(dz1.cpu(), off, w1.cpu())
    check(dxp, u, sum_error(F, s), "dxp")
    u, s = R.input_gradient(dout.cpu(), [0, T], s2.cpu()[None])
    check(dzs, u * R.act_slope(zs.cpu(), "silu"), 1.13 * sum_error(d, s) + 1e-5 * u.abs(), "dzs")
    u, s = R.input_gradient(dzs.cpu(), [0, T], s1.cpu()[None])
    check(dh, u + dout.cpu().double(), sum_error(Fs, s) + 2.0 ** -22 * (u.abs() + dout.cpu().double().abs()), "dh")
    most = max(b - a for _, (a, b) in R.groups(off))
    for got, want, rows in ((dw2, R.weight_gradient(dyp.cpu(), off, a1.cpu()), most),
                            (dw1, R.weight_gradient(dz1.cpu(), off, xp.cpu()), most),
                            (ds2[None], R.weight_gradient(dout.cpu(), [0, T], hs.cpu()), T),
                            (ds1[None], R.weight_gradient(dzs.cpu(), [0, T], h.cpu()), T)):
        close(got, want[0], rounded(sum_error(rows, want[2]), want[0], F32), "dw")
    want = R.weight_gradient(dyp.cpu(), off, a1.cpu())
    close(db2, want[1], rounded(sum_error(most, want[3]), want[1], F32), "db2")


def test_binding_refuses_on_the_device():
    x, w = torch.zeros((4, 16), device=DEV), torch.zeros((8, 16), device=DEV)
    with pytest.raises(ValueError, match="shape"):
        M.moe_linear(x, w[:, :8])
    with pytest.raises(ValueError, match="dtype"):
        M.moe_linear(x, w.to(BF16))
    with pytest.raises(ValueError, match="cpu"):
        M.moe_linear(x, w, bias=torch.zeros(8))
    with pytest.raises(ValueError, match="act"):
        M.moe_linear(x, w, act="tanh")
    with pytest.raises(ValueError, match="dtype"):
        M.moe_linear(x.half(), w.half())
    with pytest.raises(M.MoeError) as e:  # odd bf16 widths need padded rows
        M.moe_linear(x.to(BF16)[:, :13].contiguous(), w.to(BF16)[:, :13].contiguous())
    assert e.value.code == M.MOE_ERR_UNSUPPORTED
    with pytest.raises(M.MoeError) as e:
        M.moe_dropout(x, 1.0, torch.zeros(2, dtype=torch.int64, device=DEV))
    assert e.value.code == M.MOE_ERR_INVALID_ARG
