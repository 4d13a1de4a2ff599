"""The operators around the layer on the GPU where their kernels could go wrong
unseen: forms that only some shapes take, sums of any length, values far out,
and calls that the C interface allows but the binding does not make."""
import math

import pytest
import torch

import combine_router_gemm_softmax_b200 as M
from oracle import ops as R
from ops_forms import FIRST, FORMS, LONG, form_of, name_of, rows_of

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
CODE = {BF16: M.MOE_DTYPE_BF16, F32: M.MOE_DTYPE_F32}


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("off,bad", [([0, 40, 9000, 50], True), ([-5, 10, 20, 64], True), ([0, 50, 20, 64], True),
                                     ([0, 0, 10, 64], False), ([3, 20, 20, 60], False)])
def test_bias_gradient_alone_reports_bad_offsets(dt, off, bad):
    """The C interface's weight gradient without dw: the bias sums are the only kernel, and right (small integers,
    so exactly), or the status says that the offsets were not."""
    g = torch.Generator().manual_seed(1)
    dy = torch.randint(-3, 4, (64, 48), generator=g).to(dt).to(DEV)
    x = torch.zeros((64, 40), dtype=dt, device=DEV)
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    db = torch.full((3, 48), math.nan, device=DEV)
    cfg = M.MoeGemmConfig(rows=64, n=48, k=40, groups=3, dtype=CODE[dt])
    assert M.lib().moe_grouped_gemm_wgrad(cfg, dy.data_ptr(), o.data_ptr(), x.data_ptr(), None, db.data_ptr(),
                                          status.data_ptr(), stream()) == M.MOE_OK
    assert int(status.item()) == (M.MOE_STATUS_BAD_OFFSETS if bad else 0)
    if not bad:
        want = torch.stack([dy[a:b].float().sum(0) for _, (a, b) in R.groups(off)])
        assert torch.equal(db, want)


def far_act(u, name):
    """The activations in 64 bits without cancellation far out (1 + tanh loses its digits from -6 on)."""
    c = math.sqrt(2 / math.pi)
    return {"gelu": lambda: u * 0.5 * torch.special.erfc(-u / math.sqrt(2)), "silu": lambda: u * torch.sigmoid(u),
            "gelu_tanh": lambda: u * torch.sigmoid(2 * c * (u + 0.044715 * u ** 3))}[name]()


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("act,least", [("gelu", -12.75), ("gelu_tanh", -9.5), ("silu", -80.0)])
def test_negative_tails_keep_their_digits(dt, act, least):
    """Activations and slopes against their own small values, down to `least` (the values stay above 1e-36, inside
    the types' normal range). Relative errors: half a step of the type, and the evaluation's, whose largest part is
    the exponent: up to 125 in base 2, five roundings of 2^-24 of it at most, times ln 2: 2.6e-5 with GELU's tanh
    form, less with the others; 3e-5 with the function's own error. A slope is the sum of two such terms; where it
    is tested it is at least 0.43 of the larger one, so its bound is three times that."""
    u = torch.cat([torch.linspace(least, -2.0, 250), torch.linspace(2.0, 12.0, 150)]).to(dt).reshape(25, 16).to(DEV)
    ud = u.cpu().double().requires_grad_()
    want = far_act(ud, act)
    slope, = torch.autograd.grad(want.sum(), ud)
    want = want.detach()
    half = torch.finfo(dt).eps / 2
    eye = torch.eye(16, dtype=dt, device=DEV)
    for name, got, ref, err in (("rows", M.moe_linear(u[:8], eye, act=act), want[:8], 3e-5),
                                ("tiles", M.moe_linear(u.repeat(300, 1), eye, act=act)[-25:], want, 3e-5),
                                ("slope", M.moe_act_backward(torch.ones_like(u), u, act), slope, 9e-5)):
        off = (got.cpu().double() - ref).abs() / ref.abs()
        assert float(off.max()) <= half + err, (name, float(off.max()), float(u.cpu().reshape(-1)[int(off.argmax())]))


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("act", R.ACTS)
def test_activations_far_from_zero(act, dt):
    """Any finite argument: past 100 every activation is its argument or zero and its slope one or zero, exactly,
    up to the largest numbers of the type (whose squares and cubes are infinite), and NaN stays in its place."""
    big = [100.0, 1e10, 1.8e19, 2e19, 1e20, 1e38, torch.finfo(dt).max]
    z = torch.tensor([big + [-v for v in big] + [math.nan, 0.0]], device=DEV).to(dt)
    ones = torch.ones_like(z)
    pos = torch.cat([torch.ones(7), torch.full((7,), 1.0 if act == "none" else 0.0)]).to(dt)
    slopes = [M.moe_act_backward(ones, z, act), M.moe_linear_dgrad(ones, torch.eye(16, device=DEV).to(dt), z=z, act=act)]
    for got in slopes:
        assert torch.equal(got[0, :14].cpu(), pos)
        assert act == "relu" or act == "none" or bool(got[0, 14].isnan())
    v = M.moe_linear(torch.nan_to_num(z, nan=0.0), torch.eye(16, device=DEV).to(dt), act=act)[0, :14].cpu()
    assert torch.equal(v, pos * z[0, :14].cpu())


@pytest.mark.parametrize("dgrad", [False, True], ids=["forward", "dgrad"])
@pytest.mark.parametrize("sizes,length,width", [c[:3] for c in LONG])
def test_long_reductions_are_not_biased(sizes, length, width, dgrad):
    """bf16 products of one sign over long reductions. Tensor cores truncate when they add, so that the error of one
    accumulator grows with the length (7e-4 at 2^20); kept to 16384 elements, 1024 steps of 16, it is at most
    1024 steps of 2^-23, and the partial sums add a rounding each (at most 64 here). A residual takes the bulk of
    the sum away, so that the rounding of the output does not hide it."""
    g = torch.Generator(device=DEV).manual_seed(3)
    off = [0]
    for s in sizes:
        off.append(off[-1] + s)
    E, rows = len(sizes), off[-1]
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    a = (torch.rand((rows, length), generator=g, device=DEV) + 0.5).to(BF16)
    w = (torch.rand((E, length, width) if dgrad else (E, width, length), generator=g, device=DEV) + 0.5).to(BF16)
    want = torch.zeros((rows, width), dtype=torch.float64, device=DEV)
    for e, (r0, r1) in R.groups(off):
        for i in range(0, length, 1 << 14):
            we = w[e, i:i + (1 << 14)] if dgrad else w[e, :, i:i + (1 << 14)].T
            want[r0:r1] += a[r0:r1, i:i + (1 << 14)].double() @ we.double()
    bulk = (-want).to(BF16)
    y = M.moe_grouped_gemm_dgrad(a, o, w, residual=bulk) if dgrad else M.moe_grouped_gemm(a, o, w, residual=bulk)
    left = want + bulk.double()
    tol = (1024 + 64 + 4) * 2.0 ** -23 * want
    off_by = (y.double() - left).abs() - tol - torch.finfo(BF16).eps / 2 * (left.abs() + tol)
    assert float(off_by.max()) <= 0, float(((y.double() - left) / want).abs().max())


@pytest.mark.parametrize("rows,n,k", [(500, 512, 640), (1000, 1408, 512), (4099, 264, 136), (8191, 1024, 1024), (20000, 136, 264)])
def test_weight_gradient_is_as_exact_as_promised(rows, n, k):
    """include/moe.h: within 6e-7 of its size, root mean square, for normally distributed bf16 rows at any length."""
    g = torch.Generator(device=DEV).manual_seed(4)
    dy = torch.randn((rows, n), generator=g, device=DEV).to(BF16)
    x = torch.randn((rows, k), generator=g, device=DEV).to(BF16)
    want = dy.double().T @ x.double()
    assert float((M.moe_linear_wgrad(dy, x).double() - want).norm() / want.norm()) <= 6e-7


def calls_on_a_stream():
    g = torch.Generator().manual_seed(5)
    rnd = lambda *shape: torch.randn(shape, generator=g).to(BF16).to(DEV)
    x, w, dy, z = rnd(1000, 256), rnd(2, 256, 256), rnd(1000, 256), rnd(1000, 256)
    o, rng = torch.tensor([0, 400, 1000], dtype=torch.int32, device=DEV), torch.tensor([1, 2], device=DEV)
    cfg = M.config(500, 256, 4, 2, 128, "bf16", "identity")
    dest = torch.randperm(1000, generator=g).reshape(500, 2).to(torch.int32).to(DEV)
    gate = torch.rand((500, 2), generator=g).to(DEV)
    return {
        "grouped": lambda s: M.moe_grouped_gemm(x, o, w, stream=s),
        "grouped_dgrad": lambda s: M.moe_grouped_gemm_dgrad(dy, o, w, stream=s),
        "grouped_wgrad": lambda s: M.moe_grouped_gemm_wgrad(dy, o, x, stream=s),
        "linear": lambda s: M.moe_linear(x, w[0], stream=s),
        "linear_dgrad": lambda s: M.moe_linear_dgrad(dy, w[0], stream=s),
        "linear_wgrad": lambda s: M.moe_linear_wgrad(dy, x, stream=s),
        "act_backward": lambda s: M.moe_act_backward(dy, z, "silu", stream=s),
        "dropout": lambda s: M.moe_dropout(x, 0.5, rng, stream=s),
        "combine_dropout": lambda s: M.moe_unpermute_combine_dropout(cfg, x, dest, gate, 0.5, rng, stream=s),
    }


def written_on_another_stream(call):
    """The call's output, made by the call on another stream, while the current stream still has to write memory that
    was freed just before, and read again on the current stream after a wait, while the other stream goes on."""
    ref = call(None).clone()
    side = torch.cuda.Stream()
    call(side)  # any first-call set-up
    torch.cuda.synchronize()
    freed = torch.empty_like(ref)
    torch.cuda._sleep(100_000_000)  # some 50 ms
    freed.fill_(7)
    del freed
    y = call(side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(y, ref)
    side.wait_stream(torch.cuda.current_stream())
    y = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(100_000_000)
    copy = y.clone()
    del y
    with torch.cuda.stream(side):
        for _ in range(3):
            torch.empty_like(ref).fill_(9)
    torch.cuda.synchronize()
    assert torch.equal(copy, ref)


@pytest.mark.parametrize("name", ["grouped", "grouped_dgrad", "grouped_wgrad", "linear", "linear_dgrad", "linear_wgrad",
                                  "act_backward", "dropout", "combine_dropout"])
def test_outputs_made_for_another_stream(name):
    written_on_another_stream(calls_on_a_stream()[name])


def layer_calls_on_a_stream():
    g = torch.Generator().manual_seed(6)
    rnd = lambda *shape: (torch.randn(shape, generator=g) / 8).to(BF16).to(DEV)
    T, d, E, k, F = 512, 256, 8, 2, 256
    cfg = M.config(T, d, E, k, F)
    h, wr, wg, wu, wd = rnd(T, d), rnd(E, d), rnd(E, F, d), rnd(E, F, d), rnd(E, d, F)
    w13 = M.moe_pack_weights(cfg, wg, wu)
    idx, gate = M.moe_route(cfg, h, wr)
    pm = M.moe_permute(cfg, h, idx)
    yp = M.moe_grouped_ffn(cfg, pm["x_perm"], pm["offsets"], w13, wd)
    fwd_ws = M.workspace(cfg, M.MOE_OP_LAYER, DEV)
    M.moe_layer_forward(cfg, h, wr, w13_packed=w13, w_down=wd, ws=fwd_ws)
    w13_t, wd_t = M.moe_pack_weights_backward(cfg, w13, wd)
    return {
        "pack": lambda s: M.moe_pack_weights(cfg, wg, wu, stream=s),
        "route": lambda s: M.moe_route(cfg, h, wr, stream=s)[1],
        "permute": lambda s: M.moe_permute(cfg, h, idx, stream=s)["x_perm"],
        "ffn": lambda s: M.moe_grouped_ffn(cfg, pm["x_perm"], pm["offsets"], w13, wd, stream=s),
        "combine": lambda s: M.moe_unpermute_combine(cfg, yp, pm["dest_row"], gate, stream=s),
        "layer": lambda s: M.moe_layer_forward(cfg, h, wr, w13_packed=w13, w_down=wd, stream=s),
        "pack_backward": lambda s: M.moe_pack_weights_backward(cfg, w13, wd, stream=s)[0],
        "backward": lambda s: M.moe_layer_backward(cfg, h, wr, w13, w13_t, wd_t, h, fwd_ws, stream=s)["dw13"],
        "quantize": lambda s: M.moe_mxfp8_quantize(h, stream=s)[1],
        "pack_mxfp8": lambda s: M.moe_pack_weights_mxfp8(cfg, w13, wd, stream=s)[0],
    }


@pytest.mark.parametrize("name", ["pack", "route", "permute", "ffn", "combine", "layer", "pack_backward", "backward",
                                  "quantize", "pack_mxfp8"])
def test_outputs_of_the_layer_made_for_another_stream(name):
    written_on_another_stream(layer_calls_on_a_stream()[name])


@pytest.mark.parametrize("cols", [(1 << 31) - 1, (1 << 31) - 3, (1 << 31) - 8])
def test_dropout_of_the_widest_rows(cols):
    """One row of up to 2^31 - 1 columns: its ends, and a piece in the middle, against the generator's words."""
    import numpy as np
    p, seed, at = 0.5, 5, 7
    x = torch.ones((1, cols), dtype=BF16, device=DEV)
    y = M.moe_dropout(x, p, torch.tensor([seed, at], device=DEV))
    for first in (0, (1 << 30) - 32, cols // 4 * 4 - 64):
        last = min(first + 68, cols)
        quads = np.arange(first // 4, (last + 3) // 4, dtype=np.uint64)
        words = np.stack(R.philox4x32([quads, np.zeros_like(quads), np.full_like(quads, at), np.zeros_like(quads)],
                                      (seed, 0)), axis=1).reshape(-1)[:last - first]
        want = torch.from_numpy((words >= 1 << 31).astype(np.float64)) * 2
        assert torch.equal(y[0, first:last].cpu().double(), want), first


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_strides_of_absent_operands_do_not_matter(dt):
    """A bias gradient beside a dw that nobody could hold, and far strides of operands that the call does not have."""
    g = torch.Generator().manual_seed(7)
    n = k = 1 << 19
    dy = torch.randint(-3, 4, (5, n), generator=g).to(dt).to(DEV)
    x = torch.zeros((5, k), dtype=dt, device=DEV)
    db = torch.full((n,), math.nan, device=DEV)
    cfg = M.MoeGemmConfig(rows=5, n=n, k=k, groups=1, dtype=CODE[dt])
    assert M.lib().moe_linear_wgrad(cfg, dy.data_ptr(), x.data_ptr(), None, db.data_ptr(), None, stream()) == M.MOE_OK
    assert torch.equal(db, dy.float().sum(0))
    x, w = torch.ones((5, 64), dtype=dt, device=DEV), torch.ones((8, 64), dtype=dt, device=DEV)
    y = torch.zeros((5, 8), dtype=dt, device=DEV)
    cfg = M.MoeGemmConfig(rows=5, n=8, k=64, groups=1, dtype=CODE[dt], ldr=1 << 40, ldz=1 << 40, w_stride=1 << 40)
    assert M.lib().moe_linear(cfg, x.data_ptr(), w.data_ptr(), None, None, None, y.data_ptr(), None, stream()) == M.MOE_OK
    assert bool((y == 64).all())


# ------------------------------------------------------------------ every form, exactly

def integers(shape, dt, g, pad=0, most=2):
    """Whole numbers of up to `most` either way; with pad, rows that lie apart with NaN between them."""
    t = torch.randint(-most, most + 1, shape, generator=g, device=DEV).to(dt)
    if not pad:
        return t
    wide = torch.full((*shape[:-1], (shape[-1] + 7) // 8 * 8 + pad), math.nan, dtype=dt, device=DEV)
    wide[..., :shape[-1]] = t
    return wide[..., :shape[-1]]


def exactly(got, want, what):
    """want: the exact result in fp32 (whole numbers below 2^24); got: that, rounded once."""
    want = want.to(got.dtype)
    if not torch.equal(got, want):
        bad = (got != want) | got.isnan()
        at = torch.nonzero(bad)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} wrong, first at {at[0].tolist()}, last at "
                             f"{at[-1].tolist()}: {float(got[bad][0])}, not {float(want[bad][0])}")


def product_setup(case):
    _, dt, sizes, n, k, pad, form, _ = case
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert form_of(case, sms)[0] == form
    g = torch.Generator(device=DEV).manual_seed(n * 31 + k)
    dense = isinstance(sizes, int)
    ends = [0, sizes] if dense else [FIRST + sum(sizes[:e]) for e in range(len(sizes) + 1)]
    rows, E = rows_of(sizes), len(ends) - 1
    o = torch.tensor(ends, dtype=torch.int32, device=DEV)
    x, dy = integers((rows, k), dt, g, pad), integers((rows, n), dt, g, pad)
    for t in (x, dy):  # rows of no group: nothing may see them
        t[:ends[0]], t[ends[-1]:] = math.nan, math.nan
    return g, dense, ends, rows, E, o, x, dy


@pytest.mark.parametrize("case", FORMS, ids=name_of)
def test_every_form_exactly(case):
    """Products of small whole numbers, whose sums every order and every accumulator holds exactly: one element that
    is missing, read twice or of another group, at any length, makes a difference."""
    product, dt, sizes, n, k, pad = case[:6]
    g, dense, ends, rows, E, o, x, dy = product_setup(case)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    inside = slice(ends[0], ends[-1])
    if product == "wgrad":
        dw, db = torch.full((E, n, k), math.nan, device=DEV), torch.full((E, n), math.nan, device=DEV)
        if dense:
            M.moe_linear_wgrad(dy, x, dw=dw[0], dbias=db[0], status=status)
        else:
            M.moe_grouped_gemm_wgrad(dy, o, x, dw=dw, dbias=db, status=status)
        for e, (a, b) in R.groups(ends):
            exactly(dw[e], dy[a:b].float().T @ x[a:b].float(), f"dw {e}")
            exactly(db[e], dy[a:b].float().sum(0), f"dbias {e}")
        assert int(status.item()) == 0
        return
    w = integers((E, n, k), dt, g, pad)
    width = n if product == "forward" else k
    res = integers((rows, width), dt, g, pad)
    out = integers((rows, width), dt, g, pad).fill_(5.0)
    if product == "forward":
        bias = torch.randint(-9, 10, (E, n), generator=g, device=DEV).float()
        pre = integers((rows, width), dt, g, pad).fill_(5.0)
        if dense:
            M.moe_linear(x, w[0], bias=bias[0], act="relu", residual=res, preact=pre, y=out, status=status)
        else:
            M.moe_grouped_gemm(x, o, w, bias=bias, act="relu", residual=res, preact=pre, y=out, status=status)
    else:
        z = integers((rows, k), dt, g, pad, 1)  # relu's slope: one or zero
        if dense:
            M.moe_linear_dgrad(dy, w[0], z=z, act="relu", residual=res, dx=out, status=status)
        else:
            M.moe_grouped_gemm_dgrad(dy, o, w, z=z, act="relu", residual=res, dx=out, status=status)
    assert int(status.item()) == 0
    for e, (a, b) in R.groups(ends):
        if product == "forward":
            u = x[a:b].float() @ w[e].float().T + bias[e]
            exactly(pre[a:b], u, f"preact {e}")
            exactly(out[a:b], u.clamp(min=0) + res[a:b].float(), f"y {e}")
        else:
            exactly(out[a:b], (z[a:b] > 0) * (dy[a:b].float() @ w[e].float()) + res[a:b].float(), f"dx {e}")
    outside = torch.ones(rows, dtype=torch.bool, device=DEV)
    outside[inside] = False
    assert bool((out[outside] == 5).all())
    if product == "forward":
        assert bool((pre[outside] == 5).all())


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("sizes,n,k", [([700001], 8, 8), ([300000, 0, 1, 400000], 8, 8), ([20000], 160, 72),
                                       ([20000, 3, 0, 40001], 136, 264)])
def test_long_sums_of_rows_miss_none(dt, sizes, n, k):
    """Weight and bias gradients over very many rows, exactly (sums of whole numbers below 2^24): a bound that grows
    with the rows would let whole blocks of them go missing."""
    g = torch.Generator(device=DEV).manual_seed(8)
    ends = [FIRST + sum(sizes[:e]) for e in range(len(sizes) + 1)]
    rows, E = rows_of(sizes), len(sizes)
    o = torch.tensor(ends, dtype=torch.int32, device=DEV)
    dy, x = integers((rows, n), dt, g), integers((rows, k), dt, g)
    for t in (x, dy):
        t[:ends[0]], t[ends[-1]:] = math.nan, math.nan
    db = torch.full((E, n), math.nan, device=DEV)
    dw = M.moe_grouped_gemm_wgrad(dy, o, x, dbias=db)
    for e, (a, b) in R.groups(ends):
        exactly(dw[e], (dy[a:b].double().T @ x[a:b].double()).float(), f"dw {e}")
        exactly(db[e], dy[a:b].double().sum(0).float(), f"dbias {e}")


STALLS = [c for c in FORMS if c[1] == BF16 and c[6] != M.MOE_FORM_FEW_ROWS and c[2] in (
    331, 12293, [70, 0, 200, 1, 33, 19], 16381, [130, 0, 7], 8193, [18000, 14742], [2049, 1, 4099])]


@pytest.mark.parametrize("case", STALLS, ids=name_of)
def test_a_wait_that_runs_out_in_every_form(case):
    """The tiles' timeout path in the forms named by the case (forward single, pair and split; dgrad pair and split;
    wgrad pair and split, their zeroed rows included): the MMA warp waits on a barrier that nothing signals until its
    limit, the status says so, and the next call is right."""
    product, dt, sizes, n, k, pad = case[:6]
    g, dense, ends, rows, E, o, x, dy = product_setup(case)
    w = integers((E, n, k), dt, g, pad)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    call = {"forward": lambda: M.moe_grouped_gemm(x, o, w, status=status)[ends[0]:ends[-1]],
            "dgrad": lambda: M.moe_grouped_gemm_dgrad(dy, o, w, status=status)[ends[0]:ends[-1]],
            "wgrad": lambda: M.moe_grouped_gemm_wgrad(dy, o, x, status=status)}[product]
    ref = call().clone()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert M.lib().moe_debug_stall_next_gemms(1) == M.MOE_OK
    try:
        call()
        torch.cuda.synchronize()
    finally:
        M.lib().moe_debug_stall_next_gemms(0)
    assert int(status.item()) == M.MOE_STATUS_TIMEOUT
    status.zero_()
    assert torch.equal(call(), ref)
    assert int(status.item()) == 0


def test_binding_names_what_is_no_tensor():
    x, w, o = torch.zeros((4, 16), device=DEV), torch.zeros((2, 8, 16), device=DEV), torch.tensor([0, 2, 4], device=DEV)
    dy, cfg = torch.zeros((4, 8), device=DEV), M.config(2, 16, 4, 2, 128, "f32", "identity")
    d, g = torch.zeros((2, 2), dtype=torch.int32, device=DEV), torch.zeros((2, 2), device=DEV)
    for name, call in (("w", lambda: M.moe_linear(x, None)), ("w", lambda: M.moe_linear(x, [[0.0] * 16] * 8)),
                       ("w", lambda: M.moe_linear_dgrad(dy, None)), ("offsets", lambda: M.moe_grouped_gemm(x, [0, 2, 4], w)),
                       ("bias", lambda: M.moe_linear(x, w[0], bias=[0.0] * 8)), ("x", lambda: M.moe_linear_wgrad(dy, None)),
                       ("residual", lambda: M.moe_linear(x, w[0], residual=1.0)), ("z", lambda: M.moe_act_backward(x, None, "relu")),
                       ("status", lambda: M.moe_linear(x, w[0], status=0)), ("rng", lambda: M.moe_dropout(x, 0.5, [1, 2])),
                       ("dest_row", lambda: M.moe_unpermute_combine_dropout(cfg, x, None, g, 0.0)),
                       ("topk_gate", lambda: M.moe_unpermute_combine_dropout(cfg, x, d, None, 0.0))):
        with pytest.raises(TypeError, match=f"^{name}: "):
            call()


@pytest.mark.parametrize("case", [c for c in FORMS if c[0] != "wgrad"], ids=name_of)
def test_a_residual_in_place_in_every_form(case):
    """residual = y (dx), the same buffer: each element is read before it is written, whichever kernel runs."""
    product, dt, sizes, n, k, pad = case[:6]
    g, dense, ends, rows, E, o, x, dy = product_setup(case)
    w = integers((E, n, k), dt, g, pad)
    forward = product == "forward"
    res = integers((rows, n if forward else k), dt, g, pad)
    z = integers((rows, k), dt, g, pad, 1)
    inside = slice(ends[0], ends[-1])

    def call(residual, out):
        if forward:
            return M.moe_grouped_gemm(x, o, w, act="silu", residual=residual, y=out)[inside]
        return M.moe_grouped_gemm_dgrad(dy, o, w, z=z, act="silu", residual=residual, dx=out)[inside]

    apart = call(res, integers((rows, res.shape[1]), dt, g, pad)).clone()
    assert torch.equal(call(res, res), apart)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_experts_over_the_padded_layout(dt):
    """The fixed-capacity layout: its padding rows (zero in x_perm) belong to the groups. The experts' outputs there
    are those of zero rows and nothing reads them; gradients that are zero there add nothing to dw and dbias, exactly
    as without padding (whole numbers)."""
    g = torch.Generator(device=DEV).manual_seed(9)
    T, d, E, k, F, cap = 203, 128, 8, 2, 136, 40
    h, wr = integers((T, d), dt, g), torch.randn((E, d), generator=g, device=DEV).to(dt)
    w1, b1 = integers((E, F, d), dt, g), torch.randint(-9, 10, (E, F), generator=g, device=DEV).float()
    outs = []
    for layout in ("compact", "padded"):
        cfg = M.config(T, d, E, k, 128, dt, "identity", capacity=cap, layout=layout)
        idx, gate = M.moe_route(cfg, h, wr)
        pm = M.moe_permute(cfg, h, idx)
        y = M.moe_grouped_gemm(pm["x_perm"], pm["offsets"], w1, bias=b1, act="relu")
        dest = pm["dest_row"].reshape(-1).long()
        kept = dest >= 0
        dy = torch.zeros_like(y)
        dy[dest[kept]] = (torch.arange(T * k, device=DEV)[kept, None] % 5 - 2).to(dt).expand(-1, F)
        db = torch.empty((E, F), device=DEV)
        dw = M.moe_grouped_gemm_wgrad(dy, pm["offsets"], pm["x_perm"], dbias=db)
        dx = M.moe_grouped_gemm_dgrad(dy, pm["offsets"], w1)
        if layout == "padded":
            assert pm["offsets"].tolist() == [e * cap for e in range(E + 1)]
            used = torch.zeros(E * cap, dtype=torch.bool, device=DEV)
            used[dest[kept]] = True
            assert bool(kept.any()) and not bool(used.all())
            exactly(y[~used], b1.repeat_interleave(cap, 0)[~used].clamp(min=0), "padding rows")
            assert not dx[~used].any()
        outs.append((kept, y[dest[kept]], dw, db, dx[dest[kept]]))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("act", R.ACTS)
def test_activations_of_nan_and_infinity(act, dt):
    """NaN in a token's row makes all of its outputs NaN and no other token's; plus infinity stays what it is."""
    for rows in (3, 700):
        x = torch.ones((rows, 8), dtype=dt, device=DEV)
        x[0, 3], x[1] = math.nan, math.inf
        y = M.moe_linear(x, torch.ones((16, 8), dtype=dt, device=DEV), act=act)
        assert bool(y[0].isnan().all()) and bool((y[1] == math.inf).all())
        exactly(y[2:], torch.full((rows - 2, 16), 8.0, device=DEV).to(dt).float(), act) if act in ("none", "relu") else None
        assert bool(y[2:].isfinite().all())


def test_a_captured_fork_makes_its_outputs():
    """Calls on a second stream of a capture, with outputs made and dropped there, replayed twice beside other work."""
    calls = calls_on_a_stream()
    refs = {name: call(None).clone() for name, call in calls.items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    got = {}
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        for name, call in calls.items():
            call(side)  # its output is dropped at once
            got[name] = call(side)
        main.wait_stream(side)
        beside = calls["linear"](None)
    for _ in range(2):
        graph.replay()
        torch.full_like(beside, 3.0)
    torch.cuda.synchronize()
    for name, y in got.items():
        assert torch.equal(y, refs[name]), name
    assert torch.equal(beside, refs["linear"])
