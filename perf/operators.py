"""The operators that surround the expert layer, as they are measured.

    grouped           y = act(x W_e^T + b_e) + r over ragged expert groups (moe_grouped_gemm)
    grouped_backward  its input and weight gradients (moe_grouped_gemm_dgrad, moe_grouped_gemm_wgrad)
    linear            y = act(x W^T + b) + r (moe_linear)
    linear_backward   its input and weight gradients (moe_linear_dgrad, moe_linear_wgrad)
    dropout           y = r + dropout(x), the mask drawn from a counter and never stored (moe_dropout)
    combine_dropout   y = r + dropout(combine of the expert rows) (moe_unpermute_combine_dropout)

Each case is one pass through one of them. `run` computes it in plain torch
operations, or, where `own` is true, with this framework's entry points.
Layer shapes are those of the repository's workloads.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ROW_BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token of the 128-expert layer: eight experts' gate projections, one row each
        dict(name="grouped_decode", op="grouped", T=1, topk=8, E=128, route="none", cap=-1, K=2048, N=768,
             dtype="bf16", act="silu", bias=True, residual=False, preact=False, pad=False),
        # the smallest test layer, fp32
        dict(name="grouped_tiny_f32", op="grouped", T=64, topk=2, E=4, route="none", cap=-1, K=32, N=64,
             dtype="f32", act="relu", bias=True, residual=False, preact=False, pad=False),
        # prompt or training forward of the skewed 64-expert layer under its capacity, GELU experts with a
        # bias that keep their pre-activations; three experts stay empty and the rows past the kept ones
        # are left alone
        dict(name="grouped_skewed", op="grouped", T=16384, topk=6, E=64, route="zipf", cap=1920, K=2048, N=1408,
             dtype="bf16", act="gelu", bias=True, residual=False, preact=True, pad=False),
        # training backward of the scaled 8-expert layer's down projection, through the activation before it
        dict(name="grouped_backward_8", op="grouped_backward", T=4096, topk=2, E=8, route="none", cap=-1, K=3584,
             N=1024, dtype="bf16", act="gelu_tanh", dbias=True, pad=False),
        # training backward with many small experts, 16 of them hot and 8 empty, at an odd token count
        dict(name="grouped_backward_128", op="grouped_backward", T=2051, topk=8, E=128, route="hot", cap=-1,
             K=2048, N=768, dtype="bf16", act="silu", dbias=False, pad=False),
        # one decoded token through a wide dense projection
        dict(name="linear_decode", op="linear", M=1, K=4096, N=14336, dtype="bf16", act="silu", bias=True,
             residual=False, preact=False, pad=False),
        # a decode batch through a shared expert's down projection, added to the routed experts' output
        dict(name="linear_batch", op="linear", M=77, K=1408, N=2048, dtype="bf16", act="none", bias=True,
             residual=True, preact=False, pad=False),
        # a long prompt through a dense layer's down projection with the residual stream added
        dict(name="linear_prefill", op="linear", M=8192, K=14336, N=4096, dtype="bf16", act="none", bias=True,
             residual=True, preact=False, pad=False),
        # training backward of a shared expert's up projection at an odd token count
        dict(name="linear_backward", op="linear_backward", M=4099, K=2048, N=1408, dtype="bf16", act="none",
             dbias=True, pad=False),
        # fp32 at sizes that are no multiple of a tile
        dict(name="linear_f32", op="linear", M=333, K=768, N=1000, dtype="f32", act="gelu", bias=True,
             residual=True, preact=True, pad=False),
        # the skewed layer's combine with residual dropout, assignments over the capacity dropped
        dict(name="combine_dropout_skewed", op="combine_dropout", T=16384, topk=6, E=64, route="zipf", cap=1920,
             d=2048, dtype="bf16", p=0.1, residual=True),
        # residual dropout over the hidden states of the largest layer
        dict(name="dropout_residual", op="dropout", rows=32768, cols=4096, dtype="bf16", p=0.1, residual=True,
             pad=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "grouped_backward", "linear", "linear", "linear_backward", "dropout",
                     "combine_dropout"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
    if op == "dropout":
        cols = _log(rng, 64, 8192)
        rows = _log(rng, 1, max(2, min(40000, (1 << 26) // cols)))
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, p=rng.choice([0.0, 0.05, 0.1, 0.5, 0.9]),
                    residual=rng.random() < 0.6, pad=rng.random() < 0.3)
    E = rng.choice([1, 4, 8, 13, 40, 64, 128, 256])
    topk = rng.randint(1, min(8, E))
    route = rng.choice(["none", "zipf", "hot"]) if E >= 64 else "none"
    if op == "combine_dropout":
        T = _log(rng, 1, 16384)
        cap = rng.choice([-1, -1, max(1, T * topk * 5 // (4 * E))])
        d = 128 * rng.randint(1, 16) if dtype == "bf16" else 4 * rng.randint(1, 512)
        return dict(op=op, T=T, topk=topk, E=E, route=route, cap=cap, d=d, dtype=dtype,
                    p=rng.choice([0.0, 0.1, 0.5]), residual=rng.random() < 0.7)
    # a quarter has odd widths in rows that are padded to a multiple of eight elements
    pad = rng.random() < 0.25
    K, N = _log(rng, 8, 6000), _log(rng, 8, 6000)
    if not pad:
        K, N = (K + 7) // 8 * 8, (N + 7) // 8 * 8
    most = 2 * 10 ** 11 if dtype == "bf16" else 2 * 10 ** 10  # products
    if op in ("linear", "linear_backward"):
        M = _log(rng, 1, max(2, min(16384, most // (K * N))))
        c = dict(op=op, M=M, K=K, N=N, dtype=dtype, act=act, pad=pad)
    else:
        while E * K * N > 3 * 10 ** 8:
            K, N = max(8, K // 16 * 8), max(8, N // 16 * 8)
        T = _log(rng, 1, max(2, min(16384, most // (K * N * topk))))
        cap = rng.choice([-1, -1, max(1, T * topk * 5 // (4 * E))])
        c = dict(op=op, T=T, topk=topk, E=E, route=route, cap=cap, K=K, N=N, dtype=dtype, act=act, pad=pad)
    if op in ("linear", "grouped"):
        c.update(bias=rng.random() < 0.7, residual=rng.random() < 0.4, preact=rng.random() < 0.4)
    else:
        c.update(dbias=rng.random() < 0.6)
    return c


# ------------------------------------------------------------------ inputs

def _router_bias(route, E):
    """Added to the router scores: "zipf" -2 ln(e + 1) with experts 1, 31 and 63 shut, "hot" lifts the first 16 and shuts the last 8."""
    b = torch.zeros(E)
    if route == "zipf":
        b = -2.0 * torch.log(torch.arange(1, E + 1, dtype=torch.float32))
        b[torch.tensor([1, 31, 63])] = -math.inf
    elif route == "hot":
        b[:16] = 1.1
        b[E - 8:] = -math.inf
    return b


def _routing(case, g, device):
    """Routes of T tokens, and the rows that each kept assignment takes: experts in order, tokens in order within each."""
    T, E, topk = case["T"], case["E"], case["topk"]
    scores = torch.randn(T, E, generator=g, device=device) + _router_bias(case["route"], E).to(device)
    top = torch.topk(scores, topk, dim=1)
    idx = top.indices.reshape(-1)
    routed = torch.bincount(idx, minlength=E)
    kept = routed if case["cap"] < 0 else routed.clamp(max=case["cap"])
    zero = torch.zeros(1, dtype=torch.int64, device=device)
    offsets, first = torch.cat([zero, kept.cumsum(0)]), torch.cat([zero, routed.cumsum(0)])
    order = torch.argsort(idx, stable=True)
    rank = torch.empty_like(order)
    rank[order] = torch.arange(T * topk, device=device) - first[idx[order]]
    dest = torch.where(rank < kept[idx], offsets[idx] + rank, -1)
    gate = torch.softmax(top.values, dim=1)
    return offsets.to(torch.int32), dest.reshape(T, topk).to(torch.int32).contiguous(), gate.contiguous()


def _rows(shape, dtype, pad, g, scale=1.0):
    """Normal values; with `pad` in rows of a wider buffer (a multiple of eight elements, so that rows start on 16 bytes)."""
    width = shape[-1]
    if pad:
        shape = (*shape[:-1], (width + 7) // 8 * 8 + 8)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)[..., :width]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    op = case["op"]
    s = {"case": case}
    if op in ("dropout", "combine_dropout"):
        # the seed and the step count of the random numbers, in device memory
        s["rng"] = torch.randint(0, 1 << 62, (2,), generator=g, device="cuda", dtype=torch.int64)
        s["offset"] = 7
    if op == "dropout":
        shape = (case["rows"], case["cols"])
        s["x"] = _rows(shape, dt, case["pad"], g)
        s["residual"] = _rows(shape, dt, case["pad"], g) if case["residual"] else None
        s["y"] = torch.zeros(shape, dtype=dt, device="cuda")
        return s
    if op == "combine_dropout":
        T, d = case["T"], case["d"]
        _, s["dest_row"], s["gate"] = _routing(case, g, "cuda")
        s["y_perm"] = _rows((T * case["topk"], d), dt, False, g)
        s["residual"] = _rows((T, d), dt, False, g) if case["residual"] else None
        s["y"] = torch.zeros((T, d), dtype=dt, device="cuda")
        return s
    K, N, pad = case["K"], case["N"], case["pad"]
    if op in ("grouped", "grouped_backward"):
        E, P = case["E"], case["T"] * case["topk"]
        s["offsets"], _, _ = _routing(case, g, "cuda")
        wshape, bshape = (E, N, K), (E, N)
    else:
        P, wshape, bshape = case["M"], (N, K), (N,)
    s["w"] = _rows(wshape, dt, pad, g, 1.0 / math.sqrt(K))
    if op in ("grouped", "linear"):
        s["x"] = _rows((P, K), dt, pad, g)
        s["bias"] = torch.randn(bshape, generator=g, device="cuda") * 0.5 if case["bias"] else None
        s["residual"] = _rows((P, N), dt, pad, g) if case["residual"] else None
        s["y"] = _rows((P, N), dt, pad, g, 0.0)
        s["preact"] = _rows((P, N), dt, pad, g, 0.0) if case["preact"] else None
    else:
        s["dy"] = _rows((P, N), dt, pad, g)
        s["x"] = _rows((P, K), dt, pad, g)
        # the pre-activations that the layer's input x came from
        s["z"] = _rows((P, K), dt, pad, g) if case["act"] != "none" else None
        s["dx"] = _rows((P, K), dt, pad, g, 0.0)
        s["dw"] = torch.zeros(wshape, device="cuda")
        s["dbias"] = torch.zeros(bshape, device="cuda") if case["dbias"] else None
    return s


# ------------------------------------------------------------------ plain form

def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _dact(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def _product(x, w, bias, residual, act, y, preact):
    z = x.float() @ w.float().T
    if bias is not None:
        z = z + bias
    if preact is not None:
        preact.copy_(z)
    out = _act(z, act)
    if residual is not None:
        out = out + residual.float()
    y.copy_(out)


def _product_backward(dy, x, w, z, act, dx, dw, dbias):
    dyf = dy.float()
    out = dyf @ w.float()
    if z is not None:
        out = out * _dact(z.float(), act)
    dx.copy_(out)
    torch.mm(dyf.T, x.float(), out=dw)
    if dbias is not None:
        dbias.copy_(dyf.sum(0))


def _part(t, a, b):
    return None if t is None else t[a:b]


def _nth(t, e):
    return None if t is None else t[e]


def _keep(rng, offset, rows, cols, p, device):
    """Philox4x32 with ten rounds (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", 2011): the element (r, c) takes
    word c % 4 of the block with counter (c // 4, r, offset) under the seed as the key; it is kept where the word is at least p 2^32."""
    m32 = 0xFFFFFFFF
    at = rng[1] + offset
    quads = (cols + 3) // 4
    c0 = torch.arange(quads, device=device).expand(rows, quads)
    c1 = torch.arange(rows, device=device)[:, None].expand(rows, quads)
    c2, c3 = (at & m32).expand(rows, quads), ((at >> 32) & m32).expand(rows, quads)
    k0, k1 = rng[0] & m32, (rng[0] >> 32) & m32

    def mul(a, m):  # high and low words of the 64-bit product
        high = ((a >> 16) * m + (((a & 0xFFFF) * m) >> 16)) >> 16
        return high, (a * m) & m32

    for _ in range(10):
        h0, l0 = mul(c0, 0xD2511F53)
        h1, l1 = mul(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & m32, (k1 + 0xBB67AE85) & m32
    words = torch.stack([c0, c1, c2, c3], dim=2).reshape(rows, quads * 4)[:, :cols]
    return words >= int(math.floor(p * 4294967296.0))


def _dropped(x, rng, offset, p):
    """dropout(x) in 32 bits: kept elements over 1 - p, the others zero whatever they hold."""
    if p == 0.0:
        return x
    keep = _keep(rng, offset, x.shape[0], x.shape[1], p, x.device)
    return torch.where(keep, x * (1.0 / (1.0 - p)), torch.zeros_like(x))


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    op = case["op"]
    if op == "dropout":
        y = _dropped(s["x"].float(), s["rng"], s["offset"], case["p"])
        return s["y"].copy_(y if s["residual"] is None else y + s["residual"].float())
    if op == "combine_dropout":
        dest, T = s["dest_row"].long(), case["T"]
        y = torch.zeros((T, case["d"]), device="cuda")
        for j in range(case["topk"]):  # slot by slot: all slots' rows at once would be k times the output
            row = s["y_perm"][dest[:, j].clamp(min=0)].float()
            y = y + torch.where((dest[:, j] >= 0)[:, None], s["gate"][:, j:j + 1] * row, torch.zeros_like(row))
        y = _dropped(y, s["rng"], s["offset"], case["p"])
        return s["y"].copy_(y if s["residual"] is None else y + s["residual"].float())
    if op == "linear":
        _product(s["x"], s["w"], s["bias"], s["residual"], case["act"], s["y"], s["preact"])
        return {"y": s["y"], "preact": s["preact"]}
    if op == "linear_backward":
        _product_backward(s["dy"], s["x"], s["w"], s["z"], case["act"], s["dx"], s["dw"], s["dbias"])
        return {"dx": s["dx"], "dw": s["dw"], "dbias": s["dbias"]}
    off = s["offsets"].tolist()
    for e, (a, b) in enumerate(zip(off, off[1:])):  # ragged groups: one product for each expert that has rows
        if op == "grouped" and b > a:
            _product(s["x"][a:b], s["w"][e], _nth(s["bias"], e), _part(s["residual"], a, b), case["act"], s["y"][a:b],
                     _part(s["preact"], a, b))
        elif op == "grouped_backward":
            if b > a:
                _product_backward(s["dy"][a:b], s["x"][a:b], s["w"][e], _part(s["z"], a, b), case["act"], s["dx"][a:b],
                                  s["dw"][e], _nth(s["dbias"], e))
            else:
                s["dw"][e].zero_()
                if s["dbias"] is not None:
                    s["dbias"][e].zero_()
    if op == "grouped":
        return {"y": s["y"], "preact": s["preact"]}
    return {"dx": s["dx"], "dw": s["dw"], "dbias": s["dbias"]}


def _run_own(s):
    import combine_router_gemm_softmax_b200 as M
    case = s["case"]
    op = case["op"]
    if op == "dropout":
        return M.moe_dropout(s["x"], case["p"], s["rng"], s["offset"], residual=s["residual"], y=s["y"])
    if op == "combine_dropout":
        cfg = M.config(case["T"], case["d"], case["E"], case["topk"], 128, case["dtype"], "identity", case["cap"])
        return M.moe_unpermute_combine_dropout(cfg, s["y_perm"], s["dest_row"], s["gate"], case["p"], s["rng"],
                                               s["offset"], residual=s["residual"], y=s["y"])
    if op == "linear":
        M.moe_linear(s["x"], s["w"], bias=s["bias"], act=case["act"], residual=s["residual"], preact=s["preact"],
                     y=s["y"])
        return {"y": s["y"], "preact": s["preact"]}
    if op == "grouped":
        M.moe_grouped_gemm(s["x"], s["offsets"], s["w"], bias=s["bias"], act=case["act"], residual=s["residual"],
                           preact=s["preact"], y=s["y"])
        return {"y": s["y"], "preact": s["preact"]}
    if op == "linear_backward":
        M.moe_linear_dgrad(s["dy"], s["w"], z=s["z"], act=case["act"], dx=s["dx"])
        M.moe_linear_wgrad(s["dy"], s["x"], dw=s["dw"], dbias=s["dbias"])
    else:
        M.moe_grouped_gemm_dgrad(s["dy"], s["offsets"], s["w"], z=s["z"], act=case["act"], dx=s["dx"])
        M.moe_grouped_gemm_wgrad(s["dy"], s["offsets"], s["x"], dw=s["dw"], dbias=s["dbias"])
    return {"dx": s["dx"], "dw": s["dw"], "dbias": s["dbias"]}


# ------------------------------------------------------------------ what a pass cannot do without

def _expected(case):
    """Kept rows and experts that have any, for one drawing of the routes."""
    g = torch.Generator()
    g.manual_seed(1)
    offsets, dest, _ = _routing(case, g, "cpu")
    return int(offsets[-1]), int((offsets[1:] > offsets[:-1]).sum())


def work(case):
    op, size = case["op"], ROW_BYTES[case["dtype"]]
    if op == "dropout":
        n = case["rows"] * case["cols"]
        return {"bytes": n * size * (3 if case["residual"] else 2), "flops": 2 * n}
    if op == "combine_dropout":
        kept, _ = _expected(case)
        n = case["T"] * case["d"]
        return {"bytes": kept * case["d"] * size + n * size * (2 if case["residual"] else 1) + 8 * case["T"] * case["topk"],
                "flops": 2 * kept * case["d"] + 2 * n}
    K, N = case["K"], case["N"]
    rows, groups, of = (case["M"], 1, 1) if "M" in case else (*_expected(case), case["E"])
    if op in ("linear", "grouped"):
        moved = rows * K + groups * N * K + rows * N * (1 + case["residual"] + case["preact"])
        return {"bytes": moved * size + (groups * N * 4 if case["bias"] else 0), "flops": 2 * rows * N * K}
    moved = rows * N + groups * N * K + rows * K * (3 if case["act"] != "none" else 2)
    return {"bytes": moved * size + of * N * K * 4 + (of * N * 4 if case["dbias"] else 0), "flops": 4 * rows * N * K}


# ------------------------------------------------------------------ the same in 64 bits

def _gate64(z, act):
    """The activation by torch's own functions in 64 bits (nothing here is shared with the plain form)."""
    f = torch.nn.functional
    return {"none": lambda t: t * 1.0, "relu": f.relu, "gelu": f.gelu, "silu": f.silu,
            "gelu_tanh": lambda t: f.gelu(t, approximate="tanh")}[act](z)


def _mask64(rng, offset, rows, cols, p):
    """The kept elements, from the block function on 64-bit unsigned integers on the host."""
    u = np.uint64
    seed, at = (int(v) for v in rng.tolist())
    at = (at + offset) % (1 << 64)
    low, cut = u(0xFFFFFFFF), math.floor(p * 2 ** 32)
    quads = -(-cols // 4)
    keep = np.empty((rows, quads, 4), dtype=bool)
    for lo in range(0, rows, 2048):
        n = min(2048, rows - lo)
        x = [np.broadcast_to(np.arange(quads, dtype=u), (n, quads)), np.broadcast_to(np.arange(lo, lo + n, dtype=u)[:, None], (n, quads)),
             np.full((n, quads), at & 0xFFFFFFFF, dtype=u), np.full((n, quads), at >> 32, dtype=u)]
        key = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
        for r in range(10):
            a, b = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
            ka, kb = ((key[0] + r * 0x9E3779B9) & 0xFFFFFFFF), ((key[1] + r * 0xBB67AE85) & 0xFFFFFFFF)
            x = [(b >> u(32)) ^ x[1] ^ u(ka), b & low, (a >> u(32)) ^ x[3] ^ u(kb), a & low]
        for w in range(4):
            keep[lo:lo + n, :, w] = x[w] >= u(cut)
    return torch.from_numpy(keep.reshape(rows, quads * 4)[:, :cols].copy())


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("dropout", "combine_dropout"):
        if op == "dropout":
            y = s["x"].double()
        else:
            padded = torch.cat([s["y_perm"].double(), s["y_perm"].new_zeros((1, case["d"])).double()])
            y = torch.zeros((case["T"], case["d"]), dtype=torch.float64, device="cuda")
            for j in range(case["topk"]):
                y.addcmul_(padded[s["dest_row"][:, j].long()], s["gate"][:, j, None].double())
        if case["p"] > 0:
            y = y.masked_fill(~_mask64(s["rng"], s["offset"], y.shape[0], y.shape[1], case["p"]).to("cuda"), 0.0) / (1.0 - case["p"])
        return y if s["residual"] is None else y + s["residual"].double()
    grouped = op.startswith("grouped")
    ends = s["offsets"].tolist() if grouped else [0, case["M"]]
    w = s["w"] if grouped else s["w"][None]
    if op in ("linear", "grouped"):
        y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
        z = torch.zeros_like(y)
        for e in range(len(ends) - 1):
            a, b = ends[e], ends[e + 1]
            t = torch.einsum("rk,nk->rn", s["x"][a:b].double(), w[e].double())
            if case["bias"]:
                t += (s["bias"][e] if grouped else s["bias"]).double()
            z[a:b] = t
            y[a:b] = _gate64(t, case["act"])
            if case["residual"]:
                y[a:b] += s["residual"][a:b].double()
        return {"y": y, "preact": z if case["preact"] else None}
    dx = torch.zeros(s["dx"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros(w.shape, dtype=torch.float64, device="cuda")
    db = torch.zeros(w.shape[:2], dtype=torch.float64, device="cuda")
    for e in range(len(ends) - 1):
        a, b = ends[e], ends[e + 1]
        dy = s["dy"][a:b].double()
        t = torch.einsum("rn,nk->rk", dy, w[e].double())
        if s["z"] is not None:
            z = s["z"][a:b].double().requires_grad_()
            t = torch.autograd.grad(_gate64(z, case["act"]), z, t)[0]
        dx[a:b] = t
        dw[e] = torch.einsum("rn,rk->nk", dy, s["x"][a:b].double())
        db[e] = dy.sum(0)
    return {"dx": dx, "dw": dw if grouped else dw[0], "dbias": (db if grouped else db[0]) if case["dbias"] else None}
