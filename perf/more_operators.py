"""The row operators around the experts' products at the sizes that a user meets them.

Each case names one operator:

  norm      the residual's addition and the root-mean-square norm that follows
            it, with a copy in 8 bits (E4M3, one scale a row) or in MXFP4 if
            wanted; in training the gradient of all that too;
  dispatch  tokens' rows copied into expert order;
  collect   rows in expert order summed back per token, with routing weights;
            in training the gradient by the rows and by the weights too;
  swiglu    silu(gate) * up over rows [gate | up] in expert order, in 8 bits if
            wanted; in training the gradient too.

Sizes are those of the GLM-5.2-shaped layer (hidden 6144, inter 2048, 256
experts, 8 per token), of the tiny layer of the tests, and generic odd ones.
"""
import math

import torch

own = False

_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
_SIZE = {"f32": 4, "bf16": 2, "e4m3": 1, "mxfp4": 0.53125, "none": 0}
_EPS = 1e-6


def listed():
    return [
        # one token on its way into the layer: latency
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 6144, "x": "bf16", "residual": "bf16", "y": "bf16",
         "q": "none", "train": False},
        # 64 draft tokens: the float32 sum of a layer onto a bf16 stream, a copy in MXFP4 for products in 4 bits
        {"name": "norm_verify", "op": "norm", "rows": 64, "cols": 6144, "x": "f32", "residual": "bf16", "y": "bf16",
         "q": "mxfp4", "train": False},
        # 16384 tokens of prompts, rows in 8 bits beside the router's bf16 ones
        {"name": "norm_prefill", "op": "norm", "rows": 16384, "cols": 6144, "x": "bf16", "residual": "bf16", "y": "bf16",
         "q": "e4m3", "train": False},
        # an odd matrix in float32, no residual, forward and backward
        {"name": "norm_train_odd", "op": "norm", "rows": 1027, "cols": 2057, "x": "f32", "residual": "none", "y": "f32",
         "q": "none", "train": True},
        # a training batch, forward and backward
        {"name": "norm_train", "op": "norm", "rows": 16384, "cols": 6144, "x": "bf16", "residual": "bf16", "y": "bf16",
         "q": "none", "train": True},
        # 64 draft tokens in 8 bits to their 8 experts' rows
        {"name": "dispatch_verify", "op": "dispatch", "tokens": 64, "top_k": 8, "experts": 256, "cols": 6144,
         "x": "e4m3", "rows": "e4m3", "drop": 0.0},
        # 16384 tokens of prompts
        {"name": "dispatch_prefill", "op": "dispatch", "tokens": 16384, "top_k": 8, "experts": 256, "cols": 6144,
         "x": "bf16", "rows": "bf16", "drop": 0.0},
        # one token's 8 rows in float32 and the shared expert's
        {"name": "collect_token", "op": "collect", "tokens": 1, "top_k": 8, "experts": 256, "cols": 6144,
         "rows": "f32", "y": "bf16", "addend": "f32", "drop": 0.0, "train": False},
        # a training batch, forward and backward
        {"name": "collect_train", "op": "collect", "tokens": 4096, "top_k": 8, "experts": 256, "cols": 6144,
         "rows": "bf16", "y": "bf16", "addend": "bf16", "drop": 0.0, "train": True},
        # one token's gate and up of 8 experts, 8-bit rows for the down product
        {"name": "swiglu_token", "op": "swiglu", "rows": 8, "cols": 2048, "x": "bf16", "y": "e4m3", "drop": 0.0,
         "train": False},
        # ragged: an odd width, the last rows of no expert
        {"name": "swiglu_train_odd", "op": "swiglu", "rows": 777, "cols": 1001, "x": "f32", "y": "f32", "drop": 0.1,
         "train": True},
        # gate and up of a training batch of 4096 tokens, forward and backward
        {"name": "swiglu_train", "op": "swiglu", "rows": 32768, "cols": 2048, "x": "bf16", "y": "bf16", "drop": 0.0,
         "train": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "dispatch", "collect", "swiglu"])
    while True:
        if op == "norm":
            c = {"op": op, "rows": _log(rng, 1, 32768), "cols": _log(rng, 16, 12288), "x": rng.choice(["f32", "bf16"]),
                 "residual": rng.choice(["none", "f32", "bf16"]), "y": rng.choice(["f32", "bf16"]),
                 "q": rng.choice(["none", "e4m3", "mxfp4"]), "train": rng.random() < 0.5}
            most, n = 16384 * 6144, c["rows"] * c["cols"]
            if c["train"]:
                c["q"] = "none"
            size = 4 if "f32" in (c["x"], c["residual"], c["y"]) else 2
        elif op == "swiglu":
            c = {"op": op, "rows": _log(rng, 1, 65536), "cols": _log(rng, 16, 8192), "x": rng.choice(["f32", "bf16"]),
                 "y": rng.choice(["f32", "bf16", "e4m3"]), "drop": rng.choice([0.0, 0.2]), "train": rng.random() < 0.5}
            if c["train"] and c["y"] == "e4m3":
                c["y"] = "bf16"
            most, n, size = 32768 * 2048, c["rows"] * c["cols"], 4 if "f32" in (c["x"], c["y"]) else 2
        else:
            e = _log(rng, 1, 256)
            c = {"op": op, "tokens": _log(rng, 1, 16384), "top_k": rng.randint(1, min(e, 12)), "experts": e,
                 "cols": _log(rng, 16, 8192), "drop": rng.choice([0.0, 0.0, 0.2])}
            n = c["tokens"] * c["top_k"] * c["cols"]
            if op == "dispatch":
                c["x"], c["rows"] = rng.choice([("f32", "f32"), ("bf16", "bf16"), ("e4m3", "e4m3"), ("f32", "bf16")])
                most, size = 16384 * 8 * 6144, 2 if c["rows"] == "e4m3" else _SIZE[c["rows"]]
            else:
                c["rows"], c["y"] = rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"])
                c["addend"] = rng.choice(["none", "f32", "bf16"])
                c["train"] = rng.random() < 0.5
                most, size = 4096 * 8 * 6144, 4 if "f32" in (c["rows"], c["y"], c["addend"]) else 2
        if n * size <= most * 2:
            return c


# ---- inputs ----------------------------------------------------------------
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _activations(gen, rows, cols):
    """Normal activations, a few columns larger than the rest."""
    hot = torch.rand(cols, generator=gen, device="cuda") < 0.004
    return _normal(gen, rows, cols) * torch.where(hot, 4.0, 1.0)


def _route(gen, c):
    """Slot of each pick (top_k distinct experts a token) in expert order, -1
    for a dropped one, and the routing weights."""
    t, e, k = c["tokens"], c["experts"], c["top_k"]
    pull = 0.3 * _normal(gen, e)
    ids = (pull + torch.rand(t, e, generator=gen, device="cuda") * 2 - 1).topk(k, dim=1).indices
    gone = torch.rand(t, k, generator=gen, device="cuda") < c["drop"]
    ids[gone] = e                                             # sorts behind every expert
    order = torch.argsort(ids.reshape(-1), stable=True)
    inv = torch.empty(t * k, dtype=torch.int32, device="cuda")
    inv[order] = torch.arange(t * k, dtype=torch.int32, device="cuda")
    share = torch.rand(t, k, generator=gen, device="cuda") + 0.1
    share = torch.where(gone, 0.0, share)
    return torch.where(gone, -1, inv.view(t, k)), 2.5 * share / share.sum(1, keepdim=True).clamp(min=0.1)


def _eight_bits(x):
    """float32 rows to E4M3 and one scale a row."""
    scale = (x.abs().amax(1) / 448).clamp(min=2.0 ** -126)
    return (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"case": case}
    if own:
        import quantized_moe_02_amd
        st["lib"] = quantized_moe_02_amd
    empty = lambda *shape, type: torch.empty(*shape, dtype=_DTYPE[type], device="cuda")
    cols = case["cols"]
    if case["op"] == "norm":
        rows = case["rows"]
        st["x"] = _activations(gen, rows, cols).to(_DTYPE[case["x"]])
        st["w"] = (1 + 0.2 * _normal(gen, cols)).to(torch.bfloat16)
        stream = case["x"]
        st["residual"] = st["h"] = st["dh"] = st["q"] = st["scale"] = st["values"] = None
        if case["residual"] != "none":
            stream = case["residual"]
            st["residual"] = (2 * _activations(gen, rows, cols)).to(_DTYPE[stream])
            st["h"] = empty(rows, cols, type=stream)
        st["y"] = empty(rows, cols, type=case["y"])
        if case["q"] == "e4m3":
            st["q"], st["scale"] = empty(rows, cols, type="e4m3"), empty(rows, type="f32")
        elif case["q"] == "mxfp4":
            nb = (cols + 31) // 32
            st["q"] = torch.empty(rows, 16 * nb, dtype=torch.uint8, device="cuda")
            st["scale"] = torch.empty(rows, nb, dtype=torch.uint8, device="cuda")
            st["values"] = empty(rows, cols, type="bf16")
        if case["train"]:
            st["dy"] = (1e-3 * _normal(gen, rows, cols)).to(_DTYPE[case["y"]])
            if case["residual"] != "none":
                st["dh"] = (1e-3 * _normal(gen, rows, cols)).to(_DTYPE[stream])
            st["dx"] = empty(rows, cols, type=stream)
            st["dw"] = empty(cols, type="f32")
            if own:
                st["ws"] = st["lib"].rmsnorm_workspace(rows, cols)
        return st
    if case["op"] == "swiglu":
        rows = case["rows"]
        kept = int(round(rows * (1 - case["drop"])))
        st["offsets"] = torch.tensor([0, kept // 2, kept], dtype=torch.int32, device="cuda") if case["drop"] else None
        st["gu"] = (1.5 * _normal(gen, rows, 2 * cols)).to(_DTYPE[case["x"]])
        st["out"] = torch.zeros(rows, cols, dtype=torch.float32, device="cuda").to(_DTYPE[case["y"]])
        st["scale"] = torch.zeros(rows, device="cuda") if case["y"] == "e4m3" else None
        st["kept"] = kept
        if case["train"]:
            st["dh"] = (1e-3 * _normal(gen, rows, cols)).to(_DTYPE[case["y"]])
            st["dgu"] = torch.zeros_like(st["gu"])
        return st
    t, k = case["tokens"], case["top_k"]
    st["inv"], st["weights"] = _route(gen, case)
    if case["op"] == "dispatch":
        x = _activations(gen, t, cols)
        st["scale"] = st["row_scale"] = None
        if case["x"] == "e4m3":
            st["x"], st["scale"] = _eight_bits(x)
            st["row_scale"] = torch.zeros(t * k, device="cuda")
        else:
            st["x"] = x.to(_DTYPE[case["x"]])
        st["rows"] = torch.zeros(t * k, cols, dtype=torch.uint8 if case["rows"] == "e4m3" else _DTYPE[case["rows"]],
                                 device="cuda")
        if case["rows"] == "e4m3":
            st["rows"] = st["rows"].view(torch.float8_e4m3fn)
        return st
    st["rows"] = _normal(gen, t * k, cols).to(_DTYPE[case["rows"]])
    st["addend"] = None if case["addend"] == "none" else _normal(gen, t, cols).to(_DTYPE[case["addend"]])
    st["y"] = empty(t, cols, type=case["y"])
    if case["train"]:
        st["dy"] = (1e-3 * _normal(gen, t, cols)).to(_DTYPE[case["y"]])
        st["drows"] = torch.zeros_like(st["rows"])
        st["dweights"] = empty(t, k, type="f32")
    return st


# ---- plain forms -------------------------------------------------------------
def _mxfp4_values(x):
    """float32 rows as MXFP4 holds them: one power-of-two scale per 32, E2M1 codes."""
    rows, cols = x.shape
    v = torch.nn.functional.pad(x, (0, -cols % 32)).view(rows, -1, 32)
    top = v.abs().amax(2)
    _, e = torch.frexp(top)
    s = torch.where(top == 0, torch.full_like(e, -127), (e - 3).clamp(-127, 127))
    a = v.abs() * torch.exp2(-s.float())[:, :, None]
    code = ((a > 0.25).to(torch.int64) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=x.device)[code]
    return (torch.where(v < 0, -grid, grid) * torch.exp2(s.float())[:, :, None]).view(rows, -1)[:, :cols]


def _plain_norm(st):
    c = st["case"]
    out = {}
    h = st["x"]
    if c["residual"] != "none":
        h = out["h"] = (st["x"].float() + st["residual"].float()).to(st["residual"].dtype)
    h, w = h.float(), st["w"].float()
    rstd = torch.rsqrt(h.double().square().mean(1, keepdim=True) + _EPS).float()
    y = h * rstd * w
    out["y"] = y.to(st["y"].dtype)
    if c["q"] == "e4m3":
        out["q"], out["scale"] = _eight_bits(y)
    elif c["q"] == "mxfp4":
        out["q"] = _mxfp4_values(y).to(torch.bfloat16)
    if c["train"]:
        dy = st["dy"].float()
        g, n = dy * w, h * rstd
        dx = rstd * (g - n * (g * n).double().mean(1, keepdim=True).float())
        if st["dh"] is not None:
            dx = dx + st["dh"].float()
        out["dx"] = dx.to(st["dx"].dtype)
        out["dw"] = (dy * n).sum(0, dtype=torch.float64).float()
    return out


def _plain_swiglu(st):
    c, n, cols = st["case"], st["kept"], st["case"]["cols"]
    gate, up = st["gu"][:n, :cols].float(), st["gu"][:n, cols:].float()
    sig = torch.sigmoid(gate)
    y = gate * sig * up
    out = {}
    if c["y"] == "e4m3":
        q, scale = _eight_bits(y)
        st["out"].view(torch.uint8)[:n] = q.view(torch.uint8)
        st["scale"][:n] = scale
        out["scale"] = st["scale"]
    else:
        st["out"][:n] = y.to(st["out"].dtype)
    out["out"] = st["out"]
    if c["train"]:
        dh = st["dh"][:n].float()
        st["dgu"][:n, :cols] = (dh * up * sig * (1 + gate * (1 - sig))).to(st["dgu"].dtype)
        st["dgu"][:n, cols:] = (dh * gate * sig).to(st["dgu"].dtype)
        out["dgu"] = st["dgu"]
    return out


def _plain_dispatch(st):
    t, k = st["inv"].shape
    pick = (st["inv"].reshape(-1) >= 0).nonzero()[:, 0]
    slot, token = st["inv"].reshape(-1)[pick].long(), pick // k
    if st["case"]["rows"] == "e4m3":
        st["rows"].view(torch.uint8)[slot] = st["x"].view(torch.uint8)[token]
        st["row_scale"][slot] = st["scale"][token]
        return {"rows": st["rows"], "scale": st["row_scale"]}
    st["rows"][slot] = st["x"][token].to(st["rows"].dtype)
    return {"rows": st["rows"]}


def _plain_collect(st):
    kept = st["inv"] >= 0
    picked = st["rows"][st["inv"].clamp(min=0).long()].float()            # [T][k][cols]
    picked = torch.where(kept[:, :, None], picked, 0.0)
    w = torch.where(kept, st["weights"], 0.0)
    y = (w[:, :, None] * picked).sum(1)
    if st["addend"] is not None:
        y = y + st["addend"].float()
    out = {"y": y.to(st["y"].dtype)}
    if st["case"]["train"]:
        dy = st["dy"].float()
        out["dweights"] = (picked * dy[:, None, :]).sum(2)
        pick = kept.reshape(-1).nonzero()[:, 0]
        slot, token = st["inv"].reshape(-1)[pick].long(), pick // kept.shape[1]
        st["drows"][slot] = (w.reshape(-1)[pick][:, None] * dy[token]).to(st["drows"].dtype)
        out["drows"] = st["drows"]
    return out


# ---- the operators -----------------------------------------------------------
def run(st):
    c = st["case"]
    if not own:
        return {"norm": _plain_norm, "swiglu": _plain_swiglu, "dispatch": _plain_dispatch, "collect": _plain_collect}[c["op"]](st)
    lib = st["lib"]
    if c["op"] == "norm":
        lib.moe_rmsnorm(st["x"], st["w"], _EPS, y=st["y"], residual=st["residual"], h=st["h"], q=st["q"], q_scale=st["scale"])
        out = {"y": st["y"]}
        if st["h"] is not None:
            out["h"] = st["h"]
        if c["q"] == "e4m3":
            out["q"], out["scale"] = st["q"], st["scale"]
        elif c["q"] == "mxfp4":
            lib.moe_mxfp4_dequantize(st["q"], st["scale"], st["values"])
            out["q"] = st["values"]
        if c["train"]:
            h = st["x"] if st["h"] is None else st["h"]
            lib.moe_rmsnorm_grad(st["dy"], h, st["w"], _EPS, st["dx"], dh=st["dh"], dweight=st["dw"], ws=st["ws"])
            out["dx"], out["dw"] = st["dx"], st["dw"]
        return out
    if c["op"] == "swiglu":
        lib.moe_swiglu(st["gu"], st["out"], out_scale=st["scale"], expert_offsets=st["offsets"])
        out = {"out": st["out"]}
        if st["scale"] is not None:
            out["scale"] = st["scale"]
        if c["train"]:
            lib.moe_swiglu_grad(st["gu"], st["dh"], st["dgu"], expert_offsets=st["offsets"])
            out["dgu"] = st["dgu"]
        return out
    if c["op"] == "dispatch":
        lib.moe_dispatch(st["x"], st["inv"], st["rows"], x_scale=st["scale"], row_scale=st["row_scale"])
        return {"rows": st["rows"]} if st["scale"] is None else {"rows": st["rows"], "scale": st["row_scale"]}
    lib.moe_collect(st["rows"], st["inv"], st["y"], weights=st["weights"], addend=st["addend"])
    if not c["train"]:
        return {"y": st["y"]}
    lib.moe_collect_grad(st["dy"], st["inv"], drows=st["drows"], weights=st["weights"], rows=st["rows"],
                         dweights=st["dweights"])
    return {"y": st["y"], "drows": st["drows"], "dweights": st["dweights"]}


def work(case):
    cols = case["cols"]
    if case["op"] == "norm":
        n = case["rows"] * cols
        stream = case["x"] if case["residual"] == "none" else case["residual"]
        per = _SIZE[case["x"]] + 2 * _SIZE[case["residual"]] + _SIZE[case["y"]] + _SIZE[case["q"]]
        if case["q"] == "mxfp4":
            per += _SIZE["mxfp4"] + 2             # the values that the codes stand for
        if case["train"]:
            per += _SIZE[case["y"]] + 2 * _SIZE[stream] + _SIZE[case["residual"]]
        return {"bytes": int(n * per) + 6 * cols, "flops": n * (20 if case["train"] else 8)}
    if case["op"] == "swiglu":
        n = int(case["rows"] * (1 - case["drop"])) * cols
        per = 2 * _SIZE[case["x"]] + _SIZE[case["y"]]
        return {"bytes": n * (2 * per + 2 * _SIZE[case["x"]] if case["train"] else per), "flops": n * (20 if case["train"] else 6)}
    tokens, picks = case["tokens"] * cols, int(case["tokens"] * case["top_k"] * (1 - case["drop"])) * cols
    if case["op"] == "dispatch":
        return {"bytes": tokens * _SIZE[case["x"]] + picks * _SIZE[case["rows"]], "flops": 0}
    n = picks * _SIZE[case["rows"]] + tokens * (_SIZE[case["addend"]] + _SIZE[case["y"]])
    if case["train"]:
        n += tokens * _SIZE[case["y"]] + 2 * picks * _SIZE[case["rows"]]
    return {"bytes": n, "flops": picks * (6 if case["train"] else 2)}


# ---- 64-bit definitions --------------------------------------------------------
def _on_e4m3(v):
    """Nearest E4M3 value, by the spacing of the numbers around each: 2^-9 below
    2^-6, an eighth of the power of two below it elsewhere."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return (torch.round(v / step) * step).clamp(-448, 448)


def _on_mxfp4(x):
    """Each value as MXFP4 holds it: the scale brings the largest magnitude of a
    block into [4, 8), the spacing of E2M1 is 0.5, 1 and 2 from 0, 2 and 4 on."""
    rows, cols = x.shape
    v = torch.nn.functional.pad(x, (0, -cols % 32)).view(rows, -1, 32)
    top = v.abs().amax(2, keepdim=True)
    _, e = torch.frexp(top)
    scale = torch.exp2(torch.where(top > 0, (e - 3).clamp(min=-127), torch.full_like(e, -127)).double())
    a = v.abs() / scale
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    a = (torch.round(a / step) * step).clamp(max=6)
    return (torch.sign(v) * a * scale).view(rows, -1)[:, :cols]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "norm":
        return _exact_norm(case, st)
    if case["op"] == "swiglu":
        return _exact_swiglu(case, st)
    inv = st["inv"]
    t, k = inv.shape
    if case["op"] == "dispatch":
        rows = torch.zeros(t * k, case["cols"], dtype=torch.float64, device="cuda")
        scale = torch.zeros(t * k, dtype=torch.float64, device="cuda")
        for i in range(k):
            on = inv[:, i] >= 0
            rows[inv[on, i].long()] = st["x"].double()[on]
            if st["scale"] is not None:
                scale[inv[on, i].long()] = st["scale"].double()[on]
        return {"rows": rows} if st["scale"] is None else {"rows": rows, "scale": scale}
    y = torch.zeros(t, case["cols"], dtype=torch.float64, device="cuda")
    if st["addend"] is not None:
        y += st["addend"].double()
    out = {"y": y}
    if case["train"]:
        out["drows"] = torch.zeros(t * k, case["cols"], dtype=torch.float64, device="cuda")
        out["dweights"] = torch.zeros(t, k, dtype=torch.float64, device="cuda")
    for i in range(k):
        on = (inv[:, i] >= 0).nonzero()[:, 0]
        slot = inv[on, i].long()
        w, rows = st["weights"][on, i].double()[:, None], st["rows"][slot].double()
        y[on] += w * rows
        if case["train"]:
            dy = st["dy"][on].double()
            out["drows"][slot] = w * dy
            out["dweights"][on, i] = (dy * rows).sum(1)
    return out


def _exact_norm(case, st):
    w, out = st["w"].double(), {}
    h = st["x"].double()
    if case["residual"] != "none":
        h = h + st["residual"].double()
        h = out["h"] = h.to(st["residual"].dtype).double()       # the stream's own rounding is part of the definition
    inner = (h * h).sum(1, keepdim=True) / case["cols"] + _EPS
    n = h / inner.sqrt()
    y = out["y"] = n * w
    if case["q"] == "e4m3":
        scale = out["scale"] = y.abs().amax(1) / 448
        out["q"] = _on_e4m3(y / scale[:, None])
    elif case["q"] == "mxfp4":
        out["q"] = _on_mxfp4(y)
    if case["train"]:
        dy = st["dy"].double()
        out["dw"] = (dy * n).sum(0)
        g = dy * w
        dx = (g - n * ((g * n).sum(1, keepdim=True) / case["cols"])) / inner.sqrt()
        out["dx"] = dx if st["dh"] is None else dx + st["dh"].double()
    return out


def _exact_swiglu(case, st):
    n, cols = st["kept"], case["cols"]
    whole = lambda v: torch.cat([v, v.new_zeros(case["rows"] - n, *v.shape[1:])])
    gu = st["gu"][:n].double()
    gate, up = gu[:, :cols], gu[:, cols:]
    s = 1 / (1 + torch.exp(-gate))
    y = gate * s * up
    out = {}
    if case["y"] == "e4m3":
        scale = y.abs().amax(1) / 448
        out["scale"], y = whole(scale), _on_e4m3(y / scale[:, None])
    out["out"] = whole(y)
    if case["train"]:
        dh = st["dh"][:n].double()
        out["dgu"] = whole(torch.cat([dh * up * (s + gate * s * (1 - s)), dh * gate * s], 1))
    return out
