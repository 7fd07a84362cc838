"""Row operators without a GPU: the float64 oracle's own pins (hand examples,
differences), and every refusal of the entry points, which come before any HIP
call."""
import ctypes

import numpy as np
import pytest
import torch

import quantized_moe_02_amd as q
from oracle import rows as ref

FAKE = ctypes.c_void_p(0x100000)      # non-null, 256-byte aligned, never dereferenced
ODD = ctypes.c_void_p(0x100001)
TWO = ctypes.c_void_p(0x100002)       # aligned for bf16 alone
BAD, UNS, SMALL, OK = (q.MOE_ERR_INVALID_ARG, q.MOE_ERR_UNSUPPORTED, q.MOE_ERR_WORKSPACE_TOO_SMALL, q.MOE_OK)
F32, BF16, F16, MX, E4 = q.MOE_DT_F32, q.MOE_DT_BF16, q.MOE_DT_F16, q.MOE_DT_MXFP4, q.MOE_DT_E4M3


# ---- oracle pins --------------------------------------------------------------
def _slope(f, x, i, step=1e-5):
    a, b = x.copy(), x.copy()
    a[i] += step
    b[i] -= step
    return (f(a) - f(b)) / (2 * step)


def test_norm_by_hand():
    y, m = ref.rmsnorm(np.array([[3.0, -4.0], [0.0, 0.0]]), np.array([1.0, 0.5]), 0.0 + 1e-300)
    assert np.allclose(y[0], [3 / np.sqrt(12.5), -2 / np.sqrt(12.5)]) and (y[1] == 0).all() and m.shape == (2, 1)


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(0)
    h, w, dy, dh = rng.normal(size=(3, 7)), rng.normal(size=7), rng.normal(size=(3, 7)), rng.normal(size=(3, 7))
    dx, dw, mag, dwmag = ref.rmsnorm_grad(dy, h, w, 0.3, dh)
    loss = lambda h, w: (dy * ref.rmsnorm(h, w, 0.3)[0] + dh * h).sum()
    for i in np.ndindex(h.shape):
        assert abs(_slope(lambda v: loss(v, w), h, i) - dx[i]) < 1e-8
    for i in np.ndindex(w.shape):
        assert abs(_slope(lambda v: loss(h, v), w, i) - dw[i]) < 1e-8
    assert (np.abs(dx) <= mag + 1e-12).all() and (np.abs(dw) <= dwmag + 1e-12).all()


def test_collect_gradient_against_differences():
    rng = np.random.default_rng(1)
    inv = np.array([[2, -1], [0, 4], [9, 1]])
    rows, w, dy, add = rng.normal(size=(5, 6)), rng.normal(size=(3, 2)), rng.normal(size=(3, 6)), rng.normal(size=(3, 6))
    drows, dw, _ = ref.collect_grad(dy, inv, rows, w)
    loss = lambda r, w: (dy * ref.collect(r, inv, w, add)[0]).sum()
    for i in np.ndindex(rows.shape):
        assert abs(_slope(lambda v: loss(v, w), rows, i) - drows[i]) < 1e-8
    for i in np.ndindex(w.shape):
        assert abs(_slope(lambda v: loss(rows, v), w, i) - dw[i]) < 1e-8


def test_dispatch_is_the_transpose_of_collect():
    rng = np.random.default_rng(2)
    inv = np.array([[2, -1], [0, 4], [7, 1]])
    x, r = rng.normal(size=(3, 4)), rng.normal(size=(5, 4))
    out = ref.dispatch(x, inv, np.zeros((5, 4)))
    assert (out[3] == 0).all() and (out[4] == x[1]).all()
    assert np.isclose((out * r).sum(), (x * ref.collect(r, inv)[0]).sum())


def test_swiglu_gradient_against_differences():
    rng = np.random.default_rng(3)
    gu, dh = 3 * rng.normal(size=(2, 10)), rng.normal(size=(2, 5))
    dgu, mag = ref.swiglu_grad(gu, dh)
    for i in np.ndindex(gu.shape):
        assert abs(_slope(lambda v: (dh * ref.swiglu(v)).sum(), gu, i) - dgu[i]) < 1e-8
    assert (np.abs(dgu) <= mag + 1e-12).all()


def test_e4m3_grid_is_the_type():
    grid = ref.e4m3_grid()
    held = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(grid, held)


def test_e4m3_rows():
    x = np.random.default_rng(4).normal(size=(50, 33))
    codes, scale = ref.e4m3_rows(x)
    assert np.array_equal(np.abs(codes).max(1), np.full(50, 448.0))
    want = torch.from_numpy(x / scale[:, None]).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.mean(codes != want) < 1e-3            # torch rounds by way of fp32
    codes, scale = ref.e4m3_rows(np.array([[448.0, 17.0, 19.0, -27.0, 2.0 ** -10, 3 * 2.0 ** -10], [0, 0, 0, 0, 0, 0],
                                           [1, np.inf, 0, 0, 0, 0]]))
    assert codes[0].tolist() == [448, 16, 20, -28, 0, 2.0 ** -8] and scale[0] == 1
    assert (codes[1:] == 0).all() and scale[1] == 2.0 ** -126 and np.isnan(scale[2])


# ---- refusals -------------------------------------------------------------------
def _norm(**over):
    d = dict(rows=4, cols=64, xt=BF16, rt=BF16, wt=F32, yt=BF16, qt=E4, eps=1e-6, ldx=64, ldr=64, ldh=64, ldy=64, x=FAKE,
             residual=FAKE, weight=FAKE, h=FAKE, y=FAKE, q=FAKE, scale=FAKE)
    d.update(over)
    c = q.MoeRmsnormConfig(*[d[k] for k in ("rows", "cols", "xt", "rt", "wt", "yt", "qt", "eps", "ldx", "ldr", "ldh", "ldy")])
    return q.lib().moe_rmsnorm(ctypes.byref(c), *[d[k] for k in ("x", "residual", "weight", "h", "y", "q", "scale")], None)


@pytest.mark.parametrize("over,status", [
    ({"rows": -1}, BAD), ({"cols": 0}, BAD), ({"cols": 65537, "ldx": 65537, "ldr": 65537, "ldh": 65537, "ldy": 65537}, UNS),
    ({"rows": 16 * q.MOE_MAX_TOKENS + 1}, UNS), ({"rows": 0}, OK), ({"rows": 0, "x": None, "q": None, "scale": None}, OK),
    ({"xt": F16}, BAD), ({"xt": E4}, BAD), ({"rt": MX}, BAD), ({"wt": -1}, BAD), ({"yt": 5}, BAD), ({"qt": BF16}, BAD),
    ({"rows": 0, "qt": F32, "q": None, "scale": None}, OK),
    ({"eps": 0.0}, BAD), ({"eps": -1.0}, BAD), ({"eps": float("nan")}, BAD), ({"eps": float("inf")}, BAD),
    ({"ldx": 63}, BAD), ({"ldr": 63}, BAD), ({"ldh": 63}, BAD), ({"ldy": 63}, BAD), ({"ldx": 2 ** 62}, UNS), ({"ldx": -1}, BAD),
    ({"x": None}, BAD), ({"weight": None}, BAD), ({"x": ODD}, BAD), ({"xt": F32, "x": TWO}, BAD), ({"weight": TWO}, BAD),
    ({"residual": ODD}, BAD), ({"h": ODD}, BAD), ({"y": ODD}, BAD), ({"yt": F32, "y": TWO}, BAD),
    ({"residual": None}, BAD),                                       # h without a residual
    ({"h": None, "y": None, "q": None, "scale": None}, BAD), ({"q": None}, BAD), ({"scale": None}, BAD),
    ({"q": ctypes.c_void_p(0x100004)}, BAD), ({"scale": TWO}, BAD), ({"qt": MX, "q": ctypes.c_void_p(0x100008)}, BAD)])
def test_norm_refusals(over, status):
    assert _norm(**over) == status


def test_norm_refusal_of_no_config():
    L = q.lib()
    assert L.moe_rmsnorm(None, *[FAKE] * 7, None) == BAD
    assert L.moe_rmsnorm_grad(None, *[FAKE] * 7, 1 << 30, None) == BAD
    assert L.moe_dispatch(None, *[FAKE] * 5, None) == L.moe_collect(None, *[FAKE] * 5, None) == BAD
    assert L.moe_collect_grad(None, *[FAKE] * 6, None) == BAD
    assert L.moe_swiglu(None, *[FAKE] * 4, None) == L.moe_swiglu_grad(None, *[FAKE] * 4, None) == BAD


def _norm_grad(**over):
    d = dict(rows=4, cols=64, ht=BF16, wt=F32, yt=BF16, xt=BF16, eps=1e-6, ldh=64, lddy=64, lddh=64, lddx=64, dy=FAKE, h=FAKE,
             weight=FAKE, dh=FAKE, dx=FAKE, dw=FAKE, ws=FAKE, n=1 << 30)
    d.update(over)
    c = q.MoeRmsnormGradConfig(*[d[k] for k in ("rows", "cols", "ht", "wt", "yt", "xt", "eps", "ldh", "lddy", "lddh", "lddx")])
    return q.lib().moe_rmsnorm_grad(ctypes.byref(c), *[d[k] for k in ("dy", "h", "weight", "dh", "dx", "dw", "ws", "n")], None)


@pytest.mark.parametrize("over,status", [
    ({"rows": -1}, BAD), ({"cols": 0}, BAD), ({"rows": 16 * q.MOE_MAX_TOKENS + 1}, UNS), ({"rows": 0, "dw": None}, OK),
    ({"ht": MX}, BAD), ({"wt": F16}, BAD), ({"yt": E4}, BAD), ({"xt": 7}, BAD), ({"eps": 0.0}, BAD),
    ({"ldh": 63}, BAD), ({"lddy": 63}, BAD), ({"lddh": 63}, BAD), ({"lddx": 63}, BAD), ({"lddx": 2 ** 62}, UNS),
    ({"dy": None}, BAD), ({"h": None}, BAD), ({"weight": None}, BAD), ({"dx": None}, BAD), ({"dy": ODD}, BAD), ({"h": ODD}, BAD),
    ({"dh": ODD}, BAD), ({"dx": ODD}, BAD), ({"weight": TWO}, BAD), ({"dw": TWO}, BAD), ({"ws": None}, BAD),
    ({"ws": ctypes.c_void_p(0x100080)}, BAD), ({"n": 4 * 64}, SMALL)])
def test_norm_grad_refusals(over, status):
    assert _norm_grad(**over) == status


def test_norm_workspace():
    n = lambda r, c: q.moe_rmsnorm_workspace_size(r, c)
    sizes = [1, 3, 4, 5, 300, 1023, 1024, 1025, 4096, 4097, 70000, 16 * q.MOE_MAX_TOKENS]
    cols = [1, 7, 511, 512, 513, 2048, 2049, 6144, 8192, 8193, 16384, 16385, 65536]
    for r in sizes:
        for c in cols:
            ld = dict(rows=r, cols=c, ldh=c, lddy=c, lddh=c, lddx=c)
            assert n(r, c) % 256 == 0 and n(r, c) >= 4 * c and _norm_grad(**ld, n=n(r, c) - 1) == SMALL
    # enough for every call of no more rows and columns
    grid = np.array([[n(r, c) for c in cols] for r in sizes])
    assert (np.diff(grid, axis=0) >= 0).all() and (np.diff(grid, axis=1) >= 0).all() and n(0, 4) > 0
    for r, c, s in ((-1, 4, BAD), (4, 0, BAD), (4, 65537, UNS), (16 * q.MOE_MAX_TOKENS + 1, 4, UNS)):
        with pytest.raises(q.QmoeError) as ei:
            n(r, c)
        assert ei.value.status == s
    assert q.lib().moe_rmsnorm_workspace_size(4, 4, None) == BAD


def _rows(fn, **over):
    d = dict(tokens=4, cols=64, k=2, slots=8, tt=BF16, rt=BF16, at=BF16, ldt=64, ldr=64, lda=64, x=FAKE, xs=None, inv=FAKE, rows=FAKE,
             rs=None, w=FAKE, add=FAKE, y=FAKE, dy=FAKE, drows=FAKE, dw=FAKE)
    d.update(over)
    c = q.MoeRowsConfig(*[d[k] for k in ("tokens", "cols", "k", "slots", "tt", "rt", "at", "ldt", "ldr", "lda")])
    args = {"dispatch": ("x", "xs", "inv", "rows", "rs"), "collect": ("rows", "inv", "w", "add", "y"),
            "collect_grad": ("dy", "rows", "inv", "w", "drows", "dw")}[fn]
    return getattr(q.lib(), "moe_" + fn)(ctypes.byref(c), *[d[k] for k in args], None)


ALL = ("dispatch", "collect", "collect_grad")


@pytest.mark.parametrize("fn", ALL)
@pytest.mark.parametrize("over,status", [
    ({"tokens": -1}, BAD), ({"slots": -1}, BAD), ({"cols": 0}, BAD), ({"k": 0}, BAD), ({"k": 17}, UNS),
    ({"tokens": q.MOE_MAX_TOKENS + 1}, UNS), ({"slots": 16 * q.MOE_MAX_TOKENS + 1}, UNS), ({"cols": 65537, "ldt": 65537, "ldr": 65537}, UNS),
    ({"tokens": 0}, OK), ({"tt": F16}, BAD), ({"rt": F16}, BAD), ({"tt": -1}, BAD), ({"rt": E4}, BAD), ({"ldt": 63}, BAD), ({"ldr": 63}, BAD),
    ({"ldt": 2 ** 62}, UNS), ({"inv": None}, BAD), ({"inv": TWO}, BAD), ({"rows": None}, BAD), ({"rows": ODD}, BAD),
    ({"x": None, "y": None, "dy": None}, BAD), ({"x": ODD, "y": ODD, "dy": ODD}, BAD)])
def test_rows_refusals(fn, over, status):
    assert _rows(fn, **over) == status


def test_rows_refusals_of_one_entry_point():
    assert _rows("dispatch", slots=0) == OK
    assert _rows("dispatch", xs=FAKE) == BAD and _rows("dispatch", rs=FAKE) == BAD
    for t in (E4, MX):
        coded = dict(tt=t, rt=t, xs=FAKE, rs=FAKE)
        assert _rows("dispatch", tokens=0, **coded) == OK
        assert _rows("dispatch", **dict(coded, xs=None)) == _rows("dispatch", **dict(coded, rs=None)) == BAD
        assert _rows("dispatch", **dict(coded, x=ctypes.c_void_p(0x100004))) == BAD
        assert _rows("dispatch", **dict(coded, ldt=65)) == _rows("dispatch", **dict(coded, ldr=65)) == BAD
        assert _rows("dispatch", **dict(coded, rt=BF16)) == _rows("dispatch", **dict(coded, tt=F32)) == BAD
        assert _rows("collect", tt=t) == _rows("collect", rt=t) == _rows("collect_grad", rt=t) == BAD
    assert _rows("collect", at=E4) == _rows("collect", lda=63) == _rows("collect", add=ODD) == _rows("collect", w=TWO) == BAD
    assert _rows("collect_grad", drows=None, dw=None) == _rows("collect_grad", dw=TWO) == _rows("collect_grad", drows=ODD) == BAD


def _swiglu(fn, **over):
    d = dict(rows=4, cols=64, E=3, gt=BF16, ot=BF16, ldg=128, ldo=64, gu=FAKE, off=FAKE, out=FAKE, scale=None, dgu=FAKE)
    d.update(over)
    c = q.MoeSwigluConfig(*[d[k] for k in ("rows", "cols", "E", "gt", "ot", "ldg", "ldo")])
    args = ("gu", "off", "out", "scale") if fn == "swiglu" else ("gu", "out", "off", "dgu")
    return getattr(q.lib(), "moe_" + fn)(ctypes.byref(c), *[d[k] for k in args], None)


@pytest.mark.parametrize("fn", ["swiglu", "swiglu_grad"])
@pytest.mark.parametrize("over,status", [
    ({"rows": -1}, BAD), ({"cols": 0}, BAD), ({"E": 0}, BAD), ({"rows": 16 * q.MOE_MAX_TOKENS + 1}, UNS),
    ({"cols": 65537, "ldg": 2 * 65537, "ldo": 65537}, UNS), ({"rows": 0}, OK), ({"gt": F16}, BAD), ({"gt": E4}, BAD), ({"ot": F16}, BAD),
    ({"ldg": 127}, BAD), ({"ldo": 63}, BAD), ({"ldg": 2 ** 62}, UNS), ({"gu": None}, BAD), ({"gu": ODD}, BAD), ({"out": None}, BAD),
    ({"out": ODD}, BAD), ({"off": TWO}, BAD)])
def test_swiglu_refusals(fn, over, status):
    assert _swiglu(fn, **over) == status


def test_swiglu_refusals_of_one_direction():
    assert _swiglu("swiglu", scale=FAKE) == BAD
    for t in (E4, MX):
        assert _swiglu("swiglu", ot=t) == _swiglu("swiglu", ot=t, scale=FAKE, ldo=65) == BAD
        assert _swiglu("swiglu", ot=t, scale=FAKE, out=ctypes.c_void_p(0x100004)) == _swiglu("swiglu_grad", ot=t) == BAD
        assert _swiglu("swiglu", ot=t, scale=FAKE, rows=0) == OK
    assert _swiglu("swiglu_grad", dgu=None) == _swiglu("swiglu_grad", dgu=ODD) == BAD


def test_binding_refuses_host_tensors():
    x, w, inv = torch.zeros(2, 64), torch.zeros(64), torch.zeros(2, 1, dtype=torch.int32)
    for call in (lambda: q.moe_rmsnorm(x, w, 1e-6, y=x.clone()), lambda: q.moe_rmsnorm_grad(x, x, w, 1e-6, x.clone()),
                 lambda: q.moe_dispatch(x, inv, x.clone()), lambda: q.moe_collect(x, inv, x.clone()),
                 lambda: q.moe_collect_grad(x, inv, drows=x.clone()), lambda: q.moe_swiglu(x, torch.zeros(2, 32)),
                 lambda: q.moe_swiglu_grad(x, torch.zeros(2, 32), x.clone())):
        with pytest.raises(q.QmoeError) as ei:
            call()
        assert ei.value.status == BAD
