"""MXFP4 and router-balance operators without a GPU: the float64 oracle's own
pins (hand examples, differences), and every refusal of the entry points, which
come before any HIP call."""
import ctypes

import numpy as np
import pytest
import torch

import quantized_moe_02_amd as q
from oracle import operators as ref

FAKE = ctypes.c_void_p(0x100000)      # non-null, 256-byte aligned, never dereferenced
ODD = ctypes.c_void_p(0x100002)
BAD, UNS, SMALL, OK = (q.MOE_ERR_INVALID_ARG, q.MOE_ERR_UNSUPPORTED, q.MOE_ERR_WORKSPACE_TOO_SMALL,
                       q.MOE_OK)


# ---- oracle pins --------------------------------------------------------------
def test_quantize_hand_block():
    """Largest magnitude 13 in [8, 16): scale 2; ties of x / 2 go to the even code."""
    x = np.zeros((1, 34))
    x[0, :12] = [13.0, -12.0, 0.5, 1.5, 2.5, 3.5, 5.0, 7.0, 10.0, -0.49, 0.51, 11.0]
    x[0, 32] = 3.0
    codes, scale = ref.mx_quantize(x)
    assert scale.tolist() == [[128, 126]]
    got = [c & 15 if i % 2 == 0 else c >> 4 for i, c in
           ((i, int(codes[0, i // 2])) for i in range(12))]
    assert got == [7, 15, 0, 2, 2, 4, 4, 6, 6, 8, 1, 7]
    v = ref.mx_values(codes, scale)
    assert v.shape == (1, 64) and v[0, 32] == 3.0 and v[0, 0] == 12.0 and (v[0, 33:] == 0).all()


@pytest.mark.parametrize("value,byte,held", [
    (0.0, 0, 0.0), (2.0 ** -149, 0, 0.0), (2.0 ** -125, 0, 2.0 ** -125), (2.0 ** -124, 1, 2.0 ** -124),
    (1.0, 125, 1.0), (1.9999, 125, 1.5),       # 8 - eps units: E2M1 ends at 6
    (2.0 ** 127, 252, 2.0 ** 127), (np.inf, 255, np.nan), (np.nan, 255, np.nan)])
def test_quantize_scale_byte(value, byte, held):
    codes, scale = ref.mx_quantize(np.array([[value, 0.0, -0.0]]))
    assert scale[0, 0] == byte
    v = ref.mx_values(codes, scale)[0]
    assert v[0] == held and (v[1:] == 0).all() if byte != 255 else np.isnan(v).all()


def test_quantize_is_idempotent_and_nearest():
    x = np.random.default_rng(0).normal(size=(20, 96))
    codes, scale = ref.mx_quantize(x)
    v = ref.mx_values(codes, scale)
    again = ref.mx_quantize(v)
    assert np.array_equal(ref.mx_values(*again), v)
    s = np.ldexp(1.0, scale.astype(int) - 127).repeat(32, 1)
    grid = np.concatenate([-ref.E2M1, ref.E2M1])
    best = np.abs(x[..., None] - grid * s[..., None]).min(-1)
    assert np.array_equal(np.abs(x - v), best)


def test_grouped_matmul_rows():
    rng = np.random.default_rng(1)
    a, w = rng.normal(size=(4, 32)), rng.normal(size=(3, 5, 32))
    out, _ = ref.grouped_matmul(a, w, [0, 2, 2, 5], index=[3, 0, 9, 1, 1, 2], rows=6)
    assert np.allclose(out[0], w[0] @ a[3]) and np.allclose(out[4], w[2] @ a[1])
    assert (out[2] == 0).all() and (out[5] == 0).all()


def test_product_gradient_against_differences():
    """sum(dy * out(a)) changes by dx when a does."""
    rng = np.random.default_rng(2)
    a, w, dy = rng.normal(size=(4, 8)), rng.normal(size=(2, 6, 8)), rng.normal(size=(4, 6))
    off = [0, 1, 3]
    dx, _ = ref.grouped_matmul(dy, w, off, transpose=True)
    for r in range(4):
        for i in range(8):
            hi, lo = a.copy(), a.copy()
            hi[r, i] += 0.5
            lo[r, i] -= 0.5
            d = (dy[:3] * (ref.grouped_matmul(hi, w, off)[0] - ref.grouped_matmul(lo, w, off)[0])[:3]).sum()
            assert abs(d - dx[r, i]) < 1e-12 * 100


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_balance_gradient_against_differences(score):
    rng = np.random.default_rng(3)
    T, E, k = 11, 5, 2
    x = rng.normal(size=(T, E)) * 2
    ids = np.argsort(-x, 1)[:, :k]
    ids[4] = -1
    ids[6, 0] = -1
    seq = [0, 3, 3, 5, 11]
    loss, counts, tokens, g = ref.balance(x, ids, seq, 0.7, score)
    assert tokens.tolist() == [3, 0, 1, 6] and counts.sum() == 2 * 10 - 1
    assert (g[4] == 0).all()
    h = 1e-6
    for t in range(T):
        for e in range(E):
            hi, lo = x.copy(), x.copy()
            hi[t, e] += h
            lo[t, e] -= h
            d = (ref.balance(hi, ids, seq, 0.7, score)[0] - ref.balance(lo, ids, seq, 0.7, score)[0]) / (2 * h)
            # central differences: 0.7 * f'''/6 * h^2 (1e-12) and cancellation 1e-16 * 2 / 2e-6 (1e-10)
            assert abs(d - g[t, e]) < 1e-8


def test_balance_of_a_balanced_router_is_coef():
    """Every expert picked equally often: f = 1, and shares add up to 1."""
    x = np.random.default_rng(4).normal(size=(8, 4))
    ids = np.arange(8)[:, None] % 4
    for score in ("sigmoid", "softmax"):
        loss, _, _, g = ref.balance(x, ids, [0, 8], 0.25, score)
        assert abs(loss - 0.25) < 1e-15 and np.abs(g).max() < 1e-16


def test_shares_where_every_sigmoid_underflows():
    p = ref.shares(np.array([[-900.0, -901.0, -np.inf]]), "sigmoid")
    assert np.allclose(p, [[1 / (1 + np.exp(-1)), 1 / (1 + np.e), 0]])


# ---- refusals -----------------------------------------------------------------
@pytest.mark.parametrize("over,status", [
    (dict(dtype=3), BAD), (dict(dtype=-1), BAD), (dict(rows=-1), BAD), (dict(cols=0), BAD),
    (dict(ld=63), BAD), (dict(x=None), BAD), (dict(codes=None), BAD), (dict(scale=None), BAD),
    (dict(x=ctypes.c_void_p(0x100001)), BAD), (dict(x=ODD, dtype=0), BAD),
    (dict(codes=ctypes.c_void_p(0x100008)), BAD), (dict(cols=1 << 25, ld=1 << 25), UNS),
    (dict(rows=1 << 31), UNS), (dict(ld=1 << 60), UNS), (dict(rows=0), OK),
    (dict(rows=0, x=None, codes=None, scale=None), OK)])
def test_quantize_refusals(over, status):
    a = dict(x=FAKE, dtype=1, rows=5, cols=64, ld=64, codes=FAKE, scale=FAKE)
    a.update(over)
    L = q.lib()
    assert L.moe_mxfp4_quantize(a["x"], a["dtype"], a["rows"], a["cols"], a["ld"], a["codes"], a["scale"],
                                None) == status
    assert L.moe_mxfp4_dequantize(a["codes"], a["scale"], a["rows"], a["cols"], a["x"], a["dtype"], a["ld"],
                                  None) == status


def _mm(fn="matmul", **over):
    a = dict(rows=0, n=64, k=96, E=4, a_rows=None, adt=1, odt=0, lda=96, ldo=64, a=FAKE, a_scale=None, wq=FAKE,
             ws=FAKE, off=FAKE, index=None, out=FAKE)
    if fn == "dx":
        a.update(lda=64, ldo=96)
    a.update(over)
    if a["a_rows"] is None:
        a["a_rows"] = a["rows"]
    c = q.MoeMatmulConfig(a["rows"], a["n"], a["k"], a["E"], a["a_rows"], a["adt"], a["odt"], a["lda"], a["ldo"])
    L = q.lib()
    if fn == "dx":
        return L.moe_mxfp4_matmul_dx(ctypes.byref(c), a["a"], a["wq"], a["ws"], a["off"], a["out"], None)
    return L.moe_mxfp4_matmul(ctypes.byref(c), a["a"], a["a_scale"], a["wq"], a["ws"], a["off"], a["index"],
                              a["out"], None)


@pytest.mark.parametrize("fn", ["matmul", "dx"])
@pytest.mark.parametrize("over,status", [
    (dict(), OK), (dict(rows=-1), BAD), (dict(n=0), BAD), (dict(k=0), BAD), (dict(k=48), BAD), (dict(E=0), BAD),
    (dict(adt=2), BAD), (dict(adt=0), BAD), (dict(odt=2), BAD), (dict(odt=3), BAD), (dict(lda=56), BAD),
    (dict(lda=100), BAD), (dict(ldo=32), BAD), (dict(E=257), UNS), (dict(n=65568, lda=65568, ldo=65568), UNS),
    (dict(k=65568, lda=65568, ldo=65568), UNS), (dict(rows=(1 << 22) + 1), UNS), (dict(ldo=1 << 60), UNS),
    (dict(rows=2, a=None), BAD), (dict(rows=2, wq=None), BAD), (dict(rows=2, ws=None), BAD),
    (dict(rows=2, out=None), BAD), (dict(rows=2, off=None), BAD), (dict(rows=2, a=ODD), BAD),
    (dict(rows=2, wq=ODD), BAD), (dict(rows=2, ws=ODD), BAD), (dict(rows=2, out=ODD), BAD)])
def test_matmul_refusals(fn, over, status):
    assert _mm(fn, **over) == status


def test_matmul_refusals_of_one_direction():
    assert _mm(rows=2, a_rows=3) == BAD                       # no index: one input row per output row
    assert _mm(rows=2, a_scale=FAKE) == BAD                   # bf16 rows have no scales
    assert _mm(rows=2, adt=3) == BAD                          # MXFP4 rows need them
    assert _mm(rows=2, adt=3, a_scale=ODD) == BAD
    assert _mm(adt=3, lda=128) == BAD                         # MXFP4 rows are packed
    assert _mm(adt=3, a_rows=5, index=FAKE) == OK
    assert _mm(a_rows=-1, index=FAKE) == BAD
    assert _mm("dx", n=48, lda=48) == BAD                     # its sums run over n
    assert _mm("dx", adt=3) == BAD
    assert _mm("dx", a_rows=1) == BAD
    assert q.lib().moe_mxfp4_matmul(None, FAKE, None, FAKE, FAKE, FAKE, None, FAKE, None) == BAD
    assert q.lib().moe_mxfp4_matmul_dx(None, FAKE, FAKE, FAKE, FAKE, FAKE, None) == BAD


@pytest.mark.parametrize("over,status", [
    (dict(tokens=-1), BAD), (dict(n_experts=0), BAD), (dict(top_k=0), BAD), (dict(n_seq=0), BAD), (dict(score=2), BAD),
    (dict(logits_dtype=2), BAD), (dict(coef=float("nan")), BAD), (dict(coef=float("inf")), BAD),
    (dict(n_experts=257), UNS), (dict(top_k=17), UNS), (dict(n_seq=65537), UNS),
    (dict(tokens=q.MOE_MAX_TOKENS + 1), UNS), (dict(tokens=0), OK), (dict(), OK)])
def test_balance_config(over, status):
    c = q.make_balance_config(100, 16, 4, 3)
    for k, v in over.items():
        setattr(c, k, v)
    n = ctypes.c_size_t(7)
    L = q.lib()
    assert L.moe_balance_workspace_size(ctypes.byref(c), ctypes.byref(n)) == status
    if status == OK:
        assert n.value > 0 and n.value % 256 == 0
        return
    assert n.value == 7
    assert L.moe_balance_loss(ctypes.byref(c), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40, None) == status
    assert L.moe_balance_loss_grad(ctypes.byref(c), FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, None) == status


def test_balance_refusals():
    L = q.lib()
    c = q.make_balance_config(100, 16, 4, 3)
    n = q.moe_balance_workspace_size(c)
    ok = [FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE]
    for i in range(7):                 # logits, ids, seq, counts, tokens, loss, ws
        a = list(ok)
        a[i] = None
        assert L.moe_balance_loss(ctypes.byref(c), *a, n, None) == BAD, i
    assert L.moe_balance_loss(ctypes.byref(c), ctypes.c_void_p(0x100004), *ok[1:], n, None) == BAD
    assert L.moe_balance_loss(ctypes.byref(c), *ok[:6], ctypes.c_void_p(0x100040), n, None) == BAD
    assert L.moe_balance_loss(ctypes.byref(c), *ok, n - 1, None) == SMALL
    assert L.moe_balance_workspace_size(ctypes.byref(c), None) == BAD
    g = [FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE]       # logits, ids, seq, counts, tokens, dloss, dlogits
    for i in (0, 1, 2, 3, 4, 6):
        a = list(g)
        a[i] = None
        assert L.moe_balance_loss_grad(ctypes.byref(c), *a, None) == BAD, i
    assert L.moe_balance_loss_grad(ctypes.byref(c), *g[:6], ctypes.c_void_p(0x100004), None) == BAD
    c.tokens = 0
    assert L.moe_balance_loss_grad(ctypes.byref(c), None, None, FAKE, None, None, None, None, None) == OK


def test_binding_refuses_host_tensors():
    x, (codes, scales) = torch.zeros(2, 64), q.mxfp4_empty(2, 64, device="cpu")
    assert codes.shape == (2, 32) and scales.shape == (2, 2)
    w = torch.zeros(1, 4, 32, dtype=torch.uint8)
    ws = torch.zeros(1, 4, 2, dtype=torch.uint8)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    for call in (lambda: q.moe_mxfp4_quantize(x, codes, scales),
                 lambda: q.moe_mxfp4_dequantize(codes, scales, x),
                 lambda: q.moe_mxfp4_matmul(x.bfloat16(), w, ws, torch.zeros(2, 4)),
                 lambda: q.moe_mxfp4_matmul_dx(torch.zeros(2, 4).bfloat16(), w, ws, x),
                 lambda: q.moe_balance_loss(x, i32(2, 2), i32(1, 64), i32(1), torch.zeros(1), coef=1.0),
                 lambda: q.moe_balance_loss_grad(x, i32(2, 2), i32(1, 64), i32(1), x, coef=1.0)):
        with pytest.raises(q.QmoeError) as ei:
            call()
        assert ei.value.status == BAD


def test_layout_sizes_round_up():
    codes, scales = q.mxfp4_empty(3, 33, device="cpu")
    assert codes.shape == (3, 32) and scales.shape == (3, 2)
