"""Row operators on the GPU against float64 (oracle/rows.py)."""
import numpy as np
import pytest
import torch

import quantized_moe_02_amd as q
from oracle import rows as ref
from row_cases import BF, F, HALF, U, close, f64, picks, pitched, silu_bound

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.lib()


def _gen(*seed):
    return torch.Generator().manual_seed(hash(seed) & 0x7FFFFFFF)


def _held(h, w, codes, scale, y32):
    """E4M3 rows against y in fp32 as the same call wrote it."""
    y = f64(y32)
    want, s = ref.e4m3_rows(y)
    got_s, got = f64(scale), f64(codes)
    bad = np.isnan(s)
    assert np.array_equal(np.isnan(got_s), bad)
    ok = ~bad
    assert (np.abs(got_s[ok] - s[ok]) <= 2 * U * s[ok]).all()         # one division in fp32
    # nearest to y / scale, where reciprocal, product and scale are each rounded once
    v = np.abs(y[ok] / got_s[ok, None])
    step = np.exp2(np.clip(np.floor(np.log2(np.maximum(v, 2.0 ** -20))), -6, 8) - 3)
    assert (np.abs(np.abs(got[ok]) - np.minimum(v, 448)) <= step / 2 + 4 * U * v).all()
    assert (got[bad] == 0).all()
    assert np.mean(got[ok] != want[ok]) < 1e-3 if got[ok].size > 1000 else True


# ---- norm ------------------------------------------------------------------------
# one wave a row, a workgroup a row with 1 to 4 units a lane, rows read again
COLS = [1, 7, 8, 31, 33, 256, 512, 513, 2048, 2057, 4096, 4104, 6144, 6150, 8192, 8193, 16384, 16500, 65536]


def _check_norm(rows, cols, xt, rt, wt, yt, pad=0, in_place=False, scale=1.0):
    gen = _gen(rows, cols, pad)
    x = pitched((rows, cols), xt, pad, gen=gen, scale=scale)
    r = None if rt is None else pitched((rows, cols), rt, pad, gen=gen, scale=scale)
    w = (1 + 0.3 * torch.randn(cols, generator=gen)).to(wt).cuda()
    h0 = x.float() if r is None else (x.float() + r.float()).to(rt)
    h = None if r is None else r if in_place else pitched((rows, cols), rt, pad)
    y, y32 = pitched((rows, cols), yt, pad), pitched((rows, cols), F, pad)
    codes, sc = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(rows, device="cuda")
    mx, mxs = q.mxfp4_empty(rows, cols)
    keep = r.clone() if in_place else None
    q.moe_rmsnorm(x, w, EPS, y=y, residual=r, h=h, q=codes, q_scale=sc)
    if h is not None:
        assert torch.equal(h, h0)
    if in_place:
        r.copy_(keep)
    q.moe_rmsnorm(x, w, EPS, y=y32, residual=r, q=mx, q_scale=mxs)
    want, _ = ref.rmsnorm(f64(h0), f64(w), EPS)
    bound = 3.01 * U * np.abs(want)              # m, h m and its product with w
    close(y, want, bound, yt, "y")
    close(y32, want, bound, F, "y32")
    _held(h0, w, codes, sc, y32)
    a, b = q.mxfp4_empty(rows, cols)
    q.moe_mxfp4_quantize(y32, a, b)
    assert torch.equal(mx, a) and torch.equal(mxs, b)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("rows", [1, 6])
def test_norm_bf16(rows, cols):
    _check_norm(rows, cols, BF, BF, BF, BF)


@pytest.mark.parametrize("cols", COLS)
def test_norm_f32_without_residual(cols):
    _check_norm(5, cols, F, None, F, F, pad=3)


@pytest.mark.parametrize("cols", [9, 520, 2057, 4100, 6145, 8190, 9000])
@pytest.mark.parametrize("types", [(F, BF, F, BF), (BF, F, BF, F), (BF, None, F, BF), (F, F, BF, BF)])
@pytest.mark.parametrize("in_place", [False, True])
def test_norm_mixed_types_and_strides(cols, types, in_place):
    _check_norm(3, cols, *types, pad=5, in_place=in_place and types[1] is not None)


def test_norm_many_rows():
    _check_norm(1500, 300, BF, BF, F, BF)
    _check_norm(700, 2100, F, BF, F, BF, pad=1)


@pytest.mark.parametrize("cols", [40, 700, 6144, 9000])
@pytest.mark.parametrize("scale", [1e-30, 1e25, 3e37])
def test_norm_at_the_ends_of_the_range(cols, scale):
    """Squares leave fp32's range on both sides; the norm does not."""
    gen = _gen(cols)
    x = (torch.rand(3, cols, generator=gen) + 0.5).mul(scale).cuda()
    w = torch.ones(cols, device="cuda")
    y = torch.empty_like(x)
    q.moe_rmsnorm(x, w, 1e-37, y=y)
    eps = float(np.float32(1e-37))
    want, m = ref.rmsnorm(f64(x), np.ones(cols), eps)
    # 1/rms of the largest is a subnormal: a step of 2^-149
    close(y, want, 3.01 * U * np.abs(want) + np.abs(f64(x)) * 2.0 ** -149, F)
    assert (want != 0).any()


@pytest.mark.parametrize("cols", [24, 600, 6144, 9000])
def test_norm_of_infinities_nan_and_zeros(cols):
    x = torch.randn(5, cols, generator=_gen(cols)).to(BF)
    x[0, 3], x[1, cols - 1], x[2] = float("inf"), float("nan"), 0.0
    x[3, 0] = -float("inf")
    x, w = x.cuda(), torch.ones(cols, device="cuda")
    y, sc = torch.empty(5, cols, device="cuda"), torch.empty(5, device="cuda")
    codes = torch.empty(5, cols, dtype=torch.float8_e4m3fn, device="cuda")
    mx, mxs = q.mxfp4_empty(5, cols)
    q.moe_rmsnorm(x, w, EPS, y=y, q=codes, q_scale=sc)
    q.moe_rmsnorm(x, w, EPS, q=mx, q_scale=mxs)
    a, b = q.mxfp4_empty(5, cols)
    q.moe_mxfp4_quantize(y, a, b)
    assert torch.equal(mx, a) and torch.equal(mxs, b)
    y, sc, codes = y.cpu(), sc.cpu(), codes.float().cpu()
    for r, c in ((0, 3), (3, 0)):
        assert torch.isnan(y[r, c]) and (y[r][torch.arange(cols) != c] == 0).all()
    assert torch.isnan(y[1]).all() and (y[2] == 0).all() and torch.isfinite(y[4]).all()
    assert torch.isnan(sc[[0, 1, 3]]).all() and sc[2] == 2.0 ** -126 and (codes[:4] == 0).all()


def test_norm_h_alone_and_nothing_else_is_written():
    x, r = torch.randn(4, 72).cuda().to(BF), torch.randn(4, 72).cuda().to(BF)
    h, w = torch.empty_like(x), torch.ones(72, device="cuda")
    q.moe_rmsnorm(x, w, EPS, residual=r, h=h)
    assert torch.equal(h, (x.float() + r.float()).to(BF))
    q.moe_rmsnorm(x, w, EPS, residual=r, h=x)             # h over x
    assert torch.equal(h, x)


@pytest.mark.parametrize("cols", [33, 520, 4097, 9001])
def test_norm_leaves_the_gaps_between_rows(cols):
    gen = _gen(cols)
    x = pitched((4, cols), BF, 9, gen=gen)
    buf = torch.full((6, cols + 9), 7.0, device="cuda", dtype=BF)
    hb = torch.full((6, cols + 9), 7.0, device="cuda", dtype=BF)
    q.moe_rmsnorm(x, torch.ones(cols, device="cuda"), EPS, y=buf[1:5, 4:4 + cols], residual=x, h=hb[1:5, 4:4 + cols])
    for b in (buf, hb):
        b[1:5, 4:4 + cols] = 7.0
        assert (b == 7.0).all()


# ---- its gradient ------------------------------------------------------------------
def _check_norm_grad(rows, cols, ht, wt, yt, xt, dh=True, pad=0, dw=True, alias=None):
    gen = _gen(rows, cols, pad, dh)
    h = pitched((rows, cols), ht, pad, gen=gen)
    dy = pitched((rows, cols), yt, pad, gen=gen, scale=0.1)
    d = pitched((rows, cols), xt, pad, gen=gen, scale=0.1) if dh else None
    w = (1 + 0.3 * torch.randn(cols, generator=gen)).to(wt).cuda()
    want = ref.rmsnorm_grad(f64(dy), f64(h), f64(w), EPS, None if d is None else f64(d))
    dx = {None: pitched((rows, cols), xt, pad), "dh": d, "dy": dy}[alias]
    dweight = torch.full((cols,), float("nan"), device="cuda") if dw else None
    q.moe_rmsnorm_grad(dy, h, w, EPS, dx, dh=d, dweight=dweight, ws=q.rmsnorm_workspace(rows, cols) if dw else None)
    # g, its product with h, m, k, h k, the difference, its product with m, dh's addition
    close(dx, want[0], 8 * U * want[2], xt, "dx")
    if dw:
        chain = -(-rows // 256) + 8              # terms that one workgroup adds in fp32, waves and roundings of a term
        close(dweight, want[1], chain * U * want[3], F, "dweight")


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("rows", [1, 6])
def test_norm_grad_bf16(rows, cols):
    _check_norm_grad(rows, cols, BF, BF, BF, BF)


@pytest.mark.parametrize("cols", COLS)
def test_norm_grad_f32(cols):
    _check_norm_grad(5, cols, F, F, F, F, dh=False, pad=3)


@pytest.mark.parametrize("cols", [9, 520, 2057, 4100, 6145, 8190, 9000])
@pytest.mark.parametrize("types", [(F, BF, F, BF), (BF, F, BF, F), (F, F, BF, BF), (BF, BF, F, F)])
@pytest.mark.parametrize("alias", [None, "dh"])
def test_norm_grad_mixed_types_and_strides(cols, types, alias):
    _check_norm_grad(3, cols, *types, pad=5, alias=alias)


@pytest.mark.parametrize("rows,cols", [(1025, 40), (4099, 512), (5000, 17), (2049, 520), (1100, 4100), (1030, 8200)])
def test_norm_grad_many_rows(rows, cols):
    _check_norm_grad(rows, cols, BF, F, BF, BF, pad=1)


def test_norm_grad_without_weight_gradient():
    _check_norm_grad(7, 2056, BF, F, BF, BF, dw=False)
    _check_norm_grad(7, 136, F, F, F, F, dw=False, alias="dy")


def test_norm_grad_of_no_rows():
    e, w = torch.empty(0, 777, device="cuda"), torch.ones(777, device="cuda")
    dw = torch.full((777,), 3.0, device="cuda")
    q.moe_rmsnorm_grad(e, e, w, EPS, e.clone(), dweight=dw)
    assert (dw == 0).all()


def test_norm_grad_against_differences():
    """The loss in float64 from the kernel's own inputs, each input moved by itself."""
    gen = _gen(5)
    h, w, dy = torch.randn(2, 37, generator=gen), torch.rand(37, generator=gen) + 0.5, torch.randn(2, 37, generator=gen)
    dx, dw = torch.empty(2, 37, device="cuda"), torch.empty(37, device="cuda")
    q.moe_rmsnorm_grad(dy.cuda(), h.cuda(), w.cuda(), EPS, dx, dweight=dw)
    H, W, D = f64(h), f64(w), f64(dy)
    loss = lambda h, w: (D * ref.rmsnorm(h, w, EPS)[0]).sum()
    step = 1e-4                                  # third differences: step^2 * |f'''| / 6 < 1e-7
    for i in np.ndindex(H.shape):
        e = np.zeros_like(H)
        e[i] = step
        assert abs((loss(H + e, W) - loss(H - e, W)) / (2 * step) - float(dx[i])) < 1e-5
    for i in range(37):
        e = np.zeros_like(W)
        e[i] = step
        assert abs((loss(H, W + e) - loss(H, W - e)) / (2 * step) - float(dw[i])) < 1e-5


# ---- dispatch ------------------------------------------------------------------------
SHAPES = [(1, 8, 6144, 256), (1, 1, 1, 1), (5, 3, 7, 4), (64, 8, 264, 16), (37, 16, 33, 20), (9, 2, 2057, 3), (3, 4, 8192, 8), (2, 2, 65536, 4),
          (300, 5, 130, 9), (13, 12, 1000, 12), (4, 2, 257, 2), (70, 2, 520, 5)]


@pytest.mark.parametrize("T,K,cols,E", SHAPES)
@pytest.mark.parametrize("xt,rt", [(BF, BF), (F, F), (F, BF), (BF, F)])
@pytest.mark.parametrize("drop,pad", [(0.0, 0), (0.4, 3)])
def test_dispatch(T, K, cols, E, xt, rt, drop, pad):
    gen = _gen(T, K, cols)
    x, inv = pitched((T, cols), xt, pad, gen=gen), picks(T, K, E, gen, drop)
    rows = pitched((T * K, cols), rt, pad, fill=5.0)
    want = torch.from_numpy(ref.dispatch(f64(x), inv.numpy(), np.full((T * K, cols), 5.0)))
    q.moe_dispatch(x, inv.cuda(), rows)
    assert torch.equal(rows.cpu(), want.to(torch.float32).to(rt))
    rows.fill_(5.0)
    if pad:                                      # the memory around the rows
        whole = rows.as_strided((T * K, cols + pad), (cols + pad, 1))
        q.moe_dispatch(x, inv.cuda(), rows)
        assert torch.equal(rows.cpu(), want.to(torch.float32).to(rt)) and (whole[:-1, cols:] == 5.0).all()


@pytest.mark.parametrize("T,K,cols,E", SHAPES)
@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_dispatch_of_codes(T, K, cols, E, drop):
    gen = _gen(T, K, cols, 1)
    inv = picks(T, K, E, gen, drop)
    nb = (cols + 31) // 32
    b = lambda *s: torch.randint(0, 255, s, generator=gen, dtype=torch.uint8)
    for codes, scale, fill in ((b(T, cols), torch.rand(T, generator=gen), 9), (b(T, 16 * nb), b(T, nb), 9)):
        rows = torch.full((T * K, codes.shape[1]), fill, dtype=torch.uint8, device="cuda")
        rscale = torch.full((T * K, *scale.shape[1:]), fill, dtype=scale.dtype, device="cuda")
        e4 = scale.dtype is F
        v = (lambda t: t.view(torch.float8_e4m3fn)) if e4 else (lambda t: t)
        q.moe_dispatch(v(codes.cuda()), inv.cuda(), v(rows), x_scale=scale.cuda(), row_scale=rscale)
        assert np.array_equal(rows.cpu().numpy(), ref.dispatch(codes.numpy(), inv.numpy(), np.full(rows.shape, fill, np.uint8)))
        s = scale.numpy().reshape(T, -1)
        want = ref.dispatch(s, inv.numpy(), np.full((T * K, s.shape[1]), fill, s.dtype))
        assert np.array_equal(rscale.cpu().numpy().reshape(T * K, -1), want)


@pytest.mark.parametrize("fn", ["dispatch", "collect", "collect_grad"])
def test_slots_outside_take_no_part(fn):
    T, K, cols, R = 3, 3, 40, 4
    inv = torch.tensor([[0, 4, -1], [-2147483648, 2147483647, 3], [-7, -1, 100000]], dtype=torch.int32)
    gen = _gen(3)
    x, rows, w = torch.randn(T, cols, generator=gen), torch.randn(R, cols, generator=gen), torch.rand(T, K, generator=gen)
    if fn == "dispatch":
        out = rows.cuda()
        q.moe_dispatch(x.cuda(), inv.cuda(), out)
        assert np.array_equal(f64(out), ref.dispatch(f64(x), inv.numpy(), f64(rows)))
    elif fn == "collect":
        y = torch.empty(T, cols, device="cuda")
        q.moe_collect(rows.cuda(), inv.cuda(), y, weights=w.cuda())
        want, mag = ref.collect(f64(rows), inv.numpy(), f64(w))
        close(y, want, 4 * U * mag, F)
        assert (y[2] == 0).all()
    else:
        drows, dw = torch.full((R, cols), 2.0, device="cuda"), torch.empty(T, K, device="cuda")
        q.moe_collect_grad(x.cuda(), inv.cuda(), drows=drows, weights=w.cuda(), rows=rows.cuda(), dweights=dw)
        want, dww, mag = ref.collect_grad(f64(x), inv.numpy(), f64(rows), f64(w), np.full((R, cols), 2.0))
        close(drows, want, 0.0, F)
        close(dw, dww, (cols + 8) * U * mag, F)
        assert (dw[2] == 0).all()


def test_no_slots_and_no_tokens():
    inv = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    none, x = torch.empty(0, 16, device="cuda"), torch.randn(3, 16, device="cuda")
    q.moe_dispatch(x, inv, none)
    y, dw = torch.empty(3, 16, device="cuda"), torch.full((3, 2), 5.0, device="cuda")
    q.moe_collect(none, inv, y, addend=x)
    assert torch.equal(y, x)
    q.moe_collect_grad(x, inv, drows=none.clone(), rows=none, dweights=dw)
    assert (dw == 0).all()
    e, i0 = torch.empty(0, 16, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda")
    rows = torch.full((4, 16), 3.0, device="cuda")
    q.moe_dispatch(e, i0, rows)
    q.moe_collect(rows, i0, e)
    q.moe_collect_grad(e, i0, drows=rows)
    q.moe_rmsnorm(e, torch.ones(16, device="cuda"), EPS, y=e.clone())
    q.moe_swiglu(e, torch.empty(0, 8, device="cuda"))
    q.moe_swiglu_grad(e, torch.empty(0, 8, device="cuda"), e.clone())
    assert (rows == 3.0).all()


# ---- collect and its gradient -----------------------------------------------------------
@pytest.mark.parametrize("T,K,cols,E", SHAPES)
@pytest.mark.parametrize("rt,yt,at", [(BF, BF, BF), (F, F, None), (BF, F, F), (F, BF, BF)])
@pytest.mark.parametrize("drop,pad", [(0.0, 0), (0.4, 3)])
def test_collect(T, K, cols, E, rt, yt, at, drop, pad):
    gen = _gen(T, K, cols, 2)
    inv, rows = picks(T, K, E, gen, drop), pitched((T * K, cols), rt, pad, gen=gen)
    w = None if at is None else torch.rand(T, K, generator=gen)
    add = None if at is None else pitched((T, cols), at, pad, gen=gen)
    y = pitched((T, cols), yt, pad)
    q.moe_collect(rows, inv.cuda(), y, weights=None if w is None else w.cuda(), addend=add)
    want, mag = ref.collect(f64(rows), inv.numpy(), None if w is None else f64(w), None if add is None else f64(add))
    close(y, want, (K + 2) * U * mag, yt)


@pytest.mark.parametrize("cols", [5, 70, 513, 1030, 2049, 6145])       # a row's last lane in a wave of its own, too
def test_collect_onto_its_addend(cols):
    gen = _gen(8, cols)
    inv, rows, y = picks(9, 3, 5, gen), torch.randn(27, cols, generator=gen).cuda(), torch.randn(9, cols, generator=gen).cuda()
    want, mag = ref.collect(f64(rows), inv.numpy(), None, f64(y))
    q.moe_collect(rows, inv.cuda(), y, addend=y)
    close(y, want, 5 * U * mag, F)


def test_dropped_picks_are_not_multiplied():
    """What a dropped pick's weight or another row holds stays out of the sum."""
    rows = torch.full((4, 24), float("nan"), device="cuda")
    rows[1] = 2.0
    inv = torch.tensor([[-1, 1], [-1, -1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[float("inf"), 3.0], [float("nan"), 0.0]], device="cuda")
    y = torch.empty(2, 24, device="cuda")
    q.moe_collect(rows, inv, y, weights=w)
    assert (y[0] == 6.0).all() and (y[1] == 0).all()


@pytest.mark.parametrize("T,K,cols,E", SHAPES)
@pytest.mark.parametrize("rt,yt,weighted", [(BF, BF, True), (F, F, False), (BF, F, True), (F, BF, True)])
@pytest.mark.parametrize("drop,pad", [(0.0, 0), (0.4, 3)])
def test_collect_grad(T, K, cols, E, rt, yt, weighted, drop, pad):
    gen = _gen(T, K, cols, 3)
    inv, rows = picks(T, K, E, gen, drop), pitched((T * K, cols), rt, pad, gen=gen)
    dy, w = pitched((T, cols), yt, pad, gen=gen), torch.rand(T, K, generator=gen) if weighted else None
    drows, dw = pitched((T * K, cols), rt, pad, fill=2.0), torch.empty(T, K, device="cuda")
    wc = None if w is None else w.cuda()
    q.moe_collect_grad(dy, inv.cuda(), drows=drows, weights=wc, rows=rows, dweights=dw)
    want, dww, mag = ref.collect_grad(f64(dy), inv.numpy(), f64(rows), None if w is None else f64(w), np.full((T * K, cols), 2.0))
    close(drows, want, U * np.abs(want), rt, "drows")
    chain = cols / 64 + 16                       # products that one lane adds in turn, then lanes and waves
    close(dw, dww, chain * U * mag, F, "dweights")
    # each by itself, and the rows' gradient over the rows
    alone, dw2 = pitched((T * K, cols), rt, pad, fill=2.0), torch.empty(T, K, device="cuda")
    q.moe_collect_grad(dy, inv.cuda(), drows=alone, weights=wc)
    q.moe_collect_grad(dy, inv.cuda(), weights=wc, rows=rows, dweights=dw2)
    assert torch.equal(alone, drows) and torch.equal(dw2, dw)
    on = torch.zeros(T * K, dtype=torch.bool)
    on[inv[inv >= 0].long()] = True
    keep = rows.clone()
    q.moe_collect_grad(dy, inv.cuda(), drows=rows, weights=wc, rows=rows, dweights=dw2)
    assert torch.equal(rows[on], drows[on]) and torch.equal(dw2, dw) and torch.equal(rows[~on], keep[~on])


# ---- SwiGLU ----------------------------------------------------------------------------
SW = [(1, 1), (3, 7), (8, 2048), (5, 256), (33, 1001), (2, 65536), (6, 8200), (100, 40), (257, 33), (9, 4096), (7, 4104), (6, 1300), (3, 5001), (2, 9001), (2, 14001)]


@pytest.mark.parametrize("rows,cols", SW)
@pytest.mark.parametrize("gt,ot", [(BF, BF), (F, F), (BF, F), (F, BF)])
@pytest.mark.parametrize("pad,end", [(0, None), (3, 0.6)])
def test_swiglu(rows, cols, gt, ot, pad, end):
    gen = _gen(rows, cols)
    gu = pitched((rows, 2 * cols), gt, pad, gen=gen, scale=4.0)
    n = rows if end is None else int(rows * end)
    off = None if end is None else torch.tensor([0, n // 2, n], dtype=torch.int32, device="cuda")
    out = pitched((rows, cols), ot, pad, fill=3.0)
    q.moe_swiglu(gu, out, expert_offsets=off)
    g = f64(gu)
    want = np.concatenate([ref.swiglu(g[:n]), np.full((rows - n, cols), 3.0)])
    close(out, want, (silu_bound(g[:, :cols]) + 2 * U) * np.abs(want), ot)
    y32 = pitched((rows, cols), F, pad, fill=3.0)
    q.moe_swiglu(gu, y32, expert_offsets=off)
    codes = torch.full((rows, cols), 3.0, device="cuda").to(torch.float8_e4m3fn)
    sc = torch.full((rows,), 3.0, device="cuda")
    q.moe_swiglu(gu, codes, out_scale=sc, expert_offsets=off)
    _held(None, None, codes[:n], sc[:n], y32[:n])
    assert (codes[n:].float() == 3.0).all() and (sc[n:] == 3.0).all()
    mx, mxs = q.mxfp4_empty(rows, cols)
    mx.fill_(9), mxs.fill_(9)
    q.moe_swiglu(gu, mx, out_scale=mxs, expert_offsets=off)
    a, b = q.mxfp4_empty(rows, cols)
    q.moe_mxfp4_quantize(y32, a, b)
    assert torch.equal(mx[:n], a[:n]) and torch.equal(mxs[:n], b[:n]) and (mx[n:] == 9).all() and (mxs[n:] == 9).all()


@pytest.mark.parametrize("rows,cols", SW)
@pytest.mark.parametrize("gt,ht", [(BF, BF), (F, F), (BF, F), (F, BF)])
@pytest.mark.parametrize("pad,end", [(0, None), (3, 0.6)])
def test_swiglu_grad(rows, cols, gt, ht, pad, end):
    gen = _gen(rows, cols, 1)
    gu, dh = pitched((rows, 2 * cols), gt, pad, gen=gen, scale=4.0), pitched((rows, cols), ht, pad, gen=gen)
    n = rows if end is None else int(rows * end)
    off = None if end is None else torch.tensor([0, n // 2, n], dtype=torch.int32, device="cuda")
    dgu = pitched((rows, 2 * cols), gt, pad, fill=3.0)
    q.moe_swiglu_grad(gu, dh, dgu, expert_offsets=off)
    g = f64(gu)
    want, mag = ref.swiglu_grad(g[:n], f64(dh)[:n])
    tail = np.full((rows - n, 2 * cols), 3.0)
    rel = np.concatenate([silu_bound(g[:n, :cols])] * 2, 1) * 2 + 6 * U       # s and 1 - s
    close(dgu, np.concatenate([want, tail]), np.concatenate([rel * mag, tail * 0]), gt)
    keep = gu.clone()
    q.moe_swiglu_grad(gu, dh, gu, expert_offsets=off)
    assert torch.equal(gu[:n], dgu[:n]) and torch.equal(gu[n:], keep[n:])


def test_swiglu_gates_far_out():
    g = torch.tensor([0.0, -0.0, 88.0, -88.0, 200.0, -200.0, 1e38, -1e38, 3e38, float("inf"), float("nan"), 1e-30])
    gu = torch.cat([g, torch.full_like(g, 2.0)])[None].cuda()
    out, dgu = torch.empty(1, 12, device="cuda"), torch.empty(1, 24, device="cuda")
    q.moe_swiglu(gu, out)
    want = torch.nn.functional.silu(g.double()) * 2
    want[7:9] = torch.tensor([0.0, 6e38])
    out = out.cpu().double()[0]
    assert torch.equal(out[[0, 1, 4, 6, 7]], torch.tensor([0.0, 0.0, 400.0, 2 * float(g[6]), 0.0], dtype=torch.float64))
    assert torch.isinf(out[8]) and torch.isinf(out[9]) and torch.isnan(out[10])
    near = [2, 3, 5, 11]                          # e^-|g| below fp32's normal range may count as 0
    assert ((out[near] - want[near]).abs() <= 200 * U * want[near].abs() + 2.0 ** -126 * 2 * 200).all()
    q.moe_swiglu_grad(gu, torch.ones(1, 12, device="cuda"), dgu)
    d = dgu.cpu()[0]
    assert torch.equal(d[[0, 4, 6, 7]], torch.tensor([1.0, 2.0, 2.0, 0.0])) and torch.equal(d[12:][[0, 4, 7]], torch.tensor([0.0, 200.0, 0.0]))


@pytest.mark.parametrize("end", [0, 3, 5, 9, -4])
def test_rows_that_count(end):
    """The last offset is taken as it is, cut to the rows."""
    gu = torch.randn(5, 32, device="cuda")
    off = torch.tensor([0, 0, end], dtype=torch.int32, device="cuda")
    n = min(max(end, 0), 5)
    gu[n:] = float("nan")
    out, dgu = torch.full((5, 16), 2.0, device="cuda"), torch.full((5, 32), 2.0, device="cuda")
    q.moe_swiglu(gu, out, expert_offsets=off)
    q.moe_swiglu_grad(gu, torch.ones(5, 16, device="cuda"), dgu, expert_offsets=off)
    assert torch.isfinite(out).all() and (out[n:] == 2.0).all() and (dgu[n:] == 2.0).all() and (out[:n] != 2.0).all()


def test_swiglu_gradient_against_differences():
    gen = _gen(6)
    gu, dh = 2 * torch.randn(2, 26, generator=gen), torch.randn(2, 13, generator=gen)
    dgu = torch.empty(2, 26, device="cuda")
    q.moe_swiglu_grad(gu.cuda(), dh.cuda(), dgu)
    G, D, step = f64(gu), f64(dh), 1e-4
    for i in np.ndindex(G.shape):
        e = np.zeros_like(G)
        e[i] = step
        assert abs(((D * ref.swiglu(G + e)).sum() - (D * ref.swiglu(G - e)).sum()) / (2 * step) - float(dgu[i])) < 2e-5
