"""Row operators as a program uses them: many tokens and rows, offsets past 32
bits, streams, graphs, repeated runs, and all of them together as one block."""
import os
import sys

import numpy as np
import pytest
import torch

import quantized_moe_02_amd as q
import synth
from oracle import rows as ref
from row_cases import BF, F, U, close, f64, picks, pitched, silu_bound

pytestmark = pytest.mark.gpu
EPS = 1e-5
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.lib()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ---- every norm kernel with every pair of types ---------------------------------------
NARROW = [5, 24, 60, 100, 250, 500, 1000, 1500, 2040, 3100, 6100, 8100, 8201, 12300, 16385, 24600, 32800]


@pytest.mark.parametrize("cols", NARROW)
@pytest.mark.parametrize("xt,rt", [(F, BF), (BF, F), (F, F), (BF, BF)])
def test_norm_of_each_shape_and_type(cols, xt, rt):
    gen = _gen(cols)
    rows = 3
    x, r = pitched((rows, cols), xt, gen=gen), pitched((rows, cols), rt, gen=gen)
    w = (1 + 0.3 * torch.randn(cols, generator=gen)).to(BF).cuda()
    y, h = torch.empty(rows, cols, device="cuda"), torch.empty(rows, cols, device="cuda", dtype=rt)
    q.moe_rmsnorm(x, w, EPS, y=y, residual=r, h=h)
    assert torch.equal(h, (x.float() + r.float()).to(rt))
    want, _ = ref.rmsnorm(f64(h), f64(w), EPS)
    close(y, want, 3.01 * U * np.abs(want), F)
    dy, dx, dw = pitched((rows, cols), xt, gen=gen), torch.empty_like(h), torch.empty(cols, device="cuda")
    q.moe_rmsnorm_grad(dy, h, w, EPS, dx, dh=r, dweight=dw)
    want = ref.rmsnorm_grad(f64(dy), f64(h), f64(w), EPS, f64(r))
    close(dx, want[0], 8 * U * want[2], rt)
    close(dw, want[1], (rows + 8) * U * want[3], F)
    # types that have no kernel of their own
    dx = torch.empty(rows, cols, device="cuda", dtype=xt)
    q.moe_rmsnorm_grad(dy, h, w.float(), EPS, dx)
    want = ref.rmsnorm_grad(f64(dy), f64(h), f64(w), EPS)
    close(dx, want[0], 8 * U * want[2], xt)


@pytest.mark.parametrize("cols", [64, 192, 320, 960, 1984, 4032, 8128, 16320, 32704, 40000])
def test_large_inputs_give_the_bits_of_small_ones(cols):
    """Large bf16 inputs are read past the caches; no value of a row depends on it."""
    gen = torch.Generator(device="cuda").manual_seed(cols)
    rows = (100 << 20) // (2 * cols) // 32 * 32
    step = rows // 4
    x, r = (torch.randn(rows, cols, generator=gen, device="cuda").to(BF) for _ in range(2))
    w = (1 + 0.3 * torch.randn(cols, generator=gen, device="cuda")).to(BF)

    def quarters(call, *mats):
        """The outputs of one call, and of four calls over quarters of the rows."""
        one, four = ([torch.zeros_like(m) for m in mats] for _ in range(2))
        call(slice(0, rows), *one)
        for i in range(0, rows, step):
            call(slice(i, i + step), *(m[i:i + step] for m in four))
        for a, b in zip(one, four):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))

    quarters(lambda at, y, h: q.moe_rmsnorm(x[at], w, EPS, y=y, residual=r[at], h=h), x, x)
    quarters(lambda at, c, s: q.moe_rmsnorm(x[at], w, EPS, q=c, q_scale=s),
           torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(rows, device="cuda"))
    quarters(lambda at, dx: q.moe_rmsnorm_grad(r[at], x[at], w, EPS, dx, dh=r[at]), x)
    dw, part = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    dx, total, size = torch.empty_like(x), torch.zeros(cols, device="cuda", dtype=torch.float64), torch.zeros(cols, device="cuda", dtype=torch.float64)
    q.moe_rmsnorm_grad(r, x, w, EPS, dx, dweight=dw)
    for i in range(0, rows, step):
        q.moe_rmsnorm_grad(r[i:i + step], x[i:i + step], w, EPS, dx[i:i + step], dweight=part)
        total += part
        n = x[i:i + step].double() / (x[i:i + step].double().square().mean(1, keepdim=True) + EPS).sqrt()
        size += (r[i:i + step].double() * n).abs().sum(0)
    # at most (rows of a part + 8) roundings either way
    assert ((dw.double() - total).abs() <= 2 * (-(-rows // 256) + 8) * U * size + 1e-30).all()
    if cols % 128 == 0:
        half = cols // 2
        quarters(lambda at, o: q.moe_swiglu(x[at], o), r[:, :half].contiguous())
        quarters(lambda at, c, s: q.moe_swiglu(x[at], c, s),
               torch.empty(rows, half, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(rows, device="cuda"))
        quarters(lambda at, d: q.moe_swiglu_grad(x[at], r[at, :half], d), x)
    else:
        quarters(lambda at, o: q.moe_swiglu(torch.cat([x[at], r[at]], 1), o), x)
    K = 4
    T = rows // K
    inv = torch.randperm(rows, generator=gen, device="cuda").reshape(T, K).to(torch.int32)
    weights = torch.rand(T, K, generator=gen, device="cuda")
    one, four, dws, dws4 = torch.empty(T, cols, dtype=BF, device="cuda"), torch.empty(T, cols, dtype=BF, device="cuda"), torch.empty_like(weights), torch.empty_like(weights)
    d, d4 = torch.empty_like(x), torch.empty_like(x)
    q.moe_collect(x, inv, one, weights)
    q.moe_collect_grad(r[:T], inv, d, weights, rows=x, dweights=dws)
    for i in range(0, T, T // 4):
        at = slice(i, i + T // 4)
        q.moe_collect(x, inv[at], four[at], weights[at])
        q.moe_collect_grad(r[at], inv[at], d4, weights[at], rows=x, dweights=dws4[at])
    assert torch.equal(one, four) and torch.equal(d, d4) and torch.equal(dws, dws4)


# ---- many tokens: a workgroup takes a token's picks, not one of them -----------------------
@pytest.mark.parametrize("T,K,cols", [(16400, 3, 30), (8200, 5, 100), (2100, 9, 300), (2050, 16, 513), (600, 6, 2050), (520, 16, 1600),
                                      (16400, 2, 5), (2100, 4, 200)])
@pytest.mark.parametrize("rt,yt", [(BF, BF), (F, F), (BF, F)])
def test_collect_of_many_tokens(T, K, cols, rt, yt):
    gen = _gen(T + cols)
    inv = picks(T, K, 16, gen, 0.2)
    rows, dy = pitched((T * K, cols), rt, gen=gen), pitched((T, cols), yt, gen=gen)
    w = torch.rand(T, K, generator=gen).cuda()
    drows, dw, y = torch.full_like(rows, 2.0), torch.empty(T, K, device="cuda"), torch.empty(T, cols, device="cuda", dtype=yt)
    iv = inv.cuda()
    q.moe_collect(rows, iv, y, weights=w)
    q.moe_collect_grad(dy, iv, drows=drows, weights=w, rows=rows, dweights=dw)
    on, at = inv >= 0, inv.clamp(min=0).long()
    R, D, W = rows.double().cpu(), dy.double().cpu(), w.double().cpu() * on
    want, mag = torch.zeros(T, cols, dtype=torch.float64), torch.zeros(T, cols, dtype=torch.float64)
    wdw, wmag = torch.zeros(T, K, dtype=torch.float64), torch.zeros(T, K, dtype=torch.float64)
    wrows = torch.full((T * K, cols), 2.0, dtype=torch.float64)
    for i in range(K):
        picked = R[at[:, i]]
        want += W[:, i, None] * picked
        mag += (W[:, i, None] * picked).abs()
        wdw[:, i], wmag[:, i] = (D * picked).sum(1) * on[:, i], (D * picked).abs().sum(1)
        wrows[at[on[:, i], i]] = (W[:, i, None] * D)[on[:, i]]
    close(y, want.numpy(), (K + 2) * U * mag.numpy(), yt, "y")
    close(drows, wrows.numpy(), U * wrows.abs().numpy(), rt, "drows")
    close(dw, wdw.numpy(), (cols / 64 + 16) * U * wmag.numpy(), F, "dweights")
    # over the rows themselves
    keep = rows.clone()
    dw2 = torch.empty_like(dw)
    q.moe_collect_grad(dy, iv, drows=rows, weights=w, rows=rows, dweights=dw2)
    taken = torch.zeros(T * K, dtype=torch.bool)
    taken[at[on]] = True
    assert torch.equal(dw2, dw) and torch.equal(rows[taken], drows[taken]) and torch.equal(rows[~taken], keep[~taken])


# ---- large ---------------------------------------------------------------------------------
def test_offsets_past_32_bits():
    """Rows 2^23 values apart: the last ones lie past 2^32 of them."""
    pitch, n, cols = 1 << 23, 521, 1001
    buf = torch.empty((n - 1) * pitch + 2 * cols, dtype=BF, device="cuda")
    far = lambda c: buf.as_strided((n, c), (pitch, 1))
    gen = torch.Generator(device="cuda").manual_seed(1)
    near = torch.randn(n, 2 * cols, generator=gen, device="cuda").to(BF)
    w = torch.ones(cols, device="cuda")
    a = lambda c=cols: near[:, :c].contiguous()
    inv = torch.arange(n, dtype=torch.int32, device="cuda").flip(0)[:, None].contiguous()

    y = [torch.empty(n, cols, dtype=BF, device="cuda") for _ in range(4)]
    far(cols).copy_(a())
    q.moe_rmsnorm(far(cols), w, EPS, y=y[0])
    q.moe_rmsnorm(a(), w, EPS, y=y[1])
    assert torch.equal(y[0], y[1])
    q.moe_rmsnorm_grad(far(cols), far(cols), w, EPS, y[2], dh=far(cols))
    q.moe_rmsnorm_grad(a(), a(), w, EPS, y[3], dh=a())
    assert torch.equal(y[2], y[3])
    q.moe_rmsnorm(a(), w, EPS, y=far(cols))
    assert torch.equal(far(cols), y[1])
    q.moe_dispatch(a(), inv, far(cols))
    assert torch.equal(far(cols), a().flip(0))
    q.moe_collect(far(cols), inv, y[0])
    assert torch.equal(y[0], a())
    dw = [torch.empty(n, 1, device="cuda") for _ in range(2)]
    q.moe_collect_grad(a(), inv, rows=far(cols), dweights=dw[0])
    q.moe_collect_grad(a(), inv, rows=a().flip(0).contiguous(), dweights=dw[1])
    assert torch.equal(dw[0], dw[1])
    far(2 * cols).copy_(near)
    q.moe_swiglu(far(2 * cols), y[0])
    q.moe_swiglu(near, y[1])
    assert torch.equal(y[0], y[1])
    d = torch.empty_like(near)
    q.moe_swiglu_grad(near, a(), d)
    q.moe_swiglu_grad(far(2 * cols), a(), far(2 * cols))
    assert torch.equal(far(2 * cols), d)


def test_calls_of_several_launches():
    """More work items than one launch takes."""
    T, cols = 131074, 65536                                  # 2^31 and more over chunks of 16 bytes
    x, rows = torch.empty(T, cols, device="cuda"), torch.empty(T, cols, device="cuda")
    at = [0, 1, 131070, 131071, 131072, 131073]
    for i in at:
        x[i] = float(i)
    inv = torch.arange(T, dtype=torch.int32, device="cuda")[:, None].contiguous()
    q.moe_dispatch(x, inv, rows)
    for i in at:
        assert (rows[i] == float(i)).all()
    del x, rows, inv
    torch.cuda.empty_cache()
    R, cols = (1 << 21) + 3, 8200                            # 1024 lanes a row
    x, y = torch.empty(R, cols, dtype=BF, device="cuda"), torch.zeros(R, cols, dtype=BF, device="cuda")
    at = [0, (1 << 21) - 1, 1 << 21, R - 1]
    for i in at:
        x[i] = 3.0
    q.moe_rmsnorm(x, torch.ones(cols, device="cuda"), EPS, y=y)
    for i in at:
        assert (y[i] == 1.0).all()
    del x, y
    torch.cuda.empty_cache()


# ---- streams, graphs, repeats ----------------------------------------------------------------
class Step:
    """One pass through every operator on buffers of its own."""

    def __init__(self, seed, T=37, K=3, H=264, I=136):
        gen = torch.Generator().manual_seed(seed)
        n = lambda *s, dt=BF: torch.randn(*s, generator=gen).to(dt).cuda()
        e = lambda *s, dt=BF: torch.zeros(*s, dtype=dt, device="cuda")
        self.x, self.r, self.w = n(T, H), n(T, H), n(H, dt=F)
        self.inv, self.tw = picks(T, K, 8, gen, 0.1).cuda(), torch.rand(T, K, generator=gen).cuda()
        self.h, self.y, self.q, self.s = e(T, H), e(T, H), torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda"), e(T, dt=F)
        self.rows, self.qr = e(T * K, H), e(T * K, H, dt=torch.uint8).view(torch.float8_e4m3fn)
        self.sr, self.act = e(T * K, dt=F), e(T * K, H // 2)
        self.z, self.drows, self.dtw = e(T, H, dt=F), e(T * K, H), e(T, K, dt=F)
        self.dgu, self.dx, self.dw = e(T * K, H), e(T, H), e(H, dt=F)
        self.ws = q.rmsnorm_workspace(T, H)

    def outputs(self):
        return [self.h, self.y, self.q.view(torch.uint8), self.s, self.rows, self.qr.view(torch.uint8), self.sr, self.act, self.z,
                self.drows, self.dtw, self.dgu, self.dx, self.dw]

    def run(self, stream=None, ws=True):
        k = dict(stream=stream)
        q.moe_rmsnorm(self.x, self.w, EPS, y=self.y, residual=self.r, h=self.h, q=self.q, q_scale=self.s, **k)
        q.moe_dispatch(self.y, self.inv, self.rows, **k)
        q.moe_dispatch(self.q, self.inv, self.qr, x_scale=self.s, row_scale=self.sr, **k)
        q.moe_swiglu(self.rows, self.act, **k)
        q.moe_collect(self.rows, self.inv, self.z, weights=self.tw, addend=self.y, **k)
        q.moe_collect_grad(self.z, self.inv, drows=self.drows, weights=self.tw, rows=self.rows, dweights=self.dtw, **k)
        q.moe_swiglu_grad(self.rows, self.act, self.dgu, **k)
        q.moe_rmsnorm_grad(self.z, self.h, self.w, EPS, self.dx, dh=self.y, dweight=self.dw, ws=self.ws if ws else None, **k)

    def clear(self):
        for o in self.outputs():
            o.zero_()

    def result(self):
        torch.cuda.synchronize()
        return [o.clone() for o in self.outputs()]


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_the_same_bits_every_time():
    s = Step(1)
    s.run()
    first = s.result()
    assert all(o.float().abs().sum() > 0 for o in first)
    for _ in range(3):
        s.clear()
        s.run(ws=False)
        assert _same(first, s.result())


def test_on_another_stream_and_two_at_once():
    a, b = Step(1), Step(2)
    a.run(), b.run()
    want = a.result(), b.result()
    a.clear(), b.clear()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a.run(stream=sa, ws=False)
        b.run(stream=sb, ws=False)
    assert _same(want[0], a.result()) and _same(want[1], b.result())
    with torch.cuda.stream(sa):                      # the current stream, when none is given
        a.clear()
        a.run()
    assert _same(want[0], a.result())


def test_graphs_that_share_a_workspace():
    a, b = Step(3), Step(4)
    b.ws = a.ws
    a.run(), b.run()
    want = a.result(), b.result()
    graphs = []
    for s in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    for turn in range(4):
        a.clear(), b.clear()
        graphs[turn % 2].replay()
        graphs[1 - turn % 2].replay()
        assert _same(want[0], a.result()) and _same(want[1], b.result())
        Step(5).run()                                # the program's own work between the replays
    a.x.mul_(2.0)                                    # new inputs in the captured buffers
    a.clear()
    a.run()
    want = a.result()
    a.clear()
    graphs[0].replay()
    assert _same(want, a.result())


def test_a_workspace_of_the_largest_call_serves_smaller_ones():
    ws = q.rmsnorm_workspace(700, 6144)
    for rows, cols in ((700, 6144), (513, 40), (1, 6144), (700, 33), (2, 1000)):
        gen = _gen(rows)
        dy, h, w = (torch.randn(rows, cols, generator=gen).cuda() for _ in range(2)), None, torch.ones(cols, device="cuda")
        dy, h = dy
        dx, dw = torch.empty_like(h), torch.empty(cols, device="cuda")
        q.moe_rmsnorm_grad(dy, h, w, EPS, dx, dweight=dw, ws=ws)
        want = ref.rmsnorm_grad(f64(dy), f64(h), np.ones(cols), EPS)
        close(dw, want[1], (rows / 256 + 12) * U * want[3], F)


# ---- together ------------------------------------------------------------------------------------
def _decoded(codes, scales):
    E, n, kb = codes.shape
    w = torch.empty(E * n, kb * 2, device="cuda")
    q.moe_mxfp4_dequantize(codes.view(E * n, kb), scales.view(E * n, -1), w)
    return w.view(E, n, kb * 2).double().cpu()


@pytest.mark.parametrize("T", [1, 9, 70])
def test_block_against_torch(T):
    """Norm, router, experts, sum and balance loss, all gradients, against float64
    autograd over the decoded weights (the picks as the kernels took them)."""
    import mxfp4_moe_step as ex
    geom = synth.WORKLOADS["tiny"]["geom"]
    H, I, E, k = geom["hidden"], geom["moe_inter"], geom["n_routed_experts"], geom["top_k"]
    layer = ex.make_layer(geom, seed=T, score_coef=0.5)
    gen = torch.Generator().manual_seed(T)
    x, r = torch.randn(T, H, generator=gen).to(BF), torch.randn(T, H, generator=gen).to(BF)
    nw = 1 + 0.2 * torch.randn(H, generator=gen)
    dy, dh = torch.randn(T, H, generator=gen), torch.randn(T, H, generator=gen).to(BF)
    block = ex.NormMoEBlock(layer, nw.cuda())
    y, h, loss = block.forward(x.cuda(), r.cuda())
    dx, dw, d_router = block.backward(dy.cuda(), dh.cuda())

    ids = layer.saved[1].cpu().long()
    gate_up, down = _decoded(*layer.gate_up), _decoded(*layer.down)
    hr = h.double().cpu().requires_grad_(True)
    w, rw = nw.double().requires_grad_(True), layer.router_w.double().cpu().requires_grad_(True)
    n = hr * torch.rsqrt(hr.square().mean(1, keepdim=True) + 1e-6) * w
    s = torch.sigmoid(n @ rw.T)
    at = s.gather(1, ids)
    tw = geom["routed_scaling_factor"] * at / at.sum(1, keepdim=True)
    out = []
    for t in range(T):
        acc = torch.zeros(H, dtype=torch.float64)
        for j in range(k):
            g = gate_up[ids[t, j]] @ n[t]
            acc = acc + tw[t, j] * (down[ids[t, j]] @ (torch.nn.functional.silu(g[:I]) * g[I:]))
        out.append(acc)
    out = torch.stack(out)
    p = s / s.sum(1, keepdim=True)
    c = torch.bincount(ids.reshape(-1), minlength=E).double()
    bal = 0.5 * (E * c / c.sum() * p.mean(0)).sum()
    ((out * dy.double()).sum() + (hr * dh.double()).sum() + bal).backward()

    assert torch.equal(h.cpu(), (x.float() + r.float()).to(BF))
    rel = lambda got, want: float((got.double().cpu() - want).norm() / want.norm())
    # roundings to bf16 (2^-8 each): n, h of the experts, their rows; and on the way back the
    # rows' gradient, the gate's and up's, dx.  Norm-wise, so each counts at most once
    assert rel(y, out.detach()) <= 3 * 2 ** -8
    assert abs(loss.item() - bal.item()) <= 2 ** -8 * bal.item()
    assert rel(dx, hr.grad) <= 6 * 2 ** -8
    assert rel(dw, w.grad) <= 6 * 2 ** -8
    assert rel(d_router, rw.grad) <= 8 * 2 ** -8           # through products of two rounded rows


def test_example_runs(capsys):
    import mxfp4_moe_step as ex
    ex.main()
    assert "block behind its norm" in capsys.readouterr().out
