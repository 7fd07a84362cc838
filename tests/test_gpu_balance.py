"""The router's balance loss, counts and gradient on the GPU against the
float64 oracle.

Counts have to be equal.  With u = 2^-24 and L the largest finite |logit|, a
share's exponent a - m is off by a few u of its magnitude (2 L and the log's own
rounding) and the exponentials, the sum over 256 experts and the division by a
few u each, so a share is off by at most (4 L + 40) u of itself; a chunk's sum of
shares adds at most 64 u.  The gradient's f - sum f p carries the same error of
both parts, relative to f + sum f p."""
import numpy as np
import pytest
import torch

import quantized_moe_02_amd as q
from oracle import operators as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.lib()


def _call(x, ids, seq, coef, score, dloss=None, seq_arg=True):
    T, E = x.shape
    S = len(seq) - 1
    xd, idd = x.cuda(), ids.cuda()
    sd = torch.tensor(seq, dtype=torch.int32, device="cuda") if seq_arg else None
    counts = torch.full((S, E), -7, dtype=torch.int32, device="cuda")
    tokens = torch.full((S,), -7, dtype=torch.int32, device="cuda")
    loss = torch.full((1,), 9.0, device="cuda")
    dl = torch.full((T, E), 9.0, dtype=x.dtype, device="cuda")
    ws = q.balance_workspace(T, E, S)
    ws.fill_(0xFF)
    q.moe_balance_loss(xd, idd, counts, tokens, loss, coef=coef, score=score, seq_offsets=sd, ws=ws)
    g = None if dloss is None else torch.tensor([dloss], device="cuda")
    q.moe_balance_loss_grad(xd, idd, counts, tokens, dl, coef=coef, score=score, seq_offsets=sd, dloss=g)
    torch.cuda.synchronize()
    return counts, tokens, loss, dl


def _check(x, ids, seq, coef, score, dloss=None, seq_arg=True):
    counts, tokens, loss, dl = _call(x, ids, seq, coef, score, dloss, seq_arg)
    x64 = x.double().numpy()
    rl, rc, rt, rg = ref.balance(x64, ids.numpy(), seq, coef, score, 1.0 if dloss is None else dloss)
    assert np.array_equal(counts.cpu().numpy(), rc)
    assert np.array_equal(tokens.cpu().numpy(), rt)
    fin = x64[np.isfinite(x64)]
    rel = (4 * (np.abs(fin).max() if fin.size else 0) + 40) * U
    assert abs(loss.item() - rl) <= (rel + 64 * U) * abs(rl)
    T, E = x.shape
    s_of = np.searchsorted(np.asarray(seq)[1:], np.arange(T), side="right")
    f = E * rc / np.maximum(rc.sum(1, keepdims=True), 1)
    ok = ((ids.numpy() >= 0) & (ids.numpy() < E)).any(1)
    p = np.zeros((T, E))
    p[ok] = ref.shares(x64[ok], score)
    ft = f[s_of] if T else np.zeros((0, E))
    dot = (ft * p).sum(1, keepdims=True)
    n = np.maximum(rt, 1)[s_of][:, None] if T else np.ones((0, 1))
    scale = abs(coef * (1.0 if dloss is None else dloss)) / (len(seq) - 1) / n
    with np.errstate(invalid="ignore"):
        tol = 4 * rel * scale * p * (ft + dot) + 1e-38
    got = dl.double().cpu().numpy()
    lo, hi = rg - tol, rg + tol
    if x.dtype == torch.bfloat16:       # the rounding of a value in [lo, hi]
        lo, hi = (torch.from_numpy(v).float().to(torch.bfloat16).double().numpy() for v in (lo, hi))
    bad = ~((lo <= got) & (got <= hi))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], rg[bad][:4])
    assert (got[~ok] == 0).all()


def _inputs(T, E, k, seed, dtype="f32", pad=0.0, drop=0.0, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, E, generator=g) * spread).to(DT[dtype])
    ids = (x.float() + torch.randn(T, E, generator=g)).topk(k, dim=1).indices.to(torch.int32)
    ids[torch.rand(T, k, generator=g) < drop] = -1
    ids[torch.rand(T, generator=g) < pad] = -1
    return x, ids


def _seqs(T, S, seed):
    cuts = np.sort(np.random.default_rng(seed).integers(0, T + 1, S - 1)).tolist()
    return [0] + cuts + [T]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k,S,pad,drop", [
    (1, 1, 1, 1, 0, 0), (1, 256, 8, 1, 0, 0), (3, 2, 1, 2, 0, 0), (37, 16, 4, 1, 0, 0), (64, 64, 8, 5, .2, .1),
    (65, 63, 3, 3, 0, .3), (200, 100, 16, 7, .5, 0), (513, 256, 8, 40, .1, .1), (1000, 255, 2, 1, .1, 0),
    (777, 8, 2, 300, .1, .1), (5000, 128, 8, 9, .1, 0), (130, 65, 4, 4, 1.0, 0), (300, 160, 6, 2, 0, 0)])
def test_against_oracle(T, E, k, S, pad, drop, dtype, score):
    x, ids = _inputs(T, E, k, T + E, dtype, pad, drop)
    _check(x, ids, _seqs(T, S, T), 1e-3, score)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_many_chunks(score):
    """More tokens than the smallest chunks cover, sequences of 0, 1 and most."""
    T = 70001
    x, ids = _inputs(T, 32, 2, 5, "f32", 0.1)
    _check(x, ids, [0, 0, 1, 60000, 60000, T - 1, T], 0.01, score)


def test_no_offsets_is_one_sequence():
    x, ids = _inputs(150, 48, 4, 1)
    _check(x, ids, [0, 150], 0.5, "sigmoid", seq_arg=False)


def test_upstream_gradient_scales():
    x, ids = _inputs(150, 48, 4, 1)
    _check(x, ids, [0, 100, 150], 0.5, "softmax", dloss=-3.5)


def test_coefficient_zero():
    x, ids = _inputs(20, 8, 2, 1)
    _, _, loss, dl = _call(x, ids, [0, 20], 0.0, "sigmoid")
    assert loss.item() == 0 and (dl == 0).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_no_tokens(score):
    x, ids = torch.empty(0, 16), torch.empty(0, 4, dtype=torch.int32)
    counts, tokens, loss, _ = _call(x, ids, [0, 0, 0], 1.0, score)
    assert (counts == 0).all() and (tokens == 0).all() and loss.item() == 0


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_padding_may_hold_anything(score):
    """Tokens without a pick: their logits are not used, their gradient is 0."""
    x, ids = _inputs(90, 70, 3, 2)
    ids[10], ids[50:60] = -1, 70            # 70: not an expert
    x[10], x[50:60] = float("nan"), float("inf")
    seq = [0, 50, 60, 90]                   # the middle sequence is padding only
    counts, tokens, loss, dl = _call(x, ids, seq, 1e-2, score)
    keep = torch.ones(90, dtype=torch.bool)
    keep[10], keep[50:60] = False, False
    clean = torch.where(keep[:, None], x, 0.0)
    rl, rc, rt, rg = ref.balance(clean.double().numpy(), ids.numpy(), seq, 1e-2, score)
    assert np.array_equal(counts.cpu().numpy(), rc) and rt[1] == 0 and np.array_equal(tokens.cpu().numpy(), rt)
    assert abs(loss.item() - rl) <= 200 * U * rl
    assert (dl.cpu()[~keep] == 0).all() and torch.isfinite(dl).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_masked_experts_and_large_logits(score):
    """Experts at -inf have share and gradient 0; logits of +-90 and sigmoids
    that all underflow are no special case; a NaN stays in its token's row."""
    x, ids = _inputs(40, 24, 2, 3, spread=5.0)
    x[:, 20:] = -float("inf")
    x[3] = x[3] * 0 - 200.0 if score == "softmax" else x[3].clamp(min=-20) - 200.0
    x[5, 2], x[5, 4] = 90.0, -90.0
    x[3, 20:] = -float("inf")
    ids.clamp_(max=19)
    _check(x, ids, [0, 40], 1.0, score)
    x[7, 1] = float("nan")
    _, _, loss, dl = _call(x, ids, [0, 40], 1.0, score)
    assert np.isnan(loss.item()) and torch.isnan(dl[7]).all()
    dl[7] = 0
    assert torch.isfinite(dl).all()
    x[7, 1] = float("inf")
    _, _, loss, dl = _call(x, ids, [0, 40], 1.0, score)
    if score == "softmax":
        assert np.isnan(loss.item()) and torch.isnan(dl[7]).all()
    else:
        assert np.isfinite(loss.item()) and torch.isfinite(dl).all()     # sigmoid(+inf) = 1
    x[7] = -float("inf")
    _, _, loss, dl = _call(x, ids, [0, 40], 1.0, score)
    assert np.isnan(loss.item()) and torch.isnan(dl[7]).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_gradient_against_differences(score):
    """Central differences of the loss kernel over steps of 1/4: the loss is
    smooth on the scale of 1, its third derivative along a logit at most
    coef / n, so they miss by at most h^2 / 6 of that, beside the loss's own
    float32 rounding (64 + 60 u of it, twice, over 2 h)."""
    x, ids = _inputs(6, 10, 2, 8, spread=1.0)
    coef, h = 4.0, 0.25
    _, _, _, dl = _call(x, ids, [0, 6], coef, score)
    dl = dl.cpu()
    for t in (0, 3, 5):
        for e in (0, 4, 9):
            ls = []
            for d in (h, -h):
                y = x.clone()
                y[t, e] += d
                ls.append((_call(y, ids, [0, 6], coef, score)[2].item(), float(y[t, e])))
            diff = (ls[0][0] - ls[1][0]) / (ls[0][1] - ls[1][1])
            f_max = 10.0      # f <= E / 1: an expert picked by all
            tol = h * h / 6 * coef / 6 * f_max + 2 * 124 * U * coef * f_max / (2 * h)
            assert abs(diff - dl[t, e].item()) <= tol


def test_repeats_bit_for_bit_and_in_a_graph():
    x, ids = _inputs(3000, 256, 8, 6, pad=0.1)
    seq = _seqs(3000, 20, 1)
    a = _call(x, ids, seq, 1e-3, "sigmoid")
    for _ in range(3):
        assert all(torch.equal(u, v) for u, v in zip(a, _call(x, ids, seq, 1e-3, "sigmoid")))
    xd, idd = x.cuda(), ids.cuda()
    sd = torch.tensor(seq, dtype=torch.int32, device="cuda")
    out = [torch.empty_like(t) for t in a]
    ws = q.balance_workspace(3000, 256, 20)

    def step():
        q.moe_balance_loss(xd, idd, out[0], out[1], out[2], coef=1e-3, seq_offsets=sd, ws=ws)
        q.moe_balance_loss_grad(xd, idd, out[0], out[1], out[3], coef=1e-3, seq_offsets=sd)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        xd.copy_(torch.randn(3000, 256, generator=torch.Generator().manual_seed(i)))
        step()
        want = [t.clone() for t in out]
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(want, out)), i


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,S", [(60, 16, 4, 4), (64, 130, 8, 4), (128, 64, 8, 2), (100, 40, 2, 4), (40, 33, 3, 60),
                                     (300, 256, 8, 90), (1500, 12, 2, 47)])
def test_short_sequences(T, E, k, S, score):
    """One workgroup, small chunks, sequences without a token."""
    x, ids = _inputs(T, E, k, T + S, "f32", 0.1, 0.1)
    _check(x, ids, _seqs(T, S, S), 1e-3, score)
