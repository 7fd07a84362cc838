"""Further forms of the router's balance loss on the GPU against the float64
oracle (bounds as in test_gpu_balance.py)."""
import numpy as np
import pytest
import torch

import quantized_moe_02_amd as q
from oracle import operators as ref
from test_gpu_balance import U, _call, _check, _inputs, _seqs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.lib()


def test_one_workspace_for_every_smaller_batch():
    """Sized once, used by batches of fewer tokens and sequences that cut
    them into more chunks."""
    ws = q.balance_workspace(600, 40, 48)
    for T, S in ((600, 48), (575, 48), (576, 48), (300, 20), (100, 3), (129, 48), (1, 1)):
        x, ids = _inputs(T, 40, 4, T, "f32", 0.1, 0.1)
        seq = _seqs(T, S, T)
        ws.fill_(0xFF)
        counts = torch.full((S, 40), -7, dtype=torch.int32, device="cuda")
        tokens = torch.full((S,), -7, dtype=torch.int32, device="cuda")
        loss = torch.full((1,), 9.0, device="cuda")
        q.moe_balance_loss(x.cuda(), ids.cuda(), counts, tokens, loss, coef=0.5,
                           seq_offsets=torch.tensor(seq, dtype=torch.int32, device="cuda"), ws=ws)
        rl, rc, rt, _ = ref.balance(x.double().numpy(), ids.numpy(), seq, 0.5, "sigmoid")
        assert np.array_equal(counts.cpu().numpy(), rc) and np.array_equal(tokens.cpu().numpy(), rt)
        assert abs(loss.item() - rl) <= (4 * x.abs().max().item() + 104) * U * rl


@pytest.mark.parametrize("graph", [False, True])
def test_a_workspace_of_its_own(graph):
    """Without one the call takes a workspace from torch's allocator, of its
    own stream's memory: what other streams are done with does not reach it."""
    T, E, S = 3000, 256, 20
    x, ids = _inputs(T, E, 8, 6, pad=0.1)
    xd, idd, seq = x.cuda(), ids.cuda(), torch.tensor(_seqs(T, S, 1), dtype=torch.int32, device="cuda")
    out = lambda: (torch.empty(S, E, dtype=torch.int32, device="cuda"), torch.empty(S, dtype=torch.int32, device="cuda"),
                   torch.empty(1, device="cuda"))
    want = out()
    q.moe_balance_loss(xd, idd, *want, coef=1e-3, seq_offsets=seq, ws=q.balance_workspace(T, E, S))
    torch.cuda.synchronize()
    if graph:
        got, g = out(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q.moe_balance_loss(xd, idd, *got, coef=1e-3, seq_offsets=seq)
        for _ in range(3):
            for t in got:
                t.zero_()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(u, v) for u, v in zip(want, got))
        return
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        res = [out() for _ in range(4)]
        torch.cuda.synchronize()
        for r in res:
            q.moe_balance_loss(xd, idd, *r, coef=1e-3, seq_offsets=seq, stream=stream)
            q.balance_workspace(T, E, S).fill_(0xFF)        # freed at once, on the current stream
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for r in res for u, v in zip(want, r))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_every_gradient_against_differences(score):
    """Central differences of the loss kernel along every logit, beside a bound
    that a wrong gradient does not meet.  Along l_j a token's part of the loss
    has the slope m' = p (f_j - m) d, with p_j, m = sum f p and d = 1 (softmax) or
    sigmoid(-l_j).  For the softmax m''' = m' (1 - 6 p + 6 p^2); for the sigmoid
    m'' = m' c, c = (1 - 2 p) d - (1 - d) in [-1, 1], |c'| <= 1/2, so in either
    case |m'''| <= 3/2 |m'|, and m' grows by e^h at most over a step.  The
    difference misses the slope by h^2 / 6 of that: h^2 e^h / 4 of the slope
    itself, beside the loss's own rounding over h."""
    T, E, coef, h = 3, 8, 4.0, 0.25
    x, ids = _inputs(T, E, 2, 8, spread=1.0)
    _, _, _, dl = _call(x, ids, [0, T], coef, score)
    dl = dl.double().cpu().numpy()
    loss_err = (4 * (x.abs().max().item() + h) + 104) * U
    for t in range(T):
        for e in range(E):
            ls = []
            for d in (h, -h):
                y = x.clone()
                y[t, e] += d
                ls.append((_call(y, ids, [0, T], coef, score)[2].item(), float(y[t, e])))
            diff = (ls[0][0] - ls[1][0]) / (ls[0][1] - ls[1][1])
            slope = dl[t, e]
            tol = h * h * np.exp(h) / 4 * abs(slope) + loss_err * max(ls[0][0], ls[1][0]) / h
            assert tol < abs(slope) / 4, (t, e)          # the bound says something
            assert abs(diff - slope) <= tol, (t, e, diff, slope)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,S", [(90, 2), (300, 3)])       # one workgroup, and three launches
@pytest.mark.parametrize("E", [3, 4, 13, 16, 18, 32, 61, 64, 67, 128, 129, 254, 256])
def test_every_kernel(E, T, S, dtype, score):
    """4 to 64 lanes to a token, rows loaded whole and one by one."""
    x, ids = _inputs(T, E, min(E, 3), T + E, dtype, 0.1, 0.1)
    _check(x, ids, _seqs(T, S, T + E), 1e-2, score)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_very_many_sequences(score):
    """Most of one token or none, and hundreds of empty ones in the middle of a
    chunk of tokens."""
    x, ids = _inputs(3000, 20, 3, 1, "f32", 0.1, 0.1)
    _check(x, ids, _seqs(3000, 4000, 2), 0.3, score)
    x, ids = _inputs(700, 20, 3, 2, "f32", 0.1, 0.1)
    _check(x, ids, [0] * 300 + [501] * 700 + [700] * 3, 0.3, score)
