"""The norm's gradient captured into graphs without a workspace of the caller's: each
graph keeps the one that the call took."""
import pytest
import torch

import quantized_moe_02_amd as q

pytestmark = pytest.mark.gpu
EPS = 1e-5


class Call:
    def __init__(self, seed, rows, cols):
        gen = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=gen).cuda()
        self.dy, self.h, self.w = n(rows, cols), n(rows, cols), n(cols)
        self.dx, self.dw = torch.zeros(rows, cols, device="cuda"), torch.zeros(cols, device="cuda")

    def run(self, stream=None):
        q.moe_rmsnorm_grad(self.dy, self.h, self.w, EPS, self.dx, dweight=self.dw, stream=stream)

    def result(self):
        torch.cuda.synchronize()
        return self.dx.clone(), self.dw.clone()


@pytest.mark.parametrize("rows,cols", [(700, 600), (1300, 2056), (40, 20000), (2000, 17000)])
@pytest.mark.parametrize("named", [False, True])
def test_captured_without_a_workspace(rows, cols, named):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    calls, graphs, want = [Call(s, rows, cols) for s in (1, 2)], [], []
    for c in calls:
        c.run()
        want.append(c.result())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(stream=torch.cuda.current_stream() if named else None)
            torch.empty(1 << 22, device="cuda").fill_(float("nan"))       # takes what the call gave back
        graphs.append(g)
    for turn in range(4):
        for c in calls:
            c.dx.zero_(), c.dw.zero_()
        graphs[turn % 2].replay(), graphs[1 - turn % 2].replay()
        for c, w in zip(calls, want):
            assert all(torch.equal(a, b) for a, b in zip(c.result(), w))
        Call(3, 900, 1000).run()                                          # the program's own work between the replays
        torch.full((1 << 22,), float("nan"), device="cuda")
