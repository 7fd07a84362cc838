"""Row operators whose kernels take 1024 lanes a row, over more rows than one launch
takes: the rows of the second launch are the right ones.  (That these sizes take
two launches is checked without a GPU, test_row_launch_cases.py.)"""
import pytest
import torch

import quantized_moe_02_amd as q
from launch_cases import CASES, LAUNCH_ROWS

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("op,cols,to", CASES)
def test_calls_of_several_launches(op, cols, to):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rows = LAUNCH_ROWS + 3
    width = cols * (2 if op == "swiglu" else 1)
    coded = {"bf16": 2 * cols, "e4m3": cols, "mxfp4": 17 * (-(-cols // 32))}[to]
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < rows * (2 * width + coded) + (4 << 30):
        pytest.skip("needs %d GB of free GPU memory" % (rows * (2 * width + coded) >> 30))
    at = [0, 1, 2, 3, LAUNCH_ROWS - 1, LAUNCH_ROWS, LAUNCH_ROWS + 1, rows - 1]
    gen = torch.Generator(device="cuda").manual_seed(cols)
    some = torch.randn(len(at), width, generator=gen, device="cuda").to(BF)
    x = torch.empty(rows, width, dtype=BF, device="cuda")
    x[at] = some
    w = (1 + 0.3 * torch.randn(cols, generator=gen, device="cuda")).to(BF)

    def out(n):
        """An output of n rows, and its scales."""
        if to == "bf16":
            return torch.full((n, cols), 5.0, dtype=BF, device="cuda"), None
        if to == "e4m3":
            return torch.full((n, cols), 85, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn), torch.full((n,), 5.0, device="cuda")
        codes, scales = q.mxfp4_empty(n, cols)
        return codes.fill_(85), scales.fill_(85)

    def run(x, o, s):
        if op == "swiglu":
            q.moe_swiglu(x, o, out_scale=s)
        elif s is None:
            q.moe_rmsnorm(x, w, 1e-5, y=o)
        else:
            q.moe_rmsnorm(x, w, 1e-5, q=o, q_scale=s)

    want, want_s = out(len(at))
    run(some, want, want_s)
    got, got_s = out(rows)
    run(x, got, got_s)
    raw = lambda t: t.view(torch.uint8)
    for i, r in enumerate(at):
        assert torch.equal(raw(got[r]), raw(want[i])), r
        assert got_s is None or torch.equal(got_s[r], want_s[i]), r
    del x, got, got_s
    torch.cuda.empty_cache()
