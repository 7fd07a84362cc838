"""What the binding of the row operators says of arguments that are no sizes or
numbers its structs can hold: a status that names the fault.  Without a GPU."""
import pytest
import torch

import quantized_moe_02_amd as q
from quantized_moe_02_amd import binding
from test_operator_binding import On

BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _device(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0)
    monkeypatch.setattr(binding, "_current_device", lambda: 0)


def _status(call):
    with pytest.raises(q.QmoeError) as ei:
        call()
    return ei.value.status


@pytest.mark.parametrize("eps", [None, "1e-6", [1e-6], 1e39, -1e39, float("inf"), float("nan"), 0.0, -1.0])
def test_an_eps_that_is_no_positive_fp32_number(eps):
    x, w = On.of(torch.zeros(2, 8, dtype=BF)), On.of(torch.zeros(8, dtype=BF))
    assert _status(lambda: q.moe_rmsnorm(x, w, eps, y=x)) == q.MOE_ERR_INVALID_ARG
    assert _status(lambda: q.moe_rmsnorm_grad(x, x, w, eps, x)) == q.MOE_ERR_INVALID_ARG


def test_sizes_past_32_bits():
    far = lambda *s: On.of(torch.empty(s, dtype=BF, device="meta"))
    one = On.of(torch.zeros(1))
    rows = 3 << 31
    for call in (lambda: q.moe_rmsnorm(far(rows, 1), one, 1e-6, y=far(rows, 1)),
                 lambda: q.moe_rmsnorm_grad(far(rows, 1), far(rows, 1), one, 1e-6, far(rows, 1)),
                 lambda: q.moe_swiglu(far(rows, 2), far(rows, 1)),
                 lambda: q.moe_collect(far(rows, 1), On.of(torch.zeros(1, 1, dtype=torch.int32)), far(1, 1))):
        assert _status(call) == q.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("rows,cols,status", [((1 << 32) + 4, 64, "UNSUPPORTED"), (4, (1 << 32) + 64, "UNSUPPORTED"), (1 << 31, 64, "UNSUPPORTED"),
                                              (4 - (1 << 32), 64, "INVALID_ARG"), (4, 64 - (1 << 32), "INVALID_ARG")])
def test_a_workspace_of_sizes_past_32_bits(rows, cols, status):
    for size in (q.moe_rmsnorm_workspace_size, q.rmsnorm_workspace):
        assert _status(lambda: size(rows, cols)) == getattr(q, "MOE_ERR_" + status)
