"""The MXFP4 step's use of the row operators: what it holds between them, and the
gradients that it takes."""
import os
import sys

import pytest
import torch

import quantized_moe_02_amd as q
import synth
from oracle import rows as ref
from row_cases import BF, F, U, close, f64

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.lib()


def _layer(T):
    import mxfp4_moe_step as ex
    layer = ex.make_layer(synth.WORKLOADS["tiny"]["geom"], seed=T, score_coef=0.5)
    return layer, torch.randn(T, layer.geom["hidden"], generator=torch.Generator().manual_seed(T)).to(BF).cuda()


@pytest.mark.parametrize("T", [1, 9, 70])
def test_the_experts_rows_reach_their_sum_in_fp32(T):
    layer, x = _layer(T)
    y, _, _ = layer.forward(x)
    _, _, tw, offs, _, inv, gu = layer.saved[:7]
    k, I = tw.shape[1], layer.geom["moe_inter"]
    h, rows = torch.empty(T * k, I, dtype=BF, device="cuda"), torch.empty(T * k, x.shape[1], device="cuda")
    q.moe_swiglu(gu, h, expert_offsets=offs)
    q.moe_mxfp4_matmul(h, *layer.down, rows, expert_offsets=offs)
    want, mag = ref.collect(f64(rows), inv.cpu().numpy(), f64(tw))
    close(y, want, (k + 2) * U * mag, F)                   # the products and sums of k rows


@pytest.mark.parametrize("through_router", [False, True])
def test_the_weights_gradient_is_taken_where_it_is_asked_for(through_router, monkeypatch):
    """It reads every expert's row again."""
    layer, x = _layer(9)
    y, _, _ = layer.forward(x)
    asked, call = [], q.moe_collect_grad
    monkeypatch.setattr(q, "moe_collect_grad", lambda *a, **k: (asked.append(k.get("dweights") is not None), call(*a, **k))[1])
    layer.backward(torch.ones_like(y), through_router=through_router)
    assert any(asked) == through_router


@pytest.mark.parametrize("layout", ["broadcast over tokens", "broadcast over columns", "transposed", "float64"])
def test_a_gradient_in_any_layout(layout):
    T = 9
    layer, x = _layer(T)
    y, _, _ = layer.forward(x)
    gen = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=gen).cuda()
    H = y.shape[1]
    dy = {"broadcast over tokens": lambda: n(1, H).expand(T, H), "broadcast over columns": lambda: n(T, 1).expand(T, H),
          "transposed": lambda: n(H, T).t(), "float64": lambda: n(T, H).double()}[layout]()
    plain = torch.empty(T, H, device="cuda").copy_(dy)
    for got, want in zip(layer.backward(dy), layer.backward(plain)):
        assert torch.equal(got, want)
