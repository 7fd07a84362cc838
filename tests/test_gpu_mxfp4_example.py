"""The training step of examples/mxfp4_moe_step.py against the same layer
written in torch (float64, autograd) with the experts' decoded weights."""
import os
import sys

import pytest
import torch

import quantized_moe_02_amd as q
import synth

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.lib()


def _decoded(codes, scales):
    E, n, kb = codes.shape
    w = torch.empty(E * n, kb * 2, device="cuda")
    q.moe_mxfp4_dequantize(codes.view(E * n, kb), scales.view(E * n, -1), w)
    return w.view(E, n, kb * 2).double().cpu()


def _close(got, want, tol):
    err = (got.double().cpu() - want).norm() / want.norm()
    assert err <= tol, err


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [1, 7, 96])
def test_step_against_torch(T, mx):
    import mxfp4_moe_step as ex
    geom = synth.WORKLOADS["tiny"]["geom"]
    H, I, E, k = geom["hidden"], geom["moe_inter"], geom["n_routed_experts"], geom["top_k"]
    layer = ex.make_layer(geom, seed=T, score_coef=0.5, tokens_in_mxfp4=mx)
    gen = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=gen).to(torch.bfloat16)
    dy = torch.randn(T, H, generator=gen)
    y, loss, counts = layer.forward(x.cuda())
    dx, d_router = layer.backward(dy.cuda())

    ids, tw = layer.saved[1].cpu().long(), layer.saved[2].cpu().double()
    gate_up, down = _decoded(*layer.gate_up), _decoded(*layer.down)
    xr = x.double()
    if mx:      # the product sees the tokens in MXFP4; the gradient passes straight through
        codes, scales = q.mxfp4_empty(T, H)
        q.moe_mxfp4_quantize(x.cuda(), codes, scales)
        xr = _decoded(codes.view(1, T, -1), scales.view(1, T, -1))[0]
    xr.requires_grad_(True)
    out = []
    for t in range(T):
        acc = torch.zeros(H, dtype=torch.float64)
        for j in range(k):
            e = ids[t, j]
            g = gate_up[e] @ xr[t]
            acc = acc + tw[t, j] * (down[e] @ (torch.nn.functional.silu(g[:I]) * g[I:]))
        out.append(acc)
    out = torch.stack(out)
    # bf16 h and gradients: 2^-8 each, two in a row
    _close(y, out.detach(), 2 ** -8)
    (out * dy.double()).sum().backward()
    _close(dx, xr.grad, 3 * 2 ** -8)

    w = layer.router_w.double().cpu().requires_grad_(True)
    s = torch.sigmoid(x.double() @ w.T)
    p = s / s.sum(1, keepdim=True)
    n = torch.bincount(ids.reshape(-1), minlength=E).double()
    assert torch.equal(counts[0].cpu().long(), n.long())
    ref = 0.5 * (E * n / n.sum() * p.mean(0)).sum()
    assert abs(loss.item() - ref.item()) <= 1e-5 * ref.item()
    ref.backward()
    _close(d_router, w.grad, 1e-4)
