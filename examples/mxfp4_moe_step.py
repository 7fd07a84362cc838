"""One training step through an MoE layer whose experts are frozen in MXFP4.

What is trained lies around the experts: the router (through its balance loss,
and through the routing weights), the norm before the layer and whatever comes
before that (through the gradient of its input), as in fine-tuning with adapters.
The step runs on the library's entry points:

  norm                   moe_rmsnorm with the residual's addition, moe_rmsnorm_grad
  route, permute         moe_route, moe_permute
  experts, forward       moe_mxfp4_matmul (gate and up on the tokens as they
                         are, or brought to MXFP4 first; down on bf16), moe_swiglu
  combine                moe_collect, moe_collect_grad
  balance loss           moe_balance_loss, moe_balance_loss_grad
  experts, backward      moe_mxfp4_matmul_dx, moe_swiglu_grad, moe_collect without weights

    python examples/mxfp4_moe_step.py            (needs an MI355X)
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_moe_02_amd as q  # noqa: E402


def quantize_experts(w: torch.Tensor):
    """[E][n][k] weights (fp32 or bf16) to MXFP4 codes [E][n][k/2] and scales."""
    E, n, k = w.shape
    codes, scales = q.mxfp4_empty(E * n, k, w.device)
    q.moe_mxfp4_quantize(w.reshape(E * n, k), codes, scales)
    return codes.view(E, n, k // 2), scales.view(E, n, k // 32)


class Mxfp4MoE:
    """Router [E][H] fp32 and SwiGLU experts: gate and up [E][2 I][H], down [E][H][I]."""

    def __init__(self, geom: dict, router_w, gate_up, down, score_coef=1e-3, tokens_in_mxfp4=False):
        self.geom = dict(geom, n_shared_experts=0, shared_inter=0)
        self.cfg = q.make_config(self.geom, "nvfp4")     # routing and combine do not look at the format
        self.router_w = router_w
        self.gate_up, self.down = quantize_experts(gate_up), quantize_experts(down)
        self.coef, self.mx = score_coef, tokens_in_mxfp4

    def forward(self, x, seq_offsets=None):
        """x bf16 [T][H] -> y fp32 [T][H]; keeps what the backward pass needs."""
        g, T, dev = self.geom, x.shape[0], x.device
        H, I, E, k = g["hidden"], g["moe_inter"], g["n_routed_experts"], g["top_k"]
        i32 = dict(dtype=torch.int32, device=dev)
        ws = q.workspace(self.cfg, T, dev)
        ids, tw = torch.empty(T, k, **i32), torch.empty(T, k, device=dev)
        q.moe_route(self.cfg, T, x, self.router_w, None, ids, tw, ws)
        offs, tok, inv = torch.empty(E + 1, **i32), torch.empty(T * k, **i32), torch.empty(T * k, **i32)
        act, na = torch.empty(E, **i32), torch.empty(1, **i32)
        q.moe_permute(self.cfg, T, ids, offs, tok, inv, act, na, ws)

        gu = torch.empty(T * k, 2 * I, device=dev)
        if self.mx:
            xq, xs = q.mxfp4_empty(T, H, dev)
            q.moe_mxfp4_quantize(x, xq, xs)
            q.moe_mxfp4_matmul(xq, *self.gate_up, gu, a_scale=xs, expert_offsets=offs, row_index=tok)
        else:
            q.moe_mxfp4_matmul(x, *self.gate_up, gu, expert_offsets=offs, row_index=tok)
        h = torch.empty(T * k, I, dtype=torch.bfloat16, device=dev)
        q.moe_swiglu(gu, h, expert_offsets=offs)
        out = torch.empty(T * k, H, device=dev)
        q.moe_mxfp4_matmul(h, *self.down, out, expert_offsets=offs)
        y = torch.empty(T, H, device=dev)
        inv = inv.view(T, k)
        q.moe_collect(out, inv, y, weights=tw)

        logits = x.float() @ self.router_w.T
        S = 1 if seq_offsets is None else seq_offsets.numel() - 1
        counts, n_tok = torch.empty(S, E, **i32), torch.empty(S, **i32)
        loss = torch.empty(1, device=dev)
        q.moe_balance_loss(logits, ids, counts, n_tok, loss, coef=self.coef, seq_offsets=seq_offsets,
                           ws=q.balance_workspace(T, E, S, dev))
        self.saved = (x, ids, tw, offs, tok, inv, gu, out, logits, counts, n_tok, seq_offsets)
        return y, loss, counts

    def backward(self, dy, through_router=False):
        """dy fp32 [T][H], in any layout -> (gradient of x through the experts, fp32 [T][H];
        gradient of the router weights from the balance loss, [E][H]).  With
        through_router both hold all of it: the routing weights' share and, in x, the
        way through the router."""
        x, ids, tw, offs, tok, inv, gu, out, logits, counts, n_tok, seq = self.saved
        g, T, dev = self.geom, x.shape[0], x.device
        H, I, k = g["hidden"], g["moe_inter"], g["top_k"]
        dy = dy.float().contiguous()                             # one broadcast over rows or columns, too
        d_out = torch.empty(T * k, H, dtype=torch.bfloat16, device=dev)
        q.moe_collect_grad(dy, inv, drows=d_out, weights=tw)
        dh = torch.empty(T * k, I, device=dev)
        q.moe_mxfp4_matmul_dx(d_out, *self.down, dh, expert_offsets=offs)
        d_gu = torch.empty_like(gu)
        q.moe_swiglu_grad(gu, dh, d_gu, expert_offsets=offs)
        d_rows = torch.empty(T * k, H, device=dev)
        q.moe_mxfp4_matmul_dx(d_gu.to(torch.bfloat16), *self.gate_up, d_rows, expert_offsets=offs)
        dx = torch.empty(T, H, device=dev)
        q.moe_collect(d_rows, inv, dx)
        dlogits = torch.empty_like(logits)
        q.moe_balance_loss_grad(logits, ids, counts, n_tok, dlogits, coef=self.coef, seq_offsets=seq)
        if through_router:
            # weights rsf s_i / sum s over a token's picks, s = sigmoid(logits)
            d_tw, at = torch.empty_like(tw), ids.long()
            q.moe_collect_grad(dy, inv, rows=out, dweights=d_tw)
            s = torch.sigmoid(logits.gather(1, at))
            ds = (g["routed_scaling_factor"] * d_tw - (d_tw * tw).sum(1, keepdim=True)) / s.sum(1, keepdim=True)
            dlogits.scatter_add_(1, at, ds * s * (1 - s))
            dx += dlogits @ self.router_w
        return dx, dlogits.T @ x.float()


class NormMoEBlock:
    """The layer behind its norm: h = x + residual, y = layer(norm(h)); y and h go
    on to the next block as its x and residual."""

    def __init__(self, layer: Mxfp4MoE, norm_w, eps=1e-6):
        self.layer, self.norm_w, self.eps = layer, norm_w, eps

    def forward(self, x, residual, seq_offsets=None):
        """x, residual bf16 [T][H] -> y fp32 [T][H], h bf16 [T][H], the balance loss."""
        h, n = torch.empty_like(residual), torch.empty_like(residual)
        q.moe_rmsnorm(x, self.norm_w, self.eps, y=n, residual=residual, h=h)
        y, loss, _ = self.layer.forward(n, seq_offsets)
        self.h = h
        return y, h, loss

    def backward(self, dy, dh):
        """Gradients dy fp32 and dh bf16 [T][H] -> that of x and of residual (one
        tensor, bf16), of the norm's weight and of the router."""
        dn, d_router = self.layer.backward(dy, through_router=True)
        dx, dw = torch.empty_like(dh), torch.empty(self.norm_w.shape, device=dh.device)
        q.moe_rmsnorm_grad(dn, self.h, self.norm_w, self.eps, dx, dh=dh, dweight=dw)
        return dx, dw, d_router


def make_layer(geom: dict, device="cuda", seed=0, **kw) -> Mxfp4MoE:
    gen = torch.Generator(device=device).manual_seed(seed)
    H, I, E = geom["hidden"], geom["moe_inter"], geom["n_routed_experts"]
    normal = lambda *s: torch.randn(*s, generator=gen, device=device) * H ** -0.5
    return Mxfp4MoE(geom, normal(E, H), normal(E, 2 * I, H).to(torch.bfloat16),
                    normal(E, H, I).to(torch.bfloat16), **kw)


def main():
    import synth
    geom = synth.WORKLOADS["tiny"]["geom"]
    layer = make_layer(geom, score_coef=0.5)
    T = 512
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, geom["hidden"], generator=gen, device="cuda").to(torch.bfloat16)
    seq = torch.tensor([0, 200, T], dtype=torch.int32, device="cuda")
    layer.router_w[:4] *= 3.0                                    # a router that favours four experts
    for step in range(5):
        y, loss, counts = layer.forward(x, seq)
        dx, d_router = layer.backward(torch.ones_like(y) / y.numel())
        layer.router_w -= 20.0 * d_router
        print(f"step {step}: balance loss {loss.item():.4f}, busiest expert {int(counts.sum(0).max())} of "
              f"{int(counts.sum())} picks, |y| {y.norm().item():.3f}, |dx| {dx.norm().item():.5f}")
    block = NormMoEBlock(layer, torch.ones(geom["hidden"], device="cuda"))
    y, h, _ = block.forward(x, x, seq)
    dx, dw, d_router = block.backward(torch.ones_like(y) / y.numel(), torch.zeros_like(h))
    print(f"block behind its norm: |y| {y.norm().item():.3f}, |dx| {dx.float().norm().item():.5f}, |dw| {dw.norm().item():.5f}, "
          f"|d router| {d_router.norm().item():.5f}")


if __name__ == "__main__":
    main()
