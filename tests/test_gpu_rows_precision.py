"""How exactly the row operators hold what they compute in fp32, against float64:
bounds that count the roundings of each form, whatever the size of the inputs."""
import numpy as np
import pytest
import torch

import quantized_moe_02_amd as q
from oracle import rows as ref
from row_cases import BF, F, U, close, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.lib()


# ---- SwiGLU ------------------------------------------------------------------------
# s = 1 / (1 + x), x = e^-g: the hardware's power of two 2, the product by 1 - c 1 (c holds
# what its argument's rounding lost); 1 + x 1; the hardware's reciprocal 2.  1 - s = x s: x's
# share, the others and the product.
S_BOUND, REST_BOUND = 6 * U, 7 * U


def _gates(lo, hi, t, rows=64, cols=520):
    gen = torch.Generator().manual_seed(int(10 * lo))
    g = (torch.rand(rows, cols, generator=gen) * (hi - lo) + lo).to(t)
    g[::2] *= -1
    up, dh = torch.randn(rows, cols, generator=gen).to(t), torch.randn(rows, cols, generator=gen)
    return torch.cat([g, up], 1).cuda(), dh.cuda()


@pytest.mark.parametrize("lo,hi", [(0, 1), (1, 4), (4, 10), (10, 20), (20, 50), (50, 87), (87, 95)])
@pytest.mark.parametrize("t", [F, BF])
def test_swiglu_at_every_gate(lo, hi, t):
    """As exact for gates far from 0 as for those near it."""
    gu, dh = _gates(lo, hi, t)
    out, dgu = torch.empty_like(dh), torch.empty_like(gu)
    q.moe_swiglu(gu, out)
    g, up = np.split(f64(gu), 2, axis=1)
    lost = 2.0 ** -126                            # an s below that counts as 0
    want = ref.swiglu(f64(gu))
    close(out, want, (S_BOUND + 2 * U) * np.abs(want) + lost * np.abs(g * up), F)
    q.moe_swiglu_grad(gu, dh, dgu)
    want, mag = ref.swiglu_grad(f64(gu), f64(dh))
    d = np.abs(f64(dh))
    # dgate: s, rest in the slope, the slope's sum and three products; dup: s and two products
    rel = np.concatenate([np.full(g.shape, S_BOUND + REST_BOUND + 4 * U), np.full(g.shape, S_BOUND + 2 * U)], 1)
    close(dgu, want, rel * mag + lost * np.concatenate([d * np.abs(up) * (1 + np.abs(g)), d * np.abs(g)], 1), t)


def test_codes_are_those_of_the_exact_values():
    """E4M3 and MXFP4 rows of bf16 gates are made of the same fp32 values."""
    gu, _ = _gates(0, 20, BF, cols=512)
    y, mx, codes = torch.empty(64, 512, device="cuda"), q.mxfp4_empty(64, 512), q.mxfp4_empty(64, 512)
    q.moe_swiglu(gu, y)
    q.moe_swiglu(gu, mx[0], out_scale=mx[1])
    q.moe_mxfp4_quantize(y, *codes)
    assert torch.equal(mx[0], codes[0]) and torch.equal(mx[1], codes[1])


# ---- the norm's weight gradient ------------------------------------------------------
# A term dy h m: m, h m and the product. Eight terms added in fp32: 7 roundings. A workgroup's
# sum 1; everything else is float64, the result's own rounding is close()'s.
DW_BOUND = (3 + 7 + 1) * U


@pytest.mark.parametrize("rows,cols", [(64 * 32768 + 5, 24), (64 * 2048 + 1, 500), (64 * 2048, 1100), (64 * 2048 + 3, 2000), (64 * 512 + 1, 2056),
                                       (64 * 512, 5003), (64 * 256 + 2, 9000), (64 * 256, 16380), (64 * 256 + 1, 16392)])
@pytest.mark.parametrize("t,wt", [(BF, BF), (BF, F), (F, F)])
def test_norm_weight_gradient_of_long_batches(rows, cols, t, wt):
    """A few large terms in front of many that vanish beside them one by one: 64
    and more rows a workgroup, the large ones first in each."""
    if t is F and rows * cols > 150 << 20:
        rows //= 2
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    rand = lambda *s: torch.rand(*s, generator=gen, device="cuda")
    h = (0.5 + rand(rows, cols)).to(t)
    dy = (0.5 + rand(rows, cols)).mul_(2.0 ** -25)
    dy[:-(-rows // 64)] *= 2.0 ** 25
    dy = dy.to(t)
    w = (0.5 + rand(cols)).to(wt)
    dx, dw = torch.empty_like(h), torch.empty(cols, device="cuda")
    q.moe_rmsnorm_grad(dy, h, w, 1e-5, dx, dweight=dw, ws=q.rmsnorm_workspace(rows, cols))
    want = torch.zeros(cols, dtype=torch.float64, device="cuda")
    eps = float(np.float32(1e-5))
    for i in range(0, rows, 4096):
        hh = h[i:i + 4096].double()
        want += (dy[i:i + 4096].double() * hh * (hh.square().mean(1, keepdim=True) + eps).rsqrt()).sum(0)
    want = f64(want)
    close(dw, want, DW_BOUND * want, F, "dweight")          # every term is positive


@pytest.mark.parametrize("rows,cols", [(1025, 40), (5000, 17), (4099, 512), (6150, 700), (6500, 1300), (2500, 1537), (6161, 2000), (4200, 2048),
                                       (2049, 2056), (1100, 5003), (1100, 8000), (800, 8200), (700, 14000), (1300, 16400)])
@pytest.mark.parametrize("types", [(BF, BF, BF), (BF, BF, F), (F, F, F), (BF, F, BF)])
def test_norm_gradient_of_many_rows(rows, cols, types):
    """Several workgroups of several rows each, joined: every shape, bf16 rows beside
    bf16 weights, dy in fp32, all in fp32, and types without a kernel of their own."""
    ht, wt, yt = types
    gen = torch.Generator(device="cuda").manual_seed(rows)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    h, dy, dh, w = n(rows, cols).to(ht), (0.1 * n(rows, cols)).to(yt), (0.1 * n(rows, cols)).to(ht), (1 + 0.3 * n(cols)).to(wt)
    dx, dw = torch.empty_like(h), torch.empty(cols, device="cuda")
    q.moe_rmsnorm_grad(dy, h, w, 1e-5, dx, dh=dh, dweight=dw, ws=q.rmsnorm_workspace(rows, cols))
    H, D, W = h.double(), dy.double(), w.double()
    m = (H.square().mean(1, keepdim=True) + float(np.float32(1e-5))).rsqrt()
    g, k = D * W, m * m
    want = dh.double() + m * (g - H * (k * (g * H).mean(1, keepdim=True)))
    mag = dh.double().abs() + m * (g.abs() + H.abs() * (k * (g * H).abs().mean(1, keepdim=True)))
    # g, its product with h, m, k, h k, the difference, its product with m, dh's addition
    close(dx, f64(want), 8 * U * f64(mag), ht, "dx")
    t = D * H * m
    close(dw, f64(t.sum(0)), DW_BOUND * f64(t.abs().sum(0)), F, "dweight")
