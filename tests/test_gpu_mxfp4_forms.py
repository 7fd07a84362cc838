"""MXFP4 operators on the GPU at sizes that reach every kernel and every branch
of it, against the float64 oracle (bounds as in test_gpu_mxfp4.py)."""
import numpy as np
import pytest
import torch

import quantized_moe_02_amd as q
from oracle import operators as ref
from test_gpu_mxfp4 import Problem, _close, _quantize

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.lib()


def test_matrix_of_more_than_one_launch():
    """2^30 rows of one column, 2^32 chunks of eight inputs and more: the
    launches' bounds lie at no multiple of the rows' period."""
    period, rows = 251, (1 << 30) + 5
    table = torch.randn(period, 1, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    src = table.cuda().repeat(rows // period + 1, 1)[:rows]
    codes, scales = q.mxfp4_empty(rows, 1)
    codes.fill_(0xEE)
    scales.fill_(0xEE)
    q.moe_mxfp4_quantize(src, codes, scales)
    del src
    back = torch.full((rows, 1), 7.0, dtype=torch.bfloat16, device="cuda")
    q.moe_mxfp4_dequantize(codes, scales, back)
    rc, rs = ref.mx_quantize(table.double().numpy())
    held = torch.from_numpy(ref.mx_values(rc, rs)[:, :1]).to(torch.bfloat16).cuda()
    rc, rs = torch.from_numpy(rc).cuda(), torch.from_numpy(rs).cuda()
    step = period << 18
    for lo in range(0, rows, step):
        n = min(step, rows - lo)
        for got, want in ((codes, rc), (scales, rs), (back, held)):
            part = got[lo:lo + n]
            whole = n // period * period
            assert (part[:whole].view(-1, period, part.shape[1]) == want).all(), lo
            assert torch.equal(part[whole:], want[:n - whole]), lo


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
def test_sources_past_32_bit_offsets(act):
    """Rows gathered from a matrix of more than 2^32 bytes: its first and last
    rows, those around 2^32 and beside either end."""
    k, rows = (544, 1 << 22) if act == "bf16" else (2080, 1 << 22)
    P = Problem([290, 10], 4100, k, seed=k, gather=1)
    edge = 2 ** 32 // (2 * k if act == "bf16" else k // 2)
    P.index = torch.randint(0, rows, (P.R,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    P.index[:8] = torch.tensor([0, rows - 1, edge, edge + 1, edge - 1, -1, rows, 2 ** 31 - 1])
    o = torch.full((P.R, P.n), 77.0, device="cuda")
    idx, wq, ws = P.index.cuda(), P.wq.cuda(), P.ws.cuda()
    inside = (P.index >= 0) & (P.index < rows)
    at = torch.where(inside, P.index, 0).long()
    if act == "bf16":
        a = torch.empty(rows, k, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(2))
        q.moe_mxfp4_matmul(a, wq, ws, o, expert_offsets=P.offsets(), row_index=idx)
        x64 = a[at.cuda()].double().cpu().numpy()
    else:
        gen = torch.Generator("cuda").manual_seed(2)
        a = torch.randint(0, 256, (rows, k // 2), generator=gen, dtype=torch.uint8, device="cuda")
        s = torch.randint(120, 130, (rows, k // 32), generator=gen, dtype=torch.uint8, device="cuda")
        q.moe_mxfp4_matmul(a, wq, ws, o, a_scale=s, expert_offsets=P.offsets(), row_index=idx)
        x64 = ref.mx_values(a[at.cuda()].cpu().numpy(), s[at.cuda()].cpu().numpy())
    x64[~inside.numpy()] = 0
    want, mag = ref.grouped_matmul(x64, P.w64, P.off)
    _close(o, want, mag, k, False)


def test_product_of_more_than_one_launch():
    """Few-row units enough for two launches: 270000 rows, gathered from past
    2^32 bytes, of 65536 outputs.  Every row at three outputs, and every output
    of the rows around the launches' bound and the ends."""
    n, k, R, rows = 65536, 32, 270000, 1 << 22
    gen = torch.Generator("cuda").manual_seed(3)
    wide = torch.empty(rows, 512, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    wq = torch.randint(0, 256, (1, n, k // 2), generator=gen, dtype=torch.uint8, device="cuda")
    ws = torch.randint(120, 130, (1, n, 1), generator=gen, dtype=torch.uint8, device="cuda")
    idx = torch.randint(0, rows, (R,), generator=gen, dtype=torch.int32, device="cuda")
    o = torch.full((R, n), 77.0, dtype=torch.bfloat16, device="cuda")
    q.moe_mxfp4_matmul(wide[:, :k], wq, ws, o, row_index=idx)
    x = wide[:, :k][idx.long()].double().cpu().numpy()
    w = ref.mx_values(wq[0].cpu().numpy(), ws[0].cpu().numpy())
    cols = [0, 4097, n - 1]
    _close(o[:, cols], x @ w[cols].T, np.abs(x) @ np.abs(w[cols]).T, k, True)
    for lo in (0, (1 << 18) - 16, (1 << 18), R - 16):
        a = x[lo:lo + 16]
        _close(o[lo:lo + 16], a @ w.T, np.abs(a) @ np.abs(w).T, k, True)
