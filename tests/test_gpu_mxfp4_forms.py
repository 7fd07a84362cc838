"""MXFP4 operators on the GPU at sizes that reach every kernel and every branch
of it, against the float64 oracle (bounds as in test_gpu_mxfp4.py)."""
import numpy as np
import pytest
import torch

import quantized_moe_02_amd as q
from oracle import operators as ref

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
