"""Over the stand-in for the HIP runtime: the calls of launch_cases take several
launches."""
import ctypes

import pytest

import quantized_moe_02_amd as q
from launch_cases import CASES, LAUNCH_ROWS
from test_row_launches import BF16, E4, F, MX, record  # noqa: F401


@pytest.mark.parametrize("op,cols,to", CASES)
def test_calls_of_several_launches(record, op, cols, to):  # noqa: F811
    rows, ot = LAUNCH_ROWS + 3, {"bf16": BF16, "e4m3": E4, "mxfp4": MX}[to]
    if op == "rmsnorm":
        c = q.MoeRmsnormConfig(rows, cols, BF16, BF16, BF16, BF16, ot, 1e-6, cols, cols, cols, cols)
        coded = ot != BF16
        status = record.lib.moe_rmsnorm(ctypes.byref(c), F, None, F, None, None if coded else F, F if coded else None, F if coded else None, None)
    else:
        c = q.MoeSwigluConfig(rows, cols, 1, BF16, ot, 2 * cols, cols)
        status = record.lib.moe_swiglu(ctypes.byref(c), F, None, F, F, None)
    assert status == q.MOE_OK
    ls = record.take()
    assert [l.first for l in ls] == [0, LAUNCH_ROWS] and [l.blocks for l in ls] == [LAUNCH_ROWS, 3]
    assert all(l.threads == 1024 for l in ls)
