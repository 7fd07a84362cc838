"""Shapes of the operators' launches, without a GPU (tests/launches.py)."""
import ctypes

import pytest

import launches as rec
import quantized_moe_02_amd as q

X, CODES, SCALE = 1 << 60, 1 << 50, 1 << 40          # never dereferenced


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    if not rec.Recorder.available():
        pytest.skip("needs the regular build (_build/*.o) and the ROCm clang")
    return rec.Recorder(tmp_path_factory.mktemp("record"))


@pytest.fixture
def record(recorder):
    recorder.take()
    return recorder


# matrices of 2^32 chunks of eight inputs and more among them; they fit the card
@pytest.mark.parametrize("rows,cols", [(1, 1), (4099, 2057), (98304, 2048), (1 << 30, 1), ((1 << 31) - 1, 1),
                                       ((1 << 31) - 1, 33), (2200, 1 << 24), (5_000_001, 6144)])
@pytest.mark.parametrize("dtype,size", [(q.MOE_DT_F32, 4), (q.MOE_DT_BF16, 2), (q.MOE_DT_F16, 2)])
def test_quantize_launches_cover_any_matrix(record, rows, cols, dtype, size):
    nb, ld = (cols + 31) // 32, cols + 3
    for call in (lambda: record.lib.moe_mxfp4_quantize(X, dtype, rows, cols, ld, CODES, SCALE, None),
                 lambda: record.lib.moe_mxfp4_dequantize(CODES, SCALE, rows, cols, X, dtype, ld, None)):
        assert call() == q.MOE_OK
        at = 0
        for l in record.take():
            assert (l.x, l.codes, l.scale) == (X + at * ld * size, CODES + at * 16 * nb, SCALE + at * nb)
            per = 8 * 4 if l.kernel.endswith(" 4>") else 8          # inputs per work item
            assert l.threads < 1 << 32 and l.threads * per >= l.rows * 32 * nb
            at += l.rows
        assert at == rows
