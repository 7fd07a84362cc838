"""Shapes of the operators' launches, without a GPU (tests/launches.py)."""
import ctypes

import pytest

import launches as rec
import product_forms
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


F = 1 << 30                                          # 16-byte aligned, never dereferenced
MAX_ROWS = 16 * q.MOE_MAX_TOKENS


def _product(record, R, n, k, E, a_rows=None, act="bf16", index=False, lda=None, dx=False):
    """The launches of one product (dx: its gradient) over fp32 outputs."""
    c = q.MoeMatmulConfig(R, n, k, E, R if a_rows is None else a_rows, q.MOE_DT_MXFP4 if act == "mxfp4" else q.MOE_DT_BF16,
                          q.MOE_DT_F32, lda or (n if dx else k), k if dx else n)
    if dx:
        s = record.lib.moe_mxfp4_matmul_dx(ctypes.byref(c), F, F, F, F, F, None)
    else:
        s = record.lib.moe_mxfp4_matmul(ctypes.byref(c), F, F if act == "mxfp4" else None, F, F, F, F if index else None,
                                        F, None)
    assert s == q.MOE_OK
    return record.take()


@pytest.mark.parametrize("S", [1, 4, 5, 39, 48, 300, 1365, 2731, 65536])
def test_balance_workspace_holds_every_slot(record, S):
    """One slot of E shares and counts, a token and a pick count for each chunk
    and sequence; a double per 32 experts of a sequence."""
    E = 33
    tokens = sorted({t for e in (1, 8 * S, 12 * S, 16 * S, 128 * S, 128, 32768, 262144) for t in range(e - 9, e + 9)
                     if 0 < t <= q.MOE_MAX_TOKENS} | set(range(1, q.MOE_MAX_TOKENS, 4999)))
    for T in tokens:
        c, n = q.make_balance_config(T, E, 1, S), ctypes.c_size_t(0)
        assert record.lib.moe_balance_workspace_size(ctypes.byref(c), ctypes.byref(n)) == q.MOE_OK
        assert record.lib.moe_balance_loss(ctypes.byref(c), F, F, F, F, F, F, F, n, None) == q.MOE_OK
        chunks = [l.blocks for l in record.take() if l.kernel.startswith("balance_partial")]
        assert len(chunks) == 1 and n.value >= (chunks[0] + S) * (8 * E + 8) + 2 * S * 8, T


@pytest.mark.parametrize("R,n,k,E,a_rows,act,index,lda,dx", [
    (MAX_ROWS, 65536, 2048, 256, MAX_ROWS, "bf16", True, None, False),     # inputs past 32-bit offsets: few-row units
    (1 << 20, 65536, 2048, 256, 1 << 21, "bf16", True, None, False),
    (MAX_ROWS, 8192, 6144, 256, MAX_ROWS, "mxfp4", True, None, False),
    (MAX_ROWS, 65536, 65536, 1, MAX_ROWS, "mxfp4", True, None, False),
    (MAX_ROWS, 65536, 2048, 256, None, "bf16", False, 1 << 24, False),
    (MAX_ROWS, 65536, 65536, 256, None, "bf16", False, 1 << 24, True),
    (MAX_ROWS, 65536, 65536, 256, None, "bf16", False, None, True),
    (MAX_ROWS, 65536, 32, 1, None, "bf16", False, None, False)])
def test_product_launches_cover_every_unit(record, R, n, k, E, a_rows, act, index, lda, dx):
    ls = _product(record, R, n, k, E, a_rows, act, index, lda, dx)
    assert all(l.threads < 1 << 32 for l in ls)
    if "thin" not in ls[0].kernel:
        assert len(ls) == 1
        return
    # workgroups of a unit: by its outputs
    outputs = k if dx else n
    if dx:
        per = -(-outputs // (128 * int(ls[0].kernel.split("<")[1][0])))
    else:
        nt = -(-outputs // (16 * int(ls[0].kernel.split(", ")[1])))
        units = R // 16 + min(E, R)
        per = -(-nt // 2) if units * nt >= 8192 else nt
    at = 0
    for l in ls:
        assert l.kernel == ls[0].kernel and l.first == at and l.blocks % per == 0
        at += l.blocks // per
    assert at >= R // 16 + (min(E, R) if E > 1 else 1)


@pytest.mark.parametrize("kernel,kind,counts,n,k,extra,gather", product_forms.PRODUCTS, ids=product_forms.NAMES)
def test_forms_reach_their_kernels(record, kernel, kind, counts, n, k, extra, gather):
    R = sum(counts) + extra
    ls = _product(record, R, n, k, len(counts), gather or None, kind, bool(gather), dx=kind == "dx")
    assert [l.kernel for l in ls] == [kernel]


def test_forms_name_every_kernel(record):
    """Every product's kernel that the objects hold is reached by some form."""
    assert {kernel for kernel, *_ in product_forms.PRODUCTS} == {k for k in record.kernels() if "matmul" in k}


@pytest.mark.parametrize("rows,cols,dtype,chunks", [
    (4099, 4097, q.MOE_DT_BF16, 4), (4099, 4097, q.MOE_DT_F16, 4), (4099, 4097, q.MOE_DT_F32, 1), (4099, 2057, q.MOE_DT_F16, 1),
    (20000, 4097, q.MOE_DT_BF16, 1)])
def test_conversions_reach_their_kernels(record, rows, cols, dtype, chunks):
    record.lib.moe_mxfp4_quantize(X, dtype, rows, cols, cols, CODES, SCALE, None)
    record.lib.moe_mxfp4_dequantize(CODES, SCALE, rows, cols, X, dtype, cols, None)
    assert [l.kernel for l in record.take()] == [f"mx_quantize<{dtype}, {chunks}>", f"mx_dequantize<{dtype}, {chunks}>"]
