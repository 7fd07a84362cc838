"""MXFP4 operators on the GPU at sizes that reach every kernel and every branch
of it, against the float64 oracle (bounds as in test_gpu_mxfp4.py)."""
import numpy as np
import pytest
import torch

import product_forms
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


@pytest.mark.parametrize("kernel,kind,counts,n,k,extra,gather", product_forms.PRODUCTS, ids=product_forms.NAMES)
def test_every_kernel(kernel, kind, counts, n, k, extra, gather):
    """Values, and NaN in place: a NaN at the end of a row's inputs, NaN scales
    in an expert's first and last blocks, indices outside.  Outputs at whole
    lines and at an odd pitch."""
    far = gather == product_forms.FAR
    P = Problem(counts, n, k, seed=n + k, extra=extra, gather=1 if far else gather)
    live = int(P.off[-1])
    used = [e for e, c in enumerate(counts) if c]
    first, last = used[0], used[-1]
    off = P.offsets() if P.E > 1 else None
    if kind == "dx":
        P.dy[live - 1, n - 1] = float("nan")
        P.ws[first, n - 1, 0] = P.ws[last, 0, k // 32 - 1] = 255
        src = P.dy.double().numpy()
    else:
        P.ws[first, 7, k // 32 - 1] = P.ws[last, n - 1, 0] = 255
        if far:
            P.index = torch.randint(0, gather, (P.R,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
            a = torch.empty(gather, k, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(2))
        else:
            a = P.a.cuda()
        if P.index is not None and live > 4:
            P.index[1], P.index[live - 2] = -1, a.shape[0]
        a[live - 1 if P.index is None else int(P.index[live - 1]), k - 1] = float("nan")
        src, args = a, {}
        if kind == "mxfp4":
            codes, scales = _quantize(a)
            src = ref.mx_values(codes.cpu().numpy(), scales.cpu().numpy())
            a, args = codes, {"a_scale": scales}
        elif far:
            at = P.index.long().clamp(0, gather - 1)
            src = a[at.cuda()].double().cpu().numpy()
            src[((P.index < 0) | (P.index >= gather)).numpy()] = 0
        else:
            src = a.double().cpu().numpy()
    w64 = ref.mx_values(P.wq.numpy(), P.ws.numpy())
    index = None if P.index is None or far or kind == "dx" else P.index.numpy()
    want, mag = ref.grouped_matmul(src, w64, P.off, index, P.R, transpose=kind == "dx")
    want, mag = want[:live], mag[:live]
    nan = np.isnan(want)
    assert 0 < nan.sum() and (not nan.all() or live < 3)
    cols, terms = (k, n) if kind == "dx" else (n, k)
    wq, ws = P.wq.cuda(), P.ws.cuda()
    for out, pitch in (("f32", -(-cols // 64) * 64), ("bf16", -(-cols // 64) * 64), ("bf16", cols + 3)):
        full = torch.full((P.R, pitch), 77.0, dtype=DT[out], device="cuda")
        if kind == "dx":
            q.moe_mxfp4_matmul_dx(P.dy.cuda(), wq, ws, full[:, :cols], expert_offsets=off)
        else:
            q.moe_mxfp4_matmul(a, wq, ws, full[:, :cols], expert_offsets=off, row_index=P.dev(P.index), **args)
        got = full[:live, :cols]
        assert np.array_equal(torch.isnan(got).cpu().numpy(), nan), (out, pitch)
        _close(got[torch.from_numpy(~nan).cuda()], want[~nan], mag[~nan], terms, out == "bf16")
        assert (full[live:] == 77.0).all() and (full[:, cols:] == 77.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols,pitch", [(4099, 4097, 4097), (4099, 4097, 4102), (20000, 4097, 4097)])
def test_conversions_of_every_kernel(rows, cols, pitch, dtype):
    """One and four chunks per lane: rows of an odd length that repeat with a
    period that no workgroup's share has."""
    period = 37
    g = torch.Generator().manual_seed(cols)
    x = torch.randn(period, cols, generator=g) * torch.exp2(torch.randint(-9, 9, (period, cols), generator=g).float())
    x = x.to(DT[dtype])
    wide = torch.full((rows, pitch), float("nan"), dtype=DT[dtype], device="cuda")
    src = wide[:, :cols]
    src.copy_(x.cuda().repeat(rows // period + 1, 1)[:rows])
    codes, scales = _quantize(src)
    rc, rs = ref.mx_quantize(x.double().numpy())
    back = torch.full((rows, pitch), 7.0, dtype=DT[dtype], device="cuda")
    q.moe_mxfp4_dequantize(codes, scales, back[:, :cols])
    held = torch.from_numpy(ref.mx_values(rc, rs)[:, :cols]).to(DT[dtype])
    for got, want in ((codes, torch.from_numpy(rc)), (scales, torch.from_numpy(rs)), (back[:, :cols], held)):
        assert torch.equal(got, want.cuda().repeat(rows // period + 1, 1)[:rows])
    assert (back[:, cols:] == 7.0).all()


@pytest.mark.parametrize("ends", ["low", "high", "top"])
@pytest.mark.parametrize("kernel", sorted({p[0] for p in product_forms.PRODUCTS}))
def test_ends_of_the_scale_range(kernel, ends):
    """Weights of the smallest scales (bf16 has them as subnormals) and the
    largest, with inputs that keep the sums finite: exact products throughout.
    Weights of 2^128 and more (scales 253 and 254) are infinities beside bf16
    rows and in the gradient, and exact beside MXFP4 rows."""
    _, kind, counts, n, k, extra, gather = next(p for p in product_forms.PRODUCTS if p[0] == kernel)
    P = Problem(counts, n, k, seed=n + k, extra=extra, gather=gather)
    lo, hi = {"low": (0, 4), "high": (250, 253), "top": (240, 250)}[ends]
    P.ws = torch.randint(lo, hi, P.ws.shape, generator=torch.Generator().manual_seed(7), dtype=torch.uint8)
    if ends == "top":
        P.ws[:, 5], P.ws[:, 6, 0] = 253, 254
    if ends != "low":
        P.a, P.dy = ((t.float() * 2.0 ** -30).to(torch.bfloat16) for t in (P.a, P.dy))
    w64 = ref.mx_values(P.wq.numpy(), P.ws.numpy())
    wq, ws, off = P.wq.cuda(), P.ws.cuda(), P.offsets()
    got = torch.full((P.R, k if kind == "dx" else n), 77.0, device="cuda")
    if kind == "dx":
        src = P.dy.double().numpy()
        q.moe_mxfp4_matmul_dx(P.dy.cuda(), wq, ws, got, expert_offsets=off)
    elif kind == "bf16":
        src = P.a.double().numpy()
        q.moe_mxfp4_matmul(P.a.cuda(), wq, ws, got, expert_offsets=off, row_index=P.dev(P.index))
    else:
        codes, scales = _quantize(P.a.cuda())
        src = ref.mx_values(codes.cpu().numpy(), scales.cpu().numpy())
        q.moe_mxfp4_matmul(codes, wq, ws, got, a_scale=scales, expert_offsets=off, row_index=P.dev(P.index))
    if kind != "mxfp4":
        w64[np.abs(w64) >= 2.0 ** 128] *= np.inf
    with np.errstate(invalid="ignore"):
        want, mag = ref.grouped_matmul(src, w64, P.off, None if P.index is None or kind == "dx" else P.index.numpy(), P.R,
                                       transpose=kind == "dx")
    live = int(P.off[-1])
    got, want, mag = got[:live], want[:live], mag[:live]
    fin = np.isfinite(want)
    assert fin.any() and (fin.all() or (ends == "top" and kind != "mxfp4"))
    assert np.array_equal(got.cpu().numpy()[~fin], want[~fin].astype(np.float32), equal_nan=True)
    _close(got[torch.from_numpy(fin).cuda()], want[fin], mag[fin], n if kind == "dx" else k, False)
