"""MXFP4 operators on the GPU against the float64 oracle.

Codes, scales and their values have to be equal.  A product's terms are exact
in float32 (8 x 2 significant bits, or 2 x 2), and a sum of K of them in any
order, each addition off by at most 2^-23 of its result (truncation included),
is off by at most K 2^-23 sum |a w|.  A bfloat16 result is the rounding of such
a sum: it lies between the roundings of that interval's ends."""
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


def _quantize(x):
    codes, scales = q.mxfp4_empty(*x.shape)
    codes.fill_(0xEE)
    scales.fill_(0xEE)
    q.moe_mxfp4_quantize(x, codes, scales)
    torch.cuda.synchronize()
    return codes, scales


def _same(a, b):
    return np.array_equal(np.asarray(a), np.asarray(b), equal_nan=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 31), (2, 33), (7, 64), (5, 250), (64, 256), (37, 2080),
                                       (257, 513), (1, 6144), (1000, 96), (2, 100001)])
def test_quantize_and_back(rows, cols, dtype):
    g = torch.Generator().manual_seed(rows * 7 + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-9, 9, (rows, cols), generator=g).float())
    x = x.to(DT[dtype])
    codes, scales = _quantize(x.cuda())
    rc, rs = ref.mx_quantize(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), rc)
    held = ref.mx_values(rc, rs)[:, :cols]
    for out in ("f32", "bf16", "f16"):
        y = torch.full((rows, cols), 7.0, dtype=DT[out], device="cuda")
        q.moe_mxfp4_dequantize(codes, scales, y)
        with np.errstate(over="ignore"):
            assert torch.equal(y.cpu(), torch.from_numpy(held).to(DT[out])), out


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_strided_rows(dtype, offset):
    """Rows inside a wider matrix, from any element: neither the source's
    padding is read into a block nor the destination's written."""
    big = torch.randn(9, 301, generator=torch.Generator().manual_seed(5)).to(DT[dtype]).cuda()
    big[:, :offset] = float("nan")
    big[:, offset + 130:] = float("nan")
    src = big[:, offset:offset + 130]
    codes, scales = _quantize(src)
    rc, rs = ref.mx_quantize(src.double().cpu().numpy())
    assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(scales.cpu().numpy(), rs)
    dst = torch.full_like(big, 5.0)
    q.moe_mxfp4_dequantize(codes, scales, dst[:, offset:offset + 130])
    assert (dst[:, :offset] == 5).all() and (dst[:, offset + 130:] == 5).all()
    assert torch.equal(dst[:, offset:offset + 130].cpu(),
                       torch.from_numpy(ref.mx_values(rc, rs)[:, :130]).to(DT[dtype]))


def test_values_at_the_ends_of_the_range():
    """Blocks of one magnitude each, from float32's smallest to its largest,
    signed zeros, and blocks with an infinity or a NaN."""
    mags = [0.0, 2.0 ** -149, 2.0 ** -130, 2.0 ** -127, 2.0 ** -126, 2.0 ** -125, 2.0 ** -124, 2.0 ** -100, 1.0,
            2.0 ** 100, 2.0 ** 127, 3.4028234663852886e38]
    x = torch.zeros(len(mags) + 4, 32)
    f = torch.linspace(-1, 1, 32)
    for i, m in enumerate(mags):
        x[i] = (f.double() * m).float()
    x[-4, 3] = float("inf")
    x[-3, 31] = -float("inf")
    x[-2, 0] = float("nan")
    x[-2, 1] = 3.0
    x[-1] = -0.0
    codes, scales = _quantize(x.cuda())
    rc, rs = ref.mx_quantize(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), rc)
    for out in ("f32", "bf16"):
        y = torch.empty(x.shape, dtype=DT[out], device="cuda")
        q.moe_mxfp4_dequantize(codes, scales, y)
        assert _same(y.double().cpu(), ref.mx_values(rc, rs))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_ties_go_to_the_even_code(dtype):
    """Every multiple of 1/8 up to 8 beside a 4, at three scales."""
    v = torch.arange(-64, 64).float() / 8
    x = torch.cat([torch.full((128, 1), 4.0), v[:, None], -v[:, None], torch.zeros(128, 29)], 1)
    x = torch.cat([x, x * 0.25, x * 64]).to(DT[dtype])
    codes, scales = _quantize(x.cuda())
    rc, rs = ref.mx_quantize(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), rs) and np.array_equal(codes.cpu().numpy(), rc)


def test_every_byte_decodes():
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1).cuda()            # [256][256]: 16 blocks a row
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 16).contiguous().cuda()
    held = ref.mx_values(codes.cpu().numpy(), scales.cpu().numpy())
    for out in ("f32", "bf16", "f16"):
        y = torch.empty(256, 512, dtype=DT[out], device="cuda")
        q.moe_mxfp4_dequantize(codes, scales, y)
        with np.errstate(over="ignore"):
            want = torch.from_numpy(held).float().to(DT[out])   # 6 * 2^127 is past float32
        assert _same(y.double().cpu(), want.double()), out


def test_no_rows():
    for cols in (1, 64):
        codes, scales = q.mxfp4_empty(0, cols)
        x = torch.empty(0, cols, device="cuda")
        q.moe_mxfp4_quantize(x, codes, scales)
        q.moe_mxfp4_dequantize(codes, scales, x)


# ---- products -----------------------------------------------------------------
class Problem:
    """Random weights [E][n][k] and rows split over the experts as `counts`
    says, `extra` rows past them belonging to none."""

    def __init__(self, counts, n, k, seed=0, extra=0, gather=0, scale_span=6):
        g = torch.Generator().manual_seed(seed)
        self.E, self.n, self.k = len(counts), n, k
        self.off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.R = int(self.off[-1]) + extra
        self.wq = torch.randint(0, 256, (self.E, n, k // 2), generator=g, dtype=torch.uint8)
        self.ws = torch.randint(124 - scale_span, 124 + scale_span, (self.E, n, k // 32), generator=g,
                                dtype=torch.uint8)
        self.index = None
        rows = self.R
        if gather:
            rows = gather
            self.index = torch.randint(0, rows, (self.R,), generator=g, dtype=torch.int32)
        self.a = (torch.randn(rows, k, generator=g) * 2).to(torch.bfloat16)
        self.dy = torch.randn(self.R, n, generator=g).to(torch.bfloat16)
        self.w64 = ref.mx_values(self.wq.numpy(), self.ws.numpy())

    def dev(self, t):
        return None if t is None else t.cuda()

    def offsets(self):
        return torch.from_numpy(self.off).cuda()


def _close(got, want, mag, terms, bf16):
    got = got.double().cpu().numpy()
    tol = terms * 2.0 ** -23 * mag + 1e-40
    lo, hi = want - tol, want + tol
    if bf16:
        lo, hi = (torch.from_numpy(v).float().to(torch.bfloat16).double().numpy() for v in (lo, hi))
    bad = ~((lo <= got) & (got <= hi))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4])


def _run(P, act, out, a=None, ldo=None, offsets=True):
    o = torch.full((P.R, (ldo or P.n)), 77.0, dtype=DT[out], device="cuda")[:, :P.n]
    a = P.a if a is None else a
    if act == "bf16":
        x64 = a.double().numpy()
        q.moe_mxfp4_matmul(a.cuda(), P.wq.cuda(), P.ws.cuda(), o, expert_offsets=P.offsets() if offsets else None,
                           row_index=P.dev(P.index))
    else:
        codes, scales = _quantize(a.cuda())
        x64 = ref.mx_values(codes.cpu().numpy(), scales.cpu().numpy())
        q.moe_mxfp4_matmul(codes, P.wq.cuda(), P.ws.cuda(), o, a_scale=scales,
                           expert_offsets=P.offsets() if offsets else None, row_index=P.dev(P.index))
    torch.cuda.synchronize()
    want, mag = ref.grouped_matmul(x64, P.w64, P.off, None if P.index is None else P.index.numpy(), P.R)
    live = int(P.off[-1])
    _close(o[:live], want[:live], mag[:live], P.k, out == "bf16")
    assert (o[live:] == 77.0).all()
    return o


SHAPES = [  # counts, n, k, extra, gather
    ([1], 1, 32, 0, 0), ([1], 16, 64, 0, 0), ([1], 2048, 2080, 0, 0), ([3], 17, 96, 0, 0),
    ([0, 1, 0, 2, 0], 33, 160, 1, 0), ([1] * 8, 256, 256, 0, 1), ([4, 0, 5, 1], 130, 288, 2, 6),
    ([16, 17, 15, 1], 64, 512, 0, 0), ([31, 33, 32, 0, 1], 100, 544, 3, 40), ([63, 65, 2], 257, 128, 0, 20),
    ([127, 129], 129, 256, 0, 0), ([200, 0, 3], 96, 1056, 5, 64), ([255, 257, 1], 512, 320, 0, 100),
    ([500], 260, 96, 0, 0), ([0, 0, 0], 64, 64, 4, 0), ([700, 20, 20], 36, 64, 0, 9), ([300, 5], 384, 2080, 0, 0),
    ([1] * 256, 48, 96, 0, 3), ([2, 0] * 100, 20, 128, 0, 0), ([1000, 1], 1001, 160, 0, 0)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("counts,n,k,extra,gather", SHAPES)
def test_matmul(counts, n, k, extra, gather, act, out):
    _run(Problem(counts, n, k, seed=n + k, extra=extra, gather=gather), act, out)


LARGE = [  # large enough for the tiles of 256 outputs with MXFP4 rows; every count of column tiles
    ([1100], 4097, 128, 0, 0), ([300, 0, 129, 17, 33, 65, 97, 1, 257, 150], 4100, 160, 3, 77), ([513, 512], 4608, 672, 0, 0),
    ([190, 70, 200, 256, 90, 40, 10, 20], 5000, 1152, 0, 500), ([200, 5, 120, 255, 30], 6300, 2112, 2, 33)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("counts,n,k,extra,gather", LARGE)
def test_large_matmul(counts, n, k, extra, gather, act, out):
    _run(Problem(counts, n, k, seed=n + k, extra=extra, gather=gather), act, out, ldo=n + 3 if k == 672 else None)


@pytest.mark.parametrize("k", [128, 352])
@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
def test_large_matmul_keeps_nan_in_place(act, k):
    """As below for the large tiles: NaN scales in the row after a tile's last
    block and in the last block itself, a NaN input, an index outside."""
    P = Problem([700, 400], 4100, k, seed=k, gather=300)
    P.index[3], P.index[900] = -1, 300
    P.a[7, k - 1] = float("nan")
    P.ws[1, 4099, 0] = 255
    P.ws[0, 77, k // 32 - 1] = 255
    o = torch.empty(1100, 4100, device="cuda")
    idx = P.index.cuda()
    if act == "bf16":
        q.moe_mxfp4_matmul(P.a.cuda(), P.wq.cuda(), P.ws.cuda(), o, expert_offsets=P.offsets(), row_index=idx)
    else:
        codes, scales = _quantize(P.a.cuda())
        q.moe_mxfp4_matmul(codes, P.wq.cuda(), P.ws.cuda(), o, a_scale=scales, expert_offsets=P.offsets(),
                           row_index=idx)
    nan = torch.isnan(o).cpu()
    want = (P.index == 7)[:, None].expand(1100, 4100).clone()
    want[:700, 77] = True
    want[700:, 4099] = True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("R", [1, 5, 40, 300])
def test_matmul_of_one_expert_without_offsets(R, act):
    _run(Problem([R], 192, 224, seed=R), act, "f32", offsets=False)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("R", [3, 50, 260])
@pytest.mark.parametrize("ldo", [65, 66, 68, 72, 80])
def test_output_strides(ldo, R, out):
    """The columns past n keep what they hold, whatever the stride."""
    P = Problem([R], 65 if ldo > 65 else 64, 128, seed=ldo)
    full = torch.full((R, ldo), 77.0, dtype=DT[out], device="cuda")
    q.moe_mxfp4_matmul(P.a.cuda(), P.wq.cuda(), P.ws.cuda(), full[:, :P.n], expert_offsets=P.offsets())
    want, mag = ref.grouped_matmul(P.a.double().numpy(), P.w64, P.off)
    _close(full[:, :P.n], want, mag, P.k, out == "bf16")
    assert (full[:, P.n:] == 77.0).all()


@pytest.mark.parametrize("R", [2, 40, 300])
def test_input_strides_leave_their_padding_out(R):
    P = Problem([R], 80, 96, seed=R)
    wide = torch.full((R, 96 + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :96] = P.a.cuda()
    o = torch.empty(R, 80, device="cuda")
    q.moe_mxfp4_matmul(wide[:, :96], P.wq.cuda(), P.ws.cuda(), o)
    want, mag = ref.grouped_matmul(P.a.double().numpy(), P.w64, P.off)
    _close(o, want, mag, 96, False)


@pytest.mark.parametrize("R", [3, 40, 300])
@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
def test_indices_outside_read_zeros(R, act):
    P = Problem([R], 64, 160, seed=R, gather=7)
    P.index[0], P.index[R // 2], P.index[R - 1] = -1, 7, 2 ** 31 - 1
    o = _run(P, act, "f32")
    assert (o[0] == 0).all() and (o[R // 2] == 0).all() and (o[R - 1] == 0).all()


@pytest.mark.parametrize("R", [2, 40, 300])
@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
def test_nan_and_infinity_stay_in_their_rows(R, act):
    """A NaN weight scale reaches its output column, a non-finite input its
    row, and neither any other value."""
    k = 352                                        # 11 blocks: the last tile is part full
    P = Problem([R, R], 70, k, seed=R)
    P.a[1, k - 1] = float("nan")
    P.a[R + 1, 5] = float("inf")
    P.ws[1, 69, k // 32 - 1] = 255
    o = torch.empty(2 * R, 70, device="cuda")
    a = P.a.cuda()
    if act == "bf16":
        q.moe_mxfp4_matmul(a, P.wq.cuda(), P.ws.cuda(), o, expert_offsets=P.offsets())
    else:
        codes, scales = _quantize(a)
        q.moe_mxfp4_matmul(codes, P.wq.cuda(), P.ws.cuda(), o, a_scale=scales, expert_offsets=P.offsets())
    o = o.cpu().numpy()
    hit = np.zeros(o.shape, bool)
    hit[1] = True
    hit[R + 1] = True
    hit[R:, 69] = True
    assert np.isfinite(o[~hit]).all()
    assert np.isnan(o[R:, 69]).all() and np.isnan(o[1]).all() and not np.isfinite(o[R + 1]).any()


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
def test_extreme_weight_scales(act):
    """Scales over most of their range: the product carries them exactly."""
    P = Problem([5, 40], 48, 64, seed=3)
    P.ws[:] = torch.randint(20, 234, P.ws.shape, generator=torch.Generator().manual_seed(1), dtype=torch.uint8)
    P.a = (P.a.float() * 2.0 ** -20).to(torch.bfloat16)
    P.w64 = ref.mx_values(P.wq.numpy(), P.ws.numpy())
    _run(P, act, "f32")


DX = [([1], 32, 32, 0), ([1], 256, 256, 0), ([2, 0, 3], 96, 160, 1), ([1] * 8, 512, 544, 0), ([16, 17, 1], 128, 512, 0),
      ([33, 31, 0, 64], 160, 1056, 2), ([127, 129], 256, 96, 0), ([300, 5], 2080, 288, 0), ([0, 0], 64, 64, 3),
      ([520], 64, 1536, 0), ([1] * 200, 32, 64, 0), ([2, 1, 1, 4], 4096, 128, 0),
      # large tiles
      ([300, 0, 129, 17, 33, 65, 97, 1, 257, 150], 160, 4128, 3), ([700], 96, 6112, 0), ([512, 513], 32, 4352, 0),
      ([200, 190, 70, 90, 40, 10], 1056, 7200, 0), ([1100], 224, 4096, 1)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("counts,n,k,extra", DX)
def test_dx(counts, n, k, extra, out):
    P = Problem(counts, n, k, seed=n + k, extra=extra)
    o = torch.full((P.R, k + 4), 77.0, dtype=DT[out], device="cuda")
    q.moe_mxfp4_matmul_dx(P.dy.cuda(), P.wq.cuda(), P.ws.cuda(), o[:, :k], expert_offsets=P.offsets())
    want, mag = ref.grouped_matmul(P.dy.double().numpy(), P.w64, P.off, rows=P.R, transpose=True)
    live = int(P.off[-1])
    _close(o[:live, :k], want[:live], mag[:live], n, out == "bf16")
    assert (o[live:] == 77.0).all() and (o[:, k:] == 77.0).all()


@pytest.mark.parametrize("R", [2, 40, 300])
def test_dx_nan_and_strides(R):
    P = Problem([R, 3], 96, 352, seed=R)
    wide = torch.full((R + 3, 96 + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :96] = P.dy.cuda()
    wide[1, 95] = float("nan")
    P.ws[0, 95, 10] = 255
    o = torch.empty(R + 3, 352, device="cuda")
    q.moe_mxfp4_matmul_dx(wide[:, :96], P.wq.cuda(), P.ws.cuda(), o, expert_offsets=P.offsets())
    o = o.cpu().numpy()
    assert np.isnan(o[1]).all() and np.isnan(o[:R, 320:]).all()
    o[1] = 0
    assert np.isfinite(o[:, :320]).all() and np.isfinite(o[R:]).all()


def test_large_dx_keeps_nan_in_place():
    """NaN scales in the row after the last term of an expert's sums and in one
    column block, a NaN in dy, dy rows inside a matrix of NaN."""
    n, k = 160, 4128
    P = Problem([700, 400], n, k, seed=1)
    wide = torch.full((1100, n + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :n] = P.dy.cuda()
    wide[9, n - 1] = float("nan")
    P.ws[1, 0] = 255
    P.ws[0, 33, 128] = 255
    o = torch.empty(1100, k, device="cuda")
    q.moe_mxfp4_matmul_dx(wide[:, :n], P.wq.cuda(), P.ws.cuda(), o, expert_offsets=P.offsets())
    want = torch.zeros(1100, k, dtype=torch.bool)
    want[9] = True
    want[:700, 4096:4128] = True
    want[700:] = True
    assert torch.equal(torch.isnan(o).cpu(), want)


@pytest.mark.parametrize("R", [4, 70])
def test_dx_is_the_products_gradient(R):
    """sum(dy * (out(a + d) - out(a - d))) = 2 sum(dx * d), the product being
    linear: differences of the forward kernel against the backward kernel."""
    P = Problem([R, R + 1], 128, 192, seed=R)
    g = torch.Generator().manual_seed(9)
    d = (torch.randn(P.a.shape, generator=g)).to(torch.bfloat16)
    hi, lo = (P.a.float() + d.float()).to(torch.bfloat16), (P.a.float() - d.float()).to(torch.bfloat16)
    step = hi.double() - lo.double()
    wq, ws, off = P.wq.cuda(), P.ws.cuda(), P.offsets()
    outs = []
    for x in (hi, lo):
        o = torch.empty(P.R, 128, device="cuda")
        q.moe_mxfp4_matmul(x.cuda(), wq, ws, o, expert_offsets=off)
        outs.append(o.double().cpu())
    dx = torch.empty(P.R, 192, device="cuda")
    q.moe_mxfp4_matmul_dx(P.dy.cuda(), wq, ws, dx, expert_offsets=off)
    left = (P.dy.double() * (outs[0] - outs[1])).sum().item()
    right = (dx.double().cpu() * step).sum().item()
    w = np.abs(P.w64)
    mag = sum((np.abs(P.dy[r].double().numpy()) @ w[0 if r < R else 1]) @
              (np.abs(hi[r].double().numpy()) + np.abs(lo[r].double().numpy())) for r in range(P.R))
    assert abs(left - right) <= (192 + 128) * 2.0 ** -23 * mag


def test_products_repeat_bit_for_bit_on_any_stream():
    P = Problem([3, 0, 40, 150], 200, 416, seed=1, gather=50)
    a, wq, ws, off, idx = P.a.cuda(), P.wq.cuda(), P.ws.cuda(), P.offsets(), P.index.cuda()
    dy = torch.randn(P.R, 192).to(torch.bfloat16).cuda()
    w2, s2 = wq[:, :192].contiguous(), ws[:, :192].contiguous()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    res = []
    for s in (torch.cuda.current_stream(), side, side):
        o, d = torch.empty(P.R, 200, device="cuda"), torch.empty(P.R, 416, device="cuda")
        torch.cuda.synchronize()
        q.moe_mxfp4_matmul(a, wq, ws, o, expert_offsets=off, row_index=idx, stream=s)
        q.moe_mxfp4_matmul_dx(dy, w2, s2, d, expert_offsets=off, stream=s)
        s.synchronize()
        res.append((o, d))
    for o, d in res[1:]:
        assert torch.equal(o, res[0][0]) and torch.equal(d, res[0][1])


def test_operators_in_a_graph():
    P = Problem([2, 30], 64, 96, seed=4)
    x = P.a.cuda()
    wq, ws, off = P.wq.cuda(), P.ws.cuda(), P.offsets()
    codes, scales = q.mxfp4_empty(P.R, 96)
    o = torch.empty(P.R, 64, device="cuda")

    def step():
        q.moe_mxfp4_quantize(x, codes, scales)
        q.moe_mxfp4_matmul(codes, wq, ws, o, a_scale=scales, expert_offsets=off)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x.copy_((torch.randn(P.R, 96, generator=torch.Generator().manual_seed(i)) * 3).to(torch.bfloat16))
        step()
        want = o.clone()
        o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want), i


def test_offsets_that_do_not_ascend_stay_inside():
    """Undefined rows, but nothing is read or written past the buffers."""
    P = Problem([10, 20], 64, 64, seed=2)
    off = torch.tensor([-5, 12, 90], dtype=torch.int32, device="cuda")
    o = torch.full((P.R + 8, 64), 77.0, device="cuda")
    q.moe_mxfp4_matmul(P.a.cuda(), P.wq.cuda(), P.ws.cuda(), o[:P.R], expert_offsets=off)
    torch.cuda.synchronize()
    assert (o[P.R:] == 77.0).all()
    want, mag = ref.grouped_matmul(P.a.double().numpy(), P.w64, [0, 12, 30])
    _close(o[:P.R], want, mag, 64, False)


# Rows, outputs and sums that reach every kernel: items of 64 rows, of 256 x 256
# and of 128 x 512, with runs of every length.
MANY = [300, 0, 500, 290, 129, 170, 200, 257, 511, 640, 33, 193, 192, 800]
NARROW = [(7 * i) % 129 for i in range(256)]
FORMS = [([64, 3, 17, 33, 0, 130, 100, 81], 701, 160, 0), ([257, 1], 2050, 1056, 1), ([40] * 32, 513, 128, 2),
         ([300, 16, 33], 1000, 288, 0), (MANY, 2555, 160, 1), (MANY, 2559, 256, 0), (NARROW, 1021, 96, 3)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("gather", [0, 77])
@pytest.mark.parametrize("counts,n,k,extra", FORMS)
def test_forms(counts, n, k, extra, gather, out):
    _run(Problem(counts, n, k, seed=n, extra=extra, gather=gather), "bf16", out)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("counts,n,k,extra", [
    ([250, 1, 300, 64, 0, 885], 64, 1440, 0), ([33] * 64, 32, 1056, 1), ([700, 800], 352, 1504, 0),
    (MANY, 96, 2528, 1), (NARROW, 64, 992, 0)])
def test_forms_of_dx(counts, n, k, extra, out):
    test_dx(counts, n, k, extra, out)


@pytest.mark.parametrize("counts,n", [([200, 300], 1001), (MANY, 2555)])
@pytest.mark.parametrize("k", [128, 352])
def test_forms_keep_nan_in_place(counts, n, k):
    P = Problem(counts, n, k, seed=k, gather=200)
    c0 = counts[0]
    P.index[3], P.index[c0 + 9] = -1, 200
    P.index[7] = 7
    P.a[7, k - 1] = float("nan")
    P.ws[2 if counts[1] == 0 else 1, n - 1, 0] = 255
    P.ws[0, 77, k // 32 - 1] = 255
    o = torch.empty(P.R, n, device="cuda")
    q.moe_mxfp4_matmul(P.a.cuda(), P.wq.cuda(), P.ws.cuda(), o, expert_offsets=P.offsets(), row_index=P.index.cuda())
    e2 = slice(c0, c0 + max(counts[1], counts[2] if counts[1] == 0 else 0))
    want = torch.zeros(P.R, n, dtype=torch.bool)
    want[P.index == 7] = True
    want[:c0, 77] = True
    want[e2, n - 1] = True
    assert torch.equal(torch.isnan(o).cpu(), want)
