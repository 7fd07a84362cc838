"""Shared by the tests of the row operators: bounds from the number of roundings
(each is off by at most half a step), matrices at a pitch of their own."""
import numpy as np
import torch

U = 2.0 ** -24                       # half a step of fp32, relative
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -134}     # the types' last steps below their normal range
BF, F = torch.bfloat16, torch.float32


def pitched(shape, dtype, pad=0, fill=None, gen=None, scale=1.0):
    """A matrix on the GPU whose rows lie `pad` elements apart from each other and
    that starts `pad` elements into its memory; normal values, or `fill`."""
    r, c = shape
    buf = torch.full((pad + r * (c + pad) + pad,), float("nan") if fill is None else fill, dtype=dtype, device="cuda")
    m = buf[pad:pad + r * (c + pad)].view(r, c + pad)[:, :c] if r else buf[:0].view(0, c)
    if gen is not None:
        m.copy_((torch.randn(r, c, generator=gen) * scale).to(dtype))
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, want, bound, dtype, what=""):
    """|got - want| <= bound (of the fp32 arithmetic) + one rounding of that value
    to dtype; NaN in the same places."""
    g = f64(got)
    assert g.shape == want.shape, (what, g.shape, want.shape)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(g), nan), what
    tol = bound + HALF[dtype] * (np.abs(want) + bound) + TINY[dtype]
    with np.errstate(invalid="ignore"):
        off = np.where(nan | (g == want), 0, np.abs(g - want) - tol)
    assert (off <= 0).all(), (what, "off by", float(np.nanmax(off)), "over the bound at",
                              np.unravel_index(int(np.nanargmax(off)), off.shape))


def picks(T, K, experts, gen, drop=0.0):
    """Slots in expert order as moe_permute gives them, -1 for dropped picks."""
    ids = torch.rand(T, experts, generator=gen).topk(K, dim=1).indices
    gone = torch.rand(T, K, generator=gen) < drop
    ids[gone] = experts
    order = torch.argsort(ids.reshape(-1), stable=True)
    inv = torch.empty(T * K, dtype=torch.int32)
    inv[order] = torch.arange(T * K, dtype=torch.int32)
    return torch.where(gone, -1, inv.view(T, K)).to(torch.int32)


def silu_bound(g):
    """Relative error of sigmoid(g) as the kernels form it, from x = e^-|g| (its
    argument rounded at its own size, the constant log2(e) too, the hardware's
    power and reciprocal one unit each) and three more operations."""
    return (1.5 * np.abs(g) + 12) * U
