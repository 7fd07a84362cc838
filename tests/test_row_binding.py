"""The binding of the row operators without a GPU: where the tensors of a call have
to lie, and what of their shapes, types and layouts it refuses."""
import pytest
import torch

import quantized_moe_02_amd as q
from quantized_moe_02_amd import binding
from test_operator_binding import On, Reached, no_library  # noqa: F401

BF, F = torch.bfloat16, torch.float32


def _calls():
    """name -> (call of a list of tensors, the tensors)."""
    z = lambda *s, dt=BF: torch.zeros(*s, dtype=dt)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    e4 = lambda *s: u8(*s).view(torch.float8_e4m3fn)
    return {
        "norm": (lambda a: q.moe_rmsnorm(a[0], a[1], 1e-6, y=a[2], residual=a[3], h=a[4], q=a[5], q_scale=a[6]),
                 [z(2, 64), z(64), z(2, 64), z(2, 64), z(2, 64), e4(2, 64), z(2, dt=F)]),
        "norm to MXFP4": (lambda a: q.moe_rmsnorm(a[0], a[1], 1e-6, q=a[2], q_scale=a[3]), [z(2, 64), z(64, dt=F), u8(2, 32), u8(2, 2)]),
        "norm_grad": (lambda a: q.moe_rmsnorm_grad(*a[:3], 1e-6, a[3], dh=a[4], dweight=a[5], ws=a[6]),
                      [z(2, 64), z(2, 64), z(64), z(2, 64), z(2, 64), z(64, dt=F), u8(1 << 12)]),
        "dispatch": (lambda a: q.moe_dispatch(*a), [z(2, 64), i32(2, 3), z(6, 64)]),
        "dispatch of E4M3": (lambda a: q.moe_dispatch(*a[:3], x_scale=a[3], row_scale=a[4]),
                             [e4(2, 64), i32(2, 3), e4(6, 64), z(2, dt=F), z(6, dt=F)]),
        "dispatch of MXFP4": (lambda a: q.moe_dispatch(*a[:3], x_scale=a[3], row_scale=a[4]),
                              [u8(2, 32), i32(2, 3), u8(6, 32), u8(2, 2), u8(6, 2)]),
        "collect": (lambda a: q.moe_collect(*a[:3], weights=a[3], addend=a[4]), [z(6, 64), i32(2, 3), z(2, 64), z(2, 3, dt=F), z(2, 64)]),
        "collect_grad": (lambda a: q.moe_collect_grad(a[0], a[1], drows=a[2], weights=a[3], rows=a[4], dweights=a[5]),
                         [z(2, 64), i32(2, 3), z(6, 64), z(2, 3, dt=F), z(6, 64), z(2, 3, dt=F)]),
        "swiglu": (lambda a: q.moe_swiglu(a[0], a[1], expert_offsets=a[2]), [z(2, 64), z(2, 32), i32(4)]),
        "swiglu to E4M3": (lambda a: q.moe_swiglu(a[0], a[1], out_scale=a[2], expert_offsets=a[3]), [z(2, 64), e4(2, 32), z(2, dt=F), i32(4)]),
        "swiglu to MXFP4": (lambda a: q.moe_swiglu(a[0], a[1], out_scale=a[2]), [z(2, 64), u8(2, 16), u8(2, 1)]),
        "swiglu_grad": (lambda a: q.moe_swiglu_grad(*a[:3], expert_offsets=a[3]), [z(2, 64), z(2, 32), z(2, 64), i32(4)])}


def _refused(call):
    with pytest.raises(q.QmoeError) as ei:
        call()
    assert ei.value.status == q.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("name", _calls())
def test_tensors_lie_on_the_current_device(name, no_library, monkeypatch):  # noqa: F811
    call, tensors = _calls()[name]
    with pytest.raises(Reached):                     # all on it: nothing is refused
        call([On.of(t) for t in tensors])
    for far in [{i} for i in range(len(tensors))] + [set(range(len(tensors)))]:
        _refused(lambda: call([On.of(t, int(i in far)) for i, t in enumerate(tensors)]))
    for host in range(len(tensors)):
        _refused(lambda: call([t if i == host else On.of(t) for i, t in enumerate(tensors)]))
    monkeypatch.setattr(binding, "_several", True)
    monkeypatch.setattr(binding, "_current_device", lambda: 1)      # all on device 0, which is not the current one
    _refused(lambda: call([On.of(t) for t in tensors]))


# tensors that say a size themselves: rows in expert order, experts, picks a token
FREE_ROWS = {("dispatch", 2), ("collect", 0), ("swiglu", 2), ("swiglu to E4M3", 3), ("swiglu_grad", 3)}
FREE_COLUMNS = {("dispatch", 1), ("dispatch of E4M3", 1), ("dispatch of MXFP4", 1)}


@pytest.mark.parametrize("name", _calls())
def test_shapes_types_and_layouts(name, no_library):  # noqa: F811
    call, tensors = _calls()[name]
    for i, t in enumerate(tensors):
        other = [torch.zeros(t.shape, dtype=torch.float64), torch.zeros(t.shape, dtype=torch.float16)]
        if (name, i) != ("norm_grad", 6):                                      # a workspace of any shape
            other.append(t[None])
            if (name, i) not in FREE_ROWS:
                other.append(t[:-1].contiguous())
            if t.dim() == 1:
                other.append(torch.stack([t, t], 1)[:, 0])                     # a vector with gaps
            elif (name, i) not in FREE_COLUMNS:
                other.append(t[:, :-1].contiguous())
            if t.dim() == 2 and t.shape[1] > 1:
                other.append(t.t().contiguous().t())                           # columns apart
        for o in other:
            _refused(lambda: call([On.of(v) for v in tensors[:i] + [o] + tensors[i + 1:]]))


def test_combinations(no_library):  # noqa: F811
    on = On.of
    z = lambda *s, dt=BF: on(torch.zeros(*s, dtype=dt))
    x, w, inv = z(2, 64), z(64), on(torch.zeros(2, 3, dtype=torch.int32))
    _refused(lambda: q.moe_rmsnorm(x, w, 1e-6, y=z(2, 64), h=z(2, 64)))                         # h without a residual
    _refused(lambda: q.moe_rmsnorm(x, w, 1e-6, residual=z(2, 64), h=z(2, 64, dt=F)))            # of another type
    _refused(lambda: q.moe_rmsnorm(x, w, 1e-6, q=on(torch.zeros(2, 64, dtype=torch.uint8).view(torch.float8_e4m3fn))))   # no scales
    _refused(lambda: q.moe_rmsnorm_grad(x, x, w, 1e-6, z(2, 64), dh=z(2, 64, dt=F)))
    _refused(lambda: q.moe_dispatch(x, inv, z(6, 64), x_scale=z(2, dt=F)))
    _refused(lambda: q.moe_dispatch(x, inv, on(torch.zeros(6, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)), row_scale=z(6, dt=F)))
    _refused(lambda: q.moe_collect_grad(x, inv))
    _refused(lambda: q.moe_collect_grad(x, inv, drows=z(6, 64), dweights=z(2, 3, dt=F)))        # nothing to multiply with
    _refused(lambda: q.moe_collect_grad(x, inv, drows=z(6, 64), rows=z(6, 64, dt=F)))
    _refused(lambda: q.moe_collect_grad(x, inv, drows=z(6, 65)[:, :64], rows=z(6, 64)))         # another stride
    _refused(lambda: q.moe_swiglu(z(2, 65), z(2, 32)))
    _refused(lambda: q.moe_swiglu(x, z(2, 32), out_scale=z(2, dt=F)))
    _refused(lambda: q.moe_swiglu_grad(x, z(2, 32), z(2, 65)[:, :64]))
    for call in (lambda: q.moe_rmsnorm(z(3, 70)[:, 3:67], w, 1e-6, y=z(3, 99)[:, :64]), lambda: q.moe_swiglu(z(2, 80)[:, 8:72], z(2, 33)[:, 1:]),
                 lambda: q.moe_collect(z(6, 65)[:, 1:], inv, z(2, 66)[:, :64])):
        with pytest.raises(Reached):                 # rows at a pitch of their own are taken
            call()


def test_sizes_past_the_limits(monkeypatch):
    """A matrix of more than 2^31 rows, an eps past fp32."""
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0)
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    far = lambda *s: On.of(torch.empty(s, dtype=BF, device="meta"))
    w = On.of(torch.zeros(1))
    for call in (lambda: q.moe_rmsnorm(far(3 << 31, 1), w, 1e-6, y=far(3 << 31, 1)), lambda: q.moe_swiglu(far(3 << 31, 2), far(3 << 31, 1)),
                 lambda: q.moe_rmsnorm(On.of(torch.zeros(2, 1)), w, 1e39, y=On.of(torch.zeros(2, 1)))):
        with pytest.raises(q.QmoeError):
            call()
