"""The binding of the MXFP4 and router-balance operators without a GPU: where
the tensors of a call have to lie."""
import pytest
import torch

import quantized_moe_02_amd as q
from quantized_moe_02_amd import binding


class On(torch.Tensor):
    """A host tensor that says it lies on device `at`."""
    at = 0

    @staticmethod
    def of(t, at=0):
        t = torch.Tensor._make_subclass(On, t)
        t.at = at
        return t

    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.at


def _calls():
    """name -> (call of a list of tensors, the tensors)."""
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    x, bf = torch.zeros(2, 64), torch.zeros(2, 64).bfloat16()
    w, ws, off = u8(3, 64, 32), u8(3, 64, 2), i32(4)
    bal = [x, i32(2, 2), i32(1, 64), i32(1)]
    return {
        "quantize": (lambda a: q.moe_mxfp4_quantize(*a), [x, u8(2, 32), u8(2, 2)]),
        "dequantize": (lambda a: q.moe_mxfp4_dequantize(*a), [u8(2, 32), u8(2, 2), x]),
        "matmul": (lambda a: q.moe_mxfp4_matmul(*a[:4], expert_offsets=a[4], row_index=a[5]),
                   [bf, w, ws, x, off, i32(2)]),
        "matmul of MXFP4 rows": (lambda a: q.moe_mxfp4_matmul(*a[:4], a_scale=a[4], expert_offsets=a[5]),
                                 [u8(2, 32), w, ws, x, u8(2, 2), off]),
        "matmul_dx": (lambda a: q.moe_mxfp4_matmul_dx(*a[:4], expert_offsets=a[4]), [bf, w, ws, x, off]),
        "balance": (lambda a: q.moe_balance_loss(*a[:5], coef=1.0, seq_offsets=a[5], ws=a[6]),
                    bal + [torch.zeros(1), i32(2), u8(1 << 20)]),
        "balance_grad": (lambda a: q.moe_balance_loss_grad(*a[:5], coef=1.0, seq_offsets=a[5], dloss=a[6]),
                         bal + [x, i32(2), torch.zeros(1)])}


class Reached(Exception):
    pass


@pytest.fixture
def no_library(monkeypatch):
    class Library:
        moe_status_string = q.lib().moe_status_string

        def __getattr__(self, name):
            raise Reached
    monkeypatch.setattr(binding, "lib", Library)
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0)


@pytest.mark.parametrize("name", _calls())
def test_tensors_lie_on_the_current_device(name, no_library, monkeypatch):
    call, tensors = _calls()[name]
    with pytest.raises(Reached):                     # all on it: nothing is refused
        call([On.of(t) for t in tensors])
    for far in [{i} for i in range(len(tensors))] + [set(range(len(tensors)))]:
        with pytest.raises(q.QmoeError) as ei:
            call([On.of(t, int(i in far)) for i, t in enumerate(tensors)])
        assert ei.value.status == q.MOE_ERR_INVALID_ARG, far
    monkeypatch.setattr(binding, "_several", True)
    monkeypatch.setattr(binding, "_current_device", lambda: 1)      # all on device 0, which is not the current one
    with pytest.raises(q.QmoeError):
        call([On.of(t) for t in tensors])
    for host in range(len(tensors)):
        with pytest.raises(q.QmoeError):
            call([t if i == host else On.of(t) for i, t in enumerate(tensors)])
