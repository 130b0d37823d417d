"""Tensors of another GPU than the call's are refused (no GPU needed: stand-ins
answer what the binding asks of a tensor)."""
import pytest
import torch

import fft_long_convolution_gb300 as F


class Stand:
    """A contiguous CUDA tensor on GPU `index`, as far as the argument checks look."""
    is_cuda = True

    def __init__(self, dtype, shape, index):
        self.dtype, self.shape, self.index = dtype, torch.Size(shape), index

    def get_device(self):
        return self.index

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


def raises_device(f):
    with pytest.raises(ValueError, match="GPU"):
        f()


@pytest.fixture(autouse=True)
def current(monkeypatch):
    monkeypatch.setattr(F, "_current_device", lambda: 0, raising=False)


@pytest.mark.parametrize("other", ["q", "k", "v", "g", "beta", "offsets"])
def test_delta_rule(other):
    dt, B, T, H, D = torch.bfloat16, 1, 5, 2, 64
    plan = F.DeltaRule.__new__(F.DeltaRule)  # without a device to create a plan on
    plan.Dk = plan.Dv = D
    plan.torch_dtype, plan._scale, plan._h = dt, 1.0, None
    shapes = dict(q=(B, T, H, D), k=(B, T, H, D), v=(B, T, H, D), g=(B, T, H), beta=(B, T, H), offsets=(3,))

    def args(dev):
        x = {n: Stand(torch.int32 if n == "offsets" else dt, s, dev(n)) for n, s in shapes.items()}
        return plan._args(x["q"], x["k"], x["v"], x["g"], x["beta"], x["offsets"], None)

    assert args(lambda n: 0).nseq == 2
    raises_device(lambda: args(lambda n: 1 if n == other else 0))
    raises_device(lambda: args(lambda n: 1))  # all on a GPU that is not the current one


@pytest.mark.parametrize("what,dtype", [("state", torch.float32), ("slots", torch.int32), ("saved", torch.uint8)])
def test_other_operands(what, dtype):
    assert F._dense(Stand(dtype, (4,), 0), what, dtype, (4,), 0) == 1 << 20
    raises_device(lambda: F._dense(Stand(dtype, (4,), 1), what, dtype, (4,), 0))


@pytest.mark.parametrize("other", ["q", "k", "wq", "wk", "cos", "sin", "positions"])
def test_qk_norm(other):
    dt, B, T, H, D, R = torch.bfloat16, 1, 5, 2, 64, 32
    plan = F.QKNorm(D, dt, rotary=R)
    f32 = torch.float32
    kinds = dict(q=(dt, (B, T, H, D)), k=(dt, (B, T, H, D)), wq=(f32, (D,)), wk=(f32, (D,)), cos=(f32, (9, R // 2)),
                 sin=(f32, (9, R // 2)), positions=(torch.int32, (B, T)))

    def args(dev):
        return plan._args(*(Stand(*kinds[n], dev(n)) for n in kinds))

    assert args(lambda n: 0).T == T
    raises_device(lambda: args(lambda n: 1 if n == other else 0))
    raises_device(lambda: args(lambda n: 1))
