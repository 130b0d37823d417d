"""A step's pool of states is checked like its other tensors."""
import pytest
import torch

import fft_long_convolution_gb300 as F


def plans(monkeypatch):
    """Plans without a device to create them on."""
    for cls in (F.LinearAttention, F.DeltaRule):
        plan = cls.__new__(cls)
        plan.Dk = plan.Dv = 64
        plan.torch_dtype, plan._scale, plan._h = torch.bfloat16, 1.0, None
        monkeypatch.setattr(plan, "_args", lambda *a: None)
        yield plan


def test_missing_and_misshapen_pools_are_refused(monkeypatch):
    q = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    for plan in plans(monkeypatch):
        gates = (torch.zeros(2),) if isinstance(plan, F.LinearAttention) else (q[..., 0], q[..., 0])
        for state in (None, torch.zeros(()), torch.zeros(0), torch.zeros(2, 64, 64), torch.zeros(1, 3, 64, 64),
                      torch.zeros(1, 2, 64, 64, dtype=torch.float64)):
            with pytest.raises(ValueError, match="state"):
                plan.step(q, q, q, *gates, state)
