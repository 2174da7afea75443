"""The gated block and its gradients at shapes that reach every tile of its products (gated_cases.py), with the checks and
tolerances of test_gpu_gated.py."""

import pytest

import torch

from gated_cases import DW, DX, FORWARD
from test_gpu_gated import Case, announce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", [s for shapes in FORWARD.values() for s in shapes])
def test_forward_tiles(shape, dt):
    announce("forward tile", *shape, dt)
    for pre in (True, False):
        c = Case(*shape, dt, "gelu_tanh" if dt == "bf16" else "silu", seed=sum(shape))
        d = c.device()
        c.forward(d, pre)
        torch.cuda.synchronize()
        c.check(d, grad=False, pre=pre)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", sorted({*DX.values(), *DW.values()}))
def test_gradient_tiles(shape, dt):
    announce("gradient tile", *shape, dt)
    c = Case(*shape, dt, seed=sum(shape))
    d = c.device()
    c.forward(d, pre=dt == "bf16")
    c.backward(d, pre=dt == "bf16")
    torch.cuda.synchronize()
    c.check(d, pre=dt == "bf16")
