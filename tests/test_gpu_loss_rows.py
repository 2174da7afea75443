"""What one row of a loss call may not do to another."""

import pytest
import torch

from test_gpu_loss import Case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def announce(*what):
    print("case:", *what, flush=True)


@pytest.mark.parametrize("top", [0, 5])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_values_of_rows_that_do_not_count_change_nothing(dt, top):
    """A padding row may hold any number: the gradients are those with zeros in it, to the bit."""
    announce("huge ignored row", dt, top)
    c = Case(40, 300, 64, dt, top=top, seed=21, absent=0.0)
    c.index[[3, 17]] = -100
    d = c.device()
    want = {}
    for fill in (0.0, 3e38 if dt == "bf16" else 65504.0):
        d["h"][[3, 17]] = fill
        c.forward(d)
        c.backward(d)
        torch.cuda.synchronize()
        got = {x: d[x].clone() for x in ("loss", "dh", "dw")}
        want = want or got
        assert all(torch.equal(got[x], want[x]) for x in want), [x for x in want if not torch.equal(got[x], want[x])]
