"""Activations in 8 bits at the ends of bf16's range."""
import math

import pytest

from tests import training_ref as ref
from tests.test_training_gpu import make, same, ssa  # noqa: F401  (ssa: the fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("D", [64, 128])
def test_save_of_the_largest_values(ssa, D):  # noqa: F811
    """What is finite is restored finite: near the type's largest value, where
    the next E4M3 value times the scale would be infinite, the one below is taken."""
    top = torch.finfo(torch.bfloat16).max
    x = torch.zeros(200, 3, D, dtype=torch.bfloat16)
    steps = torch.arange(0x7F00, 0x7F80, dtype=torch.int16).view(torch.bfloat16)  # every value from 2^127 up
    x[:64, 0, 0], x[:64, 0, 1] = steps[:64], -steps[64:]
    x[64:128, 0, 2] = steps[64:]
    x[5, 1, 3], x[6, 1, 3], x[7, 1, 4] = top, math.inf, math.nan
    x[150, 2, 5], x[151, 2, 5] = -top, 1.0
    got = ssa.restore_fp8(*ssa.save_fp8(x.cuda())).cpu()
    ssa.check_device()
    assert torch.equal(torch.isnan(got), ~torch.isfinite(x)) and not torch.isinf(got).any()
    y = x.double().nan_to_num(0.0, 0.0, 0.0) / 2.0 ** 120
    want = torch.where(y.abs() >= 248, 240.0 * torch.sign(y), ref.e4m3_nearest(y)) * 2.0 ** 120
    assert torch.equal(got.double().nan_to_num(0.0), want)


def test_bwd_from_the_largest_saved_values(ssa):  # noqa: F811
    """Finite activations keep finite gradients through save_fp8."""
    q, k, v, dout, cu = make([100], 1, 1, 64, seed=44)
    v[3, 0, 5] = torch.finfo(torch.bfloat16).max
    dout *= 2.0 ** -20  # dout . v stays in fp32's range
    out, lse = ssa.fwd_lse(q, k, v, cu, 100)
    saved = [ssa.save_fp8(t) for t in (q, k, v)]
    grads = ssa.bwd_fp8(dout, *saved, out, lse, cu, 100)
    plain = ssa.bwd(dout, *[ssa.restore_fp8(*s) for s in saved], out, lse, cu, 100)
    ssa.check_device()
    assert all(torch.isfinite(g).all() for g in grads) and all(same(a, b) for a, b in zip(grads, plain))
