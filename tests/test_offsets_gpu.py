"""Offsets of a batch that cannot be: the kernels' own check reports them and
writes nothing, also where the difference of two offsets passes 32 bits."""
import numpy as np
import pytest

from tests.test_training_gpu import make, ssa  # noqa: F401  (ssa: the fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

LOW = -2 ** 31
# (offsets, 500 tokens): one sequence, two, and more than a warp has lanes
BATCHES = [[5, LOW], [1, LOW + 1], [0, LOW], [300, LOW, 500], [0, 300, LOW], [LOW, 0, 300], [300, LOW + 299, 500],
           [7 * i for i in range(40)] + [LOW, 400], [7 * i for i in range(40)] + [LOW]]


def fits(offsets, total):
    """The check in Python's unbounded integers."""
    return offsets[0] >= 0 and all(a <= b <= total for a, b in zip(offsets, offsets[1:]))


def test_differences_that_pass_32_bits_are_among_the_batches():
    with np.errstate(over="ignore"):
        wrapped = [any(np.int32(b) - np.int32(a) > 0 > b - a for a, b in zip(x, x[1:])) for x in BATCHES]
    assert sum(wrapped) >= 6 and not any(fits(x, 500) for x in BATCHES)


@pytest.mark.parametrize("offsets", BATCHES, ids=lambda x: f"{x[:3]}{len(x) - 1}")
@pytest.mark.parametrize("D", [64, 128])
def test_offsets_that_decrease_past_32_bits(ssa, offsets, D):  # noqa: F811
    q, k, v, dout, good = make([500], 2, 2, D, seed=45)
    out, lse = ssa.fwd_lse(q, k, v, good, 500)
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    fresh = lambda *ts: [torch.full_like(t, 7.0) for t in ts]
    ssa.check_device()

    def refused(made):
        assert ssa.get_error() == ssa.SSA_ERR_DEVICE_ARG
        assert all((t == 7).all() for t in made)

    for tsf in (0.0, 100.0):
        made = fresh(out, lse)
        ssa.fwd_lse(q, k, v, cu, 500, tsf, out=made[0], lse=made[1])
        refused(made)
        made = fresh(out)
        ssa.fwd(q, k, v, cu, 500, tsf, out=made[0])
        refused(made)
    made = fresh(out)
    counts = torch.full((2, 4, 2), 7, dtype=torch.int32, device="cuda")
    ssa.calibrate(q, k, v, cu, 500, [0.1, 0.5], out=made[0], counts=counts)
    refused(made + [counts])
    made = fresh(q, k, v)
    ssa.bwd(dout, q, k, v, out, lse, cu, 500, dq=made[0], dk=made[1], dv=made[2])
    refused(made)
