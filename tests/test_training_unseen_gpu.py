"""Gradients depend on what a row sees and on nothing else: keys without
probability, tiles that were skipped, rows that take no part and memory past a
sequence leave no trace, whatever stands there."""
import math

import pytest

from tests import training_ref as ref
from tests.test_training_gpu import BATCHES, bitmap_for, make, same, ssa  # noqa: F401  (ssa: the fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# Batches whose blocks are walked by one CTA each (many heads) and by clusters.
SHAPES = [([300], 2, 2, 128), ([300], 4, 2, 64), ([700, 200], 16, 16, 128), ([700, 200], 24, 12, 64)]


def formula(ssa, dout, q, k, v, out, lse, cu, lens, bitmap=None):  # noqa: F811
    grads = ssa.bwd(dout, q, k, v, out, lse, cu, max(lens), decision_bitmap=bitmap)
    ssa.check_device()
    want, bound = ref.backward(dout, q, k, v, out, lse, lens, bitmap)
    seen = ref.bound_dq(dout, q, k, v, out, lse, lens, bitmap)
    for g, w, b, name in zip(grads, want, (seen, *bound[1:]), ("dq", "dk", "dv")):
        ref.check(g, w, b, name)
    return grads


@pytest.mark.parametrize("lens", BATCHES + [[2000, 1], [1300] * 3], ids=str)
@pytest.mark.parametrize("H,Hk,D", [(2, 2, 128), (4, 2, 64), (16, 4, 128)])
@pytest.mark.parametrize("tsf", [0.0, 200.0])
def test_dq_over_the_seen_keys(ssa, lens, H, Hk, D, tsf):  # noqa: F811
    """Keys with much in common (a position code three times the noise), which
    cancels in dQ but would not in dS rounded once to bf16."""
    q, k, v, dout, cu = make(lens, H, Hk, D, seed=46, amp=3.0)
    bm = bitmap_for(ssa, lens, H) if tsf else None
    out, lse = ssa.fwd_lse(q, k, v, cu, max(lens), tsf, decision_bitmap=bm)
    formula(ssa, dout, q, k, v, out, lse, cu, lens, bm)


@pytest.mark.parametrize("lens,H,Hk,D", SHAPES, ids=str)
def test_keys_without_probability(ssa, lens, H, Hk, D):  # noqa: F811
    """Every block's first key, and a whole block of keys, at scores at which
    fp32 and fp64 exponentials are zero: their size does not matter by a bit."""
    q, k, v, dout, cu = make(lens, H, Hk, D, seed=40)
    q[..., 0] = 128.0  # scores along the first dimension: c * 128 * k[0]
    first = [t for lo, hi in zip(cu.tolist(), cu.tolist()[1:]) for t in range(lo, hi, 128)]
    for unseen in (first, list(range(128, 256))):
        seen = torch.ones(k.shape[0], dtype=torch.bool)
        seen[unseen] = False
        before = None
        for size in (1e3, 1e5, 1e30):
            kk = k.clone()
            kk[..., 0] = kk[..., 0] / 128  # the others' scores stay in an ordinary range
            kk[unseen, :, 0] = -size
            vv = v.clone()
            vv[unseen] = vv[unseen] * size ** 0.5
            out, lse = ssa.fwd_lse(q, kk, vv, cu, max(lens))
            grads = formula(ssa, dout, q, kk, vv, out, lse, cu, lens)
            assert not grads[1][unseen].any() and not grads[2][unseen].any()
            if before is not None:
                assert same(out, before[0])
                assert all(torch.equal(a, b) for a, b in zip(grads, before[1:]))
            before = (out, *grads)


@pytest.mark.parametrize("lens,H,Hk,D", SHAPES, ids=str)
def test_keys_of_skipped_tiles(ssa, lens, H, Hk, D):  # noqa: F811
    """Query block b skips tile b (its own rows), and every block of a sequence
    of three tiles or more skips tile 1: the keys there may have any size."""
    q, k, v, dout, cu = make(lens, H, Hk, D, seed=41)
    bm = bitmap_for(ssa, lens, H)
    bm.zero_()
    unit = 0
    for n in lens:
        for b in range((n + 127) // 128):
            bm[:, unit, 0] = (1 << b) | (2 if n > 256 else 0)
            unit += 1
    # out and lse of the kept tiles, by the formula
    o, L, _, _ = ref.forward(q, k, v, lens, bm)
    out, lse = o.bfloat16().cuda(), L.float().cuda()
    rows = slice(128, 256)  # tile 1 of the first sequence: skipped by every block
    before = None
    for offset in (0.0, 30.0, 1e4, 1e30):
        kk, vv = k.clone(), v.clone()
        kk[rows] += offset
        vv[rows] += offset
        grads = formula(ssa, dout, q, kk, vv, out, lse, cu, lens, bm)
        assert not grads[1][rows].any() and not grads[2][rows].any()
        if before is not None:
            assert all(torch.equal(a, b) for a, b in zip(grads, before))
        before = grads
    # each block's own keys, which other blocks see: its own dQ does not change
    kk, vv = k.clone(), v.clone()
    kk[:128] += 1e4
    vv[:128] += 1e4
    dq = ssa.bwd(dout, q, kk, vv, out, lse, cu, max(lens), decision_bitmap=bm)[0]
    ssa.check_device()
    assert torch.equal(dq[:128], before[0][:128])


@pytest.mark.parametrize("lens,H,Hk,D", SHAPES + [([1, 128, 5], 2, 1, 64)], ids=str)
@pytest.mark.parametrize("tsf", [0.0, 200.0])
def test_rows_that_take_no_part(ssa, lens, H, Hk, D, tsf):  # noqa: F811
    """A row whose lse is -inf has no gradient and no part in any other,
    whatever its q, out and dout hold: single rows (a block's first and last
    among them), a whole block, and one row of one head alone."""
    q, k, v, dout, cu = make(lens, H, Hk, D, seed=42, amp=3.0)
    bm = bitmap_for(ssa, lens, H) if tsf else None
    out, lse = ssa.fwd_lse(q, k, v, cu, max(lens), tsf, decision_bitmap=bm)
    total = sum(lens)
    dead = torch.zeros(H, total, dtype=torch.bool, device="cuda")
    dead[:, [t for t in (0, 5, 127, 130, total - 1) if t < total]] = True
    dead[:, 128:256] |= total > 256
    dead[0, total // 2] = True
    lse = lse.masked_fill(dead, -math.inf)
    rows = dead.T[..., None]
    finite = [t.masked_fill(rows, 0.0) for t in (dout, q, out)]
    want, bound = ref.backward(finite[0], finite[1], k, v, finite[2], lse, lens, bm)
    plain = ssa.bwd(finite[0], finite[1], k, v, finite[2], lse, cu, max(lens), decision_bitmap=bm)
    for g, w, b, name in zip(plain, want, bound, ("dq", "dk", "dv")):
        ref.check(g, w, b, name)
    for bad in (math.nan, math.inf, torch.finfo(torch.bfloat16).max):
        for which in ((2,), (0, 2), (0, 1, 2)):
            args = [t.masked_fill(rows, bad) if i in which else t for i, t in enumerate((dout, q, out))]
            grads = ssa.bwd(args[0], args[1], k, v, args[2], lse, cu, max(lens), decision_bitmap=bm)
            ssa.check_device()
            assert not grads[0].masked_select(rows).any()
            assert all(torch.equal(a, b) for a, b in zip(grads, plain)), (bad, which)


@pytest.mark.parametrize("tsf", [0.0, 30.0])
@pytest.mark.parametrize("H,Hk,D", [(2, 1, 128), (16, 16, 128), (16, 16, 64)])
def test_memory_past_a_sequence_while_skipping(ssa, tsf, H, Hk, D):  # noqa: F811
    """NaN and infinities behind the last sequence and in a sequence between two
    others, with the forward's own decisions: last tiles that end inside and are
    kept by both, one or none of the forward's two query blocks of a CTA."""
    lens, extra = [1100, 130, 70, 640, 1], 90
    q, k, v, dout, cu = make(lens, H, Hk, D, seed=43, extra=extra, amp=3.0)
    n, lo, hi = sum(lens), 1230, 1300
    ends = []

    def run(q, k, v, dout):
        bm = bitmap_for(ssa, lens, H)
        out, lse = torch.full_like(q, 3.0), torch.full((H, n + extra), 5.0, device="cuda")
        ssa.fwd_lse(q, k, v, cu, max(lens), tsf, out=out, lse=lse, decision_bitmap=bm)
        grads = [torch.full_like(t, 7.0) for t in (q, k, v)]
        ssa.bwd(dout, q, k, v, out, lse, cu, max(lens), decision_bitmap=bm, dq=grads[0], dk=grads[1], dv=grads[2])
        ssa.check_device()
        ends.append(bm)
        return [out, lse.T] + grads

    want = run(q, k, v, dout)
    if tsf:  # the last tile (8) of the first sequence: blocks 2i and 2i + 1 share a CTA
        last = (ends[0][:, :8, 0] >> 8) & 1
        pairs = last.view(H, 4, 2).sum(-1)
        assert all((pairs == m).any() for m in (0, 1, 2)), pairs
    units = torch.tensor([u for u, seq in enumerate([0] * 9 + [1] * 2 + [2] + [3] * 5 + [4]) if seq != 2], device="cuda")
    for bad in (math.nan, math.inf, -math.inf):
        poisoned = [t.clone() for t in (q, k, v, dout)]
        for t in poisoned:
            t[n:] = bad
        for w, g in zip(want, run(*poisoned)):
            assert same(w.contiguous(), g.contiguous())
        assert torch.equal(ends[0], ends[-1])
        for t in poisoned:
            t[lo:hi] = bad
        for w, g in zip(want, run(*poisoned)):
            for part in (slice(0, lo), slice(hi, n), slice(n, n + extra)):
                assert same(w[part].contiguous(), g[part].contiguous())
        assert torch.equal(ends[0][:, units], ends[-1][:, units])
