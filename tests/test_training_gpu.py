"""The training operators on the GPU against plain 64-bit implementations:
fwd_lse, bwd, save_fp8 / restore_fp8 / bwd_fp8, rotary and the autograd
functions over them. Tolerances are elementwise bounds computed from the
operands (tests/training_ref.py)."""
import math

import numpy as np
import pytest

from tests import training_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ssa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_flashattention_ssa_b200 as m

    return m


def make(lens, H, Hk, D, seed=0, extra=0, amp=1.0):
    """q, k, v, dout, cu_seqlens: noise plus a slow position code, so that tiles differ in weight."""
    g = torch.Generator().manual_seed(seed)
    total = sum(lens) + extra
    pos = torch.cat([torch.arange(n) for n in lens] + [torch.zeros(extra, dtype=torch.long)]).float()
    code = torch.stack([(pos[:, None] / 64 * 1.3 ** -torch.arange(D // 2)).sin(),
                        (pos[:, None] / 64 * 1.3 ** -torch.arange(D // 2)).cos()], -1).reshape(total, 1, D) * amp
    n = lambda h: torch.randn(total, h, D, generator=g)
    q, k, v, dout = n(H) + code, n(Hk) + code, n(Hk), n(H)
    cu = torch.tensor(ref.bounds(lens), dtype=torch.int32)
    return [t.bfloat16().cuda() for t in (q, k, v, dout)] + [cu.cuda()]


def bits(t):
    return t.view({2: torch.int16, 4: torch.int32, 1: torch.uint8}[t.element_size()])


def same(a, b):
    return torch.equal(bits(a), bits(b))


RAGGED = [1, 5, 127, 128, 129, 300, 0, 700]
BATCHES = [[1], [2], [127], [128], [129], [257, 0, 1], RAGGED, [0, 0, 64], [3] * 40 + [200]]


def bitmap_for(ssa, lens, H):
    return torch.full((H, ssa.num_qblocks(ref.bounds(lens)), ssa.bitmap_words(max(lens))), -1, dtype=torch.int32,
                      device="cuda")


# ------------------------------------------------------------------ forward

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tsf", [0.0, 300.0])
def test_fwd_lse_is_the_forward(ssa, D, tsf):
    lens = RAGGED
    q, k, v, _, cu = make(lens, 3, 3, D, seed=1, amp=3.0)
    bm, bm2 = bitmap_for(ssa, lens, 3), bitmap_for(ssa, lens, 3)
    sc, sc2 = (torch.full((3, bm.shape[1]), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    want = ssa.fwd(q, k, v, cu, max(lens), tsf, skip_counter=sc, decision_bitmap=bm)
    out, lse = ssa.fwd_lse(q, k, v, cu, max(lens), tsf, skip_counter=sc2, decision_bitmap=bm2)
    plain, lse2 = ssa.fwd_lse(q, k, v, cu, max(lens), tsf)
    ssa.check_device()
    assert same(out, want) and same(plain, want) and same(lse, lse2)
    assert torch.equal(bm, bm2) and torch.equal(sc, sc2)
    if tsf:
        assert int(sc.sum()) > 0


@pytest.mark.parametrize("lens", BATCHES, ids=str)
@pytest.mark.parametrize("H,Hk,D", [(2, 2, 128), (4, 2, 64), (3, 1, 128)])
def test_fwd_lse_formula(ssa, lens, H, Hk, D):
    q, k, v, _, cu = make(lens, H, Hk, D, seed=2)
    out, lse = ssa.fwd_lse(q, k, v, cu, max(lens))
    ssa.check_device()
    o, L, ob, Lb = ref.forward(q, k, v, lens)
    ref.check(out, o, ob, "out")
    ref.check(lse, L, Lb, "lse")


# ----------------------------------------------------------------- backward

@pytest.mark.parametrize("lens", BATCHES, ids=str)
@pytest.mark.parametrize("H,Hk,D", [(2, 2, 128), (4, 2, 64), (3, 1, 128)])
def test_bwd_formula(ssa, lens, H, Hk, D):
    q, k, v, dout, cu = make(lens, H, Hk, D, seed=3)
    out, lse = ssa.fwd_lse(q, k, v, cu, max(lens))
    grads = ssa.bwd(dout, q, k, v, out, lse, cu, max(lens))
    ssa.check_device()
    want, bound = ref.backward(dout, q, k, v, out, lse, lens)
    for g, w, b, name in zip(grads, want, bound, ("dq", "dk", "dv")):
        ref.check(g, w, b, name)


@pytest.mark.parametrize("lens,H,Hk,D", [([1300, 1], 16, 16, 64), ([1300, 1], 16, 8, 128), ([700], 24, 12, 64),
                                         ([2000], 3, 3, 128), ([1030], 1, 1, 128), ([400] * 3, 16, 16, 128)], ids=str)
def test_bwd_whole_and_shared_blocks(ssa, lens, H, Hk, D):
    """Batches whose blocks are walked by one CTA each, or by clusters of 2, 4 and 8."""
    q, k, v, dout, cu = make(lens, H, Hk, D, seed=20)
    out, lse = ssa.fwd_lse(q, k, v, cu, max(lens))
    grads = ssa.bwd(dout, q, k, v, out, lse, cu, max(lens))
    ssa.check_device()
    want, bound = ref.backward(dout, q, k, v, out, lse, lens)
    for g, w, b, name in zip(grads, want, bound, ("dq", "dk", "dv")):
        ref.check(g, w, b, name)


@pytest.mark.parametrize("S,H,D,times", [(5120, 24, 128, 20), (4096, 12, 64, 40), (640, 4, 64, 100)])
def test_bwd_waits_end(ssa, S, H, D, times):
    """Many passes over long walks: no wait of the kernel's pipeline is missed
    (a barrier that goes round unseen would run into the time limit), and
    every pass gives the same bits."""
    q, k, v, dout, cu = make([S], H, H, D, seed=21)
    out, lse = ssa.fwd_lse(q, k, v, cu, S)
    first = ssa.bwd(dout, q, k, v, out, lse, cu, S)
    for _ in range(times):
        again = ssa.bwd(dout, q, k, v, out, lse, cu, S)
    ssa.check_device()
    assert all(same(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hk", [(2, 2), (4, 2)])
@pytest.mark.parametrize("scale", [0.0, 0.3])
def test_bwd_on_the_kept_tiles(ssa, D, H, Hk, scale):
    lens = [1100, 130, 1, 640]
    q, k, v, dout, cu = make(lens, H, Hk, D, seed=4, amp=3.0)
    bm = bitmap_for(ssa, lens, H)
    out, lse = ssa.fwd_lse(q, k, v, cu, max(lens), 400.0, scale, decision_bitmap=bm)
    grads = ssa.bwd(dout, q, k, v, out, lse, cu, max(lens), scale, bm)
    ssa.check_device()
    assert int((bm != 0).sum()) > 0  # something was skipped
    o, L, ob, Lb = ref.forward(q, k, v, lens, bm, scale)
    ref.check(out, o, ob, "out")
    ref.check(lse, L, Lb, "lse")
    want, bound = ref.backward(dout, q, k, v, out, lse, lens, bm, scale)
    for g, w, b, name in zip(grads, want, bound, ("dq", "dk", "dv")):
        ref.check(g, w, b, name)


def test_bwd_more_than_32_tiles_and_a_sparse_map(ssa):
    """4,500 tokens: 36 tiles, two bitmap words, with a random map that leaves
    some blocks a single tile and some none at all."""
    lens, H, D = [4500, 77], 2, 128
    q, k, v, dout, cu = make(lens, H, 1, D, seed=5)
    rng = np.random.default_rng(0)
    bm = bitmap_for(ssa, lens, H)
    words = rng.integers(0, 2 ** 32, size=bm.shape, dtype=np.uint64)
    words[:, 3] = 0xFFFFFFFF          # nothing kept
    words[:, 7] = 0xFFFFFFFF
    words[:, 7, 1] = 0xFFFFFFFF ^ 4   # tile 34 only
    words[0, :] |= 1 << 9             # one K/V tile kept by head 1 alone
    words[:, :, 0] |= 1 << 20         # and one kept by nobody
    bm.copy_(torch.from_numpy(words.astype(np.uint32).view(np.int32)))
    lse = ref.forward(q, k, v, lens)[1].float().cuda()  # any lse will do: the formula takes it as given
    out = torch.randn_like(q)
    grads = ssa.bwd(dout, q, k, v, out, lse, cu, max(lens), decision_bitmap=bm)
    ssa.check_device()
    want, bound = ref.backward(dout, q, k, v, out, lse, lens, bm)
    for g, w, b, name in zip(grads, want, bound, ("dq", "dk", "dv")):
        ref.check(g, w, b, name)
    assert not grads[0][3 * 128:4 * 128].any() and not grads[1][20 * 128:21 * 128].any()


@pytest.mark.parametrize("S,H,Hk,D", [(5200, 4, 4, 128), (700, 2, 2, 128), (900, 8, 2, 64), (300, 4, 1, 128)])
def test_bwd_of_blocks_that_kept_nothing(ssa, S, H, Hk, D):
    """Zero gradients, every time, beside blocks with one tile: such a CTA is
    done before its own first loads have arrived."""
    q, k, v, dout, cu = make([S], H, Hk, D, seed=32)
    out, lse = ssa.fwd_lse(q, k, v, cu, S)
    bm = bitmap_for(ssa, [S], H)
    for _ in range(30):
        grads = [torch.full_like(t, 7.0) for t in (q, k, v)]
        ssa.bwd(dout, q, k, v, out, lse, cu, S, decision_bitmap=bm, dq=grads[0], dk=grads[1], dv=grads[2])
        assert not any(g.any() for g in grads)
    bm[:, 1, 0] = ~2  # query block 1 keeps tile 1
    for _ in range(30):
        dq, dk, dv = ssa.bwd(dout, q, k, v, out, lse, cu, S, decision_bitmap=bm)
        for g in (dq, dk, dv):
            assert not g[:128].any() and not g[256:].any() and g[128:256].any()
    ssa.check_device()


def test_bwd_of_nothing_beside_the_largest_keys(ssa):
    q, k, v, dout, cu = make([256], 2, 2, 128, seed=33)
    k.fill_(torch.finfo(torch.bfloat16).max)
    q.zero_()  # scores of zero, and sums of keys that would overflow
    out, lse = ssa.fwd_lse(q, k, v, cu, 256)
    bm = bitmap_for(ssa, [256], 2)
    for g in ssa.bwd(dout, q, k, v, out, lse, cu, 256, decision_bitmap=bm):
        assert not g.any()


def test_bwd_against_differences(ssa):
    """Directional differences of sum(dout * out) in 64 bits at the bf16 inputs."""
    lens, H, Hk, D = [70, 140], 2, 1, 64
    q, k, v, dout, cu = make(lens, H, Hk, D, seed=6)
    out, lse = ssa.fwd_lse(q, k, v, cu, max(lens))
    grads = ssa.bwd(dout, q, k, v, out, lse, cu, max(lens))
    ssa.check_device()
    # the gradients from the exact out and lse, whose bounds the kernel's differ
    # from by what the rounding of out to bf16 moves D: P |dout| U |out| in dS
    o, L, ob, _ = ref.forward(q, k, v, lens)
    exact, bound = ref.backward(dout, q, k, v, o, L, lens)
    (_, _, _), wide = ref.backward(dout, q, k, v, out, lse, lens)
    rng = torch.Generator().manual_seed(0)
    for i, (x, name) in enumerate(((q, "q"), (k, "k"), (v, "v"))):
        d = torch.randn(x.shape, generator=rng, dtype=torch.float64)
        args = [t.double().cpu() for t in (q, k, v)]
        f = []
        for h in (1e-5, -1e-5):
            moved = list(args)
            moved[i] = args[i] + h * d
            f.append(float((ref.forward(*moved, lens)[0] * dout.double().cpu()).sum()))
        slope = (f[0] - f[1]) / 2e-5
        along = float((exact[i] * d).sum())
        assert abs(slope - along) <= 1e-5 * (1 + float((exact[i] * d).abs().sum())), name
        # D off by e moves dS by P e: |dq| by at most c e max|k| summed P = 1, dk by c sum_r P e |q_r|
        e = float((dout.double().cpu().abs() * ob).sum(-1).max())
        slack = e * (lens[1] * 2 if i == 1 else 1) * float(max(q.abs().max(), k.abs().max())) / math.sqrt(D) if i < 2 else 0.0
        ref.check(grads[i], exact[i], wide[i] + bound[i] + slack, "d" + name)


def test_memory_past_a_sequence_has_no_effect(ssa):
    """NaN and infinities behind the last sequence, and a NaN sequence between
    two others: the other rows do not change by a bit, rows of no sequence are
    left as they were."""
    lens, H, Hk, D, extra = [130, 70, 200], 2, 1, 128, 90
    q, k, v, dout, cu = make(lens, H, Hk, D, seed=7, extra=extra)
    n, a, b = sum(lens), 130, 200

    def run(q, k, v, dout):
        out, lse = torch.full_like(q, 3.0), torch.full((H, n + extra), 5.0, device="cuda")
        ssa.fwd_lse(q, k, v, cu, max(lens), out=out, lse=lse)
        grads = [torch.full_like(t, 7.0) for t in (q, k, v)]
        ssa.bwd(dout, q, k, v, out, lse, cu, max(lens), dq=grads[0], dk=grads[1], dv=grads[2])
        ssa.check_device()
        return [out, lse.T] + grads

    want = run(q, k, v, dout)
    assert (want[0][n:] == 3).all() and (want[1][n:] == 5).all() and all((g[n:] == 7).all() for g in want[2:])
    for bad in (math.nan, math.inf, -math.inf):
        poisoned = [t.clone() for t in (q, k, v, dout)]
        for t in poisoned:
            t[n:] = bad
        for w, g in zip(want, run(*poisoned)):
            assert same(w[:n].contiguous(), g[:n].contiguous()) and same(w[n:].contiguous(), g[n:].contiguous())
        for t in poisoned:
            t[a:b] = bad
        for w, g in zip(want, run(*poisoned)):
            for part in (slice(0, a), slice(b, n), slice(n, n + extra)):
                assert same(w[part].contiguous(), g[part].contiguous())


def test_rows_that_saw_nothing(ssa):
    """lse = -inf (no column): no gradient from those rows."""
    lens, D = [200], 64
    q, k, v, dout, cu = make(lens, 1, 1, D, seed=8)
    out, lse = ssa.fwd_lse(q, k, v, cu, 200)
    lse[0, 5:150] = -math.inf
    grads = ssa.bwd(dout, q, k, v, out, lse, cu, 200)
    ssa.check_device()
    want, bound = ref.backward(dout, q, k, v, out, lse, lens)
    for g, w, b, name in zip(grads, want, bound, ("dq", "dk", "dv")):
        ref.check(g, w, b, name)
    assert not grads[0][5:150].any()


def test_bwd_repeats_and_runs_beside_itself(ssa):
    lens = [900, 40, 513]
    args = [make(lens, 4, 2, 128, seed=s) for s in (9, 10)]
    fw = [ssa.fwd_lse(*a[:3], a[4], max(lens)) for a in args]
    call = lambda i, s=None: ssa.bwd(args[i][3], *args[i][:3], *fw[i], args[i][4], max(lens), stream=s)
    want = [call(0), call(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [call(i, streams[i]) for i in (0, 1)]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert all(same(x, y) for x, y in zip(w, g))
    ssa.check_device()


def test_inconsistent_batches_write_nothing(ssa):
    lens = [300, 200]
    q, k, v, dout, cu = make(lens, 2, 2, 64, seed=11)
    out, lse = ssa.fwd_lse(q, k, v, cu, 300)
    bm = torch.zeros((2, 5, 1), dtype=torch.int32, device="cuda")
    ssa.check_device()
    tries = [(torch.tensor([0, 300, 200], dtype=torch.int32, device="cuda"), 300, None),   # decreasing
             (torch.tensor([0, 300, 501], dtype=torch.int32, device="cuda"), 300, None),   # past the tokens
             (torch.tensor([-1, 300, 500], dtype=torch.int32, device="cuda"), 300, None),
             (torch.tensor([0, 100, 500], dtype=torch.int32, device="cuda"), 300, bm),     # longer than max_seqlen
             (torch.tensor([0, 128, 500], dtype=torch.int32, device="cuda"), 400, bm)]     # 4 q-blocks, sized for 5
    for cu_bad, longest, bitmap in tries:
        grads = [torch.full_like(t, 7.0) for t in (q, k, v)]
        ssa.bwd(dout, q, k, v, out, lse, cu_bad, longest, decision_bitmap=bitmap, dq=grads[0], dk=grads[1], dv=grads[2])
        assert ssa.get_error() == ssa.SSA_ERR_DEVICE_ARG
        assert all((g == 7).all() for g in grads)
        o2, l2 = torch.full_like(q, 7.0), torch.full_like(lse, 7.0)
        ssa.fwd_lse(q, k, v, cu_bad, longest, out=o2, lse=l2, decision_bitmap=None if bitmap is None else bitmap.clone())
        assert ssa.get_error() == ssa.SSA_ERR_DEVICE_ARG
        assert (o2 == 7).all() and (l2 == 7).all()
    empty = [t[:0].contiguous() for t in (q, k, v, dout)]
    cu0 = torch.zeros(3, dtype=torch.int32, device="cuda")
    o, L = ssa.fwd_lse(*empty[:3], cu0, 0)
    assert [tuple(g.shape) for g in ssa.bwd(empty[3], *empty[:3], o, L, cu0, 0)] == [(0, 2, 64)] * 3
    ssa.check_device()


# --------------------------------------------------- activations in 8 bits

@pytest.mark.parametrize("T,H,D", [(1, 1, 64), (127, 3, 128), (128, 2, 64), (300, 5, 128), (1000, 1, 64)])
def test_save_and_restore(ssa, T, H, D):
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, D, generator=g) * torch.exp2(torch.randint(-40, 40, (T // 128 + 1, H, 1), generator=g).float()
                                                       ).repeat_interleave(128, 0)[:T]
    x = x.bfloat16()
    x[0, 0, :8] = torch.tensor([0.0, -0.0, 1.75, 448.0, -449.0, 1e-30, 2.0 ** -9, 3.0 * 2.0 ** -10]).bfloat16()
    if H > 1:
        x[:, 1] = 0                     # nothing but zeros
    if H > 2:
        x[:, 2] = 2.0 ** -133           # the smallest subnormals
        x[T // 2, 2, 3] = 3.0e38        # beside the largest
    if T > 130:
        x[130, 0, 5], x[131, 0, 6], x[132, 0, 7] = math.nan, math.inf, -math.inf
    codes, scales = ssa.save_fp8(x.cuda())
    got = ssa.restore_fp8(codes, scales)
    ssa.check_device()
    want, want_scales = ref.saved(x)
    assert torch.equal(scales.double().cpu(), want_scales)
    assert torch.equal(torch.isnan(got).cpu(), torch.isnan(want))
    assert torch.equal(got.double().cpu().nan_to_num(0.0), want.nan_to_num(0.0))


@pytest.mark.parametrize("H,Hk,D,tsf", [(2, 2, 128, 0.0), (4, 1, 64, 400.0)])
def test_bwd_from_saved(ssa, H, Hk, D, tsf):
    lens = [513, 1, 200]
    q, k, v, dout, cu = make(lens, H, Hk, D, seed=12, amp=2.0)
    bm = bitmap_for(ssa, lens, H) if tsf else None
    out, lse = ssa.fwd_lse(q, k, v, cu, max(lens), tsf, decision_bitmap=bm)
    saved = [ssa.save_fp8(t) for t in (q, k, v)]
    back = [ssa.restore_fp8(*s) for s in saved]
    grads = ssa.bwd_fp8(dout, *saved, out, lse, cu, max(lens), decision_bitmap=bm)
    plain = ssa.bwd(dout, *back, out, lse, cu, max(lens), decision_bitmap=bm)
    ssa.check_device()
    assert all(same(a, b) for a, b in zip(grads, plain))
    want, bound = ref.backward(dout, *[ref.saved(t)[0] for t in (q, k, v)], out, lse, lens, bm)
    for g, w, b, name in zip(grads, want, bound, ("dq", "dk", "dv")):
        ref.check(g, w, b, name)


# ------------------------------------------------------------------- rotary

ROTARY = [(1, 1, 1, 8, 8, 1), (3, 2, 1, 64, 64, 1), (129, 5, 2, 128, 128, 3), (50, 3, 3, 64, 30, 1), (33, 1, 4, 128, 2, 2),
          (17, 2, 2, 72, 56, 1), (10, 2, 1, 64, 0, 1), (1000, 24, 24, 128, 96, 3), (5, 2, 2, 256, 256, 4),
          (21, 3, 1, 256, 250, 2), (40, 2, 7, 128, 126, 1), (77, 1, 1, 128, 66, 1)]


@pytest.mark.parametrize("T,H,Hk,D,rot,axes", ROTARY)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("transpose", [False, True])
def test_rotary(ssa, T, H, Hk, D, rot, axes, interleaved, transpose):
    from block_sparse_flashattention_ssa_b200 import positions as pos

    g = torch.Generator().manual_seed(T + rot)
    q, k = torch.randn(T, H, D, generator=g).bfloat16(), torch.randn(T, Hk, D, generator=g).bfloat16()
    p = torch.randint(-2 ** 31, 2 ** 31 - 1, (T, axes), generator=g, dtype=torch.int64)
    p[: T // 2] %= 4000
    p = p.int() if axes > 1 else p[:, 0].int()
    sections = pos.sections(rot // 2, axes)
    f, s = pos.frequencies(sections, stretch=4.0, method="by_parts", original_length=1000)
    a, b = ssa.rotary(q.cuda(), k.cuda(), p.cuda(), f.cuda(), sections, interleaved, s, transpose)
    ssa.check_device()
    for got, x, name in ((a, q, "q"), (b, k, "k")):
        want, bound = ref.rotate(x, p, f, sections, interleaved, s, transpose)
        ref.check(got, want, bound, name)
        assert same(got[..., rot:].contiguous().cpu(), x[..., rot:].contiguous())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [64, 62, 60, 36, 32, 30, 0])
def test_rotary_slices_in_place_and_alone(ssa, interleaved, rot):
    """Q and K as slices of a fused projection, written in place, and Q alone."""
    from block_sparse_flashattention_ssa_b200 import positions as pos

    T, H, D = 77, 3, 64
    qkv = torch.randn(T, 3 * H, D, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    q, k = qkv[:, :H], qkv[:, H:2 * H]
    f, _ = pos.frequencies((rot // 2,), device="cuda")
    p = torch.arange(T, dtype=torch.int32, device="cuda")
    want = ssa.rotary(q.contiguous(), k.contiguous(), p, f, None, interleaved, 1.5)
    got = ssa.rotary(q, k, p, f, None, interleaved, 1.5)
    alone, none = ssa.rotary(q, None, p, f, None, interleaved, 1.5)
    assert none is None and same(alone, want[0]) and all(same(a, b) for a, b in zip(got, want))
    # an odd start: no 16-byte accesses
    flat = torch.empty(T * H * D + 3, dtype=torch.bfloat16, device="cuda")
    odd = flat[3:].view(T, H, D)
    odd.copy_(q)
    assert same(ssa.rotary(odd, None, p, f, None, interleaved, 1.5)[0], want[0])
    before = qkv.clone()
    ssa.rotary(q, k, p, f, None, interleaved, 1.5, out_q=q, out_k=k)
    ssa.check_device()
    assert same(q.contiguous(), want[0]) and same(k.contiguous(), want[1])
    assert same(qkv[:, 2 * H:].contiguous(), before[:, 2 * H:].contiguous())


def test_rotary_of_nothing(ssa):
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    p = torch.empty(0, dtype=torch.int32, device="cuda")
    q, k = ssa.rotary(e, e, p, torch.ones(32, dtype=torch.float64, device="cuda"))
    assert q.shape == k.shape == e.shape


# ----------------------------------------------------------------- together

def test_step_through_autograd(ssa):
    """rotary -> attention -> backward as autograd functions: the library's
    calls by hand give the same bits; a broadcast output gradient and rows of
    no sequence are handled."""
    from block_sparse_flashattention_ssa_b200 import positions as pos
    from block_sparse_flashattention_ssa_b200 import training

    lens, H, Hk, D, extra = [260, 100], 4, 2, 64, 30
    q, k, v, dout, cu = make(lens, H, Hk, D, seed=13, extra=extra, amp=3.0)
    total, n = q.shape[0], sum(lens)
    p = torch.arange(total, dtype=torch.int32, device="cuda")
    f, _ = pos.frequencies((D // 2,), device="cuda")
    for tsf, save_8bit, broadcast in ((0.0, False, False), (200.0, False, True), (200.0, True, False)):
        leaves = [t.clone().requires_grad_() for t in (q, k, v)]
        qr, kr = training.rotary(leaves[0], leaves[1], p, f, interleaved=True)
        out = training.attention(qr, kr, leaves[2], cu, max(lens), tsf, save_8bit=save_8bit)
        assert not out[n:].any()
        if broadcast:
            out.sum().backward()
            g_out = torch.ones_like(dout)
        else:
            out.backward(dout)
            g_out = dout
        a, b = ssa.rotary(q, k, p, f, interleaved=True)
        bm = bitmap_for(ssa, lens, H) if tsf else None
        o, lse = ssa.fwd_lse(a, b, v, cu, max(lens), tsf, decision_bitmap=bm)
        grads = [torch.zeros_like(t) for t in (q, k, v)]
        if save_8bit:
            ssa.bwd_fp8(g_out, *[ssa.save_fp8(t) for t in (a, b, v)], o, lse, cu, max(lens), 0.0, bm, *grads)
        else:
            ssa.bwd(g_out, a, b, v, o, lse, cu, max(lens), 0.0, bm, *grads)
        dq, dk = ssa.rotary(grads[0], grads[1], p, f, interleaved=True, transpose=True)
        ssa.check_device()
        assert same(out[:n].detach(), o[:n])
        for leaf, g in zip(leaves, (dq, dk, grads[2])):
            assert same(leaf.grad, g)
    # K alone needs a gradient; a gradient of one output only
    kk = k.clone().requires_grad_()
    training.rotary(q, kk, p, f)[1].float().sum().backward()
    assert kk.grad is not None
    x = q.clone().requires_grad_()
    training.rotary(x, None, p, f)[0].float().sum().backward()
    assert x.grad is not None


def test_captured_and_replayed(ssa):
    """The calls of a step in one CUDA graph, replayed on new inputs; autograd
    functions refuse capture."""
    from block_sparse_flashattention_ssa_b200 import positions as pos
    from block_sparse_flashattention_ssa_b200 import training

    lens, H, D = [300, 129], 2, 128
    first, second = make(lens, H, H, D, seed=14), make(lens, H, H, D, seed=15)
    cu = first[4]
    p = torch.arange(sum(lens), dtype=torch.int32, device="cuda")
    f, _ = pos.frequencies((D // 2,), device="cuda")

    def step(q, k, v, dout):
        a, b = ssa.rotary(q, k, p, f)
        out, lse = ssa.fwd_lse(a, b, v, cu, max(lens))
        saved = [ssa.save_fp8(t) for t in (a, b, v)]
        grads = ssa.bwd(dout, a, b, v, out, lse, cu, max(lens))
        grads8 = ssa.bwd_fp8(dout, *saved, out, lse, cu, max(lens))
        return [out, lse, *grads, *grads8, *ssa.rotary(grads[0], grads[1], p, f, transpose=True)]

    want = [step(*x[:4]) for x in (first, second)]
    torch.cuda.synchronize()
    buf = [t.clone() for t in first[:4]]
    graphs = []
    for _ in range(2):  # two graphs, replayed at the same time
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step(*buf)
            with pytest.raises(RuntimeError, match="captured"):
                training.attention(*buf[:3], cu, max(lens))
            with pytest.raises(RuntimeError, match="captured"):
                training.rotary(buf[0], buf[1], p, f)
        graphs.append((graph, got))
    for x, w in ((second, want[1]), (first, want[0])):
        for t, y in zip(buf, x):
            t.copy_(y)
        torch.cuda.synchronize()
        for (graph, _), s in zip(graphs, (torch.cuda.Stream(), torch.cuda.Stream())):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for _, got in graphs:
            assert all(same(a, b) for a, b in zip(got, w))
    ssa.check_device()


def test_other_streams(ssa):
    """Given a stream, a call runs there and its results outlive it."""
    lens = [500]
    q, k, v, dout, cu = make(lens, 2, 2, 64, seed=16)
    out, lse = ssa.fwd_lse(q, k, v, cu, 500)
    want = ssa.bwd(dout, q, k, v, out, lse, cu, 500)
    codes = ssa.save_fp8(q)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        o2, l2 = ssa.fwd_lse(q, k, v, cu, 500, stream=s)
        got = ssa.bwd(dout, q, k, v, o2, l2, cu, 500, stream=s)
        c2 = ssa.save_fp8(q, stream=s)
        junk = [torch.full((1 << 20,), 9.0, device="cuda") for _ in range(4)]  # would reuse freed memory
        torch.cuda.current_stream().wait_stream(s)
        assert same(o2, out) and same(l2, lse) and all(same(a, b) for a, b in zip(got, want))
        assert all(same(a, b) for a, b in zip(c2, codes))
        del junk
    ssa.check_device()


def test_offsets_past_32_bits(ssa):
    """2.3 G elements per tensor: the last rows are right, through every kernel."""
    from block_sparse_flashattention_ssa_b200 import positions as pos

    T, H, D, n = 70_000, 256, 128, 200
    lo = T - n
    small = make([n], H, H, D, seed=30)
    big = [torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    for b, t in zip(big, small[:4]):
        b[lo:] = t
    cu = torch.tensor([lo, T], dtype=torch.int32, device="cuda")
    q, k, v, dout = big
    out, lse = ssa.fwd_lse(q, k, v, cu, n)
    grads = ssa.bwd(dout, q, k, v, out, lse, cu, n)
    want_out, want_lse = ssa.fwd_lse(*small[:3], small[4], n)
    want = ssa.bwd(small[3], *small[:3], want_out, want_lse, small[4], n)
    assert same(out[lo:].contiguous(), want_out) and same(lse[:, lo:].contiguous(), want_lse)
    assert all(same(g[lo:].contiguous(), w) for g, w in zip(grads, want))
    del grads, out, lse, want, want_out, want_lse
    codes, scales = ssa.save_fp8(q)
    back = ssa.restore_fp8(codes, scales)
    # blocks of 128 tokens count from the first one: compare whole blocks at the end
    first = T // 128 * 128
    c2, s2 = ssa.save_fp8(q[first:])
    assert same(codes[first:].contiguous(), c2) and same(scales[-1:].contiguous(), s2)
    assert same(back[first:].contiguous(), ssa.restore_fp8(c2, s2))
    del codes, scales, back
    p = torch.arange(T, dtype=torch.int32, device="cuda")
    f, _ = pos.frequencies((D // 2,), device="cuda")
    for interleaved in (False, True):
        a = ssa.rotary(q, None, p, f, None, interleaved)[0]
        b = ssa.rotary(q[lo:], None, p[lo:].contiguous(), f, None, interleaved)[0]
        assert same(a[lo:].contiguous(), b)
        del a
    odd = ssa.rotary(q, None, p, f[:63].contiguous())[0]
    assert same(odd[lo:].contiguous(), ssa.rotary(q[lo:], None, p[lo:].contiguous(), f[:63].contiguous())[0])
    ssa.check_device()


def test_refusals(ssa):
    """Every argument is checked before a launch: types, shapes, devices,
    contiguity, alignment, overlaps, sizes."""
    lens, H, Hk, D = [200], 4, 2, 64
    q, k, v, dout, cu = make(lens, H, Hk, D, seed=31)
    out, lse = ssa.fwd_lse(q, k, v, cu, 200)
    bm = bitmap_for(ssa, lens, H)
    codes = [ssa.save_fp8(t) for t in (q, k, v)]
    p, f = torch.arange(200, dtype=torch.int32, device="cuda"), torch.ones(32, dtype=torch.float64, device="cuda")
    flat = torch.empty(q.numel() + 8, dtype=torch.bfloat16, device="cuda")
    crooked = flat[4:4 + q.numel()].view(q.shape)  # 8 bytes off a 16-byte boundary
    fwd = lambda q=q, k=k, v=v, cu=cu, **kw: ssa.fwd_lse(q, k, v, cu, 200, **kw)
    bwd = lambda dout=dout, q=q, k=k, v=v, out=out, lse=lse, cu=cu, **kw: ssa.bwd(dout, q, k, v, out, lse, cu, 200, **kw)
    bad = [
        lambda: fwd(q=q.cpu()), lambda: fwd(k=k.cpu()), lambda: fwd(q=q.float()), lambda: fwd(q=q[:, :, ::2]), lambda: fwd(q=q[0]),
        lambda: fwd(k=k[:, :1].contiguous(), v=v), lambda: fwd(k=k[:100], v=v[:100]), lambda: fwd(k=torch.cat([k, k[:, :1]], 1), v=v),
        lambda: fwd(cu=cu.long()), lambda: fwd(cu=cu[:1]), lambda: fwd(cu=cu.cpu()), lambda: fwd(out=out.float()), lambda: fwd(out=q),
        lambda: fwd(lse=lse[:, :100]), lambda: fwd(lse=lse.double()), lambda: fwd(decision_bitmap=bm[:, :, :0]), lambda: fwd(k=None),
        lambda: bwd(dout=dout[:100]), lambda: bwd(dout=None), lambda: bwd(out=out.float()), lambda: bwd(lse=lse.T), lambda: bwd(dq=q),
        lambda: bwd(dq=dout), lambda: bwd(dk=torch.empty_like(q)), lambda: bwd(dk=v), lambda: bwd(dq=out, dk=None),
        lambda: bwd(workspace=q.view(-1)), lambda: bwd(workspace=flat.cpu()), lambda: bwd(decision_bitmap=bm.float()),
        lambda: bwd(decision_bitmap=bm[:3]), lambda: bwd(k=k.transpose(0, 1)),
        lambda: ssa.bwd_fp8(dout, (codes[0][0], codes[1][1]), codes[1], codes[2], out, lse, cu, 200),
        lambda: ssa.bwd_fp8(dout, (q, codes[0][1]), codes[1], codes[2], out, lse, cu, 200),
        lambda: ssa.save_fp8(q.float()), lambda: ssa.save_fp8(q[0]), lambda: ssa.save_fp8(q, codes=q.view(torch.uint8)[..., :64]),
        lambda: ssa.save_fp8(q, scales=codes[1][1]), lambda: ssa.restore_fp8(q, codes[0][1]), lambda: ssa.restore_fp8(codes[0][0], codes[1][1]),
        lambda: ssa.rotary(q, k, p[:100], f), lambda: ssa.rotary(q, k, p.long(), f), lambda: ssa.rotary(q, k, p, f.float()),
        lambda: ssa.rotary(q, k, p, f.repeat(2)), lambda: ssa.rotary(q, k[:100], p, f), lambda: ssa.rotary(q, k, p, f, sections=(31,)),
        lambda: ssa.rotary(q, k, p[:, None].repeat(1, 2), f), lambda: ssa.rotary(q, k, p, f, out_q=k), lambda: ssa.rotary(q, k, p, f, out_k=q),
        lambda: ssa.rotary(q, None, p, f, out_k=k), lambda: ssa.rotary(q, q, p, f, out_q=q, out_k=q), lambda: ssa.rotary(q[:, ::2], None, p, f),
        lambda: ssa.rotary(q[..., :32], None, p, f[:16]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            pytest.fail(f"call {i} was accepted")
    refused = [
        lambda: fwd(q=crooked), lambda: bwd(dout=crooked), lambda: bwd(dq=crooked), lambda: ssa.save_fp8(crooked),
        lambda: bwd(workspace=torch.empty(1024, dtype=torch.uint8, device="cuda")), lambda: fwd(softmax_scale=math.nan),
        lambda: fwd(threshold_scale_factor=math.inf), lambda: ssa.save_fp8(q.view(200, 2, 128)[:, :, :96].contiguous()),
        lambda: ssa.rotary(q, k, p, f, scale=math.inf),
    ]
    for i, call in enumerate(refused):
        with pytest.raises(ssa.SSAError):
            call()
            pytest.fail(f"call {i} was accepted")
    ssa.check_device()
