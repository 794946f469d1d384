"""The training operators without a GPU: refusals of the C ABI and of the
binding before anything is launched, workspace sizes, position tables, and the
64-bit reference's own pins."""
import ctypes
import itertools
import math

import numpy as np
import pytest

from tests import training_ref as ref

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ssa():
    import __graft_entry__

    __graft_entry__._library_builder().build()
    import block_sparse_flashattention_ssa_b200 as m

    return m


FAKE = ctypes.c_void_p(0x10000)
MIS = ctypes.c_void_p(0x10008)
INVALID, UNSUPPORTED, OK = -1, -2, 0


def test_fwd_lse_refusals(ssa):
    base = dict(q=FAKE, k=FAKE, v=FAKE, cu=FAKE, batch=1, total=256, longest=256, H=4, Hk=2, D=128, scale=0.0, tsf=0.0,
                out=FAKE, lse=FAKE, sc=None, nq=2, bm=None)

    def call(**kw):
        a = dict(base, **kw)
        return ssa.lib().ssa_fwd_lse(a["q"], a["k"], a["v"], a["cu"], a["batch"], a["total"], a["longest"], a["H"],
                                     a["Hk"], a["D"], a["scale"], a["tsf"], a["out"], a["lse"], a["sc"], a["nq"],
                                     a["bm"], None)

    for kw in (dict(q=None), dict(lse=None), dict(cu=None), dict(batch=0), dict(total=-1), dict(H=0), dict(Hk=0), dict(Hk=3),
               dict(Hk=8), dict(Hk=-2), dict(tsf=math.nan), dict(tsf=math.inf), dict(scale=math.inf), dict(sc=FAKE, nq=-1),
               dict(bm=FAKE, longest=0), dict(longest=-1)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(D=96), dict(D=0), dict(k=MIS), dict(out=MIS)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(total=0) == OK
    assert call() == INVALID  # not device memory


def test_bwd_refusals(ssa):
    need = ssa.bwd_workspace_bytes(256, 1, 4)
    base = dict(dout=FAKE, q=FAKE, k=FAKE, v=FAKE, out=FAKE, lse=FAKE, cu=FAKE, batch=1, total=256, longest=256, H=4, Hk=2,
                D=128, scale=0.0, bm=None, nq=2, dq=FAKE, dk=FAKE, dv=FAKE, ws=FAKE, size=need)

    def call(**kw):
        a = dict(base, **kw)
        return ssa.lib().ssa_bwd(a["dout"], a["q"], a["k"], a["v"], a["out"], a["lse"], a["cu"], a["batch"], a["total"],
                                 a["longest"], a["H"], a["Hk"], a["D"], a["scale"], a["bm"], a["nq"], a["dq"], a["dk"],
                                 a["dv"], a["ws"], a["size"], None)

    for kw in ([{n: None} for n in ("dout", "q", "k", "v", "out", "lse", "cu", "dq", "dk", "dv", "ws")]
               + [dict(batch=0), dict(total=-1), dict(longest=-1), dict(H=0), dict(Hk=3), dict(Hk=0), dict(H=65535, Hk=1),
                  dict(scale=math.nan), dict(bm=FAKE, nq=-1), dict(bm=FAKE, longest=0), dict(size=need - 1), dict(size=-1)]):
        assert call(**kw) == INVALID, kw
    for kw in (dict(D=32), dict(dq=MIS), dict(dout=MIS), dict(ws=MIS), dict(v=MIS)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(total=0, ws=None, size=0) == OK
    assert call() == INVALID  # not device memory
    # the bound of the row values: every query block of every head, 128 rows of two floats
    assert need == (2 + 1) * 4 * 1024
    assert ssa.bwd_workspace_bytes(0, 1, 1) == 1024
    # past 32 bits
    assert ssa.bwd_workspace_bytes(2 ** 31 - 1, 2 ** 20, 64) == ((2 ** 31 + 126) // 128 + 2 ** 20) * 64 * 1024
    assert ssa.bwd_fp8_workspace_bytes(1000, 2, 4, 2, 64) == ssa.bwd_workspace_bytes(1000, 2, 4) + 1000 * 8 * 64 * 2
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 1, 0)):
        with pytest.raises(ssa.SSAError):
            ssa.bwd_workspace_bytes(*bad)
    with pytest.raises(ssa.SSAError):
        ssa.bwd_fp8_workspace_bytes(1, 1, 1, 0, 64)


def test_saved_refusals(ssa):
    L = ssa.lib()
    save = lambda x=FAKE, c=FAKE, s=FAKE, T=10, H=2, D=64: L.ssa_save_fp8(x, c, s, T, H, D, None)
    back = lambda c=FAKE, s=FAKE, x=FAKE, T=10, H=2, D=64: L.ssa_restore_fp8(c, s, x, T, H, D, None)
    for f in (save, back):
        assert f(T=-1) == INVALID and f(H=0) == INVALID and f(H=65536) == INVALID
        assert f(x=None) == INVALID and f(c=None) == INVALID and f(s=None) == INVALID
        assert f(D=96) == UNSUPPORTED and f(x=MIS) == UNSUPPORTED and f(c=MIS) == UNSUPPORTED
        assert f(T=0) == OK
        assert f() == INVALID  # not device memory
    need = ssa.bwd_fp8_workspace_bytes(256, 1, 4, 2, 128)
    f8 = lambda q=FAKE, qs=FAKE, v=FAKE, H=4, Hk=2, D=128, size=need, total=256, dq=FAKE: L.ssa_bwd_fp8(
        FAKE, q, qs, FAKE, FAKE, v, FAKE, FAKE, FAKE, FAKE, 1, total, 256, H, Hk, D, 0.0, None, 0, dq, FAKE, FAKE, FAKE,
        size, None)
    for kw in (dict(q=None), dict(qs=None), dict(v=None), dict(H=0), dict(Hk=0), dict(total=-1)):
        assert f8(**kw) == INVALID, kw
    assert f8(D=32) == UNSUPPORTED and f8(q=MIS) == UNSUPPORTED
    assert f8(total=0) == OK


def test_rotary_refusals(ssa):
    base = dict(q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, qs=256, ks=128, qos=256, kos=128, T=10, H=4, Hk=2, D=64, pos=FAKE,
                sections=[32], f=FAKE, rot=64, scale=1.0)

    def call(**kw):
        a = dict(base, **kw)
        sec = None if a["sections"] is None else (ctypes.c_int32 * max(1, len(a["sections"])))(*a["sections"])
        return ssa.lib().ssa_rotary(a["q"], a["k"], a["qo"], a["ko"], a["qs"], a["ks"], a["qos"], a["kos"], a["T"], a["H"],
                                    a["Hk"], a["D"], a["pos"], a.get("axes", len(a["sections"] or [0])), sec, a["f"], a["rot"], 0,
                                    a["scale"], 0, None)

    for kw in (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(pos=None), dict(f=None), dict(T=-1), dict(H=0),
               dict(H=65536), dict(Hk=-1), dict(D=0), dict(rot=63), dict(rot=66), dict(rot=-2), dict(sections=[31]),
               dict(sections=[33]), dict(sections=[16, 8, 4, 2, 2]), dict(sections=[40, -8]), dict(sections=None),
               dict(sections=[32], axes=0), dict(qs=255), dict(ks=127), dict(qos=0), dict(kos=-128), dict(scale=math.nan),
               dict(scale=math.inf)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(D=60, rot=60, sections=[30]), dict(D=264, qs=2000, qos=2000, ks=2000, kos=2000),
               dict(q=ctypes.c_void_p(0x10001))):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(T=0) == OK
    assert call() == INVALID  # not device memory


def test_binding_refuses_host_tensors(ssa):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    lse = torch.zeros(2, 4)
    for call in (lambda: ssa.fwd_lse(x, x, x, cu, 4), lambda: ssa.bwd(x, x, x, x, x, lse, cu, 4), lambda: ssa.save_fp8(x),
                 lambda: ssa.restore_fp8(x.view(torch.uint8), lse),
                 lambda: ssa.rotary(x, x, cu, torch.zeros(2, dtype=torch.float64))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_overlaps_are_found(ssa):
    buf = torch.zeros(100, dtype=torch.bfloat16)
    a, b, c = buf[:50], buf[50:], buf[49:60]
    ssa._no_overlap([(b, "b"), (None, "n")], [(a, "a"), (None, "m")])
    for outs, ins in (([(c, "c")], [(a, "a")]), ([(b, "b"), (c, "c")], []), ([(a, "a")], [(a, "a")])):
        with pytest.raises(ValueError, match="overlaps"):
            ssa._no_overlap(outs, ins)


def test_overlap_of_strided_rows_matches_enumeration(ssa):
    """_rows_overlap against the sets of addresses, over all small layouts
    (it may only be cautious where the strides differ)."""
    buf = torch.zeros(200, dtype=torch.bfloat16)
    D = 2
    for n, h1, h2, s1, s2, off in itertools.product((1, 2, 3), (1, 2), (1, 3), (2, 4, 6, 8, 10), (6, 8, 10), range(0, 14)):
        if (n > 1 and s1 < h1 * D) or (n > 1 and s2 < h2 * D):
            continue
        a = buf.as_strided((n, h1, D), (s1, D, 1), 20)
        b = buf.as_strided((n, h2, D), (s2, D, 1), 20 - 6 + off)
        truth = bool({20 + t * s1 + i for t in range(n) for i in range(h1 * D)} &
                     {14 + off + t * s2 + i for t in range(n) for i in range(h2 * D)})
        got = ssa._rows_overlap(a, s1, b, s2)
        assert got or not truth
        if s1 == s2:
            assert got == truth, (n, h1, h2, s1, off)


def test_rotary_outputs_over_the_tables(ssa):
    """An output may not lie over the positions or the frequencies, which other
    tokens still read."""
    cpu = torch.device("cpu")
    total, H, D = 6, 2, 8
    q = torch.zeros(total, H, D, dtype=torch.bfloat16)
    buf = torch.zeros(4 * q.numel(), dtype=torch.bfloat16)
    out = buf[: q.numel()].view(q.shape)
    wide = buf.view(total, 8, D)[:, :H]
    pos, freq = torch.zeros(total, dtype=torch.int32), torch.zeros(4, dtype=torch.float64)

    def check(o, pos=pos, freq=freq):
        ssa._check_rotary_outputs(cpu, total, D, (q, None), [H * D, 0], (o, None), [H * D, 0],
                                  ((pos, "positions"), (freq, "inv_freq")))

    n = q.numel()
    check(out)
    check(wide)
    check(out, pos=buf[n:n + 2 * total].view(torch.int32))  # right behind it
    for o, kw in ((out, dict(pos=buf[n - 2:n - 2 + 2 * total].view(torch.int32))), (out, dict(freq=buf[8:24].view(torch.float64))),
                  (wide, dict(pos=buf[64:64 + 2 * total].view(torch.int32))), (out, dict(pos=buf[:2 * total].view(torch.int32)))):
        with pytest.raises(ValueError, match="overlaps"):
            check(o, **kw)


def test_rows_checks(ssa):
    cpu = torch.device("cpu")
    t = torch.zeros(5, 6, 8, dtype=torch.bfloat16)
    assert ssa._rows(t, "t", cpu, 5, 8) == 48
    assert ssa._rows(t[:, 2:4], "t", cpu, 5, 8) == 48
    assert ssa._rows(t[:1, :2], "t", cpu, 1, 8) == 16
    for bad in (t.float(), t[:, ::2], t[..., ::2], t.transpose(0, 1), t[:1].expand(5, 6, 8), t[0]):
        with pytest.raises(ValueError):
            ssa._rows(bad, "t", cpu, 5, 8)
    with pytest.raises(TypeError):
        ssa._rows(None, "t", cpu, 5, 8)


def test_calls_run_on_their_tensors_device_and_given_stream(ssa, monkeypatch):
    """_run with stand-ins for two devices: the tensors' device is made current,
    the given stream is used, and tensors are kept for it; a stream of another
    device is refused."""
    import contextlib

    class Stream:
        def __init__(self, device, handle):
            self.device, self.cuda_stream = torch.device("cuda", device), handle

        def __eq__(self, other):
            return self.cuda_stream == other.cuda_stream

        def __ne__(self, other):
            return not self == other

    class Tensor:
        def __init__(self):
            self.kept = []

        def record_stream(self, s):
            self.kept.append(s.cuda_stream)

    log = []
    current = {0: Stream(0, 100), 1: Stream(1, 200)}

    @contextlib.contextmanager
    def enter(what, value):
        log.append((what, value))
        yield

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: current[0 if dev is None else dev.index])
    monkeypatch.setattr(torch.cuda, "device", lambda d: enter("device", d.index))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: enter("stream", s.cuda_stream))
    monkeypatch.setattr(ssa, "_current_handle", lambda t, dev: current[dev.index].cuda_stream)
    made = Tensor()
    body = lambda h: log.append(("run", h)) or (made,)
    x = Tensor()

    def run(dev, stream=None):
        log.clear()
        ssa._run(torch.device("cuda", dev), stream, (x, None), body)
        return list(log)

    assert run(0) == [("run", 100)]
    assert run(1) == [("device", 1), ("stream", 200), ("run", 200)]  # another device than the current one
    assert x.kept == [] and made.kept == []
    assert run(0, Stream(0, 101)) == [("device", 0), ("stream", 101), ("run", 101)]
    assert x.kept == [101] and made.kept == [100]
    assert run(1, Stream(1, 201)) == [("device", 1), ("stream", 201), ("run", 201)]
    assert made.kept == [100, 200]
    with pytest.raises(ValueError, match="stream is on"):
        run(0, Stream(1, 201))


def test_position_tables(ssa):
    from block_sparse_flashattention_ssa_b200 import positions as pos

    p = pos.grid_positions([(2, 3, 4), (0, 3, 4), (1, 1, 2)])
    want = [(t, y, x) for t in range(2) for y in range(3) for x in range(4)] + [(0, 0, 0), (0, 0, 1)]
    assert p.dtype == torch.int32 and p.tolist() == [list(w) for w in want]
    assert tuple(pos.grid_positions([]).shape) == (0, 3)
    assert pos.sections(64, 3) == (22, 21, 21) and pos.sections(64, 1) == (64,) and pos.sections(1, 3) == (1, 0, 0)
    f, s = pos.frequencies((4, 2), base=100.0)
    assert s == 1.0 and f.dtype == torch.float64
    np.testing.assert_allclose(f.numpy(), [1, 100 ** -0.25, 0.1, 100 ** -0.75, 1, 0.1], rtol=1e-14)
    f2, s2 = pos.frequencies((4,), base=100.0, stretch=8.0)
    np.testing.assert_allclose(f2.numpy() * 8, f[:4].numpy(), rtol=1e-14)
    f3, _ = pos.frequencies((4,), base=100.0, stretch=8.0, method="base")
    np.testing.assert_allclose([f3[0], f3[3]], [1.0, 100 ** -0.75 / 8], rtol=1e-13)  # fastest kept, slowest / stretch
    f4, s4 = pos.frequencies((64,), stretch=8.0, method="by_parts", original_length=8192)
    plain = 10000.0 ** (-np.arange(64) / 64)
    turns = 8192 * plain / (2 * math.pi)
    ratio = f4.numpy() / plain
    assert s4 == pytest.approx(0.1 * math.log(8) + 1)
    np.testing.assert_allclose(ratio[turns >= 32], 1.0, rtol=1e-14)
    np.testing.assert_allclose(ratio[turns <= 1], 1 / 8, rtol=1e-14)
    assert (np.diff(ratio) <= 1e-15).all() and ((ratio > 1 / 8) & (ratio < 1)).any()
    assert pos.frequencies((4,), method="by_parts", original_length=100)[1] == 1.0
    for bad in (dict(method="other"), dict(base=1.0), dict(stretch=0.5), dict(method="by_parts", stretch=2.0),
                dict(stretch=math.inf), dict(method="by_parts", original_length=9, turns=(3.0, 3.0))):
        with pytest.raises(ValueError):
            pos.frequencies((4,), **bad)
    with pytest.raises(ValueError):
        pos.sections(-1, 2)
    with pytest.raises(ValueError):
        pos.grid_positions([(1, -1, 2)])


def test_reference_gradients_are_the_differentiated_forward():
    """The 64-bit formulas against torch's own differentiation of a softmax attention."""
    lens, H, Hk, D = [5, 0, 9], 4, 2, 8
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(14, h, D, generator=g, dtype=torch.float64).requires_grad_() for h in (H, Hk, Hk))
    dout = torch.randn(14, H, D, generator=g, dtype=torch.float64)
    out = torch.zeros(14, H, D, dtype=torch.float64)
    parts = []
    for lo, hi in ((0, 5), (5, 14)):
        for h in range(H):
            p = torch.softmax(q[lo:hi, h] @ k[lo:hi, h // 2].T / math.sqrt(D), 1)
            parts.append((lo, hi, h, p @ v[lo:hi, h // 2]))
    loss = sum((o * dout[lo:hi, h]).sum() for lo, hi, h, o in parts)
    loss.backward()
    for lo, hi, h, o in parts:
        out[lo:hi, h] = o.detach()
    o, lse, _, _ = ref.forward(q.detach(), k.detach(), v.detach(), lens)
    torch.testing.assert_close(o, out)
    grads, _ = ref.backward(dout, q.detach(), k.detach(), v.detach(), o, lse, lens)
    for a, x in zip(grads, (q, k, v)):
        torch.testing.assert_close(a, x.grad)


def test_reference_e4m3_and_rotation():
    y = torch.linspace(-460, 460, 20001, dtype=torch.float64)
    want = y.clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
    near = (y.clamp(-448, 448).float().double() == y.clamp(-448, 448))
    assert torch.equal(ref.e4m3_nearest(y)[near], want[near])
    x = torch.randn(6, 2, 12, dtype=torch.float64)
    p = torch.randint(0, 50, (6, 2), dtype=torch.int32)
    f = torch.rand(5, dtype=torch.float64)
    for inter in (False, True):
        t, _ = ref.rotate(x, p, f, (2, 3), inter, 1.3, False)
        back, _ = ref.rotate(t, p, f, (2, 3), inter, 1 / 1.3, True)
        torch.testing.assert_close(back, x)
        y = torch.randn_like(x)  # the adjoint
        u, _ = ref.rotate(y, p, f, (2, 3), inter, 1.3, True)
        assert float((t * y).sum()) == pytest.approx(float((x * u).sum()), rel=1e-12)
