"""Plain 64-bit implementations of the training operators, with elementwise
error bounds for kernels that round P and dS to bf16 and keep sums in fp32.

U is bf16's half step (2^-8 relative), E a generous unit for one fp32
operation (2^-23: twice the half step, for accumulations that truncate). A sum
of n terms accumulated in fp32 is off by at most n E times the sum of the
terms' magnitudes.
"""
import math

import numpy as np
import torch

U = torch.finfo(torch.bfloat16).eps / 2
E = 2.0 ** -23
TILE = 128


def bounds(lens):
    return [int(x) for x in np.concatenate([[0], np.cumsum(lens)])]


def keep_of(bitmap, h, gqb0, n):
    """Kept elements [n, n] of one sequence and head from a decision bitmap."""
    T = (n + TILE - 1) // TILE
    words = bitmap[h, gqb0:gqb0 + T].cpu().numpy().astype(np.int64) & 0xFFFFFFFF
    tiles = np.array([[(int(words[i, j >> 5]) >> (j & 31)) & 1 for j in range(T)] for i in range(T)], dtype=bool)
    return torch.from_numpy(~np.repeat(np.repeat(tiles, TILE, 0), TILE, 1)[:n, :n])


def heads(lens, bitmap=None, H=1):
    """(h, first row, end, first q-block) of every head and non-empty sequence."""
    cu, gqb = bounds(lens), 0
    for lo, hi in zip(cu, cu[1:]):
        for h in range(H if hi > lo else 0):
            yield h, lo, hi, gqb
        gqb += (hi - lo + TILE - 1) // TILE


def _scores(q, k, lo, hi, h, g, c, keep):
    Q, K = q[lo:hi, h], k[lo:hi, g]
    s = c * (Q @ K.T)
    # fp32 dot product, the rounded factor, and the product with it
    err = abs(c) * (Q.shape[1] + 3) * E * (Q.abs() @ K.abs().T)
    if keep is not None:
        s = torch.where(keep, s, -math.inf)
    return s, err


def forward(q, k, v, lens, bitmap=None, scale=0.0):
    """(out, lse, bound of out, bound of lse) in float64 on the CPU."""
    q, k, v = (t.double().cpu() for t in (q, k, v))
    total, H, D = q.shape
    G = H // k.shape[1]
    c = scale if scale > 0 else D ** -0.5
    out, out_b = torch.zeros(total, H, D, dtype=torch.float64), torch.zeros(total, H, D, dtype=torch.float64)
    lse, lse_b = torch.zeros(H, total, dtype=torch.float64), torch.zeros(H, total, dtype=torch.float64)
    for h, lo, hi, gqb in heads(lens, H=H):
        keep = None if bitmap is None else keep_of(bitmap, h, gqb, hi - lo)
        s, err = _scores(q, k, lo, hi, h, h // G, c, keep)
        L = torch.logsumexp(s, 1)
        P = torch.exp(s - L[:, None])
        V = v[lo:hi, h // G]
        n = hi - lo
        # relative error of a probability against its row: score error, the
        # reference max's own rounding, the exponential (2 ulp) and the sum
        rho = (err + 8 * E * (s.abs().where(P > 0, torch.zeros_like(s)) + L.abs()[:, None]) + (n + 8) * E)
        rel = rho.amax(1, keepdim=True)
        out[lo:hi, h] = P @ V
        out_b[lo:hi, h] = (U + 2 * rel + n * E) * (P @ V.abs()) + U * out[lo:hi, h].abs() * 1.01 + 1e-30
        lse[h, lo:hi], lse_b[h, lo:hi] = L, rel[:, 0] + 4 * E * (L.abs() + 1)
    return out, lse, out_b, lse_b


def backward(dout, q, k, v, out, lse, lens, bitmap=None, scale=0.0):
    """Gradients from the given out and lse by the formula, and their bounds:
    ((dq, dk, dv), (bounds)) in float64 on the CPU."""
    dout, q, k, v, out, lse = (t.double().cpu() for t in (dout, q, k, v, out, lse))
    total, H, D = q.shape
    Hk = k.shape[1]
    G = H // Hk
    c = scale if scale > 0 else D ** -0.5
    z = lambda n: torch.zeros(total, n, D, dtype=torch.float64)
    dq, dk, dv, bq, bk, bv = z(H), z(Hk), z(Hk), z(H), z(Hk), z(Hk)
    mag_k, mag_v = z(Hk), z(Hk)
    for h, lo, hi, gqb in heads(lens, H=H):
        g, n = h // G, hi - lo
        keep = None if bitmap is None else keep_of(bitmap, h, gqb, n)
        s, err = _scores(q, k, lo, hi, h, g, c, keep)
        L = lse[h, lo:hi]
        P = torch.where(torch.isinf(L)[:, None], torch.zeros_like(s), torch.exp(s - L[:, None]))
        Q, K, V, dO, O = q[lo:hi, h], k[lo:hi, g], v[lo:hi, g], dout[lo:hi, h], out[lo:hi, h]
        dP = dO @ V.T
        delta = (dO * O).sum(1, keepdim=True)
        dS = P * (dP - delta)
        rho = err + 8 * E * (s.abs().where(P > 0, torch.zeros_like(s)) + L.abs().where(~torch.isinf(L), torch.zeros_like(L))[:, None] + 1)
        eP = P * rho                                      # fp32 P
        eS = (eP * (dP - delta).abs() + (P + eP) * (D + 2) * E * (dO.abs() @ V.abs().T + (dO.abs() * O.abs()).sum(1, keepdim=True)))
        rP, rS = eP + U * (P + eP), eS + U * (dS.abs() + eS)  # after rounding to bf16
        N = n * G
        dv[lo:hi, g] += P.T @ dO
        bv[lo:hi, g] += rP.T @ dO.abs() + N * E * ((P + rP).T @ dO.abs())
        dk[lo:hi, g] += c * (dS.T @ Q)
        bk[lo:hi, g] += c * (rS.T @ Q.abs() + N * E * ((dS.abs() + rS).T @ Q.abs()))
        dq[lo:hi, h] = c * (dS @ K)
        # What rounding adds to a row's dS, times a mean of finite keys, is taken
        # out of dQ: its error is sum_j e_j (k_j - m) with |e_j| <= U (|dS_j| + ..),
        # at most sum_j |e_j| (|k_j| + |m|), and |m| is at most the largest |k|.
        m = K.abs().where(torch.isfinite(K), torch.zeros_like(K)).amax(0)
        bq[lo:hi, h] = c * (rS @ K.abs() + n * E * ((dS.abs() + rS) @ K.abs())
                            + (1 + n * E) * U * ((dS.abs() + eS).sum(1, keepdim=True) * m))
    fin = lambda x, b: b + (U + 4 * E) * (x.abs() + b) + 1e-37  # the scale in fp32 and the rounding of the result
    return (dq, dk, dv), (fin(dq, bq), fin(dk, bk), fin(dv, bv))


def check(got, want, bound, what):
    got = got.detach().double().cpu()
    over = (got - want).abs() - bound
    assert torch.isfinite(got).all(), f"{what}: not finite"
    worst = float(over.max()) if over.numel() else 0.0
    at = np.unravel_index(int(over.argmax()), over.shape) if over.numel() else ()
    assert worst <= 0, f"{what}: |error| exceeds its bound by {worst:.3g} at {tuple(int(i) for i in at)}: got " \
                       f"{float(got[at]):.6g}, want {float(want[at]):.6g}, bound {float(bound[at]):.3g}"


def e4m3_nearest(y):
    """E4M3 value nearest to each finite float64 (ties to even, saturating),
    by comparison with the enumerated value set."""
    vals = sorted({(1 + m / 8) * 2.0 ** (e - 7) if e else m * 2.0 ** -9 for e in range(16) for m in range(8)
                   if not (e == 15 and m == 7)})
    v = torch.tensor(vals, dtype=torch.float64)
    a = y.abs().clamp(max=448.0)
    hi = torch.searchsorted(v, a).clamp(max=len(vals) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = v[hi] - a, a - v[lo]
    even = hi % 2 == 0  # codes ascend with the value: an even index is an even code
    return torch.where((up < down) | ((up == down) & even), v[hi], v[lo]) * torch.sign(y)


def saved(x):
    """(restored, scales) of save_fp8 in float64 on the CPU, non-finite values as NaN."""
    x = x.double().cpu()
    T, H, D = x.shape
    out, scales = torch.zeros_like(x), torch.ones((T + TILE - 1) // TILE, H, dtype=torch.float64)
    for b in range(scales.shape[0]):
        blk = x[b * TILE:(b + 1) * TILE]
        for h in range(H):
            t = blk[:, h]
            a = t[torch.isfinite(t)].abs()
            top = float(a.max()) if a.numel() else 0.0
            e = -100
            while top > 448.0 * 2.0 ** e:
                e += 1
            s = 2.0 ** e if top > 0 else 1.0
            scales[b, h] = s
            y = torch.where(torch.isfinite(t), t, torch.zeros_like(t)) / s
            out[b * TILE:b * TILE + t.shape[0], h] = torch.where(torch.isfinite(t), e4m3_nearest(y) * s, math.nan)
    return out, scales


def rotate(x, positions, inv_freq, sections, interleaved, scale, transpose):
    """(rotated, bound) in float64 on the CPU."""
    x = x.double().cpu()
    pos = positions.cpu().double().reshape(x.shape[0], -1)
    f = inv_freq.cpu()
    n = f.numel()
    axis = [a for a, m in enumerate(sections) for _ in range(m)]
    angle = (pos[:, axis] * f if n else pos[:, :0]) * (-1 if transpose else 1)
    c, s = scale * torch.cos(angle)[:, None], scale * torch.sin(angle)[:, None]
    left = torch.arange(n) * (2 if interleaved else 1)
    right = left + (1 if interleaved else n)
    y, b = x.clone(), torch.zeros_like(x)
    a0, b0 = x[..., left], x[..., right]
    y[..., left], y[..., right] = a0 * c - b0 * s, a0 * s + b0 * c
    # The table entry: fraction of a turn in fp32 (at most half a turn, 2^-25 of
    # one turn, 2 pi 2^-25 radians), sin and cos (2 ulp), the scale; the double
    # product is off by 2^-51 of the angle in turns; then two products, one sum.
    e = 2 * math.pi * 2.0 ** -24 + 6 * E + angle.abs()[:, None] * 2.0 ** -50
    b[..., left] = b[..., right] = (a0.abs() + b0.abs()) * abs(scale) * e
    return y, b + U * (y.abs() + b) * (1 if n else 0) + 1e-37


def bound_dq(dout, q, k, v, out, lse, lens, bitmap=None, scale=0.0):
    """dQ's bound over the keys a row sees alone: no term for any other key. dS
    enters in two bf16 parts, hi + lo: lo = dS - hi is exact in fp32 (it has the
    16 bits that hi has not) and at most U |dS|, so its own rounding leaves at
    most U U |dS|; the sum has 2 n terms. (backward()'s own bound of dQ is wider:
    it allows for one rounding of dS and for a term in the largest key, which an
    earlier form of the kernel needed.)"""
    dout, q, k, v, out, lse = (t.double().cpu() for t in (dout, q, k, v, out, lse))
    total, H, D = q.shape
    G = H // k.shape[1]
    c = scale if scale > 0 else D ** -0.5
    dq, bq = torch.zeros(total, H, D, dtype=torch.float64), torch.zeros(total, H, D, dtype=torch.float64)
    for h, lo, hi, gqb in heads(lens, H=H):
        n = hi - lo
        keep = None if bitmap is None else keep_of(bitmap, h, gqb, n)
        s, err = _scores(q, k, lo, hi, h, h // G, c, keep)
        L = lse[h, lo:hi]
        P = torch.where(torch.isinf(L)[:, None], torch.zeros_like(s), torch.exp(s - L[:, None]))
        seen = P > 0
        zero = torch.zeros_like(s)
        K, V, dO, O = k[lo:hi, h // G], v[lo:hi, h // G], dout[lo:hi, h], out[lo:hi, h]
        dev = (dO @ V.T - (dO * O).sum(1, keepdim=True)).where(seen, zero)
        dS = P * dev
        rho = (err + 8 * E * (s.abs() + L.abs()[:, None] + 1)).where(seen, zero)
        mag = (dO.abs() @ V.abs().T + (dO.abs() * O.abs()).sum(1, keepdim=True)).where(seen, zero)
        eS = P * rho * dev.abs() + P * (1 + rho) * (D + 2) * E * mag
        rS = eS + U * U * (dS.abs() + eS)
        dq[lo:hi, h] = c * (dS @ K)
        bq[lo:hi, h] = c * (rS @ K.abs() + 2 * n * E * (1 + U) * ((dS.abs() + rS) @ K.abs()))
    return bq + (U + 4 * E) * (dq.abs() + bq) + 1e-37
