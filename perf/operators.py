"""The training-side operators and the cases that they are measured on.

Three operators that make up one attention layer's training step around the
skip-softmax forward: rotary positions on Q and K (and their adjoint),
attention's backward pass (dense, or on the tiles the forward kept; alone or
behind the forward that hands it the row log-sum-exp), and 8-bit activation
checkpoints with the backward pass that reads them.

``run`` computes an operator in its plain form with elementary torch
operations in 32 bits; where ``own`` is true it makes the framework's calls.
``exact`` evaluates the definitions in 64 bits.

Tensors are packed varlen [total_tokens, heads, head_dim] in bf16; sequence b
is rows cu[b] .. cu[b+1]-1 and sees itself only, without a causal mask.
"""
import math

import torch

own = False

TILE = 128
E4M3_MAX = 448.0
FRAME = 32  # tokens per row and rows per frame of the video grids below


def _framework():
    import block_sparse_flashattention_ssa_b200 as ssa

    return ssa


# ------------------------------------------------------------------- cases

def _rotary(name, tokens, heads, kv_heads, dim, rot, interleaved, axes, far, stretch, transpose):
    return {"name": name, "op": "rotary", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot,
            "interleaved": interleaved, "axes": axes, "far": far, "stretch": stretch, "transpose": transpose}


def _attention(name, op, seqlens, heads, kv_heads, dim, tsf=0.0, kept=1.0, amp=1.0):
    return {"name": name, "op": op, "seqlens": seqlens, "heads": heads, "kv_heads": kv_heads, "dim": dim, "tsf": tsf,
            "kept": kept, "amp": amp}


def listed():
    return [
        # one token far into a long sequence: what a call costs at its smallest
        _rotary("rotary one token", 1, 24, 24, 128, 128, False, 1, 1_000_003, 1.0, False),
        # Q and K of one 8x32x32 video of 24 heads, three position axes, adjacent pairs
        _rotary("rotary 8192x24 grid", 8192, 24, 24, 128, 128, True, 3, 0, 1.0, False),
        # the 720p video: 75,600 tokens of 40 heads
        _rotary("rotary 75600x40 grid", 75600, 40, 40, 128, 128, True, 3, 0, 1.0, False),
        # the gradient of a rotation of half the head over a stretched context, K heads shared, an odd number of tokens
        _rotary("rotary gradient 16381x16", 16381, 16, 4, 128, 64, False, 1, 300_000, 8.0, True),
        # the smallest workload of the tests: a training step's backward pass bound by latency
        _attention("backward 1024x2 d64", "backward", "1024", 2, 2, 64),
        # one 8x32x32 video of 24 heads, dense
        _attention("backward 8192x24", "backward", "8192", 24, 24, 128),
        # the same with the forward's skip decisions at a threshold scale factor that leaves about two fifths of the tiles
        _attention("backward 8192x24 skip", "backward", "8192", 24, 24, 128, tsf=20000.0, kept=0.39, amp=2.0),
        # the 720p video, its 40 heads split over 8 GPUs
        _attention("backward 75600x5", "backward", "75600", 5, 5, 128),
        # forward and backward of a ragged batch with shared K/V heads: lengths of zero and one, tiles that end early
        _attention("step ragged", "step", "1,5,127,128,129,300,0,1000", 8, 2, 128),
        # forward and backward of the shortest video of the mixed batch, all its heads
        _attention("step 5120x40", "step", "5120", 40, 40, 128),
        # Q of the 720p video saved in 8 bits for the backward pass and brought back
        {"name": "checkpoint 75600x40", "op": "checkpoint", "tokens": 75600, "heads": 40, "dim": 128},
        # the backward pass from saved Q, K and V
        _attention("backward from saved 8192x24", "backward_saved", "8192", 24, 24, 128),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rotary", "rotary", "backward", "backward", "step", "checkpoint", "backward_saved"])
    dim = rng.choice([64, 128, 128])
    if op == "rotary":
        tokens = spread(1, 75600)
        kv = rng.randint(1, 10)
        rot = 2 * rng.randint(4, dim // 2)
        return {"op": op, "tokens": tokens, "heads": kv * rng.choice([1, 1, 2, 4]), "kv_heads": kv, "dim": dim, "rot": rot,
                "interleaved": rng.random() < 0.5, "axes": rng.choice([1, 1, 3]), "far": rng.choice([0, spread(1, 2_000_000)]),
                "stretch": rng.choice([1.0, rng.uniform(2.0, 16.0)]), "transpose": rng.random() < 0.5}
    if op == "checkpoint":
        return {"op": op, "tokens": spread(1, 75600), "heads": rng.randint(1, 40), "dim": dim}
    kv = rng.randint(1, 6)
    group = rng.choice([1, 1, 2, 4])
    lens = [rng.choice([spread(1, 700), spread(64, 9000)]) for _ in range(rng.choice([1, 1, 2, 3, 6]))]
    tsf = rng.choice([0.0, 0.0, float(spread(100, 5000))]) if op == "backward" else 0.0
    return {"op": op, "seqlens": ",".join(str(n) for n in lens), "heads": kv * group, "kv_heads": kv, "dim": dim, "tsf": tsf,
            "kept": 0.5 if tsf else 1.0, "amp": rng.choice([1.0, 2.0])}


def _lengths(case):
    return [int(n) for n in case["seqlens"].split(",")]


def work(case):
    if case["op"] == "rotary":
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 4.0 * n + 4.0 * case["tokens"] * case["axes"], "flops": 3.0 * n * case["rot"] / case["dim"]}
    if case["op"] == "checkpoint":
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 6.0 * n, "flops": 3.0 * n}
    lens, D, H, Hk = _lengths(case), case["dim"], case["heads"], case["kv_heads"]
    total = sum(lens)
    products = 7 if case["op"] == "step" else 5
    flops = sum(2.0 * products * n * n * D * H * case["kept"] for n in lens)
    rows_q, rows_k = total * H * D, total * Hk * D
    element = 1 if case["op"] == "backward_saved" else 2
    # Q, K, V, O, dO and the row log-sum-exp in; dQ, dK, dV out; a step also writes O and the log-sum-exp
    return {"bytes": float(element * (rows_q + 2 * rows_k) + 4 * rows_q + 2 * (rows_q + 2 * rows_k) + 4 * total * H), "flops": flops}


# ------------------------------------------------------------------ inputs

def _noise(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _grid(tokens):
    """Frame, row and column of each token of a video, int32 [tokens, 3]."""
    i = torch.arange(tokens, device="cuda", dtype=torch.int32)
    return torch.stack([i // (FRAME * FRAME), (i // FRAME) % FRAME, i % FRAME], 1)


def _code(lens, dim, amp):
    """Sinusoidal position code of each token, float32 [total, dim]: neighbours on the grid score high."""
    rows = []
    for n in lens:
        p = _grid(n).float()
        d = 2 * (dim // 6)
        parts = []
        for a, w in ((0, dim - 2 * d), (1, d), (2, d)):
            f = 10000.0 ** (-2.0 * torch.arange(w // 2, device="cuda", dtype=torch.float32) / w)
            t = p[:, a:a + 1] * f
            parts.append(torch.stack([t.sin(), t.cos()], -1).reshape(n, w))
        rows.append(torch.cat(parts, 1))
    return amp * torch.cat(rows)


def _sections(pairs, axes):
    """Pairs of each position axis: frame gets what rows and columns leave."""
    if axes == 1:
        return (pairs,)
    third = pairs // 3
    return (pairs - 2 * third, third, third)


def _frequencies(pairs, axes, stretch):
    """Angle per position of each pair, float64; for a stretched context the low frequencies are slowed down by it and the high
    ones kept, with a linear ramp between 1 and 32 turns over the original 8192 positions. Returns them and the factor on
    the rotated values that goes with the stretch."""
    out = []
    for n in _sections(pairs, axes):
        f = 10000.0 ** (-torch.arange(n, dtype=torch.float64) / max(n, 1))
        if stretch != 1.0:
            turns = 8192 * f / (2 * math.pi)
            keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
            f = f * keep + f / stretch * (1 - keep)
        out.append(f)
    return torch.cat(out).cuda(), (1.0 if stretch == 1.0 else 0.1 * math.log(stretch) + 1.0)


def _bounds(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _kept_tiles(q, k, tsf):
    """The forward's decisions on one sequence: bool [H, query blocks, tiles], from the running row maxima of the kept tiles."""
    S, H, D = q.shape
    G = H // k.shape[1]
    T = -(-S // TILE)
    limit = math.log2(tsf / S)
    c = math.log2(math.e) / math.sqrt(D)
    keep = torch.empty((H, T, T), dtype=torch.bool, device="cuda")
    for h in range(H):
        s = q[:, h].float() @ k[:, h // G].float().T
        s = torch.nn.functional.pad(s, (0, T * TILE - S), value=-math.inf).view(S, T, TILE).amax(-1) * c
        s = torch.nn.functional.pad(s, (0, 0, 0, T * TILE - S), value=-math.inf).view(T, TILE, T)
        valid = (torch.arange(T * TILE, device="cuda") < S).view(T, TILE)
        m = torch.full((T, TILE), -math.inf, device="cuda")
        for j in range(T):
            d = torch.where(valid, s[:, :, j] - m, -math.inf).amax(1)
            on = (d >= limit) if j else torch.ones_like(d, dtype=torch.bool)
            keep[h, :, j] = on
            m = torch.where(on[:, None], torch.maximum(m, s[:, :, j]), m)
    return keep


def _bitmap(keeps, H, longest):
    """Bit j & 31 of word j >> 5 is one where tile j is skipped: int32 [H, query blocks, words]."""
    words = (-(-longest // TILE) + 31) // 32
    out = []
    for keep in keeps:
        skipped = torch.nn.functional.pad(~keep, (0, words * 32 - keep.shape[2])).view(H, keep.shape[1], words, 32)
        w = (skipped.to(torch.int64) << torch.arange(32, device="cuda")).sum(-1)
        out.append(torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32))
    return torch.cat(out, 1).contiguous()


def _encode(x):
    """E4M3 codes (as bytes) and the power-of-two scale of each 128 tokens and head."""
    T, H, D = x.shape
    blocks = -(-T // TILE)
    padded = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, blocks * TILE - T)).view(blocks, TILE, H, D)
    m, e = torch.frexp(padded.abs().amax((1, 3)))
    e = torch.where(m <= 0.875, e - 9, e - 8)  # 448 = 0.875 * 2^9: the smallest power of two that holds the largest value
    scale = torch.where(m > 0, torch.ldexp(torch.ones_like(m), e.clamp(min=-100)), torch.ones_like(m))
    code = (padded / scale[:, None, :, None]).to(torch.float8_e4m3fn).view(blocks * TILE, H, D)[:T]
    return code.contiguous().view(torch.uint8), scale


def _decode(code, scale):
    T, H, D = code.shape
    rows = scale.repeat_interleave(TILE, 0)[:T, :, None]
    return code.view(torch.float8_e4m3fn).float() * rows


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    D, H = case["dim"], case["heads"]
    if case["op"] == "rotary":
        T, Hk = case["tokens"], case["kv_heads"]
        q, k = _noise((T, H, D), g).bfloat16(), _noise((T, Hk, D), g).bfloat16()
        if case["axes"] == 1:
            pos = torch.arange(T, device="cuda", dtype=torch.int32) + case["far"] + int(seed) % 1000
        else:
            pos = _grid(T) + case["far"]
        freq, factor = _frequencies(case["rot"] // 2, case["axes"], case["stretch"])
        sections = _sections(case["rot"] // 2, case["axes"])
        axis = torch.tensor([a for a, n in enumerate(sections) for _ in range(n)], device="cuda")
        return {"case": case, "q": q, "k": k, "positions": pos.contiguous(), "freq": freq, "factor": factor, "sections": sections,
                "axis": axis}
    if case["op"] == "checkpoint":
        # activations with heads of different sizes
        size = torch.exp2(_noise((1, H, 1), g) * 3)
        return {"case": case, "x": (_noise((case["tokens"], H, D), g) * size).bfloat16()}
    lens, Hk = _lengths(case), case["kv_heads"]
    total, cu = sum(lens), _bounds(lens)
    code = _code(lens, D, case["amp"])[:, None]
    q = (_noise((total, H, D), g) + code).bfloat16()
    k = (_noise((total, Hk, D), g) + code).bfloat16()
    v = _noise((total, Hk, D), g).bfloat16()
    s = {"case": case, "dout": _noise((total, H, D), g).bfloat16(), "q": q, "k": k, "v": v, "lens": lens, "cu": cu,
         "cu_seqlens": torch.tensor(cu, dtype=torch.int32, device="cuda"), "longest": max(lens), "bitmap": None, "keep": None}
    if case["op"] == "step":
        return s
    if case["tsf"] > 0:
        s["keep"] = [_kept_tiles(q[a:b], k[a:b], case["tsf"]) for a, b in zip(cu, cu[1:])]
        s["bitmap"] = _bitmap(s["keep"], H, s["longest"])
    out, s["lse"] = _forward(q, k, v, cu, s["keep"])
    s["out"] = out.bfloat16()
    if case["op"] == "backward_saved":
        for n in "qkv":
            s[n + "_saved"] = _encode(s.pop(n))
    return s


# -------------------------------------------------------------- plain forms

def _chunks(cu, Hk, G):
    """(sequence, first row, end, first and end KV head) such that a chunk's scores stay near 2^31 values."""
    for b, (lo, hi) in enumerate(zip(cu, cu[1:])):
        n = max(1, 2 ** 31 // max(1, (hi - lo) ** 2 * G))
        for h in range(0, Hk if hi > lo else 0, n):
            yield b, lo, hi, h, min(Hk, h + n)


def _heads(x, lo, hi, a, b, G):
    """Rows lo..hi of KV heads a..b, each with its G query heads: [b - a, G, rows, D] in 32 bits."""
    return x[lo:hi, a * G:b * G].float().permute(1, 0, 2).reshape(b - a, G, hi - lo, x.shape[2])


def _skipped(keep, a, b, G, n):
    on = keep[a * G:b * G].repeat_interleave(TILE, 1)[:, :n].repeat_interleave(TILE, 2)[:, :, :n]
    return ~on.reshape(b - a, G, n, n)


def _forward(q, k, v, cu, keep=None):
    """softmax(q k^T / sqrt(D)) v over the kept tiles, and the rows' log-sum-exp [H, total], in 32 bits."""
    total, H, D = q.shape
    Hk = k.shape[1]
    G = H // Hk
    out = torch.zeros((total, H, D), device="cuda")
    lse = torch.zeros((H, total), device="cuda")
    for i, lo, hi, a, b in _chunks(cu, Hk, G):
        kk, vv = _heads(k, lo, hi, a, b, 1), _heads(v, lo, hi, a, b, 1)
        s = (_heads(q, lo, hi, a, b, G) * (1.0 / math.sqrt(D))).reshape(b - a, -1, D) @ kk[:, 0].mT
        s = s.view(b - a, G, hi - lo, hi - lo)
        if keep is not None:
            s.masked_fill_(_skipped(keep[i], a, b, G, hi - lo), -math.inf)
        m = s.amax(-1, keepdim=True)
        s = s.sub_(m).exp_()
        l = s.sum(-1, keepdim=True)
        o = (s.view(b - a, -1, hi - lo) @ vv[:, 0]).view(b - a, G, hi - lo, D) / l
        out[lo:hi, a * G:b * G] = o.reshape(-1, hi - lo, D).permute(1, 0, 2)
        lse[a * G:b * G, lo:hi] = (m + l.log()).reshape(-1, hi - lo)
    return out, lse


def _backward(dout, q, k, v, out, lse, cu, keep=None):
    """dQ, dK, dV with the probabilities recomputed from the rows' log-sum-exp, in 32 bits, rounded at the end."""
    total, H, D = dout.shape
    Hk = k.shape[1]
    G = H // Hk
    scale = 1.0 / math.sqrt(D)
    dq = torch.zeros((total, H, D), device="cuda", dtype=torch.bfloat16)
    dk = torch.zeros((total, Hk, D), device="cuda", dtype=torch.bfloat16)
    dv = torch.zeros_like(dk)
    for i, lo, hi, a, b in _chunks(cu, Hk, G):
        n = hi - lo
        flat = lambda t: t.reshape(b - a, G * n, -1)  # noqa: E731
        qq, do = flat(_heads(q, lo, hi, a, b, G)), flat(_heads(dout, lo, hi, a, b, G))
        kk, vv = _heads(k, lo, hi, a, b, 1)[:, 0], _heads(v, lo, hi, a, b, 1)[:, 0]
        delta = (do * flat(_heads(out, lo, hi, a, b, G))).sum(-1, keepdim=True)
        p = (qq * scale) @ kk.mT
        if keep is not None:
            p.masked_fill_(flat(_skipped(keep[i], a, b, G, n)), -math.inf)
        p = p.sub_(lse[a * G:b * G, lo:hi].reshape(b - a, G * n, 1)).exp_()
        dv[lo:hi, a:b] = (p.mT @ do).permute(1, 0, 2).bfloat16()
        ds = (do @ vv.mT).sub_(delta).mul_(p)
        del p
        dq[lo:hi, a * G:b * G] = ((ds @ kk) * scale).view(-1, n, D).permute(1, 0, 2).bfloat16()
        dk[lo:hi, a:b] = ((ds.mT @ qq) * scale).permute(1, 0, 2).bfloat16()
    return dq, dk, dv


def _rotate(x, s):
    case = s["case"]
    angle = s["positions"].view(x.shape[0], -1).double()[:, s["axis"]] * s["freq"]
    if case["transpose"]:
        angle = -angle
    cos, sin = (angle.cos() * s["factor"]).float()[:, None], (angle.sin() * s["factor"]).float()[:, None]
    out = x.float()
    part = out[..., :case["rot"]]
    if case["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = part.chunk(2, -1)
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, out[..., case["rot"]:]], -1).bfloat16()


def _run_plain(s):
    op = s["case"]["op"]
    if op == "rotary":
        return {"q": _rotate(s["q"], s), "k": _rotate(s["k"], s)}
    if op == "checkpoint":
        code, scale = _encode(s["x"])
        return {"restored": _decode(code, scale).bfloat16(), "scales": scale}
    if op == "step":
        out, lse = _forward(s["q"], s["k"], s["v"], s["cu"])
        out = out.bfloat16()
        dq, dk, dv = _backward(s["dout"], s["q"], s["k"], s["v"], out, lse, s["cu"])
        return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    q, k, v = (_decode(*s[n + "_saved"]) for n in "qkv") if op == "backward_saved" else (s["q"], s["k"], s["v"])
    dq, dk, dv = _backward(s["dout"], q, k, v, s["out"], s["lse"], s["cu"], s["keep"])
    return {"dq": dq, "dk": dk, "dv": dv}


# --------------------------------------------------------- the framework's

def _run_own(s):
    ssa = _framework()
    case = s["case"]
    op = case["op"]
    if op == "rotary":
        q, k = ssa.rotary(s["q"], s["k"], s["positions"], s["freq"], sections=s["sections"], interleaved=case["interleaved"],
                          scale=s["factor"], transpose=case["transpose"])
        return {"q": q, "k": k}
    if op == "checkpoint":
        codes, scales = ssa.save_fp8(s["x"])
        return {"restored": ssa.restore_fp8(codes, scales), "scales": scales}
    if op == "step":
        out, lse = ssa.fwd_lse(s["q"], s["k"], s["v"], s["cu_seqlens"], s["longest"])
        dq, dk, dv = ssa.bwd(s["dout"], s["q"], s["k"], s["v"], out, lse, s["cu_seqlens"], s["longest"])
        return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    if op == "backward_saved":
        dq, dk, dv = ssa.bwd_fp8(s["dout"], s["q_saved"], s["k_saved"], s["v_saved"], s["out"], s["lse"], s["cu_seqlens"],
                                 s["longest"])
    else:
        dq, dk, dv = ssa.bwd(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["cu_seqlens"], s["longest"],
                             decision_bitmap=s["bitmap"])
    return {"dq": dq, "dk": dk, "dv": dv}


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ---------------------------------------------------------------- 64 bits

def _e4m3_values(y):
    """The E4M3 value nearest to each y, ties to the even code: 3 bits of mantissa, exponents from -6, largest 448."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    e = torch.where(torch.exp2(e + 1) <= y.abs(), e + 1, torch.where((torch.exp2(e) > y.abs()) & (e > -6), e - 1, e))
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _codes_value(code):
    """A code byte's value from the format: sign, 4 bits of exponent with bias 7, 3 bits of mantissa."""
    c = code.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    x = torch.where(e > 0, (1 + m / 8) * torch.exp2((e - 7).double()), m * 2.0 ** -9)
    return torch.where(c >= 128, -x, x)


def _exact_attention(s):
    """Every row block of every head in 64 bits; the log-sum-exp and the output that a backward pass is given are its inputs."""
    case = s["case"]
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    G, total, step = H // Hk, s["cu"][-1], case["op"] == "step"
    if case["op"] == "backward_saved":
        q, k, v = (_codes_value(c) * sc.double().repeat_interleave(TILE, 0)[:total, :, None]
                   for c, sc in (s["q_saved"], s["k_saved"], s["v_saved"]))
    else:
        q, k, v = s["q"], s["k"], s["v"]
    new = lambda heads: torch.zeros((total, heads, D), dtype=torch.float64, device="cuda")  # noqa: E731
    r = {"dq": new(H), "dk": new(Hk), "dv": new(Hk)}
    if step:
        r |= {"out": new(H), "lse": torch.zeros((H, total), dtype=torch.float64, device="cuda")}
    for i, (lo, hi) in enumerate(zip(s["cu"], s["cu"][1:])):
        for h in range(H if hi > lo else 0):
            K, V = k[lo:hi, h // G].double(), v[lo:hi, h // G].double()
            block = max(TILE, (2 ** 28 // (hi - lo)) // TILE * TILE)
            for x in range(lo, hi, block):
                y = min(hi, x + block)
                Q, dO = q[x:y, h].double(), s["dout"][x:y, h].double()
                z = torch.einsum("id,jd->ij", Q, K) / D ** 0.5
                if s["keep"] is not None:
                    on = s["keep"][i][h, torch.arange(x - lo, y - lo, device="cuda") // TILE][:, torch.arange(hi - lo, device="cuda") // TILE]
                    z = torch.where(on, z, -math.inf)
                L = torch.logsumexp(z, 1) if step else s["lse"][h, x:y].double()
                P = torch.exp(z - L[:, None])
                O = P @ V if step else s["out"][x:y, h].double()
                if step:
                    r["out"][x:y, h], r["lse"][h, x:y] = O, L
                dP = torch.einsum("id,jd->ij", dO, V)
                dZ = P * (dP - torch.einsum("id,id->i", dO, O)[:, None]) / D ** 0.5
                r["dq"][x:y, h] = dZ @ K
                r["dk"][lo:hi, h // G] += dZ.T @ Q
                r["dv"][lo:hi, h // G] += P.T @ dO
    return r


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        sign = -1.0 if case["transpose"] else 1.0
        pairs = case["rot"] // 2
        axis = [a for a, n in enumerate(s["sections"]) for _ in range(n)]
        p = s["positions"].reshape(case["tokens"], -1).double()
        angle = torch.stack([sign * p[:, a] * s["freq"][i] for i, a in enumerate(axis)], 1)
        turn = torch.polar(torch.full_like(angle, s["factor"]), angle)[:, None]
        got = {}
        for n in ("q", "k"):
            x = s[n].double()
            left = torch.arange(pairs, device="cuda") * (2 if case["interleaved"] else 1)
            right = left + (1 if case["interleaved"] else pairs)
            z = torch.complex(x[..., left], x[..., right]) * turn
            x[..., left], x[..., right] = z.real, z.imag
            got[n] = x
        return got
    if case["op"] == "checkpoint":
        x = s["x"]
        T, H, D = x.shape
        restored = torch.empty((T, H, D), dtype=torch.float64, device="cuda")
        scales = torch.ones((-(-T // TILE), H), dtype=torch.float64, device="cuda")
        for i, lo in enumerate(range(0, T, TILE)):
            y = x[lo:lo + TILE].double()
            top = y.abs().amax((0, 2))
            e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -91) / E4M3_MAX))
            e = torch.where(torch.exp2(e - 1) * E4M3_MAX >= top, e - 1, e)
            scales[i] = torch.where(top > 0, torch.exp2(e), 1.0)
            restored[lo:lo + TILE] = _e4m3_values(y / scales[i][:, None]) * scales[i][:, None]
        return {"restored": restored, "scales": scales}
    return _exact_attention(s)
