"""Cases of windowed attention (forward, backward, decode) and of caches held in 4 bits (rows in and out, decode).

Shapes are written as the package writes them: B sequences, n_q query heads on
n_kv key/value heads, d values per head, bf16 [B, L, H, d] tensors.

Window: a row at position p sees the keys j <= p with j > p - W or j < S (the
last W positions, its own among them, and the first S, the sinks).

4 bits: uint8 [B, n_kv, C, 80], one row of 80 bytes per sequence, head and
position. Each of the four groups of 32 channels has a scale and a lowest value
lo in bf16 and 32 codes of 0 .. 15; a code stands for lo + scale * code. Byte
4 * (4 t + g) on hold the eight codes of channels 32 g + 8 t .. + 7, the first
in the lowest four bits; bytes 64 + 4 g on hold scale and lo of group g. A
group that holds something not finite has scale and lo NaN.
"""

import math

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16


# ------------------------------------------------------------------ the cases


def listed():
    return [
        # A few short prompts of odd length with a small window: latency counts.
        dict(name="window tiny", op="window", B=2, Lq=333, Lk=333, n_q=4, n_kv=1, d=64, W=100, S=3),
        # A whole 8192-token prompt of a 32-head layer that sees 1024 positions and four sinks.
        dict(name="window layer", op="window", B=1, Lq=8192, Lk=8192, n_q=32, n_kv=8, d=128, W=1024,
             S=4),
        # The last chunk of a long prompt of a 36-head layer with a wide window.
        dict(name="window long", op="window", B=1, Lq=8192, Lk=131072, n_q=36, n_kv=6, d=128, W=4096,
             S=64),
        # Gradients of a short training sequence without sinks.
        dict(name="backward small", op="backward", B=1, L=1000, n_q=8, n_kv=2, d=64, W=256, S=0),
        # Gradients of the 8192-token layer.
        dict(name="backward layer", op="backward", B=1, L=8192, n_q=32, n_kv=8, d=128, W=1024, S=4),
        # One token for a few short sequences, one of them still empty.
        dict(name="step small", op="step", B=3, C=333, n_q=10, n_kv=5, W=64, S=4, low=1, empty=True),
        # One token for a serving batch: short and long sequences cost the same behind a window.
        dict(name="step layer", op="step", B=64, C=8192, n_q=32, n_kv=8, W=1024, S=4, low=100,
             empty=False),
        # A decode step's rows of a batch appended to 4-bit caches (and read back).
        dict(name="rows append", op="rows", B=64, L=1, C=2048, n_kv=8, ragged=False),
        # The rows of a batch of prompts of different lengths, into 4-bit caches and back.
        dict(name="rows prompt", op="rows", B=4, L=8192, C=8200, n_kv=8, ragged=True),
        # One token for a few short sequences with 4-bit caches, behind a window.
        dict(name="four small", op="four", B=3, C=500, n_q=8, n_kv=2, W=200, S=4, low=1, empty=True),
        # A serving batch whose sequences have very different lengths, caches in 4 bits.
        dict(name="four layer", op="four", B=16, C=8192, n_q=32, n_kv=8, W=0, S=0, low=1024,
             empty=False),
        # One sequence with a long cache in 4 bits.
        dict(name="four long", op="four", B=1, C=131072, n_q=36, n_kv=6, W=0, S=0, low=131072,
             empty=False),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _heads(rng, most):
    n_kv = rng.choice([1, 2, 3, 5, 6, 8])
    g = rng.choice([1, 2, 3, 4, 6, 7, 8, 12, 16])
    while n_kv * g > most:
        g = rng.choice([1, 2, 3, 4, 6, 8])
    return n_kv * g, n_kv


def _sinks(rng):
    return rng.choice([0, 0, 1, 4, 16, 64, rng.randint(1, 300)])


def draw(rng):
    op = rng.choice(["window", "backward", "step", "rows", "four"])
    most = 4 * 128 * 36 * 8192 * 4160
    if op in ("window", "backward"):
        while True:
            n_q, n_kv = _heads(rng, 64)
            c = dict(op=op, B=rng.choice([1, 1, 2, 3, 5]), n_q=n_q, n_kv=n_kv,
                     d=rng.choice([64, 128]), W=_log(rng, 1, 8192), S=_sinks(rng))
            if op == "window":
                c["Lk"] = _log(rng, 1, 131072)
                c["Lq"] = c["Lk"] if rng.random() < 0.4 else _log(rng, 1, min(c["Lk"], 8192))
            else:
                c["L"] = _log(rng, 1, 16384)
            rows, keys = (c["Lq"], c["Lk"]) if op == "window" else (c["L"], c["L"])
            if (work(c)["flops"] <= most // (1 if op == "window" else 2)
                    and c["B"] * rows * n_q <= 1 << 20 and c["B"] * keys * n_kv <= 1 << 20):
                return c
    if op == "rows":
        while True:
            B, L, n_kv = _log(rng, 1, 128), _log(rng, 1, 16384), rng.choice([1, 2, 3, 5, 6, 8])
            if B * L * n_kv <= 4 * 8192 * 8:
                return dict(op=op, B=B, L=L, C=L + _log(rng, 1, 300) - 1, n_kv=n_kv,
                            ragged=rng.random() < 0.6)
    while True:
        n_q, n_kv = _heads(rng, 64)
        B, C = _log(rng, 1, 128), _log(rng, 1, 131072)
        if B * C * n_kv <= 16 * 8192 * 8:
            break
    W = _log(rng, 1, 8192) if op == "step" or rng.random() < 0.4 else 0
    return dict(op=op, B=B, C=C, n_q=n_q, n_kv=n_kv, W=W, S=_sinks(rng) if W else 0,
                low=_log(rng, 1, C), empty=B > 1 and rng.random() < 0.4)


# ------------------------------------------------------------------ the inputs


def _lens(c):
    """Lengths spread evenly from the shortest to the capacity, and one of zero where asked."""
    lens = [round(c["C"] + (c["low"] - c["C"]) * b / max(1, c["B"] - 1)) for b in range(c["B"])]
    if c.get("empty"):
        lens[-1] = 0
    return lens


def _counts(c):
    """Rows that the sequences of a batch have: all of them, or different numbers, one of zero."""
    if not c["ragged"]:
        return [c["L"]] * c["B"]
    return [c["L"] * (c["B"] - b) // c["B"] for b in range(c["B"])][:-1] + [0 if c["B"] > 1 else c["L"]]


def _pack(x):
    """Rows [..., 128] as the 80 bytes that hold them in 4 bits."""
    g = x.double().unflatten(-1, (4, 32))
    low, high = g.amin(-1), g.amax(-1)
    span = high - low
    scale = (span / 15).float().to(BF16)
    scale = torch.where(span.isfinite(), scale, math.nan)
    low = torch.where(span.isfinite(), low, math.nan).to(BF16)
    step = scale.double()
    code = ((g - low.double()[..., None]) / torch.where(step > 0, step, 1.0)[..., None]).round()
    code = torch.where((step > 0)[..., None], code.clamp(0, 15), 0.0).to(torch.uint8)
    code = code.unflatten(-1, (4, 8)).transpose(-3, -2).flatten(-3)      # [group, eight] -> [eight, group]
    code = code[..., 0::2] | code[..., 1::2] << 4
    return torch.cat([code, torch.stack([scale, low], -1).flatten(-2).contiguous().view(torch.uint8)],
                     -1)


def _unpack(rows, dtype=torch.float32):
    """The values [..., 128] that rows of 80 bytes stand for."""
    code = torch.stack([rows[..., :64] & 15, rows[..., :64] >> 4], -1).flatten(-2)
    code = code.unflatten(-1, (4, 4, 8)).transpose(-3, -2).flatten(-2)   # [.., group, 32]
    pair = rows[..., 64:].contiguous().view(BF16).unflatten(-1, (4, 2)).to(dtype)
    return (pair[..., 1, None] + pair[..., 0, None] * code).flatten(-2)


def _filled(c, gen):
    """A 4-bit cache of normal rows, some channels much larger than the others (as keys have them)."""
    out = torch.empty(c["B"], c["n_kv"], c["C"], 80, dtype=torch.uint8, device=DEV)
    gain = torch.ones(128, device=DEV)
    gain[5::32] = 6.0
    for b in range(c["B"]):
        for i in range(0, c["C"], 16384):
            n = min(16384, c["C"] - i)
            x = torch.randn(c["n_kv"], n, 128, generator=gen, device=DEV) * gain
            out[b, :, i:i + n] = _pack(x.to(BF16))
    return out


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen, device=DEV).to(BF16)  # noqa: E731
    st = {"case": c}
    if c["op"] in ("window", "backward"):
        Lq, Lk = (c["Lq"], c["Lk"]) if c["op"] == "window" else (c["L"], c["L"])
        st["q"] = normal(c["B"], Lq, c["n_q"], c["d"])
        st["k"] = normal(c["B"], Lk, c["n_kv"], c["d"])
        st["v"] = normal(c["B"], Lk, c["n_kv"], c["d"])
        if c["op"] == "backward":
            out = _plain_window(st)                # what the forward returned
            st["o"], st["lse"] = out["o"], out["lse"]
            st["dout"] = normal(c["B"], Lq, c["n_q"], c["d"])
        return st
    if c["op"] == "rows":
        st["k"] = normal(c["B"], c["L"], c["n_kv"], 128)
        st["v"] = normal(c["B"], c["L"], c["n_kv"], 128)
        st["k"][..., 5::32] *= 6.0
        st["k4"] = torch.zeros(c["B"], c["n_kv"], c["C"], 80, dtype=torch.uint8, device=DEV)
        st["v4"] = torch.zeros_like(st["k4"])
        st["at"] = torch.randint(0, c["C"] - c["L"] + 1, (c["B"],), generator=gen, device=DEV,
                                 dtype=torch.int32)
        st["counts"] = torch.tensor(_counts(c), device=DEV, dtype=torch.int32)
        return st
    order = torch.randperm(c["B"], generator=gen, device=DEV)
    st["lens"] = torch.tensor(_lens(c), device=DEV, dtype=torch.int32)[order]
    st["q"] = normal(c["B"], 1, c["n_q"], 128)
    if c["op"] == "step":
        st["k"] = normal(c["B"], c["C"], c["n_kv"], 128)
        st["v"] = normal(c["B"], c["C"], c["n_kv"], 128)
    else:
        st["k4"], st["v4"] = _filled(c, gen), _filled(c, gen)
    return st


# ------------------------------------------------------- the framework's calls


def _workspace(st, size):
    """A training or decode loop keeps its workspace from step to step."""
    if "workspace" not in st:
        st["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return st["workspace"]


def _call(st):
    import causal_gqa_prefill_gb300 as cg

    c = st["case"]
    if c["op"] == "window":
        o, lse = cg.attn_prefill_window(st["q"], st["k"], st["v"], c["W"], c["S"])
        return {"o": o, "lse": lse}
    if c["op"] == "backward":
        ws = _workspace(st, cg.attn_prefill_window_bwd_workspace_bytes(
            c["B"], c["L"], c["n_q"], c["n_kv"], c["d"], c["W"], c["S"]))
        dq, dk, dv = cg.attn_prefill_window_backward(st["q"], st["k"], st["v"], st["o"], st["lse"],
                                                     st["dout"], c["W"], c["S"], workspace=ws)
        return {"dq": dq, "dk": dk, "dv": dv}
    if c["op"] == "step":
        ws = _workspace(st, cg.attn_decode_window_workspace_bytes(c["B"], c["C"], c["n_q"], c["n_kv"],
                                                                  window=c["W"], sinks=c["S"]))
        o, lse = cg.attn_decode_window(st["q"], st["k"], st["v"], st["lens"], c["W"], c["S"],
                                       workspace=ws)
        return {"o": o, "lse": lse}
    if c["op"] == "rows":
        cg.attn_pack4(st["k"], st["v"], st["k4"], st["v4"], st["at"], counts=st["counts"])
        k, v = cg.attn_unpack4(st["k4"], st["v4"], c["L"], at=st["at"])
        return {"k": k, "v": v}
    ws = _workspace(st, cg.attn_decode4_workspace_bytes(c["B"], c["C"], c["n_q"], c["n_kv"],
                                                        window=c["W"], sinks=c["S"]))
    o, lse = cg.attn_decode4(st["q"], st["k4"], st["v4"], st["lens"], window=c["W"] or None,
                             sinks=c["S"], workspace=ws)
    return {"o": o, "lse": lse}


# ------------------------------------------------------------- the plain forms


def _blocks(c, Lq, Lk, width):
    """Blocks of rows with the keys that they see: (first row, last row, key index, hidden [rows, keys])."""
    off = Lk - Lq
    i0 = 0
    while i0 < Lq:
        i1 = min(Lq, i0 + width)
        low = max(0, off + i0 - c["W"] + 1)
        keys = torch.cat([torch.arange(min(c["S"], low), device=DEV),
                          torch.arange(low, off + i1, device=DEV)])
        at = torch.arange(off + i0, off + i1, device=DEV)[:, None]
        yield i0, i1, keys, (keys > at) | ((keys <= at - c["W"]) & (keys >= c["S"]))
        i0 = i1


def _grouped(x, n_kv):
    """[B, rows, n_q, d] as fp32 [B, n_kv, heads of a group, rows, d]."""
    B, rows, n_q, d = x.shape
    return x.float().view(B, rows, n_kv, n_q // n_kv, d).permute(0, 2, 3, 1, 4)


def _plain_window(st):
    q, k, v, c = st["q"], st["k"], st["v"], st["case"]
    B, Lq, n_q, d = q.shape
    Lk, n_kv = k.shape[1:3]
    o = torch.empty_like(q)
    lse = torch.empty(B, n_q, Lq, device=DEV)
    width = max(128, (1 << 28) // (B * n_q * min(Lk, c["W"] + c["S"] + 1024)))
    for i0, i1, keys, hidden in _blocks(c, Lq, Lk, min(1024, width)):
        s = _grouped(q[:, i0:i1], n_kv) @ k[:, keys].float().permute(0, 2, 3, 1)[:, :, None]
        s = s.mul_(1.0 / math.sqrt(d)).masked_fill_(hidden, -math.inf)
        m = s.amax(-1, keepdim=True)
        p = s.sub_(m).exp_()
        total = p.sum(-1, keepdim=True)
        out = (p @ v[:, keys].float().permute(0, 2, 1, 3)[:, :, None]) / total
        o[:, i0:i1] = out.permute(0, 3, 1, 2, 4).reshape(B, i1 - i0, n_q, d)
        lse[:, :, i0:i1] = (m + total.log()).reshape(B, n_q, -1)
    return {"o": o, "lse": lse}


def _plain_backward(st):
    q, k, v, c = st["q"], st["k"], st["v"], st["case"]
    B, L, n_q, d = q.shape
    n_kv, scale = k.shape[2], 1.0 / math.sqrt(d)
    dq = torch.empty_like(q)
    dk = torch.zeros(B, L, n_kv, d, device=DEV)
    dv = torch.zeros_like(dk)
    width = max(128, (1 << 27) // (B * n_q * min(L, c["W"] + c["S"] + 1024)))
    for i0, i1, keys, hidden in _blocks(c, L, L, min(1024, width)):
        rows = slice(i0, i1)
        qb, ob, gb = (_grouped(x[:, rows], n_kv) for x in (q, st["o"], st["dout"]))
        kb, vb = (x[:, keys].float().permute(0, 2, 1, 3)[:, :, None] for x in (k, v))
        s = (qb @ kb.transpose(-1, -2)).mul_(scale)
        p = s.sub_(st["lse"][:, :, rows].reshape(B, n_kv, -1, i1 - i0, 1)).exp_()
        p = p.masked_fill_(hidden, 0.0)
        ds = p * (gb @ vb.transpose(-1, -2) - (gb * ob).sum(-1, keepdim=True)) * scale
        dq[:, rows] = (ds @ kb).permute(0, 3, 1, 2, 4).reshape(B, i1 - i0, n_q, d)
        dk.index_add_(1, keys, (ds.transpose(-1, -2) @ qb).sum(2).transpose(1, 2))
        dv.index_add_(1, keys, (p.transpose(-1, -2) @ gb).sum(2).transpose(1, 2))
    return {"dq": dq, "dk": dk.to(BF16), "dv": dv.to(BF16)}


def _plain_seen(c, lens):
    """The cache positions that one token per sequence sees: index [B, n], and which of them count."""
    at, end = torch.arange(c["C"], device=DEV)[None], lens.long()[:, None]
    if not c["W"]:
        return at.expand(c["B"], -1), at < end
    if c["S"] + c["W"] >= c["C"]:
        return at.expand(c["B"], -1), (at < end) & ((at >= end - c["W"]) | (at < c["S"]))
    first = (end - c["W"]).clamp_min(0)
    sinks = torch.arange(c["S"], device=DEV)[None].expand(c["B"], -1)
    recent = first + torch.arange(c["W"], device=DEV)
    return torch.cat([sinks, recent], 1), torch.cat([sinks < first, recent < end], 1)


def _plain_token(c, q, k, v, seen):
    """One token per sequence against the rows k, v fp32 [B, n_kv, n, 128] of which ``seen`` count."""
    B, n_kv, _, d = k.shape
    s = (q.float().view(B, n_kv, -1, d) @ k.transpose(2, 3)).mul_(1.0 / math.sqrt(d))
    s = s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / total.clamp_min(1e-37)
    return {"o": o.reshape(B, 1, -1, d).to(BF16), "lse": (m + total.log()).reshape(B, -1, 1)}


def _plain_step(st):
    index, seen = _plain_seen(st["case"], st["lens"])
    b = torch.arange(len(index), device=DEV)[:, None]
    k, v = (x[b, index].float().transpose(1, 2) for x in (st["k"], st["v"]))
    return _plain_token(st["case"], st["q"], k, v, seen)


def _plain_four(st):
    c = st["case"]
    index, seen = _plain_seen(c, st["lens"])
    k, v = st["k4"], st["v4"]
    if index.shape[1] < c["C"]:
        index = index[:, None, :, None].expand(-1, c["n_kv"], -1, 80)
        k, v = k.gather(2, index), v.gather(2, index)
    return _plain_token(c, st["q"], _unpack(k), _unpack(v), seen)


def _plain_rows(st):
    c = st["case"]
    at = st["at"].long()[:, None] + torch.arange(c["L"], device=DEV)
    index = at[:, None, :, None].expand(-1, c["n_kv"], -1, 80)
    stored = (torch.arange(c["L"], device=DEV) < st["counts"][:, None])[:, None, :, None]
    out = {}
    for name in ("k", "v"):
        cache = st[name + "4"]
        rows = torch.where(stored, _pack(st[name].transpose(1, 2)), cache.gather(2, index))
        cache.scatter_(2, index, rows)
        out[name] = _unpack(cache.gather(2, index)).transpose(1, 2).to(BF16).contiguous()
    return out


def run(state):
    if own:
        return _call(state)
    return {"window": _plain_window, "backward": _plain_backward, "step": _plain_step,
            "rows": _plain_rows, "four": _plain_four}[state["case"]["op"]](state)


# ------------------------------------------------------------------- the costs


def _pairs(Lq, Lk, W, S):
    """Keys that the rows of a chunk see, summed over its rows."""
    def upto(n):                       # rows at positions 0 .. n - 1
        whole = min(n, W + S)          # these see everything before them
        return whole * (whole + 1) // 2 + (n - whole) * (W + S)
    return upto(Lk) - upto(Lk - Lq)


def work(case):
    c = case
    if c["op"] in ("window", "backward"):
        Lq, Lk = (c["Lq"], c["Lk"]) if c["op"] == "window" else (c["L"], c["L"])
        rows = c["B"] * Lq * c["n_q"]
        first = max(0, Lk - Lq - c["W"] + 1)                 # keys before it: sinks only
        keys = c["B"] * c["n_kv"] * (Lk - first + min(c["S"], first))
        pairs = c["B"] * c["n_q"] * _pairs(Lq, Lk, c["W"], c["S"])
        if c["op"] == "window":
            return {"bytes": 2 * c["d"] * (2 * rows + 2 * keys) + 4 * rows, "flops": 4 * c["d"] * pairs}
        return {"bytes": 2 * c["d"] * (4 * rows + 4 * keys) + 4 * rows, "flops": 10 * c["d"] * pairs}
    if c["op"] == "rows":
        n = 2 * sum(_counts(c)) * c["n_kv"]                  # rows of K and V stored
        read = 2 * c["B"] * c["L"] * c["n_kv"]               # and read back
        return {"bytes": (256 + 80) * (n + read), "flops": 0}
    seen = sum(min(n, c["W"] + min(c["S"], max(0, n - c["W"]))) if c["W"] else n for n in _lens(c))
    held = 512 if c["op"] == "step" else 160
    return {"bytes": held * seen * c["n_kv"] + c["B"] * c["n_q"] * (2 * 256 + 4),
            "flops": 4 * 128 * c["n_q"] * seen}


# --------------------------------------------------- the definitions in 64 bits


def _exact_window(c, st, Lq, Lk, backward):
    """Head by head, blocks of rows against the whole span of keys from the first that one of them sees."""
    q, k, v = st["q"], st["k"], st["v"]
    B, _, n_q, d = q.shape
    g = n_q // k.shape[2]
    f64 = dict(dtype=torch.float64, device=DEV)
    o, lse = torch.zeros(q.shape, **f64), torch.zeros(B, n_q, Lq, **f64)
    dq, dk, dv = torch.zeros(q.shape, **f64), torch.zeros(k.shape, **f64), torch.zeros(k.shape, **f64)
    step = 1024
    for i in range(0, Lq, step):
        pos = torch.arange(Lk - Lq + i, Lk - Lq + min(Lq, i + step), device=DEV)
        start = max(0, int(pos[0]) - c["W"] + 1)
        at = torch.arange(start, int(pos[-1]) + 1, device=DEV)
        if start > 0:
            at = torch.cat([torch.arange(0, min(c["S"], start), device=DEV), at])
        see = (at[None] <= pos[:, None]) & ((pos[:, None] - at[None] < c["W"]) | (at[None] < c["S"]))
        for b in range(B):
            for h in range(n_q):
                u, r = h // g, slice(i, i + len(pos))
                Q, K, V = q[b, r, h].double(), k[b, at, u].double(), v[b, at, u].double()
                s = torch.einsum("id,jd->ij", Q, K) * d ** -0.5
                if not backward:
                    s = torch.where(see, s, -math.inf)
                    total = torch.logsumexp(s, 1)
                    lse[b, h, r] = total
                    o[b, r, h] = torch.einsum("ij,jd->id", torch.exp(s - total[:, None]), V)
                    continue
                p = torch.exp(s - st["lse"][b, h, r].double()[:, None]) * see
                G = st["dout"][b, r, h].double()
                ds = p * (torch.einsum("id,jd->ij", G, V)
                          - torch.einsum("id,id->i", G, st["o"][b, r, h].double())[:, None])
                dq[b, r, h] = torch.einsum("ij,jd->id", ds, K) * d ** -0.5
                dk[b, :, u].index_add_(0, at, torch.einsum("ij,id->jd", ds, Q) * d ** -0.5)
                dv[b, :, u].index_add_(0, at, torch.einsum("ij,id->jd", p, G))
    return {"dq": dq, "dk": dk, "dv": dv} if backward else {"o": o, "lse": lse}


def _stands_for(rows):
    """Rows of 80 bytes as 64-bit values, block of eight codes by block."""
    out = torch.empty(*rows.shape[:-1], 128, dtype=torch.float64, device=rows.device)
    for g in range(4):
        scale, low = (rows[..., 64 + 4 * g + 2 * i:66 + 4 * g + 2 * i].contiguous().view(BF16).double()
                      for i in (0, 1))
        for t in range(4):
            for i in range(8):
                byte = rows[..., 4 * (4 * t + g) + i // 2].to(torch.int32)
                out[..., 32 * g + 8 * t + i] = low[..., 0] + scale[..., 0] * ((byte >> 4 * (i % 2)) & 15)
    return out


def _exact_token(c, st):
    B, g = c["B"], c["n_q"] // c["n_kv"]
    o = torch.zeros(B, 1, c["n_q"], 128, dtype=torch.float64, device=DEV)
    lse = torch.full((B, c["n_q"], 1), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(st["lens"].tolist()):
        first = max(0, n - c["W"]) if c["W"] else 0
        at = torch.tensor([*range(min(c["S"], first)), *range(first, n)], dtype=torch.long, device=DEV)
        for u in range(c["n_kv"] if n else 0):
            heads = slice(u * g, u * g + g)
            if c["op"] == "step":
                K, V = st["k"][b, at, u].double(), st["v"][b, at, u].double()
            else:
                K, V = _stands_for(st["k4"][b, u, at]), _stands_for(st["v4"][b, u, at])
            s = torch.einsum("hd,jd->hj", st["q"][b, 0, heads].double(), K) * 128 ** -0.5
            total = torch.logsumexp(s, 1)
            o[b, 0, heads] = torch.einsum("hj,jd->hd", torch.exp(s - total[:, None]), V)
            lse[b, heads, 0] = total
    return {"o": o, "lse": lse}


def _exact_rows(c, st):
    """What each stored row stands for once it is in 4 bits; rows that are not stored read as zeros."""
    out = {}
    for name in ("k", "v"):
        out[name] = torch.zeros(st[name].shape, dtype=torch.float64, device=DEV)
        for b, n in enumerate(st["counts"].tolist()):
            for g in range(4):
                x = st[name][b, :n, :, 32 * g:32 * g + 32].double()
                low, high = x.min(-1, keepdim=True)[0], x.max(-1, keepdim=True)[0]
                scale = ((high - low) / 15).to(torch.float32).to(BF16).double()
                code = torch.where(scale > 0, (x - low) / scale, torch.zeros_like(x)).round()
                out[name][b, :n, :, 32 * g:32 * g + 32] = low + scale * code.clamp(0, 15)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "window":
        return _exact_window(case, st, case["Lq"], case["Lk"], False)
    if case["op"] == "backward":
        return _exact_window(case, st, case["L"], case["L"], True)
    return (_exact_rows if case["op"] == "rows" else _exact_token)(case, st)
