"""Cases of the cache operators: key weights of a prefill, ragged decode, eviction and decode behind a shared prefix.

Shapes are written as the package writes them: B sequences, n_q query heads on
n_kv key/value heads, d values per head, bf16 [B, L, H, d] tensors. A cache
has room for C positions, of which sequence b holds lens[b].
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ the cases


def listed():
    return [
        # Weights of a short prompt's keys: the smallest call, latency counts.
        dict(name="weights tiny", op="weights", B=1, Lq=256, Lk=256, n_q=4, n_kv=1, d=64,
             causal=True, accumulate=False),
        # A whole 8192-token prompt of a 32-head layer.
        dict(name="weights layer", op="weights", B=1, Lq=8192, Lk=8192, n_q=32, n_kv=8, d=128,
             causal=True, accumulate=False),
        # The same layer, the prompt's last chunk added to the earlier chunks' weights.
        dict(name="weights chunk", op="weights", B=1, Lq=2048, Lk=8192, n_q=32, n_kv=8, d=128,
             causal=True, accumulate=True),
        # Only the last rows of a long prompt vote on its keys: K is read once, little is computed.
        dict(name="weights window", op="weights", B=1, Lq=32, Lk=131072, n_q=36, n_kv=6, d=128,
             causal=True, accumulate=False),
        # A few short sequences, one of them still empty.
        dict(name="ragged small", op="ragged", B=3, C=333, n_q=10, n_kv=5, low=1, empty=True,
             weighted=True),
        # A serving batch whose sequences have very different lengths, weights kept for eviction.
        dict(name="ragged layer", op="ragged", B=16, C=8192, n_q=32, n_kv=8, low=1024, empty=False,
             weighted=True),
        # One sequence with a long cache, no weights.
        dict(name="ragged long", op="ragged", B=1, C=131072, n_q=36, n_kv=6, low=131072,
             empty=False, weighted=False),
        # The batch's caches brought down to a quarter, with room to go on.
        dict(name="evict layer", op="evict", B=16, C=8192, n_kv=8, d=128, budget=2048, recent=256,
             capacity=2560, low=1024, fp8=False),
        # One long prompt's cache brought down to an eighth: few rows, each of them long.
        dict(name="evict long", op="evict", B=1, C=131072, n_kv=6, d=128, budget=16384,
             recent=1024, capacity=16384, low=131072, fp8=False),
        # A handful of answers to one prompt of odd length.
        dict(name="shared small", op="shared", B=4, P=1000, C=64, n_q=8, n_kv=2, low=1,
             empty=True),
        # A batch behind a long system prompt: memory and arithmetic weigh about the same.
        dict(name="shared layer", op="shared", B=64, P=8192, C=512, n_q=32, n_kv=8, low=1,
             empty=False),
        # A large batch behind a document, 64 heads: bound by the products with the prefix.
        dict(name="shared large", op="shared", B=256, P=32768, C=1024, n_q=64, n_kv=8, low=1,
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


def draw(rng):
    op = rng.choice(["weights", "ragged", "evict", "shared"])
    if op == "weights":
        while True:
            n_q, n_kv = _heads(rng, 64)
            B, Lk = rng.choice([1, 1, 2, 3, 5]), _log(rng, 1, 131072)
            Lq = _log(rng, 1, min(Lk, 8192))
            if B * n_q * Lq * Lk <= 32 * 8192 * 8192 // 2 and B * n_q * Lk <= 1 << 25:
                break
        return dict(op=op, B=B, Lq=Lq, Lk=Lk, n_q=n_q, n_kv=n_kv, d=rng.choice([64, 128]),
                    causal=rng.random() < 0.75, accumulate=rng.random() < 0.4)
    if op == "ragged":
        while True:
            n_q, n_kv = _heads(rng, 64)
            B, C = _log(rng, 1, 128), _log(rng, 1, 131072)
            if B * C * n_kv <= 16 * 8192 * 8:
                break
        return dict(op=op, B=B, C=C, n_q=n_q, n_kv=n_kv, low=_log(rng, 1, C),
                    empty=B > 1 and rng.random() < 0.4, weighted=rng.random() < 0.6)
    if op == "evict":
        while True:
            n_kv = rng.choice([1, 2, 3, 5, 6, 8])
            B, C = _log(rng, 1, 128), _log(rng, 2, 131072)
            if B * C * n_kv <= 16 * 8192 * 8:
                break
        budget = _log(rng, 1, C)
        return dict(op=op, B=B, C=C, n_kv=n_kv, d=rng.choice([64, 128]), budget=budget,
                    recent=rng.randint(0, budget), capacity=budget + _log(rng, 1, 300) - 1,
                    low=_log(rng, 1, C), fp8=rng.random() < 0.3)
    while True:
        n_q, n_kv = _heads(rng, 64)
        B, P, C = _log(rng, 1, 256), _log(rng, 1, 65536), _log(rng, 1, 4096)
        if B * P * n_q <= 256 * 32768 * 64 // 2 and B * C * n_kv <= 256 * 1024 * 8:
            break
    return dict(op=op, B=B, P=P, C=C, n_q=n_q, n_kv=n_kv, low=_log(rng, 1, C),
                empty=B > 1 and rng.random() < 0.4)


# ------------------------------------------------------------------ the inputs


def _lens(c):
    """Lengths spread evenly from the shortest to the capacity, and one of zero where asked."""
    lens = np.linspace(c["C"], c["low"], c["B"]).astype(np.int64)
    if c.get("empty"):
        lens[-1] = 0
    return lens


def _lse(c, q, k):
    """The log-sum-exp that the prefill forward returns beside its output, head by head."""
    B, Lq, n_q, d = q.shape
    Lk, n_kv = k.shape[1], k.shape[2]
    out = torch.empty(B, n_q, Lq, device=DEV)
    hidden = torch.ones(Lq, Lk, dtype=torch.bool, device=DEV).triu(Lk - Lq + 1)
    for b in range(B):
        for h in range(n_q):
            s = q[b, :, h].float() @ k[b, :, h // (n_q // n_kv)].float().T / math.sqrt(d)
            if c["causal"]:
                s.masked_fill_(hidden, -math.inf)
            out[b, h] = torch.logsumexp(s, 1)
    return out


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen, device=DEV).to(torch.bfloat16)  # noqa: E731
    st = {"case": c}
    if "low" in c:
        order = torch.randperm(c["B"], generator=gen, device=DEV)
        st["lens"] = torch.from_numpy(_lens(c)).to(DEV, torch.int32)[order]
    if c["op"] == "weights":
        st["q"] = normal(c["B"], c["Lq"], c["n_q"], c["d"])
        st["k"] = normal(c["B"], c["Lk"], c["n_kv"], c["d"])
        st["lse"] = _lse(c, st["q"], st["k"])
        st["weights"] = torch.rand(c["B"], c["n_kv"], c["Lk"], generator=gen, device=DEV)
    elif c["op"] == "evict":
        shape = (c["B"], c["C"], c["n_kv"], c["d"])
        kind = torch.float8_e4m3fn if c["fp8"] else torch.bfloat16
        st["k"], st["v"] = normal(*shape).to(kind), normal(*shape).to(kind)
        # accumulated weights: heavy-tailed, many keys that nothing attended to, some ties
        w = torch.rand(c["B"], c["n_kv"], c["C"], generator=gen, device=DEV)
        w = torch.where(w < 0.1, 0.0, (-4.0 * w).exp())
        coarse = torch.rand(w.shape, generator=gen, device=DEV) < 0.2
        st["weights"] = torch.where(coarse, (w * 64).round() / 64, w)
        # the caches that the kept rows go to; zeros, so that rows behind the last one can be compared
        st["k_out"] = torch.zeros(c["B"], c["capacity"], c["n_kv"], c["d"], device=DEV).to(kind)
        st["v_out"] = torch.zeros_like(st["k_out"])
    else:
        st["q"] = normal(c["B"], 1, c["n_q"], 128)
        st["k"] = normal(c["B"], c["C"], c["n_kv"], 128)
        st["v"] = normal(c["B"], c["C"], c["n_kv"], 128)
        if c["op"] == "shared":
            st["prefix_k"] = normal(1, c["P"], c["n_kv"], 128)
            st["prefix_v"] = normal(1, c["P"], c["n_kv"], 128)
        elif c["weighted"]:
            st["weights"] = torch.rand(c["B"], c["n_kv"], c["C"], generator=gen, device=DEV)
    return st


# ------------------------------------------------------- the framework's calls


def _workspace(st, size):
    """A decode loop keeps its workspace from step to step."""
    if "workspace" not in st:
        st["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return st["workspace"]


def _call(st):
    import causal_gqa_prefill_gb300 as cg

    c = st["case"]
    if c["op"] == "weights":
        return cg.attn_key_weights(st["q"], st["k"], st["lse"], causal=c["causal"],
                                   weights=st["weights"], accumulate=c["accumulate"])
    if c["op"] == "ragged":
        ws = _workspace(st, cg.attn_decode_ragged_workspace_bytes(
            c["B"], c["C"], c["n_q"], c["n_kv"], weighted=c["weighted"]))
        o, lse = cg.attn_decode_ragged(st["q"], st["k"], st["v"], st["lens"],
                                       weights=st.get("weights"), workspace=ws)
        return {"o": o, "lse": lse, **({"weights": st["weights"]} if c["weighted"] else {})}
    if c["op"] == "evict":
        k, v, w, lens, index = cg.attn_evict(st["k"], st["v"], st["weights"], st["lens"],
                                             c["budget"], c["recent"], k_out=st["k_out"],
                                             v_out=st["v_out"])
        return _evicted(c, k, v, w, lens, index)
    ws = _workspace(st, cg.attn_decode_shared_workspace_bytes(c["B"], c["P"], c["C"], c["n_q"],
                                                              c["n_kv"]))
    o, lse = cg.attn_decode_shared(st["q"], st["prefix_k"], st["prefix_v"], st["k"], st["v"],
                                   st["lens"], workspace=ws)
    return {"o": o, "lse": lse}


def _evicted(c, k, v, w, lens, index):
    k, v = (k.float(), v.float()) if c["fp8"] else (k, v)
    return {"k": k, "v": v, "weights": w, "lens": lens, "index": index}


# ------------------------------------------------------------- the plain forms


def _plain_weights(st):
    c = st["case"]
    B, Lq, n_q, d = st["q"].shape
    Lk, n_kv = st["k"].shape[1:3]
    q = st["q"].float().view(B, Lq, n_kv, -1, d).permute(0, 2, 3, 1, 4).reshape(B, n_kv, -1, d)
    s = q @ st["k"].float().permute(0, 2, 3, 1)
    s = s.view(B, n_kv, -1, Lq, Lk).mul_(1.0 / math.sqrt(d))
    s.sub_(st["lse"].view(B, n_kv, -1, Lq, 1)).exp_()
    if c["causal"]:
        s.masked_fill_(torch.ones(Lq, Lk, dtype=torch.bool, device=DEV).triu(Lk - Lq + 1), 0.0)
    w = s.sum((2, 3))
    if c["accumulate"]:
        st["weights"].add_(w)
    else:
        st["weights"].copy_(w)
    return st["weights"]


def _plain_softmax(s):
    """exp(s - max), its sum (at least the smallest number, for rows without a key) and the log of that sum."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    return p, total.clamp_min(1e-37), (m + total.log()).squeeze(-1)


def _plain_scores(st):
    """The scores of the sequences' own positions, -inf past their lengths: [B, n_kv, g, C]."""
    B, C, n_kv, d = st["k"].shape
    q = st["q"].float().view(B, n_kv, -1, d)
    s = (q @ st["k"].float().permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(d))
    hidden = torch.arange(C, device=DEV) >= st["lens"][:, None]
    return s.masked_fill_(hidden[:, None, None], -math.inf)


def _plain_ragged(st):
    B, C, n_kv, d = st["k"].shape
    p, total, lse = _plain_softmax(_plain_scores(st))
    o = (p @ st["v"].float().permute(0, 2, 1, 3)) / total
    out = {"o": o.reshape(B, 1, -1, d).to(torch.bfloat16), "lse": lse.reshape(B, -1, 1)}
    if "weights" in st:
        out["weights"] = st["weights"].add_((p / total).sum(2))
    return out


def _plain_shared(st):
    B, C, n_kv, d = st["k"].shape
    P = st["prefix_k"].shape[1]
    q = st["q"].float().view(B, n_kv, -1, d)
    rows = q.transpose(0, 1).reshape(n_kv, -1, d)
    first = (rows @ st["prefix_k"][0].float().permute(1, 2, 0)).mul_(1.0 / math.sqrt(d))
    first = first.view(n_kv, B, -1, P).transpose(0, 1)
    p, total, lse = _plain_softmax(torch.cat([first, _plain_scores(st)], -1))
    shared = p[..., :P].transpose(0, 1).reshape(n_kv, -1, P) @ st["prefix_v"][0].float().transpose(0, 1)
    o = shared.view(n_kv, B, -1, d).transpose(0, 1) + p[..., P:] @ st["v"].float().permute(0, 2, 1, 3)
    return {"o": (o / total).reshape(B, 1, -1, d).to(torch.bfloat16), "lse": lse.reshape(B, -1, 1)}


def _plain_evict(st):
    c, w = st["case"], st["weights"]
    B, n_kv, C = w.shape
    N, lens = c["budget"], st["lens"].long()[:, None, None]
    at = torch.arange(C, device=DEV)
    rank = torch.where(at >= lens - c["recent"], math.inf, w)
    rank = torch.where(at < lens, rank, -math.inf)
    index = rank.sort(dim=-1, descending=True, stable=True).indices[..., :N]
    kept = torch.arange(N, device=DEV) < lens                                # [B, 1, N]
    index = torch.where(kept, index, C).sort(-1).values
    source = torch.where(kept, index, 0)
    rows = source.transpose(1, 2)[..., None].expand(-1, -1, -1, c["d"])
    live = kept.transpose(1, 2)[..., None]
    held = torch.uint8 if c["fp8"] else torch.bfloat16
    k, v = (torch.where(live, x.view(held).gather(1, rows), torch.zeros((), dtype=held, device=DEV))
            for x in (st["k"], st["v"]))
    st["k_out"].view(held)[:, :N] = k
    st["v_out"].view(held)[:, :N] = v
    kept_w = torch.zeros(B, n_kv, c["capacity"], device=DEV)
    kept_w[..., :N] = torch.where(kept, w.gather(2, source), 0.0)
    return _evicted(c, st["k_out"], st["v_out"], kept_w, st["lens"].clamp(max=N),
                    torch.where(kept, index, -1).to(torch.int32))


def run(state):
    if own:
        return _call(state)
    return {"weights": _plain_weights, "ragged": _plain_ragged, "evict": _plain_evict,
            "shared": _plain_shared}[state["case"]["op"]](state)


# ------------------------------------------------------------------- the costs


def work(case):
    c = case
    if c["op"] == "weights":
        seen = c["Lq"] * c["Lk"]
        if c["causal"]:
            seen -= c["Lq"] * (c["Lq"] - 1) // 2
        rows, keys = c["B"] * c["Lq"] * c["n_q"], c["B"] * c["Lk"] * c["n_kv"]
        return {"bytes": 2 * c["d"] * (rows + keys) + 4 * rows
                + 4 * keys * (2 if c["accumulate"] else 1),
                "flops": 2 * c["d"] * c["B"] * c["n_q"] * seen}
    total = int(_lens(c).sum())
    if c["op"] == "evict":
        kept = int(np.minimum(_lens(c), c["budget"]).sum()) * c["n_kv"]
        held = c["d"] * (1 if c["fp8"] else 2)
        return {"bytes": 4 * held * kept + 4 * total * c["n_kv"]
                + 4 * c["B"] * c["n_kv"] * (c["capacity"] + c["budget"]), "flops": 0}
    rows = c["B"] * c["n_q"]
    size = 512 * total * c["n_kv"] + rows * (2 * 256 + 4)
    if c["op"] == "ragged":
        return {"bytes": size + (8 * total * c["n_kv"] if c["weighted"] else 0),
                "flops": 4 * 128 * c["n_q"] * total}
    return {"bytes": size + 512 * c["P"] * c["n_kv"],
            "flops": 4 * 128 * c["n_q"] * (total + c["B"] * c["P"])}


# --------------------------------------------------- the definitions in 64 bits


def _exact_weights(c, st):
    out = torch.zeros(c["B"], c["n_kv"], c["Lk"], dtype=torch.float64, device=DEV)
    g, off = c["n_q"] // c["n_kv"], c["Lk"] - c["Lq"]
    keys = torch.arange(c["Lk"], device=DEV)
    step = max(1, (1 << 27) // c["Lk"])
    for b in range(c["B"]):
        for h in range(c["n_q"]):
            k = st["k"][b, :, h // g].double()
            for i in range(0, c["Lq"], step):
                q = st["q"][b, i:i + step, h].double()
                e = torch.exp(torch.einsum("id,jd->ij", q, k) * c["d"] ** -0.5
                              - st["lse"][b, h, i:i + step].double()[:, None])
                if c["causal"]:
                    at = torch.arange(i, i + len(q), device=DEV) + off
                    e *= keys[None, :] <= at[:, None]
                out[b, h // g] += e.sum(0)
    return out + st["weights"].double() if c["accumulate"] else out


def _exact_decode(c, st):
    B, g = c["B"], c["n_q"] // c["n_kv"]
    o = torch.zeros(B, 1, c["n_q"], 128, dtype=torch.float64, device=DEV)
    lse = torch.full((B, c["n_q"], 1), -math.inf, dtype=torch.float64, device=DEV)
    w = st["weights"].double().clone() if "weights" in st else None
    lens = st["lens"].tolist()
    for u in range(c["n_kv"]):
        heads = slice(u * g, u * g + g)
        if c["op"] == "shared":
            pk, pv = st["prefix_k"][0, :, u].double(), st["prefix_v"][0, :, u].double()
        for b in range(B):
            k, v = st["k"][b, :lens[b], u].double(), st["v"][b, :lens[b], u].double()
            if c["op"] == "shared":
                k, v = torch.cat([pk, k]), torch.cat([pv, v])
            if not len(k):
                continue
            s = torch.einsum("hd,jd->hj", st["q"][b, 0, heads].double(), k) * 128 ** -0.5
            top = torch.logsumexp(s, 1)
            p = torch.exp(s - top[:, None])
            o[b, 0, heads] = torch.einsum("hj,jd->hd", p, v)
            lse[b, heads, 0] = top
            if w is not None:
                w[b, u, :lens[b]] += p.sum(0)
    return {"o": o, "lse": lse, **({} if w is None else {"weights": w})}


def _exact_evict(c, st):
    w, lens = st["weights"].cpu().numpy(), st["lens"].tolist()
    k, v = (x.float().cpu().numpy() for x in (st["k"], st["v"]))
    k2, v2 = (np.zeros((c["B"], c["capacity"], c["n_kv"], c["d"])) for _ in range(2))
    w2 = np.zeros((c["B"], c["n_kv"], c["capacity"]))
    index = np.full((c["B"], c["n_kv"], c["budget"]), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        old = max(0, n - c["recent"])
        for u in range(c["n_kv"]):
            keep = np.arange(n)
            if n > c["budget"]:
                best = np.lexsort((np.arange(old), -w[b, u, :old]))[:c["budget"] - (n - old)]
                keep = np.sort(np.concatenate([best, np.arange(old, n)]))
            m = len(keep)
            index[b, u, :m] = keep
            w2[b, u, :m] = w[b, u, keep]
            k2[b, :m, u], v2[b, :m, u] = k[b, keep, u], v[b, keep, u]
    return {"k": k2, "v": v2, "weights": w2,
            "lens": np.minimum(np.array(lens), c["budget"]).astype(np.int32), "index": index}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "weights":
        return _exact_weights(case, st)
    return (_exact_evict if case["op"] == "evict" else _exact_decode)(case, st)
