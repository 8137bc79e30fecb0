"""Cases for timing the mixture-of-experts operators: routing, grouped Q4_K
products (single tokens in f32, prompts in fp16) and the weighted combination.

A case names one operator and its sizes. `run` computes it in its plain form
(elementary torch operations in 32 bits) where `own` is false, and calls the
library where it is true. Weights are Q4_K superblocks (144 bytes per 256
weights: d, dmin, twelve bytes of 6-bit scales and mins, 128 bytes of 4-bit
quants).

Vocabulary: pair p = token * top_k + j is the j-th choice of a token; the
routed pairs, sorted by expert (then by p), fill the slots 0, 1, ...:
offsets[e] .. offsets[e + 1] are expert e's slots, order[s] the pair of slot s
(-1 behind the last). A pair without an expert (a padded token, or fewer
experts left than choices) has id -1 and no slot; its output rows stay as they
were.
"""
import math

import torch

own = False

SB = 256          # weights per superblock
SB_BYTES = 144    # bytes per superblock


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a decode step's routing: a small batch, many narrow experts
        dict(name="route_decode", op="route", tokens=24, experts=64, top_k=8, renorm=True, masked=0, pad=0),
        # a prompt batch's routing, some experts switched off, padded tokens at the end
        dict(name="route_prompts", op="route", tokens=8191, experts=128, top_k=8, renorm=False, masked=5, pad=77),
        # one token through two wide experts: gate and up with SwiGLU, then down
        dict(name="gemv_swiglu_1tok", op="gemv_swiglu", tokens=1, experts=8, top_k=2, n=14336, k=4096, pad=0),
        dict(name="gemv_down_1tok", op="gemv", tokens=1, experts=8, top_k=2, n=4096, k=14336, pad=0),
        # a decode batch over many narrow experts (ragged: 0 to ~10 tokens each)
        dict(name="gemv_swiglu_24tok", op="gemv_swiglu", tokens=24, experts=64, top_k=4, n=1536, k=2048, pad=1),
        dict(name="gemv_down_24tok", op="gemv", tokens=24, experts=64, top_k=4, n=2048, k=1536, pad=1),
        # prompts through wide experts
        dict(name="gemm_swiglu_2048tok", op="gemm_swiglu", tokens=2048, experts=8, top_k=2, n=14336, k=4096, pad=0),
        dict(name="gemm_down_2048tok", op="gemm", tokens=2048, experts=8, top_k=2, n=4096, k=14336, pad=0),
        # a short prompt over many narrow experts: ragged groups of some tens of tokens
        dict(name="gemm_swiglu_777tok", op="gemm_swiglu", tokens=777, experts=64, top_k=4, n=1536, k=2048, pad=9),
        dict(name="gemm_down_777tok", op="gemm", tokens=777, experts=64, top_k=4, n=2048, k=1536, pad=9),
        # the end of the layer: a decode batch, and a prompt batch with the residual stream
        dict(name="combine_24tok", op="combine", tokens=24, top_k=4, hidden=4096, pad=1, residual=True),
        dict(name="combine_4096tok", op="combine", tokens=4096, top_k=4, hidden=4096, pad=33, residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "gemv", "gemv_swiglu", "gemm", "gemm_swiglu", "combine"))
    if op == "route":
        experts = _log(rng, 2, 256)
        top_k = rng.randint(1, min(8, experts))
        tokens = _log(rng, 1, 8192)
        return dict(op=op, tokens=tokens, experts=experts, top_k=top_k, renorm=rng.random() < 0.5,
                    masked=rng.randint(0, max(0, experts - top_k)) // 4, pad=rng.randint(0, tokens // 8))
    if op == "combine":
        tokens = _log(rng, 1, 4096)
        return dict(op=op, tokens=tokens, top_k=rng.randint(1, 4), hidden=4 * _log(rng, 64, 1024),
                    pad=rng.randint(0, tokens // 8), residual=rng.random() < 0.5)
    decode = op.startswith("gemv")
    tokens = _log(rng, 1, 32) if decode else _log(rng, 64, 2048)
    if rng.random() < 0.5:      # a few wide experts
        experts, top_k = rng.randint(4, 8), rng.randint(1, 2)
        hidden, inter = SB * rng.randint(8, 16), SB * rng.randint(16, 56)
    else:                       # many narrow ones
        experts, top_k = rng.randint(16, 64), rng.randint(2, 4)
        hidden, inter = SB * rng.randint(4, 10), SB * rng.randint(2, 8)
    n, k = (inter, hidden) if op.endswith("swiglu") else (hidden, inter)
    if rng.random() < 0.4:      # a number of rows that fills no tile
        n -= rng.randint(1, 127)
    return dict(op=op, tokens=tokens, experts=experts, top_k=top_k, n=n, k=k, pad=rng.randint(0, tokens // 8))


def work(case):
    t, op = case["tokens"], case["op"]
    live = t - case["pad"]
    if op == "route":
        e, k = case["experts"], case["top_k"]
        return {"bytes": 4 * (t * e + 3 * t * k + e + 1), "flops": 4 * t * e}
    if op == "combine":
        h, k = case["hidden"], case["top_k"]
        rows = live * k + t + (t if case["residual"] else 0)
        return {"bytes": 4 * rows * h + 8 * t * k, "flops": 2 * live * k * h}
    e, k = case["experts"], case["top_k"]
    mats = 2 if op.endswith("swiglu") else 1
    hit = e * (1.0 - (1.0 - k / e) ** live)     # experts some token goes to, on average
    pairs = live * k
    x_rows = live if mats == 2 else pairs
    x_bytes = 4 if op.startswith("gemv") else 2
    y_bytes = 2 if op == "gemm_swiglu" else 4
    return {"bytes": hit * mats * case["n"] * case["k"] // SB * SB_BYTES + x_rows * case["k"] * x_bytes
            + pairs * case["n"] * y_bytes + 4 * (t * k + e + 1),
            "flops": 2 * mats * pairs * case["n"] * case["k"]}


# ------------------------------------------------------------------ inputs

def _weights(gen, experts, n, k):
    """Q4_K superblocks as quantised weights have them: values around zero
    (the mins sit near the middle of the quants' range), of a few hundredths."""
    count = experts * n * (k // SB)
    raw = torch.randint(0, 256, (count, SB_BYTES), dtype=torch.uint8, device="cuda", generator=gen)
    d = torch.empty(count, device="cuda").uniform_(0.8e-4, 2.0e-4, generator=gen)
    dmin = d * torch.empty(count, device="cuda").uniform_(7.5, 8.5, generator=gen)
    raw[:, 0:2] = d.half().view(torch.uint8).view(count, 2)
    raw[:, 2:4] = dmin.half().view(torch.uint8).view(count, 2)
    sc = torch.randint(24, 64, (count, 8), dtype=torch.uint8, device="cuda", generator=gen)
    mn = (sc.float() * torch.empty(count, 8, device="cuda").uniform_(0.85, 1.0, generator=gen)).to(torch.uint8)
    raw[:, 4:8] = sc[:, :4] | ((sc[:, 4:] >> 4) << 6)
    raw[:, 8:12] = mn[:, :4] | ((mn[:, 4:] >> 4) << 6)
    raw[:, 12:16] = (sc[:, 4:] & 15) | ((mn[:, 4:] & 15) << 4)
    return raw.view(experts, n, k // SB, SB_BYTES)


def _group(ids, experts):
    """offsets [experts + 1] and order [pairs] of ids [tokens, top_k] (-1: no expert)."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, experts), flat)
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=experts + 1)[:experts]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    slot = torch.arange(flat.numel(), device=flat.device)
    order = torch.where(slot < offsets[-1], order, torch.full_like(order, -1))
    return offsets.int(), order.int()


def _routing(gen, case):
    """ids, offsets, order of a router that prefers some experts; padded tokens go nowhere."""
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    pull = 0.7 * torch.randn(e, device="cuda", generator=gen)
    logits = torch.randn(t, e, device="cuda", generator=gen) + pull
    ids = torch.topk(logits, k, dim=1).indices.int()
    if case["pad"]:
        ids[t - case["pad"]:] = -1
    return ids, *_group(ids, e)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, t = case["op"], case["tokens"]
    s = dict(case)
    if op == "route":
        e, k = case["experts"], case["top_k"]
        # a router's logits come out of a 16-bit product: equal ones are common
        logits = torch.randn(t, e, device="cuda", generator=gen) + 0.7 * torch.randn(e, device="cuda", generator=gen)
        logits = logits.bfloat16().float()
        if case["masked"]:
            logits[:, torch.randperm(e, device="cuda", generator=gen)[:case["masked"]]] = -math.inf
        if case["pad"]:
            logits[t - case["pad"]:] = -math.inf
        s["logits"] = logits
        s["ids"] = torch.empty(t, k, dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty(t, k, device="cuda")
        s["offsets"] = torch.empty(e + 1, dtype=torch.int32, device="cuda")
        s["order"] = torch.empty(t * k, dtype=torch.int32, device="cuda")
        return s
    if op == "combine":
        k, h = case["top_k"], case["hidden"]
        s["z"] = torch.randn(t * k, h, device="cuda", generator=gen)
        s["ids"] = torch.randint(0, 8, (t, k), dtype=torch.int32, device="cuda", generator=gen)
        if case["pad"]:
            s["ids"][t - case["pad"]:] = -1
        s["weights"] = torch.softmax(torch.randn(t, k, device="cuda", generator=gen), 1)
        s["res"] = torch.randn(t, h, device="cuda", generator=gen) if case["residual"] else None
        s["y"] = torch.empty(t, h, device="cuda")
        return s
    e, k_top, n, k = case["experts"], case["top_k"], case["n"], case["k"]
    ids, s["offsets"], s["order"] = _routing(gen, case)
    counts = (s["offsets"][1:] - s["offsets"][:-1])
    s["pairs"], s["cmax"] = t * k_top, max(1, int(counts.max()))
    half = op.startswith("gemm")
    s["w"] = _weights(gen, e, n, k)
    if op.endswith("swiglu"):       # the tokens' normalised activations, gathered by the operator
        s["w_up"] = _weights(gen, e, n, k)
        s["per_row"] = k_top
        x = torch.randn(t, k, device="cuda", generator=gen)
    else:                           # what gate and up gave, row = slot
        s["per_row"] = 0
        x = torch.randn(t * k_top, k, device="cuda", generator=gen) * torch.randn(t * k_top, k, device="cuda", generator=gen)
    s["x"] = x.half() if half else x
    s["y"] = torch.zeros(t * k_top, n, device="cuda", dtype=torch.float16 if op == "gemm_swiglu" else torch.float32)
    return s


# ------------------------------------------------------------------ plain forms

def _dequant(raw):
    """Q4_K superblocks [..., nsb, 144] as f32 [..., nsb * 256]: d*sc*q - dmin*m,
    the products exact, one rounding."""
    d = raw[..., 0:2].contiguous().view(torch.float16).float()
    dmin = raw[..., 2:4].contiguous().view(torch.float16).float()
    s = raw[..., 4:16]
    sc = torch.cat([s[..., 0:4] & 63, (s[..., 8:12] & 15) | ((s[..., 0:4] >> 6) << 4)], -1).float()
    mn = torch.cat([s[..., 4:8] & 63, (s[..., 8:12] >> 4) | ((s[..., 4:8] >> 6) << 4)], -1).float()
    qs = raw[..., 16:].unflatten(-1, (4, 1, 32))
    q = torch.cat([qs & 15, qs >> 4], -2).flatten(-3, -2)         # [..., 8, 32]
    w = (d * sc).unsqueeze(-1) * q - (dmin * mn).unsqueeze(-1)
    return w.flatten(-3)


def _rows(s):
    """Per slot: its expert, its place within the expert, its pair, its row of x."""
    off, order = s["offsets"].long(), s["order"].long()
    slot = torch.arange(s["pairs"], device="cuda")
    expert = torch.searchsorted(off, slot, right=True) - 1
    live = slot < off[-1]
    expert = torch.where(live, expert, torch.zeros_like(expert))
    pair = order.clamp(min=0)
    row = slot if s["per_row"] == 0 else pair // s["per_row"]
    return slot, expert, slot - off[expert], pair, row, live


def _products(s, mats, mirror):
    """One [pairs, n] f32 product per matrix, rows in slot order (rows of slots
    without a pair hold anything). mirror: weights rounded to fp16 first."""
    slot, expert, place, pair, row, live = _rows(s)
    x = s["x"].float()
    out = []
    if s["pairs"] <= s["experts"]:      # few pairs: each with its own expert's matrix
        for m in mats:
            w = _dequant(m[expert])
            w = w.half().float() if mirror else w
            out.append(torch.bmm(w, x[row].unsqueeze(-1)).squeeze(-1))
        return out, pair, live
    place = torch.where(live, place, torch.zeros_like(place))
    off = s["offsets"].long()
    at = (off[:-1, None] + torch.arange(s["cmax"], device="cuda")).clamp(max=s["pairs"] - 1)
    xp = x[row[at]]                      # [experts, cmax, k]; places past an expert's count are not read back
    for m in mats:
        w = _dequant(m)
        w = w.half().float() if mirror else w
        out.append(torch.bmm(xp, w.transpose(1, 2))[expert, place])
    return out, pair, live


def _plain(s):
    op = s["op"]
    if op == "route":
        lg, e, k = s["logits"], s["experts"], s["top_k"]
        val, idx = torch.sort(lg, dim=1, descending=True, stable=True)
        val, idx = val[:, :k], idx[:, :k].int()
        ok = val > -math.inf
        top = torch.where(val[:, :1] > -math.inf, val[:, :1], torch.zeros_like(val[:, :1]))
        w = torch.where(ok, torch.exp(val - top), torch.zeros_like(val))
        total = w.sum(1, keepdim=True) if s["renorm"] else torch.exp(lg - top).sum(1, keepdim=True)
        w = torch.where(ok, w / total, torch.zeros_like(w))
        ids = torch.where(ok, idx, torch.full_like(idx, -1))
        return (ids, w) + _group(ids, e)
    if op == "combine":
        t, k, h = s["tokens"], s["top_k"], s["hidden"]
        ok = (s["ids"] >= 0).unsqueeze(-1)
        z = torch.where(ok, s["z"].view(t, k, h), torch.zeros((), device="cuda"))
        y = (z * s["weights"].unsqueeze(-1)).sum(1)
        return y + s["res"] if s["res"] is not None else y
    mirror = op.startswith("gemm")
    if op.endswith("swiglu"):
        (g, u), pair, live = _products(s, (s["w"], s["w_up"]), mirror)
        h = g / (1.0 + torch.exp(-g)) * u
        return torch.where(live.unsqueeze(-1), h, torch.zeros((), device="cuda")).to(s["y"].dtype)
    (y,), pair, live = _products(s, (s["w"],), mirror)
    full = torch.zeros(s["pairs"] + 1, s["n"], device="cuda")
    full[torch.where(live, pair, torch.full_like(pair, s["pairs"]))] = y
    return full[:-1]


def run(s):
    if not own:
        return _plain(s)
    import gguf_quant_dequant_q4k_b200 as q4k
    op = s["op"]
    if op == "route":
        q4k.q4k_moe_route(s["logits"], s["ids"], s["weights"], s["offsets"], s["order"], s["tokens"],
                          s["experts"], s["top_k"], renorm=s["renorm"])
        return s["ids"], s["weights"], s["offsets"], s["order"]
    if op == "combine":
        q4k.q4k_moe_combine(s["z"], s["ids"], s["weights"], s["res"], s["y"], s["tokens"], s["top_k"], s["hidden"])
        return s["y"]
    sizes = (s["experts"], s["pairs"], s["per_row"], s["n"], s["k"])
    if op == "gemv":
        q4k.q4k_moe_gemv(s["w"], s["x"], s["offsets"], s["order"], s["y"], *sizes)
    elif op == "gemv_swiglu":
        q4k.q4k_moe_gemv_swiglu(s["w"], s["w_up"], s["x"], s["offsets"], s["order"], s["y"], *sizes)
    elif op == "gemm":
        q4k.q4k_moe_gemm_f16(s["w"], s["x"], s["offsets"], s["order"], s["y"], *sizes)
    else:
        q4k.q4k_moe_gemm_swiglu_f16(s["w"], s["w_up"], s["x"], s["offsets"], s["order"], s["y"], *sizes)
    return s["y"]


# ------------------------------------------------------------------ in 64 bits

def _matrix64(raw, mirror):
    """One expert's matrix [n, k] in 64 bits, field by field; mirror: the
    binary16 nearest to the f32 value, as the fp16 products use it."""
    n, nsb = raw.shape[0], raw.shape[1]
    b = raw.to(torch.int64)
    d = raw[..., :4].contiguous().view(torch.float16).to(torch.float64)
    w = torch.empty(n, nsb, 8, 32, dtype=torch.float64, device=raw.device)
    for j in range(8):
        if j < 4:
            sc, mn = b[..., 4 + j] % 64, b[..., 8 + j] % 64
        else:
            sc = b[..., 8 + j] % 16 + 16 * (b[..., j] // 64)
            mn = b[..., 8 + j] // 16 + 16 * (b[..., 4 + j] // 64)
        byte = b[..., 16 + 32 * (j // 2): 48 + 32 * (j // 2)]
        q = byte // 16 if j % 2 else byte % 16
        w[..., j, :] = (d[..., 0] * sc).unsqueeze(-1) * q - (d[..., 1] * mn).unsqueeze(-1)
    w = w.view(n, nsb * SB)
    # the weight is the f32 value; both are part of the operator's definition
    return w.float().half().double() if mirror else w.float().double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        lg = s["logits"].cpu().double()
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        ids = torch.argsort(-lg, dim=1, stable=True)[:, :k]
        picked = lg.gather(1, ids)
        base = lg if not case["renorm"] else picked
        w = torch.exp(picked - torch.logsumexp(base, 1, keepdim=True))
        return None, torch.where(picked > -math.inf, w, torch.zeros_like(w)), None, None
    if op == "combine":
        t, k = case["tokens"], case["top_k"]
        y = s["res"].double() if s["res"] is not None else torch.zeros(t, case["hidden"], dtype=torch.float64, device="cuda")
        for j in range(k):
            w = (s["weights"][:, j].double() * (s["ids"][:, j] >= 0)).unsqueeze(1)
            y = y + w * s["z"][j::k].double()
        return y
    mirror = op.startswith("gemm")
    off, order = s["offsets"].tolist(), s["order"].long()
    out = torch.zeros(s["pairs"], case["n"], dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        rows = torch.arange(a, b, device="cuda") if s["per_row"] == 0 else order[a:b] // s["per_row"]
        x = s["x"][rows].double()
        y = x @ _matrix64(s["w"][e], mirror).T
        if op.endswith("swiglu"):
            out[a:b] = y * torch.sigmoid(y) * (x @ _matrix64(s["w_up"][e], mirror).T)
        else:
            out[order[a:b]] = y
    return out
