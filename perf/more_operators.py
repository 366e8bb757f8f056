"""The expert layer of a mixture-of-experts model on packed weights, as measured cases.

Four operators, in the order in which a layer calls them:

* norm     the residual stream plus what the layer before adds to it, its RMS norm in fp32 or
           bf16 (for the router's product) and in 8 bits: e4m3 codes with one power of two for
           32 columns (for the experts);
* sort     the k largest router logits of each token, their weights, and the tokens' rows in
           the order of their experts, from bf16 or 8-bit rows;
* experts  the packed Q4_K products of each expert with its rows: one matrix per expert (down),
           or silu(gate) * up of two;
* combine  back to the order of the tokens, with the weights applied.

``run`` computes a case in its plain form (elementary torch operations in 32 bits), or with
``own`` through gguf_q4_dequant_gb300. ``exact`` is the same from the definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
WEIGHTINGS = ("softmax", "softmax_top", "sigmoid", "sigmoid_top")


# --------------------------------------------------------------------- cases ---

def listed():
    return [
        # one chat, one token: the norm before a layer's products (Qwen3-8B hidden size)
        dict(name="norm_one", op="norm", tokens=1, cols=4096, bf16=False, delta=True, out="bf16", eight=False),
        # a prompt chunk through a bf16 residual stream, 8-bit rows for the experts (Qwen3-14B hidden size)
        dict(name="norm_prompt_8bit", op="norm", tokens=4096, cols=5120, bf16=True, delta=True, out="f32", eight=True),
        # a decode batch: 48 tokens to 8 of 128 experts
        dict(name="sort_batch", op="sort", tokens=48, experts=128, top=8, cols=2048, weighting="softmax_top",
             masked=False, ties=False, eight=False, shape=1),
        # a prompt chunk, 8-bit rows
        dict(name="sort_prompt", op="sort", tokens=8192, experts=128, top=8, cols=2048, weighting="softmax_top",
             masked=False, ties=False, eight=True, shape=2),
        # an odd count of tokens and experts, some experts switched off, logits that tie
        dict(name="sort_masked", op="sort", tokens=1003, experts=61, top=4, cols=4096, weighting="sigmoid_top",
             masked=True, ties=True, eight=False, shape=3),
        # one chat, one token: 8 experts of 128, one row each
        dict(name="gated_one", op="experts", gated=True, tokens=1, experts=128, top=8, n=768, k=2048, skew=0.0, shape=4),
        # a decode batch: nearly every expert has a few rows
        dict(name="gated_batch", op="experts", gated=True, tokens=64, experts=128, top=8, n=768, k=2048, skew=0.5, shape=5),
        # a prompt chunk: some hundred rows an expert
        dict(name="gated_prompt", op="experts", gated=True, tokens=4096, experts=128, top=8, n=768, k=2048, skew=0.5, shape=6),
        # the way down for a few chats, few large experts (Qwen3-8B feed-forward sizes)
        dict(name="down_few", op="experts", gated=False, tokens=5, experts=8, top=2, n=4096, k=12288, skew=0.0, shape=7),
        # the way down for a prompt chunk
        dict(name="down_prompt", op="experts", gated=False, tokens=2048, experts=16, top=4, n=4096, k=2048, skew=0.3, shape=8),
        # a small batch back to its tokens
        dict(name="combine_batch", op="combine", tokens=48, top=8, cols=2048, base=False, missing=False, shape=9),
        # a prompt chunk back to its tokens, onto the output of a shared expert
        dict(name="combine_prompt", op="combine", tokens=8192, top=8, cols=2048, base=True, missing=True, shape=10),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    """Seconds that the work of a case takes at about this card's rates."""
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def draw(rng):
    op = rng.choice(["norm", "sort", "experts", "experts", "experts", "combine"])
    most = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        case = _drawn(rng, op)
        if _cost(case) <= most and _plain_bytes(case) <= 16e9:
            return case


def _drawn(rng, op):
    shape = rng.randrange(1, 1 << 30)
    cols = 32 * _log(rng, 2, 256)
    if op == "norm":
        out = rng.choice(["f32", "bf16", "none"])
        return dict(op=op, tokens=_log(rng, 1, 16384), cols=cols, bf16=rng.random() < 0.5, delta=rng.random() < 0.7,
                    out=out, eight=out == "none" or rng.random() < 0.5)
    experts = _log(rng, 2, 512)
    top = min(experts, rng.choice([1, 2, 3, 4, 6, 8, 10]))
    if op == "sort":
        return dict(op=op, tokens=_log(rng, 1, 20000), experts=experts, top=top, cols=cols,
                    weighting=rng.choice(WEIGHTINGS), masked=rng.random() < 0.4, ties=rng.random() < 0.4,
                    eight=rng.random() < 0.5, shape=shape)
    if op == "combine":
        return dict(op=op, tokens=_log(rng, 1, 20000), top=top, cols=cols, base=rng.random() < 0.5,
                    missing=rng.random() < 0.4, shape=shape)
    return dict(op=op, gated=rng.random() < 0.5, tokens=_log(rng, 1, 6000), experts=experts, top=top,
                n=8 * _log(rng, 8, 1024), k=256 * _log(rng, 1, 48), skew=rng.choice([0.0, 0.5, 1.5]), shape=shape)


# ------------------------------------------------- sizes that a case implies ---

def _rows(case):
    """Rows of each expert: `top` different experts for each token, some more popular than others."""
    r = np.random.RandomState(case["shape"] % (1 << 31))
    score = case["skew"] * r.standard_normal(case["experts"]) + r.gumbel(size=(case["tokens"], case["experts"]))
    ids = np.argpartition(-score, case["top"] - 1, axis=1)[:, :case["top"]]
    return np.bincount(ids.reshape(-1), minlength=case["experts"])


def _plain_bytes(case):
    """The largest intermediates of the plain form, for drawn cases."""
    if case["op"] != "experts":
        return 0.0
    rows = _rows(case)
    mats = 2 if case["gated"] else 1
    return 4.0 * int((rows > 0).sum()) * (2 * mats * case["n"] * case["k"] + int(rows.max()) * (case["k"] + mats * case["n"]))


def work(case):
    op = case["op"]
    if op == "norm":
        T, C = case["tokens"], case["cols"]
        x = 2 if case["bf16"] else 4
        per = 2 * x + (4 if case["delta"] else 0) + {"f32": 4, "bf16": 2, "none": 0}[case["out"]] + (33 / 32 if case["eight"] else 0)
        return {"bytes": int(T * C * per) + 4 * C, "flops": 5 * T * C}
    if op == "sort":
        T, E, k, C = case["tokens"], case["experts"], case["top"], case["cols"]
        row = C * 33 // 32 if case["eight"] else 2 * C
        return {"bytes": 4 * T * E + 16 * T * k + 4 * E + T * row + 2 * T * k * C, "flops": 4 * T * E}
    if op == "combine":
        T, k, C = case["tokens"], case["top"], case["cols"]
        return {"bytes": T * C * (2 * k + 4 + (4 if case["base"] else 0)) + 8 * T * k, "flops": 2 * T * k * C}
    rows = _rows(case)
    P, live, mats = int(rows.sum()), int((rows > 0).sum()), 2 if case["gated"] else 1
    N, K = case["n"], case["k"]
    return {"bytes": mats * live * N * (K // 256) * 144 + 2 * P * (K + N) + 4 * case["experts"],
            "flops": 2 * mats * P * N * K}


# -------------------------------------------------------------------- inputs ---

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def _packed(g, experts, n, k):
    """Q4_K rows [experts, n, k / 256 * 144] of weights with a mean near zero and a deviation of about
    1 / sqrt(k): 6-bit scales and mins drawn alike, dmin = 7.5 d."""
    b = torch.randint(0, 256, (experts, n, k // 256, 144), generator=g, device=DEV, dtype=torch.uint8)
    b[..., 8:12] = b[..., 4:8]                      # the mins of sub-blocks 0-3 as their scales,
    low = b[..., 12:16] & 15
    b[..., 12:16] = low | (low << 4)                # and of 4-7
    # a weight is d * sc * (q - 7.5): sc has a root mean square of 36.4, q - 7.5 of 4.6
    d = (0.5 + torch.rand(experts, n, k // 256, 1, generator=g, device=DEV)) / (36.4 * 4.6 * math.sqrt(k))
    head = torch.cat([d, 7.5 * d], -1).to(torch.float16).contiguous()
    b[..., 0:4] = head.view(torch.uint8)
    return b.view(experts, n, k // 256 * 144)


def _eight(y):
    """e4m3 codes and the exponents of their scales, for each 32 columns (plain form)."""
    v = y.view(y.shape[0], -1, 32)
    m, e = torch.frexp(v.abs().amax(-1, keepdim=True))      # amax = m * 2^e, 1/2 <= m < 1
    e = (e - 9 + (m > 0.875).to(torch.int32)).clamp(-127, 127)  # amax <= 448 * 2^e
    return torch.ldexp(v, -e).to(torch.float8_e4m3fn).view(y.shape), e.squeeze(-1)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "norm":
        T, C = case["tokens"], case["cols"]
        dt = torch.bfloat16 if case["bf16"] else torch.float32
        # a residual stream: some columns much larger than the rest
        x = _normal(g, T, C) * torch.exp(1.0 * _normal(g, C)) * 2.0
        s["x"] = x.to(dt)
        s["delta"] = _normal(g, T, C, scale=0.5) if case["delta"] else None
        s["weight"] = 1.0 + _normal(g, C, scale=0.2)
        s["sum"] = torch.empty_like(s["x"])
        s["out"] = None if case["out"] == "none" else torch.empty(T, C, device=DEV, dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16)
        s["codes"] = torch.empty(T, C, device=DEV, dtype=torch.float8_e4m3fn) if case["eight"] else None
        s["scales"] = torch.empty(T, C // 32, device=DEV, dtype=torch.uint8) if case["eight"] else None
        return s
    if op == "sort":
        T, E, k, C = case["tokens"], case["experts"], case["top"], case["cols"]
        logits = _normal(g, T, E, scale=2.0) + _normal(g, E)
        if case["ties"]:
            logits = torch.round(logits * 4) / 4
        if case["masked"]:
            r = random.Random(case["shape"])
            off = torch.tensor([r.random() < 0.3 for _ in range(E)], device=DEV)
            off[r.randrange(E)] = False
            logits = logits.masked_fill(off, float("-inf"))
            if T > 2:
                logits[1] = float("-inf")          # a token that goes nowhere
                logits[2, 1:] = float("-inf")      # and one with one expert at most
        s["logits"] = logits
        x = _normal(g, T, C, dtype=torch.bfloat16)
        s["x"], s["x_scales"] = x, None
        if case["eight"]:
            s["x"], e = _eight(x.float())
            s["x_scales"] = (e + 127).to(torch.uint8)
        i32 = dict(dtype=torch.int32, device=DEV)
        s["ids"], s["order"], s["slots"] = torch.empty(T, k, **i32), torch.empty(T * k, **i32), torch.empty(T, k, **i32)
        s["starts"] = torch.empty(E + 1, **i32)
        s["weights"] = torch.empty(T, k, device=DEV)
        s["rows"] = torch.zeros(T * k, C, dtype=torch.bfloat16, device=DEV)
        s["ws"] = torch.empty(4 * E * (-(-T // 64) + 1), dtype=torch.uint8, device=DEV)
        return s
    if op == "combine":
        T, k, C = case["tokens"], case["top"], case["cols"]
        s["y"] = _normal(g, T * k, C, dtype=torch.bfloat16)
        w = torch.rand(T, k, generator=g, device=DEV) + 0.05
        s["weights"] = w / w.sum(1, keepdim=True)
        s["slots"] = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32).view(T, k)
        if case["missing"]:
            s["slots"][torch.rand(T, k, generator=g, device=DEV) < 0.05] = -1
        s["base"] = _normal(g, T, C) if case["base"] else None
        s["out"] = torch.empty(T, C, device=DEV)
        return s
    E, N, K = case["experts"], case["n"], case["k"]
    rows = _rows(case)
    s["w"] = _packed(g, E, N, K)
    s["w2"] = _packed(g, E, N, K) if case["gated"] else None
    s["x"] = _normal(g, int(rows.sum()), K, dtype=torch.bfloat16)
    s["starts"] = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device=DEV)
    s["y"] = torch.empty(int(rows.sum()), N, dtype=torch.bfloat16, device=DEV)
    # the plan of the step, as index tensors: the experts with rows, and each row's place among its expert's
    live = np.nonzero(rows)[0]
    s["live"] = torch.tensor(live, device=DEV)
    s["row_expert"] = torch.tensor(np.repeat(np.arange(len(live)), rows[live]), device=DEV)
    s["row_at"] = torch.tensor(np.concatenate([np.arange(n) for n in rows[live]]), device=DEV)
    s["most"] = int(rows.max())
    return s


# ---------------------------------------------------------------- plain form ---

def _dequant(w):
    """fp32 weights [..., n, k] of packed rows: w = d * sc * q - dmin * m."""
    b = w.view(*w.shape[:-1], -1, 144)
    head = b[..., 0:4].contiguous().view(torch.float16).float()
    s = b[..., 4:16].to(torch.int32)
    lo, mid, hi = s[..., 0:4], s[..., 4:8], s[..., 8:12]
    sc = torch.cat([lo & 63, (hi & 15) | ((lo >> 6) << 4)], -1).float()
    mn = torch.cat([mid & 63, (hi >> 4) | ((mid >> 6) << 4)], -1).float()
    q = b[..., 16:].reshape(*b.shape[:-1], 4, 1, 32)
    q = torch.cat([q & 15, q >> 4], -2).reshape(*b.shape[:-1], 8, 32).float()
    v = (head[..., 0:1] * sc).unsqueeze(-1) * q - (head[..., 1:2] * mn).unsqueeze(-1)
    return v.reshape(*w.shape[:-1], -1)


def _plain_norm(s):
    r = s["x"].float()
    if s["delta"] is not None:
        r = r + s["delta"]
    y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    got = {"sum": r.to(s["x"].dtype)}
    if s["out"] is not None:
        got["out"] = y.to(s["out"].dtype)
    if s["codes"] is not None:
        codes, e = _eight(y)
        got["codes"], got["scales"] = codes, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return got


def _plain_sort(s):
    k, weighting = s["case"]["top"], s["case"]["weighting"]
    logits = s["logits"]
    T, E = logits.shape
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    live = top > float("-inf")
    if weighting.startswith("softmax"):
        rel = torch.where(live, torch.exp(top - top[:, :1]), 0.0)
        total = torch.exp(logits - top[:, :1]).sum(1, keepdim=True) if weighting == "softmax" else rel.sum(1, keepdim=True)
    else:
        rel = torch.where(live, 1 / (1 + torch.exp(-top)), 0.0)
        total = rel.sum(1, keepdim=True) if weighting == "sigmoid_top" else torch.ones_like(rel[:, :1])
    weights = torch.where(live, rel / total, 0.0)
    ids = torch.where(live, ids, -1)
    key = torch.where(live, ids, E).view(-1)
    counts = (key[:, None] == torch.arange(E, device=DEV)).sum(0) if T * k * E < 1 << 26 else torch.bincount(key, minlength=E + 1)[:E]
    starts = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), counts.cumsum(0)])
    place = torch.sort(key, stable=True)[1]
    used = torch.arange(T * k, device=DEV) < starts[E]
    order = torch.where(used, place, -1)
    slots = torch.empty_like(place)
    slots[place] = torch.arange(T * k, device=DEV)
    slots = torch.where(live.view(-1), slots, -1)
    x = s["x"]
    if s["x_scales"] is not None:
        x = torch.ldexp(x.float().view(T, -1, 32), s["x_scales"].to(torch.int32).unsqueeze(-1) - 127).view(T, -1)
    rows = torch.where(used[:, None], x[place // k].to(torch.bfloat16), s["rows"])
    i32 = torch.int32
    return {"ids": ids.to(i32), "weights": weights, "order": order.to(i32), "slots": slots.view(T, k).to(i32),
            "starts": starts.to(i32), "rows": rows}


def _plain_experts(s):
    x = s["x"].float()
    padded = torch.zeros(s["live"].numel(), s["most"], x.shape[1], device=DEV)
    padded[s["row_expert"], s["row_at"]] = x
    y = torch.bmm(padded, _dequant(s["w"][s["live"]]).transpose(1, 2))
    if s["w2"] is not None:
        y = y / (1 + torch.exp(-y)) * torch.bmm(padded, _dequant(s["w2"][s["live"]]).transpose(1, 2))
    return y[s["row_expert"], s["row_at"]].to(torch.bfloat16)


def _plain_combine(s):
    slots = s["slots"].long()
    live = (slots >= 0).unsqueeze(-1)
    y = torch.where(live, s["y"][slots.clamp(min=0)].float(), 0.0)
    out = (y * s["weights"].unsqueeze(-1)).sum(1)
    return out if s["base"] is None else s["base"] + out


# ----------------------------------------------------------------------- run ---

def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return {"norm": _plain_norm, "sort": _plain_sort, "experts": _plain_experts, "combine": _plain_combine}[op](s)
    import gguf_q4_dequant_gb300 as q4k
    if op == "norm":
        q4k.q4k_add_norm(s["x"], s["delta"], s["weight"], EPS, sum=s["sum"], out=s["out"], codes=s["codes"], scales=s["scales"])
        got = {"sum": s["sum"]}
        if s["out"] is not None:
            got["out"] = s["out"]
        if s["codes"] is not None:
            got["codes"], got["scales"] = s["codes"], s["scales"].view(torch.float8_e8m0fnu)
        return got
    if op == "sort":
        q4k.q4k_route(s["logits"], case["top"], WEIGHTINGS.index(case["weighting"]), 1.0, s["ids"], s["weights"], s["order"],
                      s["slots"], s["starts"], s["ws"])
        q4k.q4k_experts_gather(s["x"], s["order"], case["top"], s["rows"], scales=s["x_scales"])
        return {n: s[n] for n in ("ids", "weights", "order", "slots", "starts", "rows")}
    if op == "combine":
        q4k.q4k_experts_combine(s["y"], s["slots"], s["weights"], s["out"], base=s["base"])
        return s["out"]
    if s["w2"] is not None:
        q4k.q4k_experts_gated(s["w"], s["w2"], case["n"], case["k"], s["x"], s["starts"], s["y"])
    else:
        q4k.q4k_experts_matmul(s["w"], case["n"], case["k"], s["x"], s["starts"], s["y"])
    return s["y"]


# --------------------------------------------------------------------- exact ---

def _nearest_e4m3(v):
    """The e4m3 value nearest to each of v (ties to the even code), |v| <= 448, in 64 bits."""
    a = v.abs()
    step = torch.exp2((torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))) - 3)
    return torch.sign(v) * torch.round(a / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "norm":
        r = s["x"].to(f64) + (0 if s["delta"] is None else s["delta"].to(f64))
        y = r / torch.sqrt((r * r).sum(1, keepdim=True) / r.shape[1] + EPS) * s["weight"].to(f64)
        got = {"sum": r}
        if s["out"] is not None:
            got["out"] = y
        if s["codes"] is not None:
            b = y.reshape(y.shape[0], -1, 32)
            scale = torch.exp2(torch.ceil(torch.log2(b.abs().amax(2) / 448)))
            got["codes"], got["scales"] = _nearest_e4m3(b / scale.unsqueeze(2)).reshape(y.shape), scale
        return got
    if op == "sort":
        # the weights from each token's own logits; the rows by counting who comes before whom
        T, E, k = case["tokens"], case["experts"], case["top"]
        z = s["logits"].to(f64)
        at = torch.arange(E, device=DEV)
        weights = torch.zeros(T, k, dtype=f64, device=DEV)
        chosen = torch.full((T, k), -1, device=DEV)
        left = z.clone()
        for j in range(k):
            best = left.amax(1, keepdim=True)
            i = torch.where(left == best, at, E).amin(1, keepdim=True)
            ok = best > float("-inf")
            chosen[:, j:j + 1] = torch.where(ok, i, -1)
            left.scatter_(1, i, float("-inf"))
        picked = torch.gather(z, 1, chosen.clamp(min=0)).masked_fill(chosen < 0, float("-inf"))
        if case["weighting"] == "softmax":
            weights = torch.exp(picked - torch.logsumexp(z, 1, keepdim=True))
        elif case["weighting"] == "softmax_top":
            weights = torch.exp(picked - torch.logsumexp(picked, 1, keepdim=True))
        else:
            weights = torch.sigmoid(picked)
            if case["weighting"] == "sigmoid_top":
                weights = weights / weights.sum(1, keepdim=True)
        weights = weights.masked_fill(chosen < 0, 0.0)
        x = s["x"].to(f64)
        if s["x_scales"] is not None:
            x = x * torch.exp2(s["x_scales"].to(f64) - 127).repeat_interleave(32, 1)
        lists = [torch.nonzero(chosen == e)[:, 0] for e in range(E)]
        tokens = torch.cat(lists)
        rows = torch.zeros(T * k, case["cols"], dtype=f64, device=DEV)
        rows[:tokens.numel()] = x[tokens]
        return {"ids": None, "weights": weights, "order": None, "slots": None, "starts": None, "rows": rows}
    if op == "combine":
        out = torch.zeros(case["tokens"], case["cols"], dtype=f64, device=DEV) if s["base"] is None else s["base"].to(f64)
        for j in range(case["top"]):
            at = s["slots"][:, j].long()
            out = out + torch.where((at >= 0).unsqueeze(1), s["weights"][:, j:j + 1].to(f64) * s["y"][at.clamp(min=0)].to(f64), 0.0)
        return out
    if work(case)["flops"] > 2e12:
        return None
    y = torch.empty(s["y"].shape, dtype=f64, device=DEV)
    starts = s["starts"].tolist()
    for e in range(case["experts"]):
        a, b = starts[e], starts[e + 1]
        if a < b:
            x = s["x"][a:b].to(f64)
            first = x @ _weights64(s["w"][e]).T
            if case["gated"]:
                first = first * torch.sigmoid(first) * (x @ _weights64(s["w2"][e]).T)
            y[a:b] = first
    return y


def _weights64(rows):
    """Weights of packed rows in 64 bits, weight by weight from the format."""
    n = rows.shape[0]
    b = rows.reshape(n, -1, 144)
    i = torch.arange(256, device=rows.device)
    j = i // 32
    byte = b[:, :, 16 + 32 * (i // 64) + i % 32]
    q = torch.where(i % 64 < 32, byte % 16, byte // 16).to(torch.float64)
    s = b[:, :, 4:16].long()
    early = j < 4
    sc = torch.where(early, s[:, :, torch.where(early, j, 0)] % 64,
                     s[:, :, torch.where(early, 0, j + 4)] % 16 + 16 * (s[:, :, torch.where(early, 0, j - 4)] // 64))
    mn = torch.where(early, s[:, :, torch.where(early, j + 4, 0)] % 64,
                     s[:, :, torch.where(early, 0, j + 4)] // 16 + 16 * (s[:, :, torch.where(early, 0, j)] // 64))
    d = b[:, :, 0:4].contiguous().view(torch.float16).to(torch.float64)
    return (d[:, :, 0:1] * sc * q - d[:, :, 1:2] * mn).reshape(n, -1)
