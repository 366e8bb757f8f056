"""The decode-step operators around the packed matmuls, as measured cases.

Four operators, with what each takes from the others in a step of a served
model:

* append     the fp32 q, k and v rows of a step (the outputs of the packed
             matmuls): optional RMS norm per head, rotary positions, bf16 k and
             v into the pages of the cache, bf16 q out;
* attention  the new tokens of each sequence (one, or a chunk of a prompt)
             over its pages: causal, grouped heads, optional sliding window
             with first tokens that stay visible;
* pages      forking, freeing and compacting the sequences' pages (with the
             copies of the pages in every layer);
* pick       penalties for repeated tokens, biases and a grammar mask on the
             logits, then the greedy pick.

``run`` computes a case in its plain form (elementary torch operations in 32
bits), or with ``own`` through gguf_q4_dequant_gb300. ``exact`` is the same
from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------- cases ---

def listed():
    return [
        # one chat, one token: nothing to hide latency behind (head counts of the Qwen3-8B shape)
        dict(name="attn_one_token", op="attention", heads=32, kv_heads=8, dim=128, page=16, seqs=1,
             new=1, singles=1.0, len_lo=517, len_hi=517, window=0, sinks=0, shape=1),
        # a full serving batch, every sequence at its own length (Qwen3-14B shape: 5 query heads a kv head)
        dict(name="attn_batch_decode", op="attention", heads=40, kv_heads=8, dim=128, page=16, seqs=64,
             new=1, singles=1.0, len_lo=200, len_hi=16000, window=0, sinks=0, shape=2),
        # two very long documents, one token each: work has to be split along the length (Llama-3.2-1B shape)
        dict(name="attn_long_decode", op="attention", heads=32, kv_heads=8, dim=64, page=64, seqs=2,
             new=1, singles=1.0, len_lo=100003, len_hi=131072, window=0, sinks=0, shape=3),
        # the last chunk of a long prompt (Qwen3-8B shape)
        dict(name="attn_prompt_chunk", op="attention", heads=32, kv_heads=8, dim=128, page=64, seqs=1,
             new=4096, singles=0.0, len_lo=16384, len_hi=16384, window=0, sinks=0, shape=4),
        # a mixed step: chunks of prompts beside single tokens, sliding window with
        # first tokens kept (Llama-3.2-3B shape: 3 query heads a kv head)
        dict(name="attn_window_mixed", op="attention", heads=24, kv_heads=8, dim=128, page=32, seqs=8,
             new=515, singles=0.5, len_lo=700, len_hi=9000, window=1024, sinks=4, shape=5),
        # q, k, v of a decode batch into the cache
        dict(name="append_decode", op="append", heads=40, kv_heads=8, dim=128, page=16, seqs=64,
             new=1, singles=1.0, len_lo=1, len_hi=8192, pairs=2, norm=True, shape=6),
        # q, k, v of a prompt chunk
        dict(name="append_prompt", op="append", heads=32, kv_heads=8, dim=128, page=64, seqs=2,
             new=2048, singles=0.0, len_lo=2500, len_hi=9000, pairs=1, norm=False, shape=7),
        # a beam step: the beams are dropped and forked anew from their parents (Llama-3.2-3B shape, 28 layers)
        dict(name="pages_beam_fork", op="fork", layers=28, kv_heads=8, dim=128, page=16, pages=1024,
             seqs=20, parents=4, children=16, len_lo=300, len_hi=1500, shape=8),
        # after many requests ended: the live pages move together (Llama-3.2-1B shape, 16 layers)
        dict(name="pages_compact", op="compact", layers=16, kv_heads=8, dim=64, page=32, pages=2048,
             seqs=64, live=0.6, shape=9),
        # greedy pick of one chat with a repeat penalty, logits not kept
        dict(name="pick_one", op="pick", rows=1, vocab=128256, history=700, biases=0, mask=False,
             keep=False, shape=10),
        # a batch under grammars, processed logits kept (for sampling)
        dict(name="pick_batch", op="pick", rows=64, vocab=151936, history=4000, biases=32, mask=True,
             keep=True, shape=11),
        # a larger batch at an odd vocabulary size, picks only
        dict(name="pick_rows", op="pick", rows=200, vocab=50257, history=1000, biases=8, mask=True,
             keep=False, shape=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    """Seconds that the work of a case takes at about this card's rates."""
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "fork", "compact", "pick"])
    most = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        case = _drawn(rng, op)
        if _cost(case) <= most and _plain_bytes(case) <= 12e9:
            return case


def _drawn(rng, op):
    shape = rng.randrange(1, 1 << 30)
    dim = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 8, 8])
    if op == "attention":
        kind = rng.choice(["single", "single", "chunk", "mixed"])
        lo = _log(rng, 1, 20000)
        case = dict(op=op, heads=kv * rng.choice([1, 2, 3, 4, 5, 7, 8]), kv_heads=kv, dim=dim,
                    page=rng.choice([16, 32, 64, 128]), seqs=_log(rng, 1, 64 if kind != "chunk" else 6),
                    new=1 if kind == "single" else _log(rng, 2, 4096),
                    singles={"single": 1.0, "chunk": 0.0, "mixed": 0.5}[kind],
                    len_lo=lo, len_hi=lo + _log(rng, 1, 20000), window=0, sinks=0, shape=shape)
        if rng.random() < 0.4:
            case["window"] = _log(rng, 16, 4096)
            case["sinks"] = rng.choice([0, 1, 4, 130])
        return case
    if op == "append":
        lo = _log(rng, 1, 4000)
        return dict(op=op, heads=kv * rng.choice([1, 2, 3, 4, 5, 8]), kv_heads=kv, dim=dim,
                    page=rng.choice([16, 32, 64, 128]), seqs=_log(rng, 1, 64), new=_log(rng, 1, 2048),
                    singles=rng.choice([0.0, 0.5, 1.0]), len_lo=lo, len_hi=lo + _log(rng, 1, 8000),
                    pairs=rng.choice([0, 1, 2]), norm=rng.random() < 0.5, shape=shape)
    if op == "fork":
        parents = _log(rng, 1, 8)
        children = parents * rng.choice([1, 2, 3, 4])
        page = rng.choice([16, 32, 64])
        hi = _log(rng, 17, 3000)
        return dict(op=op, layers=_log(rng, 1, 28), kv_heads=kv, dim=dim, page=page,
                    pages=parents * (-(-hi // page)) + children + rng.randrange(0, 200),
                    seqs=parents + children, parents=parents, children=children, len_lo=1, len_hi=hi,
                    shape=shape)
    if op == "compact":
        return dict(op=op, layers=_log(rng, 1, 16), kv_heads=kv, dim=dim, page=rng.choice([16, 32, 64]),
                    pages=_log(rng, 64, 4000), seqs=_log(rng, 1, 64), live=rng.uniform(0.1, 0.95),
                    shape=shape)
    return dict(op=op, rows=_log(rng, 1, 256), vocab=_log(rng, 1000, 200000), history=_log(rng, 1, 8000),
                biases=rng.choice([0, 3, 40]), mask=rng.random() < 0.5, keep=rng.random() < 0.5,
                shape=shape)


# ------------------------------------------------- sizes that a case implies ---

def _batch(case):
    """Length (with the new tokens) and count of new tokens of each sequence."""
    r = random.Random(case["shape"])
    lens, news = [], []
    for i in range(case["seqs"]):
        n = _log(r, case["len_lo"], case["len_hi"])
        single = r.random() < case["singles"]
        m = 1 if single else r.randint(max(1, case["new"] // 2), case["new"])
        if case["seqs"] == 1:
            m = case["new"]
        elif i == 3 and not single:
            m = 0  # a sequence of the step that has nothing new
        lens.append(n)
        news.append(min(m, n))
    return lens, news


def _visible(case, n, m):
    """Sum over the m new tokens of a length-n sequence of the keys each one sees, and the keys any sees."""
    w, s = case["window"], case["sinks"]
    p = torch.arange(n - m, n, dtype=torch.int64)
    if w == 0:
        return int((p + 1).sum()), n if m else 0
    lo = (p - w + 1).clamp(min=0)
    seen = p + 1 - lo + torch.minimum(lo, torch.tensor(s))
    first = max(0, n - m - w + 1)
    return int(seen.sum()), (n - first + min(first, s)) if m else 0


def _compact_shape(case):
    """Page counts of the sequences, and the random pages they hold."""
    r = random.Random(case["shape"])
    total = max(1, min(case["pages"], int(case["pages"] * case["live"])))
    ids = r.sample(range(case["pages"]), total)
    cuts = sorted(r.randint(0, total) for _ in range(case["seqs"] - 1))
    counts = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    return counts, ids


def _fork_shape(case):
    r = random.Random(case["shape"])
    lens = [_log(r, case["len_lo"], case["len_hi"]) for _ in range(case["parents"])]
    need = sum(-(-n // case["page"]) for n in lens)
    ids = r.sample(range(case["pages"]), need)
    return lens, ids


def _plain_bytes(case):
    """The largest intermediates of the plain form, for drawn cases."""
    if case["op"] == "attention":
        lens, news = _batch(case)
        return (4.0 * case["seqs"] * max(lens) * (case["heads"] * max(1, max(news)) + 2 * case["kv_heads"] * case["dim"]))
    if case["op"] in ("fork", "compact"):
        return 4.0 * case["layers"] * case["pages"] * case["kv_heads"] * case["page"] * case["dim"]
    return 0.0


def work(case):
    op = case["op"]
    if op == "attention":
        H, G, D = case["heads"], case["kv_heads"], case["dim"]
        pairs = keys = rows = 0
        for n, m in zip(*_batch(case)):
            a, b = _visible(case, n, m)
            pairs, keys, rows = pairs + a, keys + b, rows + m
        return {"bytes": 2 * 2 * rows * H * D + 2 * 2 * keys * G * D, "flops": 4 * D * H * pairs}
    if op == "append":
        _, news = _batch(case)
        heads = case["heads"] + 2 * case["kv_heads"]
        rows = sum(news)
        return {"bytes": 6 * rows * heads * case["dim"] + (4 * rows * case["dim"] if case["pairs"] else 0),
                "flops": 8 * rows * heads * case["dim"]}
    page_bytes = 2 * 2 * case["layers"] * case["kv_heads"] * case["page"] * case["dim"] if op != "pick" else 0
    if op == "fork":
        lens, _ = _fork_shape(case)
        partial = sum(lens[i % len(lens)] % case["page"] != 0 for i in range(case["children"]))
        width = max(-(-n // case["page"]) for n in lens)
        return {"bytes": 2 * partial * page_bytes + 8 * width * case["children"] + 8 * case["pages"], "flops": 0}
    if op == "compact":
        counts, ids = _compact_shape(case)
        moved = sum(i >= len(ids) for i in ids)
        return {"bytes": 2 * moved * page_bytes + 8 * case["pages"] + 8 * len(ids), "flops": 0}
    V, R = case["vocab"], case["rows"]
    return {"bytes": R * (4 * V * (2 if case["keep"] else 1) + (V // 8 if case["mask"] else 0) + 4 * case["history"] // 2
                          + 8 * case["biases"] + 8),
            "flops": 2 * R * V}


# -------------------------------------------------------------------- inputs ---

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def _pool(g, *shape):
    out = torch.empty(*shape, dtype=torch.bfloat16, device=DEV)
    for layer in out:
        layer.copy_(torch.randn(layer.shape, generator=g, device=DEV, dtype=torch.bfloat16))
    return out


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "pick":
        R, V = case["rows"], case["vocab"]
        s["logits"] = _normal(g, R, V, scale=3.0, dtype=torch.float32)
        r = random.Random(case["shape"])
        counts = [r.randint(0, case["history"]) if R > 1 else case["history"] for _ in range(R)]
        starts = [0]
        for c in counts:
            starts.append(starts[-1] + c)
        # tokens repeat, and the likely ones are among them
        few = torch.randint(0, V, (R, 64), generator=g, device=DEV)
        few[:, 0] = s["logits"].argmax(1)
        row = torch.repeat_interleave(torch.arange(R, device=DEV), torch.tensor(counts, device=DEV),
                                      output_size=starts[-1])
        pickd = torch.randint(0, 64, (starts[-1],), generator=g, device=DEV)
        rare = torch.randint(0, V, (starts[-1],), generator=g, device=DEV)
        s["history"] = torch.where(pickd < 48, few[row, pickd], rare).to(torch.int32)
        s["starts"] = _ints(starts)
        pen = torch.rand(R, 3, generator=g, device=DEV)
        s["penalties"] = pen * torch.tensor([0.3, 0.5, 0.1], device=DEV) + torch.tensor([1.0, 0.0, 0.0], device=DEV)
        s["bias_ids"] = s["bias"] = s["bias_starts"] = s["mask"] = None
        if case["biases"]:
            B = case["biases"]
            step = V // B  # distinct ids
            s["bias_ids"] = (torch.arange(B, device=DEV) * step
                             + torch.randint(0, step, (R, B), generator=g, device=DEV)).to(torch.int32).reshape(-1)
            s["bias"] = _normal(g, R * B, scale=2.0, dtype=torch.float32)
            s["bias_starts"] = torch.arange(R + 1, dtype=torch.int32, device=DEV) * B
        if case["mask"]:
            words = -(-V // 32)
            s["mask"] = torch.randint(-(1 << 31), 1 << 31, (R, words), generator=g, device=DEV).to(torch.int32)
            if R > 2:
                s["mask"][2] = 0  # a grammar that allows nothing
        s["out"] = torch.empty_like(s["logits"]) if case["keep"] else None
        s["pick"] = torch.empty(R, dtype=torch.int64, device=DEV)
        return s

    G, D, P = case["kv_heads"], case["dim"], case["page"]
    if op in ("attention", "append"):
        lens, news = _batch(case)
        counts = [-(-n // P) for n in lens]
        pages, width, layers = sum(counts) + 3, max(counts), 1
        ids = torch.randperm(pages, generator=g, device=DEV)[:sum(counts)].tolist()
    elif op == "fork":
        lens, ids = _fork_shape(case)
        counts = [-(-n // P) for n in lens] + [0] * case["children"]
        lens = lens + [0] * case["children"]
        pages, width, layers = case["pages"], max(counts), case["layers"]
    else:
        counts, ids = _compact_shape(case)
        lens = [c * P for c in counts]
        pages, width, layers = case["pages"], max(counts), case["layers"]
    table = torch.full((len(counts), max(1, width)), -1, dtype=torch.int32)
    at = 0
    for i, c in enumerate(counts):
        table[i, :c] = torch.tensor(ids[at:at + c], dtype=torch.int32)
        at += c
    refs = torch.zeros(pages, dtype=torch.int32)
    refs[torch.tensor(ids, dtype=torch.int64)] = 1
    s["k"] = _pool(g, layers, pages, G, P, D)
    s["v"] = _pool(g, layers, pages, G, P, D)
    s["table"], s["refs"], s["lens"] = table.to(DEV), refs.to(DEV), _ints(lens)

    if op in ("attention", "append"):
        starts = [0]
        for m in news:
            starts.append(starts[-1] + m)
        T = starts[-1]
        s["seqs"], s["starts"], s["tokens"] = _ints(list(range(len(lens)))), _ints(starts), T
        s["max_new"], s["max_len"] = max(news), max(lens)
        # the plan of the step, as index tensors
        s["row_seq"] = torch.repeat_interleave(torch.arange(len(news)), torch.tensor(news)).to(DEV)
        s["row_at"] = torch.cat([torch.arange(m) for m in news]).to(DEV)
        s["row_pos"] = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, news)]).to(DEV)
    if op == "attention":
        s["q"] = _normal(g, T, case["heads"], D, scale=1.5)
        s["out"] = torch.empty_like(s["q"])
    if op == "append":
        H = case["heads"]
        for name, heads in (("yq", H), ("yk", G), ("yv", G)):
            s[name] = _normal(g, T, heads * D, scale=2.0, dtype=torch.float32)
        s["q_out"] = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
        s["rope"] = s["q_norm"] = s["k_norm"] = None
        if case["pairs"]:
            ang = (torch.arange(table.shape[1] * P, dtype=torch.float64)[:, None]
                   * 1e6 ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D)[None, :])
            s["rope"] = torch.cat([ang.cos(), ang.sin()], 1).float().to(DEV)
        if case["norm"]:
            s["q_norm"] = torch.rand(D, generator=g, device=DEV) + 0.5
            s["k_norm"] = torch.rand(D, generator=g, device=DEV) + 0.5
    if op == "fork":
        s["parents"] = _ints([i % case["parents"] for i in range(case["children"])])
        s["children"] = _ints([case["parents"] + i for i in range(case["children"])])
        s["status"] = torch.empty(case["children"], dtype=torch.int32, device=DEV)
    if op == "compact":
        s["refs0"], s["table0"] = s["refs"].clone(), s["table"].clone()
    if own:
        import gguf_q4_dequant_gb300 as q4k
        s["cache"] = q4k.Cache(s["k"], s["v"], s["refs"], s["table"], s["lens"])
        s["workspace"] = s["cache"].workspace()
    return s


# --------------------------------------------------------------------- passes ---

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_attention(s):
    import gguf_q4_dequant_gb300 as q4k
    c = s["case"]
    q4k.q4k_cache_attention(s["cache"], 0, s["seqs"], s["starts"], s["q"], s["out"], c["heads"], s["max_new"],
                            c["dim"] ** -0.5, c["window"], c["sinks"], s["workspace"])
    return s["out"]


def _own_append(s):
    import gguf_q4_dequant_gb300 as q4k
    c = s["case"]
    q4k.q4k_cache_append(s["cache"], 0, s["seqs"], s["starts"], s["yq"], s["yk"], s["yv"], s["q_out"], c["heads"],
                         s["rope"], c["pairs"], s["q_norm"], s["k_norm"], 1e-6)
    return s["q_out"], s["k"], s["v"]


def _own_fork(s):
    import gguf_q4_dequant_gb300 as q4k
    q4k.q4k_pages_free(s["cache"], s["children"])
    q4k.q4k_pages_fork(s["cache"], s["parents"], s["children"], s["status"], s["workspace"])
    return s["k"], s["v"], s["refs"], s["table"], s["lens"], s["status"]


def _own_compact(s):
    import gguf_q4_dequant_gb300 as q4k
    s["refs"].copy_(s["refs0"])  # the pass before moved them: as they were, so that this one has the same to do
    s["table"].copy_(s["table0"])
    q4k.q4k_pages_compact(s["cache"], s["workspace"])
    return s["k"], s["v"], s["refs"], s["table"]


def _own_pick(s):
    import gguf_q4_dequant_gb300 as q4k
    c = s["case"]
    q4k.q4k_logits_pick(s["logits"], c["rows"], c["vocab"], s["out"], s["pick"], s["history"], s["starts"],
                        s["penalties"], s["bias_ids"], s["bias"], s["bias_starts"], s["mask"])
    return s["out"], s["pick"]


def _plain_attention(s):
    c = s["case"]
    H, G, D, P = c["heads"], c["kv_heads"], c["dim"], c["page"]
    n, N, M = c["seqs"], s["max_len"], s["max_new"]
    rows = s["table"][:, :-(-N // P)].long().clamp(min=0)
    there = torch.arange(rows.shape[1] * P, device=DEV)[None, :] < s["lens"][:, None]
    k = s["k"][0][rows].permute(0, 2, 1, 3, 4).reshape(n, G, -1, D).float()
    v = s["v"][0][rows].permute(0, 2, 1, 3, 4).reshape(n, G, -1, D).float()
    v = torch.where(there[:, None, :, None], v, 0.0)
    q = torch.zeros(n, M, H, D, device=DEV)
    q[s["row_seq"], s["row_at"]] = s["q"].float()
    pos = torch.full((n, M), -1, device=DEV)
    pos[s["row_seq"], s["row_at"]] = s["row_pos"]
    q = q.reshape(n, M, G, H // G, D).permute(0, 2, 3, 1, 4).reshape(n, G, -1, D)
    x = torch.matmul(q, k.transpose(2, 3)).reshape(n, G, H // G, M, -1).mul_(D ** -0.5)
    j = torch.arange(x.shape[-1], device=DEV)
    sees = (j[None, None, :] <= pos[:, :, None]) & there[:, None, :]
    if c["window"]:
        sees &= (j[None, None, :] > pos[:, :, None] - c["window"]) | (j < c["sinks"])[None, None, :]
    x = x.masked_fill_(~sees[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = x.sum(-1, keepdim=True)
    y = torch.matmul(x.reshape(n, G, -1, x.shape[-1]), v).reshape(n, G, H // G, M, D)
    y = torch.where(total > 0, y / total, 0.0).permute(0, 3, 1, 2, 4).reshape(n, M, H, D)
    return y[s["row_seq"], s["row_at"]].to(torch.bfloat16)


def _rotate(x, table, pairs):
    half = x.shape[-1] // 2
    cos, sin = table[:, None, :half], table[:, None, half:]
    if pairs == 1:  # (0, 1), (2, 3), ...
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    a, b = x[..., :half], x[..., half:]  # (0, D/2), (1, D/2 + 1), ...
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _plain_append(s):
    c = s["case"]
    H, G, D, P = c["heads"], c["kv_heads"], c["dim"], c["page"]
    q, k, v = s["yq"].view(-1, H, D), s["yk"].view(-1, G, D), s["yv"].view(-1, G, D)
    if s["q_norm"] is not None:
        q = q / (q.square().mean(-1, keepdim=True) + 1e-6).sqrt() * s["q_norm"]
        k = k / (k.square().mean(-1, keepdim=True) + 1e-6).sqrt() * s["k_norm"]
    pos = s["row_pos"]
    if c["pairs"]:
        q, k = _rotate(q, s["rope"][pos], c["pairs"]), _rotate(k, s["rope"][pos], c["pairs"])
    page = s["table"][s["row_seq"], pos // P].long()
    s["k"][0][page, :, pos % P] = k.to(torch.bfloat16)
    s["v"][0][page, :, pos % P] = v.to(torch.bfloat16)
    s["q_out"].copy_(q)
    return s["q_out"], s["k"], s["v"]


def _plain_fork(s):
    P = s["case"]["page"]
    refs, table, lens, par, chi = s["refs"], s["table"], s["lens"], s["parents"].long(), s["children"].long()
    cols = torch.arange(table.shape[1], device=DEV)[None, :]
    # the children's pages go back
    old = table[chi]
    refs.index_add_(0, old.clamp(min=0).flatten().long(), -(old >= 0).flatten().int())
    table[chi] = -1
    lens[chi] = 0
    # forks: full pages are shared, a page that is partly filled is copied to the lowest free one
    n = lens[par]
    full, part = (n // P).long(), n % P > 0
    need = part.long()
    free = refs == 0
    ok = need.cumsum(0) <= free.sum()
    order = torch.sort((~free).int(), stable=True).indices
    fresh = order[(need.cumsum(0) - 1).clamp(min=0)]
    rows = table[par]
    src = rows.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0].long().clamp(min=0)
    rows = torch.where(cols < full[:, None], rows, -1)
    rows = torch.where((cols == full[:, None]) & part[:, None], fresh[:, None].int(), rows)
    table[chi] = torch.where(ok[:, None], rows, -1)
    lens[chi] = torch.where(ok, n, 0)
    refs.index_add_(0, rows.clamp(min=0).flatten().long(), ((rows >= 0) & ok[:, None]).flatten().int())
    copied = (part & ok).nonzero()[:, 0]
    s["k"][:, fresh[copied]] = s["k"][:, src[copied]]
    s["v"][:, fresh[copied]] = s["v"][:, src[copied]]
    s["status"].copy_(torch.where(ok, 0, 1))
    return s["k"], s["v"], refs, table, lens, s["status"]


def _plain_compact(s):
    s["refs"].copy_(s["refs0"])  # as in the framework's pass
    s["table"].copy_(s["table0"])
    refs, table = s["refs"], s["table"]
    live = refs > 0
    ids = torch.arange(refs.numel(), device=DEV)
    low = ids < live.sum()
    src, dst = (live & ~low).nonzero()[:, 0], (~live & low).nonzero()[:, 0]
    to = ids.clone()
    to[src] = dst
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, to[table.long().clamp(min=0)], -1))
    return s["k"], s["v"], refs, table


def _plain_pick(s):
    c = s["case"]
    R, V = c["rows"], c["vocab"]
    x = s["logits"]
    row = torch.searchsorted(s["starts"].long(), torch.arange(s["history"].numel(), device=DEV), right=True) - 1
    count = torch.zeros(R * V, device=DEV)
    count.index_add_(0, row * V + s["history"].long(), torch.ones(s["history"].numel(), device=DEV))
    count = count.view(R, V)
    rep, presence, freq = s["penalties"].split(1, 1)
    y = torch.where(x > 0, x / rep, x * rep) - count * freq - presence
    x = torch.where(count > 0, y, x)
    if s["bias"] is not None:
        brow = torch.arange(R, device=DEV).repeat_interleave(c["biases"])
        add = torch.zeros_like(x)
        add[brow, s["bias_ids"].long()] = s["bias"]
        x = x + add
    if s["mask"] is not None:
        bits = (s["mask"][:, :, None] >> torch.arange(32, dtype=torch.int32, device=DEV)) & 1
        allowed = bits.reshape(R, -1)[:, :V] == 1
        x = torch.where(allowed, x, -math.inf)
        best = torch.where(allowed.any(1), (x == x.amax(1, keepdim=True)).int().argmax(1), -1)
    else:
        best = (x == x.amax(1, keepdim=True)).int().argmax(1)
    return x if c["keep"] else None, best


_own = {"attention": _own_attention, "append": _own_append, "fork": _own_fork, "compact": _own_compact,
        "pick": _own_pick}
_plain = {"attention": _plain_attention, "append": _plain_append, "fork": _plain_fork,
          "compact": _plain_compact, "pick": _plain_pick}


# ---------------------------------------------------------------------- exact ---

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attention":
        return _exact_attention(case, s)
    if op == "append":
        return _exact_append(case, s)
    if op == "pick":
        return _exact_pick(case, s)
    return None  # copies and whole numbers: nothing is computed in floating point


def _exact_attention(case, s):
    D, P, r = case["dim"], case["page"], case["heads"] // case["kv_heads"]
    lens, news = _batch(case)
    out = torch.zeros(s["tokens"], case["heads"], D, dtype=torch.float64, device=DEV)
    at = 0
    for b, (n, m) in enumerate(zip(lens, news)):
        pages = s["table"][b, :-(-n // P)].long()
        i = torch.arange(n - m, n, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)[None, :]
        hidden = j > i
        if case["window"]:
            hidden = hidden | ((j <= i - case["window"]) & (j >= case["sinks"]))
        for h in range(case["heads"] if m else 0):
            k = s["k"][0, pages, h // r].reshape(-1, D)[:n].double()
            v = s["v"][0, pages, h // r].reshape(-1, D)[:n].double()
            e = (s["q"][at:at + m, h].double() @ k.T) / math.sqrt(D)
            e[hidden] = -math.inf
            out[at:at + m, h] = torch.softmax(e, 1) @ v
        at += m
    return out


def _exact_append(case, s):
    H, G, D, P = case["heads"], case["kv_heads"], case["dim"], case["page"]
    pos = s["row_pos"]

    def turned(y, heads, weight):
        x = y.double().view(-1, heads, D)
        if weight is not None:
            x = x * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) / D + 1e-6) * weight.double()
        if case["pairs"]:
            z = s["rope"].double()[pos]
            z = torch.complex(z[:, :D // 2], z[:, D // 2:])[:, None]
            if case["pairs"] == 1:
                x = torch.view_as_real(torch.view_as_complex(x.reshape(*x.shape[:-1], -1, 2).contiguous()) * z).flatten(-2)
            else:
                w = torch.complex(x[..., :D // 2].contiguous(), x[..., D // 2:].contiguous()) * z
                x = torch.cat([w.real, w.imag], -1)
        return x

    q, k = turned(s["yq"], H, s["q_norm"]), turned(s["yk"], G, s["k_norm"])
    pk, pv = s["k"].double(), s["v"].double()
    page = s["table"][s["row_seq"], pos // P].long()
    for h in range(G):
        pk[0, page, h, pos % P] = k[:, h]
        pv[0, page, h, pos % P] = s["yv"].double().view(-1, G, D)[:, h]
    return q, pk, pv


def _exact_pick(case, s):
    R, V = case["rows"], case["vocab"]
    starts = s["starts"].tolist()
    x = s["logits"].double()
    best = torch.empty(R, dtype=torch.int64, device=DEV)
    for m in range(R):
        ids, counts = s["history"][starts[m]:starts[m + 1]].long().unique(return_counts=True)
        rep, presence, freq = s["penalties"][m].double().tolist()
        y = x[m, ids]
        x[m, ids] = torch.where(y > 0, y / rep, y * rep) - freq * counts - presence
        if case["biases"]:
            b = slice(m * case["biases"], (m + 1) * case["biases"])
            x[m, s["bias_ids"][b].long()] += s["bias"][b].double()
        allowed = torch.ones(V, dtype=torch.bool, device=DEV)
        if case["mask"]:
            word = s["mask"][m].long() & 0xFFFFFFFF
            allowed = (word.repeat_interleave(32)[:V] >> (torch.arange(V, device=DEV) % 32)) & 1 == 1
            x[m, ~allowed] = -math.inf
        top = torch.nonzero(allowed & (x[m] == x[m].max()))
        best[m] = top[0, 0] if top.numel() else -1
    return x if case["keep"] else None, best
