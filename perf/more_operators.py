"""Timed cases of attention for trees of drafted tokens, and of attention over one shared
latent vector a token: its append, its absorbed and its expanded form.

A case is a dict of plain values.  ``run`` computes it in plain torch operations
(``own`` false) or through the library's entry points (``own`` true) on the
inputs that ``prepare`` made; ``exact`` gives the same outputs from the
operators' definitions in 64 bits.

Operators (``case["op"]``):

``tree``           rows of n drafted tokens that hang together as a tree, behind their context in a paged KV
                   cache of any format: a drafted token sees the context and its own ancestors, which a bit
                   mask per token gives
``latent_append``  a step's latent vectors and position keys into a paged latent cache, the position parts
                   of keys and queries rotated on the way
``latent``         absorbed latent attention: every head's query [512 + 64] against the cached rows
                   [512 latent | 64 position], whose first 512 elements are the values too; decode rows,
                   causal rows of a few drafted tokens, and trees of them
``expanded``       expanded latent attention of prompts: per head 128-element keys and values made of the
                   latent vectors, and one 64-element position key a token that all heads share
"""
import math
import random

import torch

own = False

PAGE = 32
DEV = "cuda"
LATENT, ROPE, NOPE, VDIM = 512, 64, 128, 128


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the smallest verify pass: two sequences, eight drafted tokens each
        {"name": "tree_2x8_f16", "op": "tree", "fmt": "f16", "hq": 4, "hkv": 1, "d": 64, "batch": 2, "lo": 100,
         "hi": 300, "nodes": 8, "window": 0, "rows": 1},
        # a batch that drafts trees of 25 tokens over long contexts
        {"name": "tree_16x25_e4m3", "op": "tree", "fmt": "e4m3", "hq": 32, "hkv": 8, "d": 128, "batch": 16,
         "lo": 2048, "hi": 32768, "nodes": 25, "window": 0, "rows": 2},
        # wide trees of 64 tokens in the block formats
        {"name": "tree_8x64_q8_0", "op": "tree", "fmt": "q8_0", "hq": 32, "hkv": 8, "d": 128, "batch": 8,
         "lo": 1000, "hi": 16384, "nodes": 64, "window": 0, "rows": 3},
        # narrow trees that fit beside one another on a decode tile
        {"name": "tree_32x6_q4_0", "op": "tree", "fmt": "q4_0", "hq": 32, "hkv": 8, "d": 128, "batch": 32,
         "lo": 1024, "hi": 8192, "nodes": 6, "window": 0, "rows": 4},
        # the append of one decode step of 16 sequences, 128 heads' queries rotated
        {"name": "latent_append_16", "op": "latent_append", "n": 16, "heads": 128, "start": 30000, "scatter": True,
         "layout": "interleaved", "scaling": "ramp"},
        # a whole prompt that ends inside a page
        {"name": "latent_append_8201", "op": "latent_append", "n": 8201, "heads": 32, "start": 5, "scatter": False,
         "layout": "half", "scaling": "none"},
        # the smallest decode step: two short sequences, 16 heads
        {"name": "latent_2x300_h16", "op": "latent", "heads": 16, "batch": 2, "lo": 100, "hi": 300, "long": 0,
         "draft": 0, "tree": False, "rows": 1},
        # a decode batch of a model cut over several devices: 16 heads, bound by the cache's bytes
        {"name": "latent_64x8192_h16", "op": "latent", "heads": 16, "batch": 64, "lo": 1024, "hi": 16384, "long": 0,
         "draft": 0, "tree": False, "rows": 2},
        # all 128 heads on one device, one session of 131072 tokens beside shorter ones
        {"name": "latent_long_h128", "op": "latent", "heads": 128, "batch": 31, "lo": 2048, "hi": 8192,
         "long": 131072, "draft": 0, "tree": False, "rows": 3},
        # trees of six drafted tokens over the latent cache, 128 heads: tensor-core bound
        {"name": "latent_tree_16x6_h128", "op": "latent", "heads": 128, "batch": 16, "lo": 2048, "hi": 16384,
         "long": 0, "draft": 6, "tree": True, "rows": 4},
        # ragged short prompts of one prefill step
        {"name": "expanded_prompts_h8", "op": "expanded", "heads": 8, "batch": 5, "lo": 17, "hi": 900, "chunk": 0,
         "offset": 0, "rows": 5},
        # a chunk of 2048 tokens behind 8192 others, beside a fresh prompt
        {"name": "expanded_chunk_h32", "op": "expanded", "heads": 32, "batch": 1, "lo": 1000, "hi": 1000,
         "chunk": 2048, "offset": 8192, "rows": 6},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "latent_append", "latent", "latent", "expanded"])
    if op == "latent_append":
        return {"op": op, "n": _log_int(rng, 1, 8192), "heads": rng.choice([8, 32, 64, 128]),
                "start": _log_int(rng, 1, 100000), "scatter": rng.random() < 0.5,
                "layout": rng.choice(["half", "interleaved"]), "scaling": rng.choice(["none", "ramp"])}
    batch = _log_int(rng, 1, 24)
    lo = _log_int(rng, 1, 4096)
    hi = _log_int(rng, lo, 12000)
    rows = rng.randint(0, 1 << 20)
    if op == "tree":
        hq, hkv = rng.choice([(4, 1), (8, 8), (8, 4), (32, 8), (16, 2)])
        return {"op": op, "fmt": rng.choice(["f16", "q8_0", "q4_0", "i8", "e4m3"]), "hq": hq, "hkv": hkv,
                "d": rng.choice([64, 128]), "batch": batch, "lo": lo, "hi": hi, "nodes": _log_int(rng, 1, 100),
                "window": rng.choice([0, 0, 0, 1000]), "rows": rows}
    if op == "latent":
        draft = rng.choice([0, 0, 2, 5])
        return {"op": op, "heads": rng.choice([8, 16, 32, 64, 128]), "batch": batch, "lo": lo, "hi": hi,
                "long": rng.choice([0, 0, 0, 60000]), "draft": draft, "tree": draft > 0 and rng.random() < 0.5,
                "rows": rows}
    batch = rng.randint(1, 6)
    lo = _log_int(rng, 1, 500)
    case = {"op": op, "heads": rng.choice([2, 5, 8, 24]), "batch": batch, "lo": lo, "hi": _log_int(rng, lo, 2000),
            "chunk": 0, "offset": 0, "rows": rows}
    if rng.random() < 0.4:
        case["chunk"], case["offset"] = _log_int(rng, 1, 1500), _log_int(rng, 1, 8000)
    return case


def _rows(case):
    """(seq_len, q_offset) of the case's rows."""
    r = random.Random(7000 + case["rows"])
    rows = []
    for _ in range(case["batch"]):
        ctx = r.randint(case["lo"], case["hi"])
        if case["op"] == "tree":
            rows.append((ctx + case["nodes"], ctx))
        elif case["op"] == "latent":
            rows.append((ctx + case["draft"], ctx) if case["draft"] else (ctx, ctx - 1))
        else:
            rows.append((ctx, 0))
    if case["op"] == "latent" and case["long"]:
        n = max(1, case["draft"])
        rows.append((case["long"], case["long"] - n))
    if case["op"] == "expanded" and case["chunk"]:
        rows.append((case["offset"] + case["chunk"], case["offset"]))
    return rows


def _parents(case):
    """Parent of each drafted token of each row, -1 for a root; a parent comes before its children."""
    r = random.Random(9000 + case["rows"])
    out = []
    for s, o in _rows(case):
        out.append([-1 if i == 0 else r.randint(max(-1, i - 9), i - 1) for i in range(s - o)])
    return out


def _ancestors(parents):
    """Per drafted token the set of its ancestors and itself, as an integer of bits."""
    sets = []
    for i, p in enumerate(parents):
        sets.append((1 << i) | (sets[p] if p >= 0 else 0))
    return sets


def _pairs(case):
    """Query-key pairs over all rows."""
    total = 0
    tree = _parents(case) if case["op"] == "tree" or case.get("tree") else None
    w = case.get("window", 0)
    for i, (s, o) in enumerate(_rows(case)):
        if tree is None:
            total += (s * (s + 1) - o * (o + 1)) // 2
        else:
            for bits in _ancestors(tree[i]):
                depth = bin(bits).count("1")
                total += (min(o, max(0, w - depth)) if w else o) + depth
    return total


_ROW_BYTES = {"f16": lambda d: 2 * d, "q8_0": lambda d: d + d // 16, "q4_0": lambda d: d // 2 + d // 16,
              "i8": lambda d: d, "e4m3": lambda d: d}


def work(case):
    op = case["op"]
    if op == "latent_append":
        n = case["n"]
        return {"bytes": n * (2 * 2 * (LATENT + ROPE) + 2 * 2 * case["heads"] * ROPE + 8),
                "flops": 3 * n * (case["heads"] + 1) * ROPE}
    rows = _rows(case)
    nq = sum(s - o for s, o in rows)
    if op == "tree":
        d, w = case["d"], case["window"]
        keys = sum(s - (max(0, o + 1 - w) if w else 0) for s, o in rows)
        b = keys * case["hkv"] * 2 * _ROW_BYTES[case["fmt"]](d)
        if case["fmt"] in ("i8", "e4m3"):
            b += -(-keys // PAGE) * case["hkv"] * 8
        return {"bytes": b + nq * case["hq"] * d * 4 + nq * 4 * -(-case["nodes"] // 32),
                "flops": 4 * d * case["hq"] * _pairs(case)}
    h = case["heads"]
    if op == "latent":
        return {"bytes": sum(s for s, _ in rows) * 2 * (LATENT + ROPE) + nq * h * 2 * (2 * LATENT + ROPE),
                "flops": 2 * h * (2 * LATENT + ROPE) * _pairs(case)}
    keys = sum(s for s, _ in rows)
    return {"bytes": keys * 2 * (h * (NOPE + VDIM) + ROPE) + nq * h * 2 * (NOPE + ROPE + VDIM),
            "flops": 2 * h * (NOPE + ROPE + VDIM) * _pairs(case)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _page_table(g, rows, pages):
    need = [-(-s // PAGE) for s, _ in rows]
    perm = torch.randperm(pages, generator=g, device=DEV).int()
    pt = torch.full((len(rows), max(need)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for r, c in enumerate(need):
        pt[r, :c] = perm[at:at + c]
        at += c
    return pt


def _mask(case):
    """int32 [drafted tokens of all rows, words]: bit j of a token's words = drafted token j of its row."""
    words = -(-max(s - o for s, o in _rows(case)) // 32)
    out = []
    for parents in _parents(case):
        for bits in _ancestors(parents):
            out.append([(bits >> (32 * w)) & 0xFFFFFFFF for w in range(words)])
    t = torch.tensor(out, dtype=torch.int64)
    return torch.where(t >= 1 << 31, t - (1 << 32), t).int().to(DEV)


def _encode(x, fmt):
    """fp32 [..., 32, d] -> (codes, scales) of a whole page of one head."""
    if fmt == "f16":
        return x.half().view(torch.uint8), None
    if fmt in ("i8", "e4m3"):
        amax = x.abs().amax(dim=(-1, -2), keepdim=True)
        if fmt == "i8":
            s = amax / 127
            return torch.round(x / s).to(torch.int8).view(torch.uint8), s[..., 0, 0]
        s = torch.exp2(torch.ceil(torch.log2(amax / 448)))
        return (x / s).to(torch.float8_e4m3fn).view(torch.uint8), s[..., 0, 0]
    b = x.unflatten(-1, (-1, 32))
    if fmt == "q8_0":
        s = b.abs().amax(-1, keepdim=True) / 127
        return torch.round(b / s).to(torch.int8).flatten(-2).view(torch.uint8), s[..., 0].half()
    at = b.abs().argmax(-1, keepdim=True)
    s = b.gather(-1, at) / -8
    c = (b / s + 8.5).clamp(0, 15).to(torch.uint8)
    return (c[..., :16] | (c[..., 16:] << 4)).flatten(-2), s[..., 0].half()


def _planes(g, num_pages, hkv, d, fmt):
    """K and V planes of a filled cache, K with three channels eight times the others, as trained keys have."""
    out = []
    for is_k in (True, False):
        gain = torch.ones(d, device=DEV)
        if is_k:
            gain[torch.randint(0, d, (3,), generator=g, device=DEV)] = 8
        codes, scales = [], []
        for p in range(0, num_pages, 2048):
            c, s = _encode(_normal(g, min(2048, num_pages - p), hkv, PAGE, d).mul_(gain), fmt)
            codes.append(c)
            scales.append(s)
        out += [torch.cat(codes), None if fmt == "f16" else torch.cat(scales)]
    return out


_SCALING = {
    "none": {"factor": 1.0, "original_ctx": 0, "low": 0.0, "high": 0.0, "base": 10000.0},
    "ramp": {"factor": 8.0, "original_ctx": 4096, "low": 1.0, "high": 32.0, "base": 10000.0},
}


def _frequencies(scaling):
    """(angular frequency of each pair of the position part, multiplier of its cosines and sines)."""
    s = _SCALING[scaling]
    f = [s["base"] ** (-2.0 * i / ROPE) for i in range(ROPE // 2)]
    if scaling == "none":
        return f, 1.0

    def pair_of(turns):
        return ROPE * math.log(s["original_ctx"] / (turns * 2 * math.pi)) / (2 * math.log(s["base"]))

    lo = max(math.floor(pair_of(s["high"])), 0)
    hi = min(math.ceil(pair_of(s["low"])), ROPE - 1)
    t = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3))) for i in range(ROPE // 2)]
    return [x * (1 - a) + x / s["factor"] * a for x, a in zip(f, t)], 0.1 * math.log(s["factor"]) + 1.0


def _softmax_scale():
    return 1.0 / math.sqrt(NOPE + ROPE)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "latent_append":
        n, h, start = case["n"], case["heads"], case["start"]
        freq, s["mscale"] = _frequencies(case["scaling"])
        s["freq"] = torch.tensor(freq, dtype=torch.float64, device=DEV)
        if case["scatter"]:  # one token of each of n sequences, each somewhere in a page of its own
            pos = torch.randint(0, start + 1, (n,), generator=g, device=DEV)
            s["pages"] = n + 8
            slots = torch.randperm(n + 8, generator=g, device=DEV)[:n] * PAGE + pos % PAGE
        else:
            pos = start + torch.arange(n, device=DEV)
            s["pages"] = (start % PAGE + n + PAGE - 1) // PAGE + 8
            perm = torch.randperm(s["pages"], generator=g, device=DEV)
            slots = perm[(pos - start // PAGE * PAGE) // PAGE] * PAGE + pos % PAGE
        s["pos"], s["slots"] = pos.int(), slots.int()
        s["c"] = _normal(g, n, LATENT).half()
        # the position keys are the end of the projection that made the latent vectors, the queries' position
        # parts the end of every head of theirs; the rotated ones go to the end of the absorbed queries
        s["kr"] = _normal(g, n, LATENT + ROPE).half()[:, LATENT:]
        s["qr"] = _normal(g, n, h, NOPE + ROPE).half()[:, :, NOPE:]
        s["q"] = torch.zeros(n, h, LATENT + ROPE, dtype=torch.float16, device=DEV)
        s["data"] = _normal(g, s["pages"], PAGE, LATENT + ROPE).half()
    elif op == "expanded":
        rows, h = _rows(case), case["heads"]
        nk, nq = sum(x[0] for x in rows), sum(x[0] - x[1] for x in rows)
        s["row_list"] = rows
        s["q"] = _normal(g, nq, h, NOPE + ROPE).half()
        kv = _normal(g, nk, h, NOPE + VDIM).half()  # one projection of the latent vectors makes both
        s["k"], s["v"] = kv[:, :, :NOPE], kv[:, :, NOPE:]
        s["kr"] = _normal(g, nk, ROPE).half()
        s["out"] = torch.empty(nq, h, VDIM, dtype=torch.float16, device=DEV)
    else:
        rows = _rows(case)
        s["row_list"] = rows
        s["pages"] = sum(-(-x[0] // PAGE) for x in rows) + 3
        s["pt"] = _page_table(g, rows, s["pages"])
        nq = sum(x[0] - x[1] for x in rows)
        if op == "tree" or case["tree"]:
            s["mask"] = _mask(case)
        if op == "tree":
            s["planes"] = _planes(g, s["pages"], case["hkv"], case["d"], case["fmt"])
            s["q"] = _normal(g, nq, case["hq"], case["d"]).half()
            s["out"] = torch.empty_like(s["q"])
        else:
            s["data"] = torch.empty(s["pages"], PAGE, LATENT + ROPE, dtype=torch.float16, device=DEV)
            for p in range(0, s["pages"], 4096):
                s["data"][p:p + 4096] = _normal(g, *s["data"][p:p + 4096].shape)
            s["q"] = _normal(g, nq, case["heads"], LATENT + ROPE).mul_(0.5).half()
            s["out"] = torch.empty(nq, case["heads"], LATENT, dtype=torch.float16, device=DEV)
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program of the library's keeps between calls: the rotary table, the cache's description, the plan."""
    import mixed_attention_quantized_gb300 as mq
    case = s["case"]
    op = case["op"]
    s["mq"] = mq
    if op == "latent_append":
        layout = {"half": mq.ROPE_HALF, "interleaved": mq.ROPE_INTERLEAVED}[case["layout"]]
        scaling = {"none": mq.ROPE_SCALE_NONE, "ramp": mq.ROPE_SCALE_RAMP}[case["scaling"]]
        s["rope"] = mq.Rope(ROPE, layout=layout, scaling=scaling, **_SCALING[case["scaling"]])
    if "data" in s:
        s["cache"] = mq.LatentCache(s["pages"], LATENT, ROPE, s["data"])
    if op == "latent_append":
        return
    seq, off = [x[0] for x in s["row_list"]], [x[1] for x in s["row_list"]]
    if op == "tree":
        fmt = {"f16": mq.F16, "q8_0": mq.Q8_0, "q4_0": mq.Q4_0, "i8": mq.I8_PAGE, "e4m3": mq.E4M3_PAGE}[case["fmt"]]
        s["cache"] = mq.KVCache(s["pages"], case["hkv"], case["d"], fmt, fmt, *s["planes"])
        s["plan"] = mq.Plan(s["cache"], case["hq"], [mq.ROW_TREE] * len(seq), seq, off, s["pt"].shape[1],
                            window=case["window"])
    elif op == "latent":
        kind = mq.ROW_TREE if case["tree"] else (mq.ROW_CHUNK if case["draft"] else mq.ROW_DECODE)
        s["plan"] = mq.LatentPlan(s["cache"], case["heads"], [kind] * len(seq), seq, off, s["pt"].shape[1],
                                  _softmax_scale())
    else:
        s["plan"] = mq.ExpandedPlan(case["heads"], seq, off, _softmax_scale())
    s["ws"] = mq.alloc_workspace(s["plan"].workspace_bytes)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        mq = s["mq"]
        if op == "latent_append":
            mq.latent_append(s["cache"], s["rope"], s["qr"], s["c"], s["kr"], s["pos"], s["slots"],
                             s["q"][:, :, LATENT:])
            return {"q": s["q"], "cache": s["data"]}
        if op == "expanded":
            s["plan"].run(s["q"], s["k"], s["kr"], s["v"], s["out"], s["ws"])
        elif "mask" in s:
            s["plan"].run(s["q"], s["pt"], s["out"], s["ws"], tree_mask=s["mask"])
        else:
            s["plan"].run(s["q"], s["pt"], s["out"], s["ws"])
        return s["out"]
    return {"tree": _tree, "latent": _latent, "expanded": _expanded, "latent_append": _latent_append}[op](s)


def _seen(s, row, at, first):
    """bool [queries, keys from `first` on]: what the queries of a row see; `at` their place in the batch."""
    seq, off = s["row_list"][row]
    kp = first + torch.arange(seq - first, device=DEV)
    if "mask" not in s:
        return kp <= off + torch.arange(seq - off, device=DEV)[:, None]
    bit = kp - off
    words = s["mask"][at:at + seq - off]
    drafted = (words[:, bit.clamp_min(0) // 32] >> (bit.clamp_min(0) % 32)) & 1
    seen = (bit < 0) | (drafted == 1)
    w = s["case"].get("window", 0)
    if w:  # a token's position is its depth in the tree behind the context
        depth = torch.where(bit >= 0, drafted, torch.zeros_like(drafted)).sum(-1, keepdim=True)
        seen = seen & ((bit >= 0) | (kp > off + depth - 1 - w))
    return seen


def _softmax(score, seen):
    """Masked softmax numerators and their sums; rows that see nothing sum to zero."""
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    score -= torch.where(top == -math.inf, torch.zeros_like(top), top)
    score.exp_()
    total = score.sum(-1, keepdim=True)
    return score, torch.where(total > 0, total, torch.ones_like(total))


def _decode(codes, scale, fmt):
    """Planes of pages [n, hkv, 32, row bytes] -> fp32 [n, hkv, 32, d]."""
    if fmt == "f16":
        return codes.view(torch.float16).float()
    if fmt in ("i8", "e4m3"):
        return codes.view(torch.int8 if fmt == "i8" else torch.float8_e4m3fn).float() * scale[..., None, None]
    if fmt == "q8_0":
        return (codes.view(torch.int8).float().unflatten(-1, (-1, 32)) * scale.float()[..., None]).flatten(-2)
    c = codes.unflatten(-1, (-1, 16))
    c = torch.cat([c & 15, c >> 4], -1).float() - 8
    return (c * scale.float()[..., None]).flatten(-2)


def _tree(s):
    case = s["case"]
    hkv, d, w = case["hkv"], case["d"], case["window"]
    group = case["hq"] // hkv
    at = 0
    for r, (seq, off) in enumerate(s["row_list"]):
        nq = seq - off
        first = max(0, off + 1 - w) // PAGE if w else 0
        pages = s["pt"][r, first:-(-seq // PAGE)].long()
        k, v = (_decode(c[pages], None if x is None else x[pages], case["fmt"]).transpose(0, 1)
                .reshape(hkv, -1, d)[:, :seq - first * PAGE] for c, x in (s["planes"][:2], s["planes"][2:]))
        q = s["q"][at:at + nq].float().view(nq, hkv, group, d).permute(1, 2, 0, 3).reshape(hkv, group * nq, d)
        score = torch.matmul(q, k.transpose(1, 2)).mul_(1.0 / math.sqrt(d)).view(hkv, group, nq, -1)
        p, total = _softmax(score, _seen(s, r, at, first * PAGE))
        o = torch.matmul(p.view(hkv, group * nq, -1), v).view(hkv, group, nq, d).div_(total)
        s["out"][at:at + nq] = o.permute(2, 0, 1, 3).reshape(nq, -1, d).half()
        at += nq
    return s["out"]


def _latent(s):
    h = s["case"]["heads"]
    at = 0
    for r, (seq, off) in enumerate(s["row_list"]):
        nq = seq - off
        k = s["data"][s["pt"][r, :-(-seq // PAGE)].long()].float().view(-1, LATENT + ROPE)[:seq]
        q = s["q"][at:at + nq].float().view(nq * h, -1)
        score = torch.matmul(q, k.t()).mul_(_softmax_scale()).view(nq, h, seq)
        p, total = _softmax(score, _seen(s, r, at, 0)[:, None, :])
        o = torch.matmul(p.view(nq * h, seq), k[:, :LATENT]).view(nq, h, LATENT).div_(total)
        s["out"][at:at + nq] = o.half()
        at += nq
    return s["out"]


def _expanded(s):
    at = first = 0
    for r, (seq, off) in enumerate(s["row_list"]):
        nq = seq - off
        q = s["q"][at:at + nq].float().transpose(0, 1)
        k, v = (x[first:first + seq].float().transpose(0, 1) for x in (s["k"], s["v"]))
        kr = s["kr"][first:first + seq].float()
        seen = _seen(s, r, at, 0)
        for h0 in range(0, q.shape[0], 4):  # a few heads at a time: the scores are kept
            part = slice(h0, h0 + 4)
            score = torch.matmul(q[part, :, :NOPE], k[part].transpose(1, 2))
            score += torch.matmul(q[part, :, NOPE:], kr.t())
            p, total = _softmax(score.mul_(_softmax_scale()), seen)
            s["out"][at:at + nq, part] = torch.matmul(p, v[part]).div_(total).transpose(0, 1).half()
        at += nq
        first += seq
    return s["out"]


def _rotate(x, c, sn, layout):
    x = x.float()
    if layout == "half":
        a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
        return torch.cat([a * c - b * sn, b * c + a * sn], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)


def _latent_append(s):
    a = s["pos"].double()[:, None] * s["freq"]  # the angles of far positions need 64 bits
    c, sn = (torch.cos(a) * s["mscale"]).float(), (torch.sin(a) * s["mscale"]).float()
    layout = s["case"]["layout"]
    s["q"][:, :, LATENT:] = _rotate(s["qr"], c[:, None], sn[:, None], layout).clamp(-65504, 65504).half()
    page, at = s["slots"].long() // PAGE, s["slots"].long() % PAGE
    s["data"][page, at, :LATENT] = s["c"]
    s["data"][page, at, LATENT:] = _rotate(s["kr"], c, sn, layout).clamp(-65504, 65504).half()
    return {"q": s["q"], "cache": s["data"]}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "latent_append":
        return _append64(s)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    trees = _parents(case) if "mask" in s else None
    at = first = 0
    for r, (seq, off) in enumerate(s["row_list"]):
        nq = seq - off
        hidden = _hidden64(case, seq, off, trees[r] if trees else None)
        for h in range(out.shape[1]):
            q = s["q"][at:at + nq, h].double()
            if case["op"] == "tree":
                kvh = h // (case["hq"] // case["hkv"])
                if h % (case["hq"] // case["hkv"]) == 0:
                    pages = s["pt"][r, :-(-seq // PAGE)].long()
                    k, v = (_values64(c[pages, kvh], None if x is None else x[pages, kvh], case["fmt"])
                            .reshape(-1, case["d"])[:seq] for c, x in (s["planes"][:2], s["planes"][2:]))
                scale = case["d"] ** -0.5
            elif case["op"] == "latent":
                if h == 0:
                    k = s["data"][s["pt"][r, :-(-seq // PAGE)].long()].flatten(0, 1)[:seq].double()
                    v = k[:, :LATENT]
                scale = 192.0 ** -0.5
            else:
                k = torch.cat([s["k"][first:first + seq, h], s["kr"][first:first + seq]], 1).double()
                v = s["v"][first:first + seq, h].double()
                scale = 192.0 ** -0.5
            for a in range(0, nq, 1024):
                logits = torch.einsum("qd,kd->qk", q[a:a + 1024], k) * scale
                p = torch.softmax(logits.masked_fill(hidden[a:a + 1024], -math.inf), -1)
                out[at + a:at + min(nq, a + 1024), h] = torch.einsum("qk,kd->qd", p, v)
        at += nq
        first += seq
    return out


def _hidden64(case, seq, off, parents):
    nq = seq - off
    if parents is None:
        return torch.ones(nq, seq, dtype=torch.bool, device=DEV).triu(off + 1)
    hide = torch.ones(nq, seq, dtype=torch.bool)
    w = case.get("window", 0)
    depth = []
    for i, p in enumerate(parents):
        depth.append(0 if p < 0 else depth[p] + 1)
        start = max(0, off + depth[i] + 1 - w) if w else 0
        hide[i, min(start, off):off] = False
        j = i
        while j >= 0:
            hide[i, off + j] = False
            j = parents[j]
    return hide.to(DEV)


def _values64(codes, scale, fmt):
    if fmt == "f16":
        return codes.view(torch.float16).double()
    if fmt in ("i8", "e4m3"):
        x = codes.view({"i8": torch.int8, "e4m3": torch.float8_e4m3fn}[fmt]).double()
        return x * scale.double().reshape(-1, 1, 1)
    block = scale.double().repeat_interleave(32, dim=-1)
    if fmt == "q8_0":
        return codes.view(torch.int8).double() * block
    x = torch.empty(block.shape, dtype=torch.float64, device=DEV)
    for b in range(scale.shape[-1]):
        part = codes[..., 16 * b:16 * b + 16]
        x[..., 32 * b:32 * b + 16] = (part % 16).double() - 8
        x[..., 32 * b + 16:32 * b + 32] = torch.div(part, 16, rounding_mode="floor").double() - 8
    return x * block


def _append64(s):
    turn = torch.polar(torch.full((len(s["pos"]), ROPE // 2), s["mscale"], dtype=torch.float64, device=DEV),
                       s["pos"].double()[:, None] * s["freq"])

    def turned(x, t):
        x = x.double()
        if s["case"]["layout"] == "half":
            z = torch.complex(x[..., :ROPE // 2].contiguous(), x[..., ROPE // 2:].contiguous()) * t
            return torch.cat([z.real, z.imag], -1)
        return torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous()) * t).flatten(-2)

    q, data = s["q"].double(), s["data"].double().flatten(0, 1)
    q[..., LATENT:] = turned(s["qr"], turn[:, None])
    data[s["slots"].long()] = torch.cat([s["c"].double(), turned(s["kr"], turn)], 1)
    return {"q": q, "cache": data.view(s["data"].shape)}
