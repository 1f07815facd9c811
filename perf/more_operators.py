"""The operators before and behind a LoRA layer: norm, 8-bit cache, attention over it: cases, plain forms, calls.

A layer of a served model normalises its input before the base product and the
adapters read it, and writes its rotated keys and its values to a cache that
the attention of all later tokens reads.

    norm       h = x + r;  y[t][c] = h[t][c] w[c] / sqrt(mean_c h[t][c]^2 + eps), each rounded to its type;
               a = max_c |y[t][c]|, s[t] = a / 127, q[t][c] = rint(127 y[t][c] / a), ties to even
    cache      the same q and s for each token and head of k and v, at a slot of a page; read back q s
    attention  o = sum_j e^(scale q.k_j) v_j / sum_j e^(scale q.k_j) over the keys j that a query sees.  Token i of
               the n last of a sequence of len is at p = len - n + i and sees j <= p with p - j < window (or no
               window) or j < sinks
    tree       of n drafted tokens the i-th sees those in its mask, and the context j < len - n as a token at
               p = len - n + (how many of the drafted ones before it it sees) does

With `own` false, run() computes these in elementary torch operations; with
`own` true it calls the library.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _norm(name, rows, d, dtype="bf16", residual=True):
    return {"name": name, "kind": "norm", "rows": rows, "d": d, "dtype": dtype, "residual": residual}


def _cache(name, kind, tokens, kv_heads, head_dim, page, dtype="bf16", spread=1):
    return {"name": name, "kind": kind, "tokens": tokens, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
            "dtype": dtype, "spread": spread}


def _attn(name, seqs, n_q, max_len, heads=32, kv_heads=8, head_dim=128, page=64, window=0, sinks=0, dtype="bf16",
          prompts=0, prompt=0, prompt_len=0, tree=False, ragged=True, lengths=1):
    """`seqs` sequences of up to max_len keys with n_q last tokens each, and `prompts` with `prompt` last tokens."""
    return {"name": name, "kind": "attention", "seqs": seqs, "n_q": n_q, "max_len": max_len, "heads": heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "window": window, "sinks": sinks, "dtype": dtype,
            "prompts": prompts, "prompt": prompt, "prompt_len": prompt_len, "tree": tree, "ragged": ragged,
            "lengths": lengths}


def listed():
    return [
        # a decode step of 64 requests: the norm before the query, key and value projections
        _norm("norm decode", 64, 4096),
        # the same norm of 32 ragged prefill requests
        _norm("norm prefill", 16997, 4096),
        # the decode step's keys and values into a large cache, and back
        _cache("cache decode", "write", 64, 8, 128, 64, spread=64),
        # those of the ragged prefill requests
        _cache("cache prefill", "write", 16997, 8, 128, 16),
        # rows of a shared prefix fetched back, fp32, heads of no power of two
        _cache("cache read", "read", 3001, 3, 80, 32, dtype="f32", spread=3),
        # one request decodes: latency
        _attn("attention 1 request", 1, 1, 4097, ragged=False),
        # 64 requests decode at ragged lengths: the cache's bytes
        _attn("attention decode", 64, 1, 32768),
        # 256 requests far beyond the window: pages between the first tokens and the window are gone
        _attn("attention window", 256, 1, 131072, page=32, window=4096, sinks=4),
        # four prompts of 512 tokens beside 256 decoding requests
        _attn("attention mixed step", 256, 1, 8192, page=16, prompts=4, prompt=512, prompt_len=4096),
        # one long prompt: the matrix units
        _attn("attention prompt", 0, 0, 0, page=64, window=4096, sinks=4, prompts=1, prompt=16384, prompt_len=16384,
              ragged=False),
        # 32 requests verify 24 drafted tokens each
        _attn("tree", 32, 24, 16384, page=16, tree=True),
        # fp32, odd head size, a window, sequences shorter than their drafts' window
        _attn("tree odd", 7, 13, 3001, heads=12, kv_heads=3, head_dim=80, page=16, window=1000, sinks=3, dtype="f32",
              tree=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm", "write", "read", "attention", "attention", "attention", "prompt", "tree", "tree"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "norm":
        d = _log(rng, 64, 16384)
        d = max(64, d // 64 * 64) if rng.random() < 0.67 else d
        return {"kind": kind, "rows": min(_log(rng, 1, 65536), 16997 * 4096 // (d * (1 if dtype == "bf16" else 2))), "d": d,
                "dtype": dtype, "residual": rng.random() < 0.7}
    head_dim = rng.choice([32, 64, 80, 96, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if kind in ("write", "read"):
        tokens = min(_log(rng, 1, 16997), 16997 * 1024 // (kv * head_dim * (1 if dtype == "bf16" else 2)))
        return {"kind": kind, "tokens": tokens, "kv_heads": kv, "head_dim": head_dim, "page": page, "dtype": dtype,
                "spread": rng.choice([1, 2, 4])}
    window = 0 if rng.random() < 0.5 else _log(rng, 16, 8192)
    c = {"kind": "attention", "seqs": 0, "n_q": 0, "max_len": 0, "heads": kv * rng.choice([1, 3, 4, 8]), "kv_heads": kv,
         "head_dim": head_dim, "page": page, "window": window, "sinks": rng.choice([0, 1, 4, 70]) if window else 0,
         "dtype": dtype, "prompts": 0, "prompt": 0, "prompt_len": 0, "tree": kind == "tree", "ragged": True,
         "lengths": rng.randrange(1 << 30)}
    row = kv * head_dim
    if kind == "prompt":
        # no more pairs than the long prompt's
        n = _log(rng, 2, 8192)
        c.update(prompts=rng.choice([1, 2, 3, 5]), prompt=n, prompt_len=n + rng.choice([0, 1, 100, 1000]))
        while c["prompts"] * c["prompt"] * c["prompt_len"] * c["heads"] * head_dim > 16384 * 4096 * 32 * 128:
            c.update(prompts=max(1, c["prompts"] // 2), prompt=1 + c["prompt"] // 2, prompt_len=1 + c["prompt_len"] // 2)
    elif kind == "tree":
        n = rng.randint(2, 64)
        c.update(seqs=_log(rng, 1, 64), n_q=n, max_len=n + _log(rng, 1, 16384))
        c["seqs"] = max(1, min(c["seqs"], 32 * 24 * 16384 * 32 * 128 // (n * c["max_len"] * c["heads"] * head_dim * 2),
                               64 * 32768 * 1024 // (c["max_len"] * row * 2)))
    else:
        c.update(seqs=_log(rng, 1, 256), n_q=rng.choice([1, 1, 2, 5]), max_len=5 + _log(rng, 1, 65536))
        c["seqs"] = max(1, min(c["seqs"], 64 * 32768 * 1024 // (c["max_len"] * row * 2)))
        if rng.random() < 0.3:
            c.update(prompts=rng.choice([1, 3]), prompt=_log(rng, 2, 1000), prompt_len=rng.choice([1000, 1777]))
    return c


# ------------------------------------------------------------------ inputs --
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _activations(g, rows, d, dtype):
    """Normal rows of different sizes, a few channels much larger than the rest, some rows of padding zeros."""
    x = torch.randn(rows, d, generator=g, device=DEV)
    x *= torch.exp(torch.randn(rows, 1, generator=g, device=DEV) * 0.5)
    x *= 1 + 15 * (torch.rand(d, generator=g, device=DEV) < 0.005)
    if rows >= 16:
        x *= torch.rand(rows, 1, generator=g, device=DEV) > 0.03
    return x.to(dtype)


def _heads(g, tokens, heads, head_dim, dtype):
    """Heads of normal values, a few channels larger than the rest, tokens of different sizes."""
    x = torch.randn(tokens, heads, head_dim, generator=g, device=DEV)
    x *= torch.exp(torch.randn(tokens, heads, 1, generator=g, device=DEV) * 0.3)
    x *= 1 + 2 * (torch.rand(heads, head_dim, generator=g, device=DEV) < 0.03)
    return x.to(dtype)


def _pitch(head_dim):
    return (head_dim + 15) // 16 * 16


def _empty_cache(n_pages, c):
    shape = (n_pages, c["kv_heads"], c["page"])
    values = [torch.zeros(*shape, _pitch(c["head_dim"]), dtype=torch.int8, device=DEV) for _ in range(2)]
    return values + [torch.zeros(*shape, device=DEV) for _ in range(2)]


def _q8(x):
    """Rows in 8 bits and their scales; in 64 bits, since values next to a half decide whole numbers."""
    x = x.double()
    a = x.abs().amax(-1, keepdim=True)
    q = torch.round(x * 127 / torch.where(a > 0, a, 1.0))
    return q.to(torch.int8), (a[..., 0] / 127).float()


def _filled_cache(g, n_pages, c):
    """A cache whose every slot holds a token, a few pages at a time."""
    cache = _empty_cache(n_pages, c)
    hk, p, d = c["kv_heads"], c["page"], c["head_dim"]
    step = max(1, (1 << 26) // (hk * p * d))
    for lo in range(0, n_pages, step):
        n = min(step, n_pages - lo)
        for value, scale in ((cache[0], cache[2]), (cache[1], cache[3])):
            x = _heads(g, n * p, hk, d, torch.float32).view(n, p, hk, d).transpose(1, 2)
            a = x.abs().amax(-1)
            value[lo:lo + n, :, :, :d] = torch.round(x * (127 / a)[..., None]).to(torch.int8)
            scale[lo:lo + n] = a / 127
    return cache


def _groups(c):
    """The batch as (sequences, last tokens of each, lengths) of the prompts and of the others, by the case alone."""
    rng = random.Random(c["lengths"])
    pick = lambda n, hi: max(n, int(hi * math.sqrt(rng.uniform(0.02, 1)))) if c["ragged"] else hi  # noqa: E731
    got = []
    for count, n, hi in ((c["prompts"], c["prompt"], c["prompt_len"]), (c["seqs"], c["n_q"], c["max_len"])):
        if count:
            got.append((count, n, [pick(n, hi) for _ in range(count)]))
    return got


def _first_seen(c, n, length):
    """The first key beyond the sinks that a sequence's last n tokens see."""
    return min(length, max(c["sinks"], length - n - c["window"] + 1)) if c["window"] else 0


def _batch(g, c):
    """Pages in shuffled order; those that no query sees are gone (-1)."""
    groups, p = _groups(c), c["page"]
    lens = [x for _, _, ls in groups for x in ls]
    counts = [n for count, n, _ in groups for _ in range(count)]
    most = max(-(-x // p) for x in lens) + 1
    table = torch.full((len(lens), most), -1, dtype=torch.int32)
    live = torch.zeros(len(lens), most, dtype=torch.bool)
    for s, (n, x) in enumerate(zip(counts, lens)):
        live[s, :-(-min(c["sinks"], x) // p)] = c["sinks"] > 0
        live[s, _first_seen(c, n, x) // p:-(-x // p)] = True
    n_pages = int(live.sum()) + 3
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32).cpu()
    table[live] = order[:n_pages - 3]
    q_off = torch.tensor([0] + counts).cumsum(0).to(torch.int32)
    return {"lens": torch.tensor(lens, dtype=torch.int32).to(DEV), "q_off": q_off.to(DEV), "table": table.to(DEV),
            "tokens": sum(counts), "max_q": max(counts), "n_pages": n_pages}


def _trees(g, c):
    """For each drafted token the tokens that it sees: itself and what its parent sees; parents lie before their children."""
    n, s = c["n_q"], c["seqs"]
    back = torch.randint(1, 4, (s, n), generator=g, device=DEV).cpu().tolist()
    masks = []
    for row in back:
        m = []
        for i in range(n):
            m.append((m[max(0, i - row[i])] if i else 0) | 1 << i)
        masks += m
    return torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64).to(DEV)


def _inputs(c, seed):
    g, t = _gen(seed), TYPES[c["dtype"]]
    if c["kind"] == "norm":
        s = {"x": _activations(g, c["rows"], c["d"], t), "w": 1 + 0.2 * torch.randn(c["d"], generator=g, device=DEV)}
        s["r"] = _activations(g, c["rows"], c["d"], t) if c["residual"] else None
        return s
    if c["kind"] in ("write", "read"):
        n_pages = -(-c["tokens"] * c["spread"] // c["page"]) + 1
        slots = torch.randperm(n_pages * c["page"], generator=g, device=DEV)[:c["tokens"]].to(torch.int32)
        if c["spread"] == 1:
            # whole pages in order
            slots = slots.sort().values
        if c["kind"] == "read":
            return {"slots": slots, "cache": _filled_cache(g, n_pages, c)}
        k, v = (_heads(g, c["tokens"], c["kv_heads"], c["head_dim"], t) for _ in range(2))
        return {"slots": slots, "k": k, "v": v, "cache": _empty_cache(n_pages, c)}
    s = _batch(g, c)
    s["q"] = (1.5 * _heads(g, s["tokens"], c["heads"], c["head_dim"], torch.float32)).to(t)
    s["cache"] = _filled_cache(g, s["n_pages"], c)
    s["tree"] = _trees(g, c) if c["tree"] else None
    return s


EPS = 1e-5


def prepare(case, seed):
    c, s = case, _inputs(case, seed)
    s["case"] = c
    t = TYPES[c["dtype"]]
    if c["kind"] == "norm":
        s["y"] = torch.empty_like(s["x"])
        s["sum"] = torch.empty_like(s["x"]) if c["residual"] else None
        s["q8"] = torch.empty(c["rows"], c["d"], dtype=torch.int8, device=DEV)
        s["scale"] = torch.empty(c["rows"], device=DEV)
    elif c["kind"] in ("write", "read"):
        s["back"] = [torch.empty(c["tokens"], c["kv_heads"], c["head_dim"], dtype=t, device=DEV) for _ in range(2)]
    else:
        s["out"] = torch.empty_like(s["q"])
    if own:
        # the handles that a serving program keeps for a layer; the plan serves every layer of a step
        import rank_sgmv_bgmv_amd as L
        if c["kind"] == "norm":
            s["norm"] = L.Norm(s["w"], EPS)
        else:
            s["handle"] = L.Cache(*s["cache"], head_dim=c["head_dim"])
        if c["kind"] == "attention":
            s["attention"] = L.Attention(c["heads"], c["head_dim"] ** -0.5, window=c["window"], sinks=c["sinks"], dtype=t)
            s["batch"] = L.AttentionBatch(s["tokens"], s["q_off"], s["lens"], s["table"], max_q=s["max_q"], tree=s["tree"])
            s["plan"] = L.new_attention_plan(s["attention"], s["handle"], s["batch"])
            L.lora_attention_plan(s["attention"], s["handle"], s["batch"], s["plan"])
            s["ws"] = L.new_attention_workspace(s["attention"], s["handle"], s["batch"])
    return s


# ------------------------------------------------------------------ passes --
def _plain_norm(x, r, w, dtype):
    h = x if r is None else (x.float() + r.float()).to(dtype)
    v = h.double()
    y = (v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * w.double()).to(dtype)
    q, scale = _q8(y)
    got = (y, q * scale[:, None], scale)
    return got if r is None else (h, *got)


def _plain_put(x, value, scale, page, at):
    q, a = _q8(x)
    value[page, :, at, :x.shape[2]] = q
    scale[page, :, at] = a


def _plain_write(s, c):
    page, at = (s["slots"] // c["page"]).long(), (s["slots"] % c["page"]).long()
    _plain_put(s["k"], s["cache"][0], s["cache"][2], page, at)
    _plain_put(s["v"], s["cache"][1], s["cache"][3], page, at)


def _plain_read(s, c):
    page, at = (s["slots"] // c["page"]).long(), (s["slots"] % c["page"]).long()
    read = lambda value, scale: (value[page, :, at, :c["head_dim"]].float() * scale[page, :, at][..., None]).to(  # noqa: E731
        TYPES[c["dtype"]])
    return read(s["cache"][0], s["cache"][2]), read(s["cache"][1], s["cache"][3])


def _plain_group(s, c, first, token, count, n, lengths):
    """Sequences first .. first + count with n last tokens each: a padded batch over every key that one of them sees."""
    p, d, hk = c["page"], c["head_dim"], c["kv_heads"]
    lo = [_first_seen(c, n, x) for x in lengths]
    sinks = c["sinks"]
    wide = max(x - y for x, y in zip(lengths, lo))
    lens = s["lens"][first:first + count].long()[:, None]
    j = torch.tensor(lo, device=DEV)[:, None] + torch.arange(wide, device=DEV)
    there = j < lens
    if sinks:
        j = torch.cat([torch.arange(sinks, device=DEV).expand(count, -1), j], 1)
        there = torch.cat([j[:, :sinks] < lens, there & (j[:, sinks:] >= sinks)], 1)
    j = torch.where(there, j, 0)
    page = s["table"][first:first + count].long().gather(1, j // p).clamp(min=0)
    fetch = lambda value, scale: (value[page, :, j % p, :d].float() * scale[page, :, j % p][..., None]).transpose(1, 2)  # noqa: E731
    k, v = fetch(s["cache"][0], s["cache"][2]), fetch(s["cache"][1], s["cache"][3]).contiguous()
    q = s["q"][token:token + count * n].view(count, n, hk, -1, d).permute(0, 2, 1, 3, 4).reshape(count, hk, -1, d).float()
    scores = torch.matmul(q, k.transpose(2, 3).contiguous()) * d ** -0.5
    j, there = j[:, None, :], there[:, None, :]
    i = torch.arange(n, device=DEV)
    context = lens[:, :, None] - n
    pos = context + i[:, None]
    seen = j <= pos
    if c["tree"]:
        mask = s["tree"].view(count, n)[..., None]
        before = (mask >> i & 1) * (i < i[:, None])
        pos = context + before.sum(-1, keepdim=True)
        draft = (mask >> (j - context).clamp(min=0) & 1).bool()
        seen = torch.where(j < context, j <= pos, draft)
    if c["window"]:
        near = (pos - j < c["window"]) | (j < sinks)
        seen = seen & (near | (j >= context) if c["tree"] else near)
    seen = (seen & there)[:, None, :, None, :].expand(count, hk, n, q.shape[2] // n, -1).reshape(scores.shape)
    scores = torch.where(seen, scores, -math.inf)
    e = torch.exp(scores - scores.amax(-1, keepdim=True).clamp(min=-1e30))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(total > 0, total, 1.0)
    return o.view(count, hk, n, -1, d).permute(0, 2, 1, 3, 4).reshape(count * n, -1, d)


def _plain_attention(s, c):
    groups = _groups(c)
    # (sequences and tokens before each group)
    starts = [(0, 0), (groups[0][0], groups[0][0] * groups[0][1])]
    return torch.cat([_plain_group(s, c, *at, *g) for at, g in zip(starts, groups)]).to(TYPES[c["dtype"]])


def run(state):
    s, c = state, state["case"]
    kind = c["kind"]
    if own:
        import rank_sgmv_bgmv_amd as L
        if kind == "norm":
            L.lora_norm_apply(s["norm"], s["x"], y=s["y"], q=s["q8"], scale=s["scale"], residual=s["r"], total=s["sum"])
            got = (s["y"], s["q8"] * s["scale"][:, None], s["scale"])
            return got if s["r"] is None else (s["sum"], *got)
        if kind == "attention":
            L.lora_attention_apply(s["attention"], s["handle"], s["batch"], s["plan"], s["q"], s["out"], s["ws"])
            return s["out"]
        if kind == "write":
            L.lora_cache_write(s["handle"], s["slots"], s["k"], s["v"])
        L.lora_cache_read(s["handle"], s["slots"], s["back"][0], s["back"][1])
        return s["back"]
    if kind == "norm":
        return _plain_norm(s["x"], s["r"], s["w"], TYPES[c["dtype"]])
    if kind == "attention":
        return _plain_attention(s, c)
    if kind == "write":
        _plain_write(s, c)
    return list(_plain_read(s, c))


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["kind"] == "norm":
        n = c["rows"] * c["d"]
        return {"bytes": n * (e * (4 if c["residual"] else 2) + 1) + 4 * c["rows"] + 4 * c["d"], "flops": 8 * n}
    row = c["kv_heads"] * c["head_dim"]
    if c["kind"] in ("write", "read"):
        one = 2 * row * e + 2 * (row + 4 * c["kv_heads"]) + 4
        return {"bytes": c["tokens"] * one * (2 if c["kind"] == "write" else 1), "flops": 4 * c["tokens"] * row}
    keys = pairs = tokens = 0
    for count, n, lengths in _groups(c):
        tokens += count * n
        for x in lengths:
            w, sinks = c["window"] or x, c["sinks"]
            lo = _first_seen(c, n, x)
            keys += x - lo + min(sinks, lo)
            for p in range(x - n, x):
                # (a drafted token counts the keys that it would see in a plain sequence)
                pairs += min(p + 1, w) + min(sinks, max(0, p + 1 - w))
    return {"bytes": 2 * keys * (row + 4 * c["kv_heads"]) + 2 * tokens * c["heads"] * c["head_dim"] * e,
            "flops": 4 * pairs * c["heads"] * c["head_dim"]}


# ------------------------------------------------------------------- exact --
def _exact_rows(x):
    top = torch.maximum(x.max(dim=-1).values, -x.min(dim=-1).values).unsqueeze(-1)
    t = 127.0 * x / torch.where(top == 0, 1.0, top)
    low = torch.floor(t)
    part = t - low
    # the nearest whole number, the even one of two that are as near
    up = (part > 0.5) | ((part == 0.5) & (low.remainder(2) == 1))
    return low + up, top / 127.0


def exact(case, seed):
    """From the definitions, in 64 bits."""
    c, s = case, _inputs(case, seed)
    t = TYPES[c["dtype"]]
    if c["kind"] == "norm":
        h = s["x"].double()
        if s["r"] is not None:
            h = h + s["r"].double()
        # (the norm is one of the sum as it is kept, the 8-bit values are those of y as it is kept)
        kept = h.to(t).double()
        size = torch.sqrt(kept.square().sum(1) / c["d"] + EPS)
        y = kept * s["w"].double() / size.unsqueeze(1)
        q, scale = _exact_rows(y.to(t).double())
        got = (y, q * scale, scale[:, 0])
        return got if s["r"] is None else (h, *got)
    if c["kind"] in ("write", "read"):
        if c["kind"] == "write":
            pairs = [_exact_rows(x.double()) for x in (s["k"], s["v"])]
            return [q * a for q, a in pairs]
        at = s["slots"].long()
        flat = lambda x: x.transpose(1, 2).flatten(0, 1)[at].double()  # noqa: E731
        return [flat(s["cache"][i])[..., :c["head_dim"]] * flat(s["cache"][i + 2]).unsqueeze(-1) for i in (0, 1)]
    if sum(count * n * n * (1 + max(ls) // n) for count, n, ls in _groups(c)) * c["heads"] * c["head_dim"] > 1 << 46:
        return None
    # sequence after sequence and head after head
    d, p, group = c["head_dim"], c["page"], c["heads"] // c["kv_heads"]
    out = torch.zeros(s["tokens"], c["heads"], d, dtype=torch.float64, device=DEV)
    offsets, lens = s["q_off"].tolist(), s["lens"].tolist()
    for b, length in enumerate(lens):
        lo, n = offsets[b], offsets[b + 1] - offsets[b]
        start = _first_seen(c, n, length)
        keys = [j for j in range(min(c["sinks"], start))] + list(range(start, length))
        at = torch.tensor(keys, device=DEV)
        slot = s["table"][b].long()[at // p] * p + at % p
        distance = torch.arange(length - n, length, device=DEV).unsqueeze(1) - at
        allowed = distance >= 0
        if c["tree"]:
            bits = torch.tensor([[(m >> i) & 1 for i in range(n)] for m in s["tree"][lo:lo + n].tolist()], device=DEV)
            depth = torch.tril(bits, -1).sum(1, keepdim=True)
            distance = (length - n + depth) - at
            allowed = torch.ones_like(distance, dtype=torch.bool)
        if c["window"]:
            allowed = allowed & ((distance < c["window"]) | (at < c["sinks"]))
        if c["tree"]:
            drafted = at >= length - n
            allowed[:, drafted] = bits[:, at[drafted] - (length - n)].bool()
        for h in range(c["kv_heads"]):
            flat = lambda i: s["cache"][i][:, h].flatten(0, 1)[slot].double()  # noqa: E731
            k, v = flat(0)[:, :d] * flat(2).unsqueeze(1), flat(1)[:, :d] * flat(3).unsqueeze(1)
            for r in range(group):
                x = s["q"][lo:lo + n, h * group + r].double() @ k.t() / math.sqrt(d)
                x = torch.softmax(x.masked_fill(~allowed, -math.inf), dim=1)
                out[lo:lo + n, h * group + r] = torch.nan_to_num(x, nan=0.0) @ v
    return out
