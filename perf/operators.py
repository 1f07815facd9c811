"""The base product, row quantisation and rotary positions around a LoRA layer: cases, plain forms, calls.

A LoRA layer adds its low-rank products to y = x W^T of the shared base model.
The cases here are what stands around that step: rows quantised to 8 bits, the
8-bit base product with a scale for each token and channel, both in one call,
and the rotation of q and k by their positions.

    quantise   a = max |x[t]|, s[t] = a / 127, q[t][c] = rint(127 x[t][c] / a), ties to even; zeros for a = 0
    product    y[t][o] = s_x[t] s_w[o] sum_c q[t][c] W[o][c] (+ bias[o])
    apply      product(quantise(x))
    rotary     pair (a, b) of a head at position p: m (a cos p f - b sin p f), m (b cos p f + a sin p f)

With `own` false, run() computes these in elementary torch operations; with
`own` true it calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gemm(name, kind, rows, d_in, d_out, dtype="bf16", bias=False):
    return {"name": name, "kind": kind, "rows": rows, "d_in": d_in, "d_out": d_out, "dtype": dtype, "bias": bias}


def _rot(name, rows, heads, kv_heads, head_dim, rot_dim, dtype="bf16", interleaved=False, heads_first=False,
         inverse=False, max_pos=8192, factor=1.0, mscale=1.0):
    return {"name": name, "kind": "rotary", "rows": rows, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "rot_dim": rot_dim, "dtype": dtype, "interleaved": interleaved, "heads_first": heads_first,
            "inverse": inverse, "max_pos": max_pos, "factor": factor, "mscale": mscale}


def listed():
    return [
        # one request decodes: its key projection, where latency counts
        _gemm("product 1 row", "product", 1, 4096, 1024),
        # a decode step of 64 requests through the widest projection: the weights' bytes
        _gemm("product decode", "product", 64, 4096, 14336),
        # four prefill requests of 512 tokens beside 256 decoding ones, the down projection
        _gemm("product mixed step", "product", 2304, 14336, 4096),
        # 32 ragged prefill requests: the matrix rate
        _gemm("product prefill", "product", 16997, 4096, 4096),
        # no size is a multiple of anything, fp32 out, with a bias
        _gemm("product odd", "product", 777, 1001, 1283, dtype="f32", bias=True),
        # the decode step's query projection from bf16 activations
        _gemm("apply decode", "apply", 64, 4096, 4096),
        # 16 images of 4096 positions through one attention projection of a diffusion model
        _gemm("apply diffusion", "apply", 65536, 1280, 1280, bias=True),
        # the activations of a decode step, quantised once for query, key and value
        {"name": "quantise decode", "kind": "quantise", "rows": 64, "d_in": 4096, "dtype": "bf16"},
        # a weight quantised when the model is loaded
        {"name": "quantise weight", "kind": "quantise", "rows": 4096, "d_in": 14336, "dtype": "f32"},
        # query and key heads of a decode step, far positions
        _rot("rotary decode", 64, 32, 8, 128, 128, max_pos=131072, factor=8.0),
        # the same heads of 32 ragged prefill requests
        _rot("rotary prefill", 16997, 32, 8, 128, 128),
        # part of the head, neighbouring pairs, heads first, fp32, the gradient's direction
        _rot("rotary part", 3001, 12, 3, 80, 34, dtype="f32", interleaved=True, heads_first=True, inverse=True,
             max_pos=1000000, factor=4.0, mscale=1.2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["product", "product", "apply", "quantise", "rotary", "rotary"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    # two sizes of three are whole 64s, the others anything
    size = lambda lo, hi: max(lo, _log(rng, lo, hi) // 64 * 64) if rng.random() < 0.67 else _log(rng, lo, hi)  # noqa: E731
    if kind == "rotary":
        head_dim = rng.choice([32, 64, 80, 96, 128, 256])
        rot_dim = head_dim if rng.random() < 0.6 else 2 * rng.randint(1, head_dim // 2)
        kv = rng.choice([1, 2, 4, 8])
        c = {"kind": kind, "rows": _log(rng, 1, 16997), "heads": kv * rng.choice([1, 3, 4, 5]), "kv_heads": kv,
             "head_dim": head_dim, "rot_dim": rot_dim, "dtype": dtype, "interleaved": rng.random() < 0.4,
             "heads_first": rng.random() < 0.3, "inverse": rng.random() < 0.25,
             "max_pos": _log(rng, 16, 2000000), "factor": rng.choice([1.0, 2.0, 8.0]),
             "mscale": rng.choice([1.0, 1.25])}
        c["rows"] = min(c["rows"], 16997 * 5120 // ((c["heads"] + kv) * head_dim))
        return c
    if kind == "quantise":
        d = size(64, 16384)
        return {"kind": kind, "rows": min(_log(rng, 1, 65536), 4096 * 14336 // d), "d_in": d, "dtype": dtype}
    d_in, d_out = size(64, 14336), size(64, 14336)
    rows = min(_log(rng, 1, 65536), 16997 * 4096 * 4096 // (d_in * d_out), 65536 * 1280 // max(d_in, d_out))
    return {"kind": kind, "rows": max(1, rows), "d_in": d_in, "d_out": d_out, "dtype": dtype,
            "bias": rng.random() < 0.4}


# ------------------------------------------------------------------ inputs --
def _activations(g, rows, d, dtype):
    """Normal rows of different sizes, a few channels much larger than the rest, some rows of padding zeros."""
    x = torch.randn(rows, d, generator=g, device=DEV)
    x *= torch.exp(torch.randn(rows, 1, generator=g, device=DEV) * 0.5)
    x *= 1 + 15 * (torch.rand(d, generator=g, device=DEV) < 0.005)
    if rows >= 16:
        x *= torch.rand(rows, 1, generator=g, device=DEV) > 0.03
    return x.to(dtype)


def _q8(x):
    """Rows in 8 bits and their scales; in 64 bits, since values next to a half decide whole numbers."""
    x = x.double()
    a = x.abs().amax(1, keepdim=True)
    q = torch.round(x * 127 / torch.where(a > 0, a, 1.0))
    return q.to(torch.int8), (a[:, 0] / 127).float()


def _inputs(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    t = TYPES[c["dtype"]]
    if c["kind"] == "rotary":
        shape = lambda h: (h, c["rows"], c["head_dim"]) if c["heads_first"] else (c["rows"], h, c["head_dim"])  # noqa: E731
        x = [torch.randn(shape(h), generator=g, device=DEV).to(t) for h in (c["heads"], c["kv_heads"])]
        if c["heads_first"]:
            x = [v.transpose(0, 1) for v in x]
        pos = torch.randint(0, c["max_pos"], (c["rows"],), generator=g, device=DEV, dtype=torch.int32)
        j = torch.arange(c["rot_dim"] // 2, dtype=torch.float64)
        freq = torch.pow(10000.0, -2 * j / c["rot_dim"]) / c["factor"]
        return {"x": x, "pos": pos, "freq": freq.to(DEV)}
    if c["kind"] == "quantise":
        return {"x": _activations(g, c["rows"], c["d_in"], t)}
    x = _activations(g, c["rows"], c["d_in"], t)
    wq, ws = _q8(torch.randn(c["d_out"], c["d_in"], generator=g, device=DEV) * 0.02)
    bias = torch.randn(c["d_out"], generator=g, device=DEV) * 0.1 if c["bias"] else None
    s = {"wq": wq, "ws": ws, "bias": bias}
    if c["kind"] == "product":
        s["xq"], s["xs"] = _q8(x)
    else:
        s["x"] = x
    return s


def prepare(case, seed):
    c, s = case, _inputs(case, seed)
    s["case"] = c
    t = TYPES[c["dtype"]]
    if c["kind"] == "rotary":
        s["out"] = [torch.empty_like(v) for v in s["x"]]
    elif c["kind"] == "quantise":
        s["q"] = torch.empty(c["rows"], c["d_in"], dtype=torch.int8, device=DEV)
        s["scale"] = torch.empty(c["rows"], dtype=torch.float32, device=DEV)
    else:
        s["y"] = torch.empty(c["rows"], c["d_out"], dtype=t, device=DEV)
    if own:
        # the handles and the workspace that a serving program keeps for a layer
        import rank_sgmv_bgmv_amd as L
        if c["kind"] == "rotary":
            s["rotary"] = L.Rotary(s["freq"], c["head_dim"], interleaved=c["interleaved"], mscale=c["mscale"])
        elif c["kind"] != "quantise":
            s["weight"] = L.BaseWeight(s["wq"], s["ws"], s["bias"])
            if c["kind"] == "apply":
                s["ws8"] = L.new_base_workspace(s["weight"], c["rows"])
    return s


# ------------------------------------------------------------------ passes --
def _plain_product(xq, xs, wq, ws, bias, dtype):
    y = (xq.float() @ wq.float().T) * xs[:, None] * ws
    return (y if bias is None else y + bias).to(dtype)


def _plain_rotary(x, pos, freq, interleaved, inverse, mscale):
    rot = 2 * freq.numel()
    angle = pos.double()[:, None, None] * freq
    cos, sin = (torch.cos(angle) * mscale).float(), (torch.sin(angle) * mscale).float()
    if inverse:
        sin = -sin
    v = x.float()
    y = v.clone()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = v[..., first], v[..., second]
    y[..., first] = a * cos - b * sin
    y[..., second] = b * cos + a * sin
    return y.to(x.dtype)


def run(state):
    s, c = state, state["case"]
    kind = c["kind"]
    if own:
        import rank_sgmv_bgmv_amd as L
        if kind == "product":
            L.lora_base_product(s["weight"], s["xq"], s["xs"], s["y"])
            return s["y"]
        if kind == "apply":
            L.lora_base_apply(s["weight"], s["x"], s["y"], s["ws8"])
            return s["y"]
        if kind == "quantise":
            L.lora_quantize_rows(s["x"], s["q"], s["scale"])
            return s["q"] * s["scale"][:, None], s["scale"]
        L.lora_rotary_apply(s["rotary"], s["pos"], s["x"], s["out"], inverse=c["inverse"])
        return s["out"]
    if kind == "product":
        return _plain_product(s["xq"], s["xs"], s["wq"], s["ws"], s["bias"], TYPES[c["dtype"]])
    if kind == "apply":
        q, scale = _q8(s["x"])
        return _plain_product(q, scale, s["wq"], s["ws"], s["bias"], TYPES[c["dtype"]])
    if kind == "quantise":
        q, scale = _q8(s["x"])
        return q * scale[:, None], scale
    return [_plain_rotary(x, s["pos"], s["freq"], c["interleaved"], c["inverse"], c["mscale"]) for x in s["x"]]


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["kind"] == "rotary":
        values = c["rows"] * (c["heads"] + c["kv_heads"])
        return {"bytes": 2 * values * c["head_dim"] * e + 4 * c["rows"], "flops": 3 * values * c["rot_dim"]}
    n, d = c["rows"], c["d_in"]
    if c["kind"] == "quantise":
        return {"bytes": n * d * (e + 1) + 4 * n, "flops": 3 * n * d}
    m = c["d_out"]
    x = n * d + 4 * n if c["kind"] == "product" else n * d * e
    return {"bytes": x + m * d + 4 * m * (2 if c["bias"] else 1) + n * m * e, "flops": 2 * n * m * d}


# ------------------------------------------------------------------- exact --
def exact(case, seed):
    """From the definitions, in 64 bits."""
    c, s = case, _inputs(case, seed)
    if c["kind"] == "rotary":
        # a rotation by an angle is a product with e^(i angle), here m e^(i angle) or m e^(-i angle)
        turn = s["pos"].to(torch.float64).reshape(-1, 1, 1) * s["freq"].reshape(1, 1, -1) * (-1 if c["inverse"] else 1)
        turn = torch.polar(torch.full_like(turn, c["mscale"]), turn)
        got = []
        for x in s["x"]:
            head, rest = x.double().split([c["rot_dim"], c["head_dim"] - c["rot_dim"]], dim=-1)
            n, h, r = head.shape
            pairs = head.reshape(n, h, r // 2, 2) if c["interleaved"] else head.reshape(n, h, 2, r // 2).transpose(2, 3)
            pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            head = (pairs if c["interleaved"] else pairs.transpose(2, 3)).reshape(n, h, r)
            got.append(torch.cat([head, rest], dim=-1))
        return got
    if c["kind"] == "product":
        xq, xs = s["xq"].double(), s["xs"].double()
    else:
        x = s["x"].to(torch.float64)
        top = torch.maximum(x.max(dim=1).values, -x.min(dim=1).values)
        xs = top / 127.0
        t = 127.0 * x / torch.where(top == 0, 1.0, top).unsqueeze(1)
        low = torch.floor(t)
        part = t - low
        # the nearest whole number, the even one of two that are as near
        up = (part > 0.5) | ((part == 0.5) & (low.remainder(2) == 1))
        xq = low + up
    if c["kind"] == "quantise":
        return xq * xs.unsqueeze(1), xs
    w = s["wq"].double() * s["ws"].double().unsqueeze(1)
    y = torch.matmul(xq * xs.unsqueeze(1), w.t())
    return y if s["bias"] is None else y.add(s["bias"].double())
