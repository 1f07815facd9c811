"""The norm, the 8-bit cache and attention over it (include/lora_layer.h)
against plain implementations in 64 bits.

Tolerances, with u = eps / 2 of the output's type, v = 2^-24 (a float32 rounding) and h = 2^-11 (a float16 one):
  norm       total is one rounding: equal.  y is float64 rounded through float32 to its type: u |y| + v |y| (and to
             bfloat16 through float32 a tie may go the other way, which is the same u).  q and scale are those of the
             kernel's own y: equal
  cache      equal
  attention  with p the exact weights, A = sum p |v| and o the exact output, to first order in the errors:
             a score off by s moves the output by sum p s |v - o|.  Scores are float32 sums of D products with scales and
             a maximum taken off: s <= (D + 8) 2v S, S = scale sum |q k|, and 4 v (|score| + |largest score|) more; in
             bfloat16 calls of many rows K is rounded to float16: h S more.
             A weight in float16 is off by h (two of them, in float32 calls, by h^2), its value too where it is rounded
             to float16 (many rows, bfloat16), exp2 and scales by 8 v.  Where the sum takes the rounded weights (many
             rows, bfloat16) theirs move the output by sum p h |v - o|, which is no more than h (A + |o|).
             The sums over n keys are off by 2 v n A.  Then u |o|.  All times 1.05, for what is not first order (s < 0.03).
"""
import math

import pytest
import torch

import rank_sgmv_bgmv_amd as L
from test_gpu_base import ref_quantize

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
V, H = 2.0 ** -24, 2.0 ** -11
TYPES = [torch.bfloat16, torch.float32]
ids = {torch.bfloat16: "bf16", torch.float32: "f32"}.get


def half(t):
    return torch.finfo(t).eps / 2


def gen(seed):
    return torch.Generator().manual_seed(seed)


def bits(t):
    return t.view({1: torch.int8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def same(a, b):
    return torch.equal(bits(a.contiguous()), bits(b.contiguous()))


# ---------------------------------------------------------------------- norm --
def place(t, pad=0, off=0, fill=7):
    """t on the device as rows of a wider buffer that begins elsewhere; returns the buffer and the view."""
    T, d = t.shape
    buf = torch.full((off + (T + 1) * (d + pad),), fill, dtype=t.dtype, device=DEV)
    v = buf[off:off + T * (d + pad)].view(T, d + pad)[:, :d]
    v.copy_(t)
    return buf, v


def check_norm(T, d, dtype, residual=True, pad=0, off=0, eps=1e-5, x=None, want=("y", "q", "total")):
    g = gen(T * 31 + d)
    x = (torch.randn(T, d, generator=g) * 2).to(dtype) if x is None else x
    r = torch.randn(T, d, generator=g).to(dtype) if residual else None
    w = 1 + 0.3 * torch.randn(d, generator=g)
    norm = L.Norm(w.to(DEV), eps)
    _, xv = place(x, pad, off)
    rv = place(r, pad, off)[1] if residual else None
    bufs = {n: place(torch.full((T, d), 7).to(t), pad, off) for n, t in (("total", dtype), ("y", dtype), ("q", torch.int8))}
    tv, yv, qv = (bufs[n][1] if n in want else None for n in ("total", "y", "q"))
    if not residual:
        tv = None
    s = torch.full((T + 2,), -5.0, device=DEV)
    L.lora_norm_apply(norm, xv, y=yv, q=qv, scale=None if qv is None else s[1:T + 1], residual=rv, total=tv)
    h = x if r is None else (x.float() + r.float()).to(dtype)
    if tv is not None:
        assert same(tv.cpu(), h)
    hd = h.double()
    ref = hd * w.double() / torch.sqrt((hd * hd).mean(1, keepdim=True) + eps)
    if yv is not None:
        y = yv.cpu()
        ok = (y.double() - ref).abs() <= (half(dtype) + V) * ref.abs() + torch.finfo(dtype).tiny * half(dtype)
        assert bool((ok | (ref.isnan() & y.isnan())).all())
        if qv is not None:
            q, scale = ref_quantize(y)
            assert torch.equal(qv.cpu(), q)
            assert same(s.cpu()[1:T + 1][~scale.isnan()], scale[~scale.isnan()])
            assert torch.equal(s.cpu()[1:T + 1].isnan(), scale.isnan())
    assert s[0] == -5 and s[-1] == -5
    for n, (buf, view) in bufs.items():
        view.fill_(7)
        assert bool((buf == 7).all()), n
    return qv, s


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("T, d", [(1, 1), (1, 4096), (3, 7), (2, 8), (5, 63), (7, 65), (64, 4096), (65, 1001), (130, 256),
                                  (9, 1280), (4, 14336), (3, 16387), (2, 40001), (2, 65536), (700, 512), (33, 2048),
                                  (300, 31)])
def test_norm(T, d, dtype):
    check_norm(T, d, dtype)
    check_norm(T, d, dtype, residual=False)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("pad, off", [(1, 0), (8, 0), (16, 16), (0, 1), (3, 5)])
def test_norm_strides_and_alignment(dtype, pad, off):
    for T, d in ((5, 512), (3, 4099), (70, 48)):
        check_norm(T, d, dtype, pad=pad, off=off)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_norm_outputs_that_are_asked_for(dtype):
    """Any of the outputs may be missing; the others keep their bits."""
    g = gen(9)
    x, r = (torch.randn(37, 1000, generator=g).to(dtype).to(DEV) for _ in range(2))
    norm = L.Norm(torch.rand(1000, generator=g).to(DEV) + 0.5, 1e-6)
    mk = lambda t=dtype: torch.empty(37, 1000, dtype=t, device=DEV)  # noqa: E731
    y, q, s, tot = mk(), mk(torch.int8), torch.empty(37, device=DEV), mk()
    L.lora_norm_apply(norm, x, y=y, q=q, scale=s, residual=r, total=tot)
    y2, q2, s2, t2 = mk(), mk(torch.int8), torch.empty(37, device=DEV), mk()
    L.lora_norm_apply(norm, x, y=y2, residual=r)
    L.lora_norm_apply(norm, x, q=q2, scale=s2, residual=r, total=t2)
    assert same(y, y2) and same(q, q2) and same(s, s2) and same(tot, t2)
    # the norm of the kept total, without a residual
    y3 = mk()
    L.lora_norm_apply(norm, tot, y=y3)
    assert same(y, y3)
    # what the separate call makes of y
    q3, s3 = mk(torch.int8), torch.empty(37, device=DEV)
    L.lora_quantize_rows(y, q3, s3)
    assert same(q, q3) and same(s, s3)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("d", [64, 1000, 5000, 65536])
def test_norm_in_place(d, dtype):
    g = gen(d)
    x, r = (torch.randn(9, d, generator=g).to(dtype).to(DEV) for _ in range(2))
    norm = L.Norm(torch.rand(d, generator=g).to(DEV) + 0.5, 1e-5)
    y, tot = torch.empty_like(x), torch.empty_like(x)
    L.lora_norm_apply(norm, x, y=y, residual=r, total=tot)
    a, b = x.clone(), r.clone()
    L.lora_norm_apply(norm, a, y=a, residual=b, total=b)
    assert same(a, y) and same(b, tot)
    a, y2 = x.clone(), torch.empty_like(x)
    L.lora_norm_apply(norm, a, y=y2, residual=r, total=a)
    assert same(a, tot) and same(y2, y)


def test_norm_of_a_row_does_not_depend_on_the_others():
    g = gen(4)
    x = torch.randn(300, 1280, generator=g).to(torch.bfloat16).to(DEV)
    norm = L.Norm(torch.ones(1280, device=DEV), 1e-5)
    y = torch.empty_like(x)
    L.lora_norm_apply(norm, x, y=y)
    for lo, n in ((0, 1), (17, 5), (200, 100)):
        part = torch.empty(n, 1280, dtype=torch.bfloat16, device=DEV)
        L.lora_norm_apply(norm, x[lo:lo + n], y=part)
        assert same(part, y[lo:lo + n])


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_norm_extremes(dtype):
    """Zero rows, tiny and huge ones, rows with an infinity or NaN: no row meets another."""
    x = torch.randn(8, 300, generator=gen(1))
    x[0] = 0
    x[1] *= 1e-30
    x[2] *= 1e37
    x[3, 17] = float("inf")
    x[4, 299] = float("nan")
    x[5] = -0.0
    x = x.to(dtype)
    q, s = check_norm(8, 300, dtype, residual=False, x=x)
    assert torch.equal(s.cpu()[1:9].isnan(), torch.tensor([False, False, False, True, True, False, False, False]))
    check_norm(8, 300, dtype, residual=False, x=x, eps=0.0)


def test_norm_more_rows_than_workgroups():
    T, d = 270001, 8
    x = torch.randn(T, d, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    y = torch.empty_like(x)
    L.lora_norm_apply(L.Norm(torch.ones(d, device=DEV), 0.0), x, y=y)
    xd = x.double()
    ref = xd / torch.sqrt((xd * xd).mean(1, keepdim=True))
    assert bool(((y.double() - ref).abs() <= 2 * V * ref.abs()).all())


# --------------------------------------------------------------------- cache --
def blank_cache(n_pages, heads, page, d, gap=0, fill=55):
    """A cache whose pages lie in wider rows, with bytes that are to stay; returns it and the buffers."""
    pitch = L.lora_cache_pitch(d)
    wide = heads * page * pitch
    raw = torch.full((n_pages, 2 * wide + 16 * gap), fill, dtype=torch.int8, device=DEV)
    k, v = (raw[:, i * wide:(i + 1) * wide].view(n_pages, heads, page, pitch) for i in (0, 1))
    raws = torch.full((n_pages, 2 * heads * page + 4 * gap), -3.0, device=DEV)
    ks, vs = (raws[:, i * heads * page:(i + 1) * heads * page].view(n_pages, heads, page) for i in (0, 1))
    return L.Cache(k, v, ks, vs, d), raw, raws


def rows_of(t, seed, dtype, heads_first=False, pad=0, off=0):
    """Heads [T][heads][d] on the device, as a view with strides of its own."""
    T, h, d = t.shape
    shape = (h, T, d + pad) if heads_first else (T, h, d + pad)
    buf = torch.full((off + T * h * (d + pad) + 8,), 3.0, dtype=dtype, device=DEV)
    v = buf[off:off + T * h * (d + pad)].view(shape)[..., :d]
    v = v.transpose(0, 1) if heads_first else v
    v.copy_(t)
    return buf, v


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("T, heads, d, page", [(1, 1, 1, 16), (1, 8, 128, 16), (5, 3, 80, 32), (64, 8, 128, 64), (3, 2, 33, 16),
                                               (40, 1, 256, 128), (130, 5, 64, 16), (7, 2, 96, 1024), (9, 1, 15, 16),
                                               (17, 2, 17, 16), (1000, 2, 32, 256)])
def test_cache_write_and_read(T, heads, d, page, dtype):
    g = gen(T + d)
    n_pages = 2 * (T // page) + 3
    cache, raw, raws = blank_cache(n_pages, heads, page, d, gap=3)
    slots = torch.randperm(n_pages * page, generator=g)[:T].to(torch.int32)
    skip = torch.rand(T, generator=g) < (0.2 if T > 2 else 0)
    named = slots.clone()
    named[skip] = torch.tensor([-1, n_pages * page, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)[torch.arange(int(skip.sum())) % 4]
    x = [(torch.randn(T, heads, d, generator=g) * 3).to(dtype) for _ in range(2)]
    x[0][T // 2] = 0
    views = [rows_of(t, 0, dtype, heads_first=i == 1, pad=i, off=i)[1] for i, t in enumerate(x)]
    L.lora_cache_write(cache, named.to(DEV), *views)
    live = ~skip
    want = torch.full_like(raw.cpu(), 55), torch.full_like(raws.cpu(), -3.0)
    pitch, wide = L.lora_cache_pitch(d), heads * page * L.lora_cache_pitch(d)
    p, a = (slots // page).long()[live], (slots % page).long()[live]
    for i, t in enumerate(x):
        q, s = ref_quantize(t.reshape(T * heads, d))
        full = torch.zeros(T, heads, pitch, dtype=torch.int8)
        full[..., :d] = q.view(T, heads, d)
        want[0][:, i * wide:(i + 1) * wide].view(n_pages, heads, page, pitch)[p, :, a] = full[live]
        want[1][:, i * heads * page:(i + 1) * heads * page].view(n_pages, heads, page)[p, :, a] = s.view(T, heads)[live]
    assert torch.equal(raw.cpu(), want[0]) and same(raws.cpu(), want[1])
    for to in TYPES:
        outs = [rows_of(torch.full((T, heads, d), 7.0), 0, to, heads_first=i == 0, pad=2 - i, off=i) for i in (0, 1)]
        L.lora_cache_read(cache, named.to(DEV), outs[0][1], outs[1][1])
        for i, (buf, out) in enumerate(outs):
            q, s = ref_quantize(x[i].reshape(T * heads, d))
            back = (q.float() * s[:, None]).view(T, heads, d).to(to)
            back[skip] = 7.0
            assert same(out.cpu(), back)
            out.fill_(3.0)
            assert bool((buf == 3.0).all())


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_cache_extremes(dtype):
    """Infinities, NaN and values from 2^64 on: scale NaN and zeros, in their head alone; tiny and zero heads."""
    d = 70
    x = torch.randn(8, 2, d, generator=gen(2))
    x[0, 0, 3] = float("inf")
    x[1, 1, 69] = float("nan")
    x[2, 0, 5] = 2.0 ** 64
    x[3, 0, 5] = 1.8e19  # below 2^64 = 1.84e19
    x[4] = 0
    x[5] *= 1e-38
    x = x.to(dtype)
    cache, *_ = blank_cache(2, 2, 16, d)
    slots = torch.arange(8, dtype=torch.int32, device=DEV) + 3
    L.lora_cache_write(cache, slots, x.to(DEV), x.to(DEV))
    ref = x.clone()
    ref[2, 0, 5] = float("inf")
    q, s = ref_quantize(ref.reshape(16, d))
    got = cache.k.transpose(1, 2).reshape(32, 2, -1)[3:11].cpu(), cache.k_scale.transpose(1, 2).reshape(32, 2)[3:11].cpu()
    assert torch.equal(got[0][..., :d].reshape(16, d), q)
    assert torch.equal(got[1].reshape(16).isnan(), s.isnan()) and int(s.isnan().sum()) == 3
    assert same(got[1].reshape(16)[~s.isnan()], s[~s.isnan()])
    back = [torch.empty(8, 2, d, dtype=dtype, device=DEV) for _ in range(2)]
    L.lora_cache_read(cache, slots, *back)
    assert torch.equal(back[1].cpu().isnan().all(2).reshape(16), s.isnan())


# ----------------------------------------------------------------- attention --
class Step:
    """A batch on the device and on the host: sequences as (queries, keys), random pages, values from a seed."""

    def __init__(self, seqs, heads, kv_heads, d, page, dtype, window=0, sinks=0, tree=None, seed=0, scale=None, extra=0,
                 max_q=None, gap=0, spread=1.0):
        g = gen(seed + 7 * len(seqs) + d)
        self.seqs, self.heads, self.kv, self.d, self.page, self.dtype = seqs, heads, kv_heads, d, page, dtype
        self.window, self.sinks, self.scale = window, sinks, d ** -0.5 if scale is None else scale
        self.T = sum(n for n, _ in seqs) + extra
        most = max([1] + [-(-x // page) for _, x in seqs]) + 1
        n_pages = sum(-(-x // page) for _, x in seqs) + 2
        order = torch.randperm(n_pages, generator=g).to(torch.int32)
        self.pages = torch.full((len(seqs), most), -1, dtype=torch.int32)
        at = 0
        for s, (_, x) in enumerate(seqs):
            n = -(-x // page)
            self.pages[s, :n] = order[at:at + n]
            at += n
        shape = (n_pages, kv_heads, page)
        self.cache = blank_cache(n_pages, kv_heads, page, d, gap)[0]
        self.k, self.v = (torch.randint(-127, 128, (*shape, L.lora_cache_pitch(d)), generator=g, dtype=torch.int8) for _ in range(2))
        size = lambda: torch.exp(torch.randn(shape, generator=g) * 0.3 * spread) * 0.02  # noqa: E731
        self.ks, self.vs = size(), size()
        self.q = (torch.randn(self.T, heads, d, generator=g) * 1.5).to(dtype)
        self.q_off = torch.tensor([0] + [n for n, _ in seqs], dtype=torch.int32).cumsum(0).to(torch.int32)
        self.lens = torch.tensor([x for _, x in seqs], dtype=torch.int32)
        self.tree = tree
        self.max_q = max(n for n, _ in seqs) if max_q is None else max_q

    def load(self):
        for to, t in ((self.cache.k, self.k), (self.cache.v, self.v), (self.cache.k_scale, self.ks), (self.cache.v_scale, self.vs)):
            to.copy_(t)
        self.attention = L.Attention(self.heads, self.scale, window=self.window, sinks=self.sinks, dtype=self.dtype)
        tree = None if self.tree is None else torch.tensor([m - (1 << 64) if m >> 63 else m for m in self.tree], dtype=torch.int64)
        self.batch = L.AttentionBatch(self.T, self.q_off.to(DEV), self.lens.to(DEV), self.pages.to(DEV), self.max_q,
                                      None if tree is None else tree.to(DEV))
        self.plan = L.new_attention_plan(self.attention, self.cache, self.batch)
        self.plan.fill_(255)
        L.lora_attention_plan(self.attention, self.cache, self.batch, self.plan)
        self.ws = L.new_attention_workspace(self.attention, self.cache, self.batch)
        self.ws.fill_(255)
        return self

    def run(self, heads_first=False, pad=0, off=0, in_place=False):
        self.load()
        q = rows_of(self.q, 0, self.dtype, heads_first, pad, off)[1]
        if in_place:
            buf, out = None, q
        else:
            buf, out = rows_of(torch.full(self.q.shape, 7.0), 0, self.dtype, heads_first, pad, off)
        L.lora_attention_apply(self.attention, self.cache, self.batch, self.plan, q, out, self.ws)
        got = out.cpu().clone()
        assert L.lora_read_device_errors(self.plan) == 0
        if buf is not None:
            assert same(q.cpu(), self.q)
            out.fill_(3.0)
            assert bool((buf == 3.0).all())
        return got

    def sees(self, s, i):
        """The keys that query i of sequence s sees, as a mask over its keys."""
        n, length = self.seqs[s]
        j = torch.arange(length)
        context = length - n
        p = context + i
        if self.tree is not None:
            m = self.tree[int(self.q_off[s]) + i] & ((1 << n) - 1)
            p = context + bin(m & ((1 << i) - 1)).count("1")
        near = (j <= p) & ((p - j < self.window) | (j < self.sinks)) if self.window else j <= p
        if self.tree is not None:
            b = j - context
            draft = torch.tensor([0 <= x < 64 and bool(m >> x & 1) for x in b.tolist()], dtype=torch.bool)
            near = torch.where(j < context, near, draft)
        page = self.pages[s].long()[j // self.page] if length else j
        return near & (page >= 0) & (page < self.k.shape[0])

    def rows(self, s):
        """K, V of sequence s in float64 [kv][keys][d]; keys of no page are zeros."""
        _, length = self.seqs[s]
        j = torch.arange(length)
        page = self.pages[s].long()[j // self.page]
        there = ((page >= 0) & (page < self.k.shape[0]))[:, None, None]
        page = page.clamp(0, self.k.shape[0] - 1)
        get = lambda t, sc: torch.where(there, t[page, :, j % self.page, :self.d].double() * sc[page, :, j % self.page][..., None].double(), 0.0).transpose(0, 1)  # noqa: E731
        return get(self.k, self.ks), get(self.v, self.vs)

    def reference(self):
        """The outputs, and how far they may be off; NaN where NaN is due, rows of no sequence not set."""
        out = torch.full((self.T, self.heads, self.d), float("nan"), dtype=torch.float64)
        tol = torch.zeros_like(out)
        group, f32 = self.heads // self.kv, self.dtype == torch.float32
        for s, (n, length) in enumerate(self.seqs):
            k, v = self.rows(s)
            seen = torch.stack([self.sees(s, i) for i in range(n)]) if n else torch.zeros(0, length, dtype=torch.bool)
            for h in range(self.heads):
                lo = int(self.q_off[s])
                q = self.q[lo:lo + n, h].double()
                kk, vv = k[h // group], v[h // group]
                x = torch.where(seen, (q @ kk.T) * self.scale, -math.inf)
                size = torch.where(seen, (q.abs() @ kk.abs().T) * self.scale, 0.0)
                top = x.amax(1, keepdim=True).clamp(min=-1e30) if length else torch.zeros(n, 1, dtype=torch.float64)
                p = torch.where(seen, torch.exp(x - top), 0.0)
                total = p.sum(1, keepdim=True)
                p = p / torch.where(total == 0, 1.0, total)
                vz = torch.where(vv.isnan(), 0.0, vv)
                poisoned = (seen & (vv.isnan().any(1) | kk.isnan().any(1))).any(1)
                o = p @ vz
                o[poisoned] = math.nan
                out[lo:lo + n, h] = o
                xs = torch.where(seen, x, 0.0)
                off = (self.d + 8) * 2 * V * size + 4 * V * (xs.abs() + top.abs())
                if not f32:
                    off = off + H * size
                weight = 8 * V + (H * H if f32 else 2 * H + H * H)
                also = 0.0 if f32 else H
                e = torch.zeros(n, self.d, dtype=torch.float64)
                for c in range(0, length, 256):
                    e += (p[:, c:c + 256, None] * off[:, c:c + 256, None] * (vz[None, c:c + 256] - o[:, None]).abs()).sum(1)
                A = p @ vz.abs()
                tol[lo:lo + n, h] = 1.05 * (e + (weight + 2 * V * length) * A + also * o.abs()) + half(self.dtype) * o.abs()
        return out, tol

    def check(self, **kw):
        got = self.run(**kw)
        ref, tol = self.reference()
        for s, (n, length) in enumerate(self.seqs):
            lo = int(self.q_off[s])
            g, r, t = got[lo:lo + n].double(), ref[lo:lo + n], tol[lo:lo + n]
            bad = ~(((g - r).abs() <= t) | (g.isnan() & r.isnan()))
            assert not bool(bad.any()), (s, n, length, int(bad.sum()), bad.nonzero()[:4].tolist(),
                                         float(((g - r).abs() / t)[~r.isnan()].max()) if t.numel() else 0)
        if self.T > int(self.q_off[-1]):
            rest = got[int(self.q_off[-1]):]
            assert bool((rest == 7.0).all()) or kw.get("in_place")
        return got


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("heads, kv, d, page", [(1, 1, 64, 16), (4, 1, 128, 16), (8, 2, 80, 32), (12, 3, 33, 64), (5, 5, 128, 128),
                                                (4, 1, 256, 16), (16, 1, 96, 16), (3, 1, 1, 16), (6, 2, 48, 1024)])
def test_attention_of_single_tokens(heads, kv, d, page, dtype):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 200, 1000]
    Step([(1, x) for x in lens], heads, kv, d, page, dtype).check()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("heads, kv, d, page", [(4, 1, 128, 16), (6, 2, 64, 32), (2, 2, 80, 16), (8, 1, 256, 16), (3, 3, 40, 64)])
def test_attention_of_prompts(heads, kv, d, page, dtype):
    Step([(1, 1), (2, 2), (17, 17), (64, 64), (65, 70), (130, 130), (200, 333), (3, 500)], heads, kv, d, page, dtype).check()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("n", [2, 4, 5, 8, 9, 16, 17, 33])
def test_attention_rows_of_every_kernel(n, dtype):
    """Few rows of one and of two blocks of 16, and many."""
    Step([(n, n + 100), (1, 40), (n, n)], 4, 1, 64, 16, dtype).check()
    Step([(n, n + 100), (1, 40), (n, n)], 4, 1, 128, 16, dtype, window=50, sinks=2).check()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("d", [64, 128, 200])
def test_attention_of_many_short_drafts(d, dtype):
    """17 to 32 rows of more sequences than go with the kernel for few rows in bfloat16."""
    Step([(8, 8 + 7 * i) for i in range(36)], 4, 1, d, 16, dtype).check()
    Step([(5 + i % 4, 8 + 5 * i) for i in range(20)] + [(1, 90)], 8, 2, d, 16, dtype, window=60, sinks=1).check()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("heads", [16, 17, 32, 33, 64, 65, 130])
def test_attention_many_query_heads(heads, dtype):
    Step([(1, 100), (1, 3), (2, 70)], heads, 1, 64, 16, dtype).check()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("window, sinks", [(1, 0), (1, 1), (2, 0), (16, 4), (63, 0), (64, 1), (65, 70), (100, 300), (1000, 4),
                                           (2 ** 31 - 1, 2 ** 31 - 1), (5, 130)])
def test_attention_windows(window, sinks, dtype):
    seqs = [(1, 1), (1, 64), (1, 500), (1, 1000), (40, 300), (70, 70), (130, 700)]
    Step(seqs, 4, 2, 64, 16, dtype, window=window, sinks=sinks).check()
    Step([(n, x) for n, x in seqs if n == 1], 4, 2, 128, 32, dtype, window=window, sinks=sinks).check()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("seqs", [[(1, 5000)], [(1, 9001), (1, 30)], [(7, 6000), (1, 1)], [(100, 7000)], [(300, 5003), (1, 4000)]])
def test_attention_in_pieces(seqs, dtype):
    """Long sequences, few of them: they are cut and joined."""
    step = Step(seqs, 4, 1, 64, 16, dtype)
    step.check()
    cuts = step.plan[:24].view(torch.int32).cpu().tolist()[4:6]
    assert sum(cuts) >= 1
    Step(seqs, 4, 2, 128, 64, dtype, window=4500, sinks=3).check()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("heads_first, pad, off, in_place", [(True, 0, 0, False), (False, 1, 0, False), (False, 8, 3, False),
                                                             (True, 3, 1, False), (False, 0, 0, True), (True, 5, 1, True)])
def test_attention_strides(heads_first, pad, off, in_place, dtype):
    for seqs in ([(1, 70), (1, 300), (1, 9)], [(40, 100), (1, 5), (90, 90)], [(1, 3000)], [(80, 2000)]):
        Step(seqs, 4, 2, 72, 16, dtype, gap=2).check(heads_first=heads_first, pad=pad, off=off, in_place=in_place)


def chain(n):
    return [(1 << (i + 1)) - 1 for i in range(n)]


def branches(n, g):
    m = []
    for i in range(n):
        parent = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
        m.append((m[parent] if parent >= 0 else 0) | 1 << i)
    return m


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("n", [1, 2, 5, 16, 24, 63, 64])
@pytest.mark.parametrize("window, sinks", [(0, 0), (20, 3)])
def test_attention_of_trees(n, window, sinks, dtype):
    g = gen(n)
    lens = [n, n + 1, n + 63, n + 300, 2 * n + 1000]
    tree = [m for _ in lens for m in branches(n, g)]
    Step([(n, x) for x in lens], 4, 2, 64, 16, dtype, window=window, sinks=sinks, tree=tree).check()


def test_attention_of_a_chain_is_that_of_a_sequence():
    """Drafted tokens each of which sees all before it: the same bits as without a tree, for kernels of few rows and many."""
    for n in (3, 40):
        a = Step([(n, 200), (n, n)], 4, 2, 64, 16, torch.bfloat16).run()
        b = Step([(n, 200), (n, n)], 4, 2, 64, 16, torch.bfloat16, tree=chain(n) * 2).run()
        assert same(a, b)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("n", [5, 50])
def test_attention_trees_of_any_bits(n, dtype):
    """Tokens that do not see themselves, bits of tokens that are not there, and rows that see nothing: zeros."""
    g = gen(n)
    tree = [int(torch.randint(0, 1 << 62, (1,), generator=g)) << 2 | 1 for _ in range(2 * n)]
    tree[3] = 0
    tree[n + 4] = 0
    step = Step([(n, n), (n, n + 70)], 4, 2, 64, 16, dtype, tree=tree)
    got = step.check()
    assert bool((got[3] == 0).all()) and bool((got[n + 4] != 0).any())


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_attention_rows_that_see_nothing(dtype):
    """More queries than keys, empty sequences, pages that are gone: zeros; rows of no sequence stay."""
    for n in (1, 3, 90):
        step = Step([(n, 0), (n, 2), (0, 50), (n, 100), (n, 40)], 4, 2, 64, 16, dtype, extra=3)
        step.pages[3] = torch.tensor([-1, 10 ** 9, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32)[torch.arange(step.pages.shape[1]) % 4]
        step.pages[4, 1] = -1
        got = step.check()
        assert bool((got[:n] == 0).all()) and bool((got[2 * n:3 * n] == 0).all())
        assert bool((got[n:n + max(0, n - 2)] == 0).all())
        assert bool((got[4 * n:] == 7).all())


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_attention_reads_no_page_that_is_not_seen(dtype):
    """Dropped pages between the first keys and the window may name anything; the cache's other slots hold NaN."""
    seqs = [(1, 1000), (1, 700), (20, 900)]
    step = Step(seqs, 4, 2, 64, 16, dtype, window=100, sinks=5)
    clean = step.check()
    for s, (n, x) in enumerate(seqs):
        live = torch.zeros(step.pages.shape[1], dtype=torch.bool)
        live[0] = True
        live[(x - n - 100 + 1) // 16:-(-x // 16)] = True
        step.pages[s, ~live] = -7
    used = step.pages[step.pages >= 0].long()
    gone = torch.ones(step.k.shape[0], dtype=torch.bool)
    gone[used] = False
    step.ks[gone] = step.vs[gone] = float("nan")
    for s, (_, x) in enumerate(seqs):  # behind a sequence's last key
        if x % 16:
            last = int(step.pages[s, x // 16])
            step.ks[last, :, x % 16:] = step.vs[last, :, x % 16:] = float("nan")
    assert same(step.run(), clean)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_attention_nan_keys_and_values(dtype):
    """A key or value that is NaN makes the rows NaN that see it, in its cache head, and no others."""
    for which in ("ks", "vs"):
        for seqs in ([(4, 150)], [(100, 150)]):
            step = Step(seqs, 4, 2, 64, 16, dtype)
            n, x = seqs[0]
            j = x - 2
            getattr(step, which)[int(step.pages[0, j // 16]), 1, j % 16] = float("nan")
            got = step.check()
            nan = got.isnan().all(2)
            want = torch.zeros(n, 4, dtype=torch.bool)
            want[n - 2:, 2:] = True
            assert torch.equal(nan, want) and torch.equal(got.isnan().any(2), want)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_attention_nan_queries_stay_in_their_row(dtype):
    for seqs in ([(4, 150)], [(100, 150)]):
        step = Step(seqs, 4, 2, 64, 16, dtype)
        clean = step.check()
        step.q[1, 2, 5] = float("inf")
        step.q[2, 0, 63] = float("nan")
        got = step.run()
        assert bool(got[1, 2].isnan().all()) and bool(got[2, 0].isnan().all())
        keep = torch.ones(seqs[0][0], 4, dtype=torch.bool)
        keep[1, 2] = keep[2, 0] = False
        assert same(got[keep], clean[keep])


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** -20, 2.0 ** 20, 2.0 ** 50])
def test_attention_sizes_of_values(size, dtype):
    """Large and small values, keys and queries: nothing leaves the range of float16 on the way."""
    for seqs in ([(1, 300), (2, 90)], [(100, 150)]):
        step = Step(seqs, 4, 2, 64, 16, dtype)
        step.vs *= size
        step.check()
        step = Step(seqs, 4, 2, 64, 16, dtype, scale=0.125 / size)
        step.ks *= size
        step.check()
        step = Step(seqs, 4, 2, 64, 16, dtype, scale=0.125 / size)
        step.q = (step.q.float() * size).to(dtype)
        step.check()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_attention_values_of_very_different_sizes(dtype):
    """Values 2^20 apart between sequences' tiles and zero values; a first key that takes most of the weight."""
    for seqs in ([(1, 400)], [(100, 400)]):
        step = Step(seqs, 4, 2, 64, 16, dtype)
        for t in range(0, 400, 64):
            for j in range(t, min(t + 64, 400)):
                step.vs[int(step.pages[0, j // 16]), :, j % 16] *= 2.0 ** (-10 if t % 128 else 10)
        step.vs[int(step.pages[0, 3])] = 0.0
        step.v[int(step.pages[0, 3])] = 0
        step.check()
        step = Step(seqs, 4, 2, 64, 16, dtype)
        first = int(step.pages[0, 0])
        step.ks[first, :, 0] *= 20
        step.vs[first, :, 0] *= 2.0 ** -12
        step.check()


def test_attention_plan_counts_what_it_leaves_out():
    step = Step([(2, 50), (1, 60), (1, 30)], 4, 2, 64, 16, torch.bfloat16, extra=2)
    good = step.run()
    cases = [("lens", 1, 16 * step.pages.shape[1] + 1), ("lens", 1, -1), ("q_off", 2, 1), ("q_off", 2, 100), ("max_q", None, 1)]
    for what, at, value in cases:
        bad = Step([(2, 50), (1, 60), (1, 30)], 4, 2, 64, 16, torch.bfloat16, extra=2)
        if what == "max_q":
            bad.max_q = value
            out_rows = [0, 1]
        else:
            getattr(bad, what)[at] = value
            out_rows = [2] if what == "lens" else [2, 3]
        bad.load()
        out = torch.full(bad.q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
        L.lora_attention_apply(bad.attention, bad.cache, bad.batch, bad.plan, bad.q.to(DEV), out, bad.ws)
        assert L.lora_read_device_errors(bad.plan) >= 1, (what, value)
        out = out.cpu()
        assert bool((out[out_rows] == 7).all()) and bool((out[4:] == 7).all()), (what, value)
        keep = [r for r in range(4) if r not in out_rows]
        assert same(out[keep], good[keep]), (what, value)


def test_attention_on_another_plan_writes_nothing():
    for n in (1, 100):
        a = Step([(n, 150), (n, n)], 4, 2, 64, 16, torch.bfloat16).load()
        for kw in (dict(window=9), dict(max_q=n + 1), dict(sinks=2)):
            b = Step([(n, 150), (n, n)], 4, 2, 64, 16, torch.bfloat16, **kw).load()
            out = torch.full(a.q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
            size = max(a.plan.numel(), b.plan.numel())
            plan = torch.zeros(size, dtype=torch.uint8, device=DEV)
            plan[:b.plan.numel()] = b.plan
            L.lora_attention_apply(a.attention, a.cache, a.batch, plan, a.q.to(DEV), out, a.ws)
            assert bool((out == 7).all()) and L.lora_read_device_errors(plan) >= 1


def test_attention_gives_the_same_bits_again():
    for seqs in ([(1, 5000), (1, 77)], [(200, 3000), (1, 10)]):
        step = Step(seqs, 4, 1, 128, 16, torch.bfloat16)
        first = step.run()
        for _ in range(3):
            assert same(step.run(), first)


def test_attention_with_nothing_to_do():
    cache, *_ = blank_cache(2, 1, 16, 64)
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    z = torch.zeros(1, dtype=torch.int32, device=DEV)
    att = L.Attention(2, 1.0)
    q = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    batch = L.AttentionBatch(0, z, e, torch.empty(0, 3, dtype=torch.int32, device=DEV), 1)
    plan, ws = L.new_attention_plan(att, cache, batch), L.new_attention_workspace(att, cache, batch)
    L.lora_attention_plan(att, cache, batch, plan)
    L.lora_attention_apply(att, cache, batch, plan, q, q, ws)
    L.lora_cache_write(cache, e, q[:, :1], q[:, :1])
    L.lora_cache_read(cache, e, q[:, :1], q[:, 1:])
    L.lora_norm_apply(L.Norm(torch.ones(8, device=DEV), 0.0), torch.empty(0, 8, device=DEV), y=torch.empty(0, 8, device=DEV))


def test_cache_beyond_4_gib():
    """Pages whose bytes lie behind 2^32 of the cache's start, and scales too."""
    n_pages, heads, page, d = 70000, 2, 256, 128
    cache = L.new_cache(n_pages, heads, page, d, DEV)
    T = 300
    g = gen(3)
    slots = (n_pages * page - 1 - torch.arange(T)).to(torch.int32)
    k, v = (torch.randn(T, heads, d, generator=g).to(torch.bfloat16) for _ in range(2))
    L.lora_cache_write(cache, slots.to(DEV), k.to(DEV), v.to(DEV))
    back = [torch.empty(T, heads, d, device=DEV) for _ in range(2)]
    L.lora_cache_read(cache, slots.to(DEV), *back)
    for x, b in zip((k, v), back):
        q, s = ref_quantize(x.reshape(-1, d))
        assert same(b.cpu().reshape(-1, d), q.float() * s[:, None])
    # the two last pages as a sequence, a third of them queries
    pages = torch.tensor([[n_pages - 2, n_pages - 1]], dtype=torch.int32, device=DEV)
    for n in (1, 60):
        att = L.Attention(4, d ** -0.5, dtype=torch.float32)
        batch = L.AttentionBatch(n, torch.tensor([0, n], dtype=torch.int32, device=DEV),
                                 torch.tensor([512], dtype=torch.int32, device=DEV), pages, n)
        plan, ws = L.new_attention_plan(att, cache, batch), L.new_attention_workspace(att, cache, batch)
        q = torch.randn(n, 4, d, generator=g).to(DEV)
        out = torch.empty_like(q)
        L.lora_attention_plan(att, cache, batch, plan)
        L.lora_attention_apply(att, cache, batch, plan, q, out, ws)
        kk, vv = torch.zeros(512, heads, d, dtype=torch.float64), torch.zeros(512, heads, d, dtype=torch.float64)
        for t, b in ((kk, back[0]), (vv, back[1])):
            t[512 - T:] = b.cpu().double().flip(0)
        for h in range(4):
            x = q[:, h].cpu().double() @ kk[:, h // 2].T * d ** -0.5
            x.masked_fill_(torch.arange(512)[None] > 512 - n + torch.arange(n)[:, None], -math.inf)
            p = torch.softmax(x, 1)
            # float32 throughout: scores to 1e-5, weights to 2^-22, sums of 512
            size = p @ vv[:, h // 2].abs() + (p @ vv[:, h // 2]).abs()
            assert bool(((out[:, h].cpu().double() - p @ vv[:, h // 2]).abs() <= 1e-4 * size).all())


def test_attention_of_single_tokens_among_as_many_tokens_as_drafts():
    """As many tokens as if every sequence had the most: a single token goes with the drafts, the rest belong to none."""
    Step([(40, 100), (1, 3000)], 4, 2, 64, 16, torch.bfloat16, extra=39).check()
    Step([(9, 100), (1, 3000), (9, 9)], 4, 1, 80, 16, torch.float32, extra=8).check()
    Step([(24, 300), (0, 10), (1, 1)], 8, 2, 128, 16, torch.bfloat16, extra=47).check()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("d", [129, 200, 256])
def test_attention_of_long_heads_in_place(d, dtype):
    """Their values are taken in halves; all of a row's queries are read before any of its outputs is written."""
    for seqs in ([(40, 300), (1, 5), (150, 150)], [(30, 3000), (1, 70)]):
        step = Step(seqs, 4, 2, d, 16, dtype)
        assert same(step.check(in_place=True), step.check())


@pytest.mark.parametrize("n, heads, dtype", [(1, 2, torch.bfloat16), (2, 40, torch.bfloat16), (1, 2, torch.float32),
                                             (2, 20, torch.float32), (2, 130, torch.bfloat16)])
def test_attention_more_sequences_than_workgroups(n, heads, dtype):
    """70000 short sequences (35000 of two units of rows each) whose queries see their own key alone: each output is that key's value, off by the rounding of
    its weight and of the value (h each in bfloat16), of the sum (8 v) and of the output."""
    S, d, page = 70000 if heads < 100 else 35000, 64, 16
    T = S * n
    g = gen(n)
    cache = L.new_cache(S, 1, page, d, DEV)
    pages = torch.randperm(S, generator=g).to(torch.int32)
    slots = (pages[:, None] * page + torch.arange(n, dtype=torch.int32)).reshape(-1).to(DEV)
    k, v = (torch.randn(T, 1, d, generator=g).to(dtype).to(DEV) for _ in range(2))
    L.lora_cache_write(cache, slots, k, v)
    back = [torch.empty(T, 1, d, device=DEV) for _ in range(2)]
    L.lora_cache_read(cache, slots, *back)
    att = L.Attention(heads, d ** -0.5, window=1, dtype=dtype)
    batch = L.AttentionBatch(T, (torch.arange(S + 1, dtype=torch.int32) * n).to(DEV),
                             torch.full((S,), n, dtype=torch.int32, device=DEV), pages[:, None].contiguous().to(DEV), n)
    plan, ws = L.new_attention_plan(att, cache, batch), L.new_attention_workspace(att, cache, batch)
    L.lora_attention_plan(att, cache, batch, plan)
    q = torch.randn(T, heads, d, generator=torch.Generator(DEV).manual_seed(n), device=DEV).to(dtype)
    out = torch.full_like(q, 7.0)
    L.lora_attention_apply(att, cache, batch, plan, q, out, ws)
    assert L.lora_read_device_errors(plan) == 0
    tol = 1.01 * (half(dtype) + 16 * V + (2 * H if dtype == torch.bfloat16 else 2 * H * H)) * back[1].abs()
    assert bool(((out.float() - back[1]).abs() <= tol).all())


# ----------------------------------------------------- as they are used together --
class LayerRun:
    """Norm, query, key and value projections with adapters, rotary positions, cache, attention: one layer's first half."""
    D, HEADS, KV, HD = 256, 8, 2, 64

    def __init__(self, seqs, tree=None, seed=0):
        self.step = st = Step(seqs, self.HEADS, self.KV, self.HD, 16, torch.bfloat16, tree=tree, seed=seed)
        st.load()
        g = gen(seed + 100)
        T, D, wide = st.T, self.D, (self.HEADS + 2 * self.KV) * self.HD
        put = lambda t: t.to(torch.bfloat16).to(DEV)  # noqa: E731
        self.x, self.r = put(torch.randn(T, D, generator=g)), put(torch.randn(T, D, generator=g))
        self.total, self.y = torch.zeros_like(self.x), torch.zeros_like(self.x)
        self.q8, self.scale = torch.zeros(T, D, dtype=torch.int8, device=DEV), torch.zeros(T, device=DEV)
        self.norm = L.Norm((1 + 0.1 * torch.randn(D, generator=g)).to(DEV), 1e-5)
        W = torch.randint(-127, 128, (wide, D), generator=g, dtype=torch.int8)
        self.base = L.BaseWeight(W.to(DEV), torch.full((wide,), 1 / (73 * D ** 0.5), device=DEV))
        self.pool = L.Pool(put(torch.randn(3, 16, D, generator=g) / 16), put(torch.randn(3, wide, 16, generator=g) / 8))
        self.adapters = L.Batch(T, torch.randint(-1, 3, (T, 1), generator=g, dtype=torch.int32).to(DEV))
        self.lora_ws = L.new_workspace(self.adapters, 3, DEV)
        self.qkv = torch.zeros(T, wide, dtype=torch.bfloat16, device=DEV)
        heads = self.qkv.view(T, -1, self.HD)
        self.q, self.k, self.v = heads[:, :self.HEADS], heads[:, self.HEADS:-self.KV], heads[:, -self.KV:]
        self.rotary = L.Rotary(torch.as_tensor(L.lora_rotary_frequencies(self.HD), dtype=torch.float64).to(DEV), self.HD)
        self.pos, self.slots = (torch.zeros(T, dtype=torch.int32, device=DEV) for _ in range(2))
        self.out = torch.full((T, self.HEADS, self.HD), 7.0, dtype=torch.bfloat16, device=DEV)
        self.set_lens([x for _, x in seqs])

    def set_lens(self, lens):
        st = self.step
        st.seqs = [(n, x) for (n, _), x in zip(st.seqs, lens)]
        p = torch.cat([torch.arange(x - n, x) for n, x in st.seqs])
        s = torch.cat([torch.full((n,), i) for i, (n, _) in enumerate(st.seqs)])
        self.pos.copy_(p)
        self.slots.copy_(st.pages[s, p // 16] * 16 + p % 16)
        st.batch.lens.copy_(torch.tensor(lens, dtype=torch.int32))

    def run(self):
        st = self.step
        L.lora_attention_plan(st.attention, st.cache, st.batch, st.plan)
        L.lora_norm_apply(self.norm, self.x, y=self.y, q=self.q8, scale=self.scale, residual=self.r, total=self.total)
        L.lora_base_product(self.base, self.q8, self.scale, self.qkv)
        L.lora_apply(self.pool, self.adapters, self.y, self.qkv, self.lora_ws)
        L.lora_rotary_apply(self.rotary, self.pos, [self.q, self.k])
        L.lora_cache_write(st.cache, self.slots, self.k, self.v)
        L.lora_attention_apply(st.attention, st.cache, st.batch, st.plan, self.q, self.out, st.ws)

    def state(self):
        c = self.step.cache
        return [t.clone() for t in (self.total, self.y, self.q8, self.scale, self.qkv, c.k, c.v, c.k_scale, c.v_scale, self.out)]


SEQS = [[(1, 200), (40, 40), (3, 70)], [(1, 5000)], [(24, 300), (24, 24)], [(200, 260), (1, 16)]]


@pytest.mark.parametrize("seqs", SEQS)
@pytest.mark.parametrize("trees", [False, True])
def test_layer(seqs, trees):
    """Each of them against its formula, on what the one before it left on the device."""
    if trees and max(n for n, _ in seqs) > 64:
        seqs = [(60, 260), (1, 16)]
    g = gen(5)
    rows = [i for n, _ in seqs for i in range(n)]
    tree = [1 << i | 1 | int(torch.randint(0, 1 << i, (1,), generator=g)) if i else 1 for i in rows] if trees else None
    run = LayerRun(seqs, tree)
    run.run()
    st = run.step
    h = run.x.cpu().double() + run.r.cpu().double()
    total = run.total.cpu()
    assert same(total, h.to(torch.bfloat16))
    t = total.double()
    y = t * run.norm.weight.cpu().double() / (t.square().mean(1, keepdim=True) + 1e-5).sqrt()
    assert bool(((run.y.cpu().double() - y).abs() <= (half(torch.bfloat16) + V) * y.abs()).all())
    q8, scale = ref_quantize(run.y.cpu())
    assert same(run.q8.cpu(), q8) and same(run.scale.cpu(), scale)
    slots = run.slots.cpu().long()
    for heads, c, s in ((run.k, st.cache.k, st.cache.k_scale), (run.v, st.cache.v, st.cache.v_scale)):
        q8, scale = ref_quantize(heads.cpu().reshape(-1, run.HD))
        assert same(c.cpu()[slots // 16, :, slots % 16].reshape(-1, run.HD), q8)
        assert same(s.cpu()[slots // 16, :, slots % 16].reshape(-1), scale)
    st.q = run.q.cpu()
    st.k, st.v, st.ks, st.vs = (x.cpu() for x in (st.cache.k, st.cache.v, st.cache.k_scale, st.cache.v_scale))
    ref, tol = st.reference()
    assert bool(((run.out.cpu().double() - ref).abs() <= tol).all())
    assert L.lora_read_device_errors(st.plan) == 0


def test_layer_in_a_graph():
    """Captured once with the plan, replayed on new inputs, lengths and slots, with eager work and synchronizations between:
    every replay leaves what an eager run leaves, in the cache too."""
    seqs = [(1, 200), (40, 60), (3, 70), (1, 1)]
    a, b = LayerRun(seqs), LayerRun(seqs)
    a.run()
    b.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
    g = gen(3)
    for lens in ([190, 45, 3, 16], [1, 40, 80, 1], [208, 64, 33, 2], [208, 64, 33, 2], [17, 50, 70, 9]):
        x = torch.randn(a.x.shape, generator=g).to(torch.bfloat16).to(DEV)
        for run in (a, b):
            run.x.copy_(x)
            run.set_lens(lens)
        graph.replay()
        b.run()
        torch.cuda.synchronize()
        assert all(same(s, t) for s, t in zip(a.state(), b.state())), lens
        assert L.lora_read_device_errors(a.step.plan) == 0


def test_layer_on_another_stream():
    seqs = [(1, 4000), (70, 90)]
    a, b = LayerRun(seqs), LayerRun(seqs)
    torch.cuda.synchronize()
    a.run()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b.run()
    torch.cuda.synchronize()
    assert all(same(s, t) for s, t in zip(a.state(), b.state()))


def test_attention_calls_at_once():
    """Two calls on two streams that share a plan and a cache, each with a workspace of its own."""
    st = Step([(1, 5000), (1, 300), (30, 3000)], 8, 2, 128, 16, torch.bfloat16).load()
    g = gen(8)
    qs = [torch.randn(st.T, 8, 128, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2)]
    outs, want = [torch.zeros_like(q) for q in qs], []
    for q in qs:
        out = torch.zeros_like(q)
        L.lora_attention_apply(st.attention, st.cache, st.batch, st.plan, q, out, st.ws)
        want.append(out)
    wss = [L.new_attention_workspace(st.attention, st.cache, st.batch) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for q, out, ws, stream in zip(qs, outs, wss, streams):
            with torch.cuda.stream(stream):
                L.lora_attention_apply(st.attention, st.cache, st.batch, st.plan, q, out, ws)
    torch.cuda.synchronize()
    assert all(same(out, w) for out, w in zip(outs, want))


def test_attention_graphs_share_a_workspace():
    """Two captured calls on one workspace, of different batches, replayed one after the other."""
    steps = [Step(seqs, 8, 2, 128, 16, torch.bfloat16).load() for seqs in ([(1, 5000), (1, 300)], [(30, 3000), (1, 70)])]
    ws = torch.empty(max(st.ws.numel() for st in steps), dtype=torch.uint8, device=DEV)
    qs = [st.q.to(DEV) for st in steps]
    outs, want, graphs = [torch.zeros_like(q) for q in qs], [], []
    for st, q, out in zip(steps, qs, outs):
        L.lora_attention_apply(st.attention, st.cache, st.batch, st.plan, q, out, ws)
        want.append(out.clone())
    torch.cuda.synchronize()
    for st, q, out in zip(steps, qs, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            L.lora_attention_apply(st.attention, st.cache, st.batch, st.plan, q, out, ws)
        graphs.append(graph)
    for k in (0, 1, 1, 0, 1):
        outs[k].zero_()
        graphs[k].replay()
        torch.cuda.synchronize()
        assert same(outs[k], want[k])
