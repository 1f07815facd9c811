"""The operators around a LoRA layer (include/lora_base.h) against plain
implementations in 64 bits.

Tolerances, with u = eps / 2 of the output's type (the one rounding to it) and
v = 2^-24 (a float32 rounding):
  quantised rows   equal; their scale is the float32 nearest to a / 127
  product          the sum is exact; float(sum), * q_scale, * scale and + bias
                   round once each: u |y| + 4 v (|product| + |bias|)
  rotary           the angle's fraction of a turn is off by 2^-27 turns (4.7e-8
                   rad < v), sine and cosine by at most 2 ulp (2 v), times m by v:
                   4 v m each; two products and a sum, 2 v more:
                   u |y| + 6 v m (|a| + |b|)
"""
import fractions

import numpy as np
import pytest
import torch

import rank_sgmv_bgmv_amd as L

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
V = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float32]
ids = {torch.bfloat16: "bf16", torch.float32: "f32"}.get


def half(t):
    return torch.finfo(t).eps / 2


def gen(seed):
    return torch.Generator().manual_seed(seed)


def i8(shape, g, lo=-127, hi=127):
    return torch.randint(lo, hi + 1, shape, generator=g, dtype=torch.int8)


# ------------------------------------------------------------------ quantise --
def ref_quantize(x):
    x = x.double()
    a = x.abs().amax(1)
    bad = ~torch.isfinite(x).all(1)
    q = torch.round(127 * x / torch.where(a > 0, a, 1.0)[:, None])
    q = torch.where(bad[:, None], 0.0, q)
    return q.to(torch.int8), torch.where(bad, torch.nan, a.float().double().div(127)).float()


def check_quantize(x, ld_extra=0, off=0):
    """x on the host; q gets a wider buffer whose other bytes have to stay."""
    T, d = x.shape
    e = torch.tensor([], dtype=x.dtype).element_size()
    buf = torch.full((off + (T + 1) * (d + ld_extra),), 3, dtype=x.dtype, device=DEV)
    xv = buf[off:off + T * (d + ld_extra)].view(T, d + ld_extra)[:, :d]
    xv.copy_(x)
    qb = torch.full((off + (T + 1) * (d + ld_extra),), 77, dtype=torch.int8, device=DEV)
    qv = qb[off:off + T * (d + ld_extra)].view(T, d + ld_extra)[:, :d]
    sb = torch.full((T + 2,), -5.0, device=DEV)
    L.lora_quantize_rows(xv, qv, sb[1:T + 1])
    q, s = ref_quantize(x)
    assert torch.equal(qv.cpu(), q), (e, T, d)
    assert torch.equal(sb.cpu()[1:T + 1].view(torch.int32)[~s.isnan()], s.view(torch.int32)[~s.isnan()])
    assert torch.equal(sb.cpu()[1:T + 1].isnan(), s.isnan())
    assert sb[0] == -5 and sb[-1] == -5
    rest = qb.clone()
    rest[off:off + T * (d + ld_extra)].view(T, d + ld_extra)[:, :d] = 77
    assert bool((rest == 77).all())


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("T, d", [(1, 1), (1, 4096), (3, 7), (2, 8), (5, 63), (64, 64), (7, 65), (65, 1001), (130, 256),
                                  (9, 1280), (4, 14336), (3, 16387), (2, 70001), (1000, 128), (4099, 31)])
def test_quantize(T, d, dtype):
    x = torch.randn(T, d, generator=gen(T * 7 + d)) * torch.rand(T, 1, generator=gen(T)) * 10
    check_quantize(x.to(dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("ld_extra, off", [(1, 0), (8, 0), (16, 0), (0, 1), (3, 5), (16, 16)])
def test_quantize_strides_and_alignment(dtype, ld_extra, off):
    for T, d in ((5, 512), (3, 4099), (70, 48)):
        check_quantize(torch.randn(T, d, generator=gen(d)).to(dtype), ld_extra, off)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_quantize_halves_go_to_the_even_number(dtype):
    """x = a (2k + 1) / 254: every quotient is a half, or for a that is no multiple of 127 next to one."""
    k = torch.arange(-127, 127).double()
    for a in (254.0, 127.0, 2.0 ** 20 * 127, 1.0, 1.0 / 3, 5.0):
        x = torch.cat([a * (2 * k + 1) / 254, torch.tensor([a, -a], dtype=torch.float64)])[None].to(dtype)
        check_quantize(x.expand(3, -1).contiguous())


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_quantize_next_to_halves(dtype):
    """Values one step of their type around every half, with maxima of many significands."""
    g = gen(5)
    k = torch.arange(0, 127).double()
    rows = []
    for _ in range(200):
        a = (1 + torch.rand(1, generator=g)).to(dtype).double()
        x = (a * (2 * k + 1) / 254).to(dtype)
        up = torch.nextafter(x.float(), torch.tensor(9.0)) if dtype == torch.float32 else (x.view(torch.int16) + 1).view(dtype)
        dn = torch.nextafter(x.float(), torch.tensor(0.0)) if dtype == torch.float32 else (x.view(torch.int16) - 1).view(dtype)
        rows.append(torch.cat([x, -up.to(dtype), dn.to(dtype), a.to(dtype)]))
    check_quantize(torch.stack(rows))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_quantize_extremes(dtype):
    """Zero rows, tiny and huge maxima, rows with an infinity or a NaN: no row meets another."""
    d = 300
    x = torch.randn(12, d, generator=gen(1))
    x[0] = 0
    x[1] = -0.0
    x[2] *= 1e-38
    x[3] *= 1e-42 if dtype == torch.float32 else 1e-39
    x[4] *= 5e37
    x[5, 17] = float("inf")
    x[6, 299] = float("-inf")
    x[7, 0] = float("nan")
    x[8] = float("nan")
    x[9] = 0
    x[9, 150] = torch.finfo(dtype).max
    x[10] = 0
    x[10, 3] = 2.0 ** -149 if dtype == torch.float32 else 2.0 ** -133
    check_quantize(x.to(dtype))


@pytest.mark.parametrize("T, d, dtype", [(270001, 8, torch.bfloat16), (66001, 1032, torch.float32)])
def test_quantize_more_rows_than_workgroups(T, d, dtype):
    x = torch.randn(T, d, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(dtype)
    q, s = torch.empty(T, d, dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    L.lora_quantize_rows(x, q, s)
    a = x.abs().amax(1).double()
    assert torch.equal(s, (a / 127).float())
    for lo in range(0, T, 20000):
        v = x[lo:lo + 20000].double()
        assert torch.equal(q[lo:lo + 20000].double(), torch.round(127 * v / a[lo:lo + 20000, None])), lo


def test_quantize_no_rows():
    x, q, s = torch.empty(0, 64, device=DEV), torch.empty(0, 64, dtype=torch.int8, device=DEV), torch.empty(0, device=DEV)
    L.lora_quantize_rows(x, q, s)


# ------------------------------------------------------------------- product --
def ref_product(q, qs, W, ws, bias):
    p = (q.double() @ W.double().T) * qs.double()[:, None] * ws.double()
    y = p if bias is None else p + bias.double()
    return y, p.abs() + (0 if bias is None else bias.double().abs())


def check_product(T, d_in, d_out, dtype, bias=True, seed=0, pad=(0, 0, 0), off=(0, 0, 0), q=None, W=None):
    """pad: further columns of q, W and y; off: their first element's place in a buffer."""
    g = gen(seed + T * 31 + d_in * 7 + d_out)
    q = i8((T, d_in), g) if q is None else q
    W = i8((d_out, d_in), g, -128, 127) if W is None else W
    qs, ws = torch.rand(T, generator=g) * 0.02, torch.rand(d_out, generator=g) * 0.01
    b = torch.randn(d_out, generator=g) if bias else None

    def place(t, p, o, fill):
        buf = torch.full((o + (t.shape[0] + 1) * (t.shape[1] + p),), fill, dtype=t.dtype, device=DEV)
        v = buf[o:o + t.shape[0] * (t.shape[1] + p)].view(t.shape[0], -1)[:, :t.shape[1]]
        v.copy_(t)
        return buf, v

    _, qv = place(q, pad[0], off[0], 99)
    _, Wv = place(W, pad[1], off[1], 99)
    yb, yv = place(torch.zeros(T, d_out, dtype=dtype), pad[2], off[2], 7.0)
    w = L.BaseWeight(Wv, ws.to(DEV), None if b is None else b.to(DEV))
    L.lora_base_product(w, qv, qs.to(DEV), yv)
    y, mag = ref_product(q, qs, W, ws, b)
    got = yv.cpu().double()
    tol = half(dtype) * y.abs() + 4 * V * mag
    bad = (got - y).abs() > tol
    assert not bad.any(), (T, d_in, d_out, int(bad.sum()), bad.nonzero()[:4].tolist())
    rest = yb.clone()
    rest[off[2]:off[2] + T * (d_out + pad[2])].view(T, -1)[:, :d_out] = 7.0
    assert bool((rest == 7.0).all())


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("T", [1, 2, 5, 15, 16, 17, 31, 33, 48, 64, 65, 127, 128, 129, 200, 257, 300, 513, 1030])
def test_product_tokens(T, dtype):
    check_product(T, 512, 384, dtype)
    check_product(T, 320, 272, dtype, bias=False)


@pytest.mark.parametrize("T", [1, 16, 40, 100, 300])
@pytest.mark.parametrize("d_in", [1, 3, 15, 16, 17, 48, 63, 64, 65, 100, 127, 128, 129, 144, 192, 250, 256, 400, 1001, 1040,
                                  2064])
def test_product_d_in(d_in, T):
    check_product(T, d_in, 70, torch.float32)


@pytest.mark.parametrize("T", [1, 20, 130, 300])
@pytest.mark.parametrize("d_out", [1, 2, 3, 4, 5, 15, 16, 17, 31, 64, 66, 127, 128, 130, 255, 256, 260, 1283])
def test_product_d_out(d_out, T):
    check_product(T, 128, d_out, torch.bfloat16)
    check_product(T, 130, d_out, torch.float32)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("T", [3, 64, 300])
@pytest.mark.parametrize("pad, off", [((1, 0, 0), (0, 0, 0)), ((0, 1, 0), (0, 0, 0)), ((0, 0, 1), (0, 0, 0)),
                                      ((16, 16, 8), (0, 0, 0)), ((0, 0, 0), (1, 0, 0)), ((0, 0, 0), (0, 4, 0)),
                                      ((0, 0, 0), (0, 0, 1)), ((5, 3, 2), (7, 9, 3)), ((0, 0, 2), (16, 16, 2))])
def test_product_strides_and_alignment(T, pad, off, dtype):
    check_product(T, 256, 192, dtype, pad=pad, off=off)


@pytest.mark.parametrize("T, d_in, d_out", [(1, 4096, 1024), (64, 4096, 4096), (5, 14336, 256), (777, 1001, 1283),
                                            (640, 1280, 1280), (2304, 1024, 4096), (1500, 4096, 640)])
def test_product_sizes_of_use(T, d_in, d_out):
    check_product(T, d_in, d_out, torch.bfloat16)


@pytest.mark.parametrize("T", [1, 17, 130, 300])
@pytest.mark.parametrize("d_in", [131071, 131056])
def test_product_largest_sums(T, d_in):
    """Every product has the largest size and one sign: the sum ends just below 2^31."""
    q = torch.full((T, d_in), -128, dtype=torch.int8)
    W = torch.full((33, d_in), -128, dtype=torch.int8)
    W[::2] = 127
    check_product(T, d_in, 33, torch.float32, bias=False, q=q, W=W)


TILES = [(16797, 656, 579), (16806, 656, 513), (13627, 656, 266), (16511, 656, 65), (9355, 656, 65), (117, 704, 63),
         (16877, 672, 130), (17045, 656, 1411), (301, 655, 130), (5001, 655, 1283)]


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("T, d_in, d_out", TILES)
def test_product_large(T, d_in, d_out, dtype):
    """Sizes that take each of the tile shapes, with ends in both directions and in the sum's axis, and one that is
    split into whole rounds and a rest; against the float64 product on the GPU (sums below 2^53: exact)."""
    g = gen(T)
    q, W = i8((T, d_in), g).to(DEV), i8((d_out, d_in), g, -128, 127).to(DEV)
    qs, ws, b = (torch.rand(n, generator=g).to(DEV) * 0.02 for n in (T, d_out, d_out))
    yb = torch.full((T + 1, d_out + 8), 7.0, dtype=dtype, device=DEV)
    L.lora_base_product(L.BaseWeight(W, ws, b), q, qs, yb[:T, :d_out])
    p = (q.double() @ W.double().T) * qs.double()[:, None] * ws.double()
    ref = p + b.double()
    bad = (yb[:T, :d_out].double() - ref).abs() > half(dtype) * ref.abs() + 4 * V * (p.abs() + b.double().abs())
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist())
    assert bool((yb[T] == 7).all()) and bool((yb[:, d_out:] == 7).all())


def test_product_nan_scale_stays_in_its_row():
    g = gen(3)
    q, W = i8((20, 64), g).to(DEV), i8((48, 64), g).to(DEV)
    qs = torch.ones(20, device=DEV)
    qs[7] = float("nan")
    q[7] = 0
    y = torch.zeros(20, 48, device=DEV)
    L.lora_base_product(L.BaseWeight(W, torch.ones(48, device=DEV)), q, qs, y)
    nan = y.isnan()
    assert bool(nan[7].all()) and not bool(nan[torch.arange(20) != 7].any())


@pytest.mark.parametrize("T", [3, 70, 300])
def test_product_rows_far_apart(T):
    """Row strides that put later rows beyond 4 GiB of each operand's start."""
    ld = ((1 << 32) // (T - 1) + 64) // 16 * 16
    g = gen(T)
    q, W = i8((T, 64), g), i8((T, 64), g)
    big = torch.empty(T * ld, dtype=torch.int8, device=DEV)
    v = big.view(T, ld)
    v[:, :64], v[:, 64:128] = q.to(DEV), W.to(DEV)
    y = torch.empty(T * ld // 4, dtype=torch.float32, device=DEV).view(T, ld // 4)[:, :T]
    qs, ws = torch.rand(T, generator=g), torch.rand(T, generator=g)
    L.lora_base_product(L.BaseWeight(v[:, 64:128], ws.to(DEV)), v[:, :64], qs.to(DEV), y)
    ref, mag = ref_product(q, qs, W, ws, None)
    assert bool(((y.cpu().double() - ref).abs() <= V * ref.abs() + 4 * V * mag).all())


def test_product_many_rows():
    """More rows than a grid's second dimension could count in tiles of 64: the last ones are right."""
    T, d = 64 * 65536 + 70, 16
    q = (torch.arange(T, device=DEV).view(-1, 1) % 251 - 125).to(torch.int8).expand(T, d).contiguous()
    W = torch.ones(2, d, dtype=torch.int8, device=DEV)
    y = torch.zeros(T, 2, device=DEV)
    L.lora_base_product(L.BaseWeight(W, torch.ones(2, device=DEV)), q, torch.ones(T, device=DEV), y)
    assert torch.equal(y, (q[:, :1].float() * d).expand(T, 2))


def test_product_of_a_row_does_not_depend_on_the_others():
    """A row's results have the same bits in a batch of any size: one kernel or another, the sum is exact and what
    follows it is the same."""
    g = gen(11)
    q, W = i8((700, 1040), g).to(DEV), i8((333, 1040), g).to(DEV)
    qs, ws, b = torch.rand(700, generator=g).to(DEV), torch.rand(333, generator=g).to(DEV), torch.randn(333, generator=g).to(DEV)
    w = L.BaseWeight(W, ws, b)
    whole = torch.empty(700, 333, device=DEV)
    L.lora_base_product(w, q, qs, whole)
    for lo, n in ((0, 1), (5, 16), (30, 31), (64, 64), (100, 100), (300, 400)):
        y = torch.empty(n, 333, device=DEV)
        L.lora_base_product(w, q[lo:lo + n], qs[lo:lo + n], y)
        assert torch.equal(y, whole[lo:lo + n]), (lo, n)
        odd = torch.zeros(n, 1041, dtype=torch.int8, device=DEV)[:, 1:]  # the same rows, at odd addresses
        odd.copy_(q[lo:lo + n])
        L.lora_base_product(w, odd, qs[lo:lo + n], y)
        assert torch.equal(y, whole[lo:lo + n]), (lo, n)


def test_product_many_channels():
    """More channels than a launch takes: the last ones are right."""
    n, d = (1 << 17) + 33, 16
    W = (torch.arange(n, device=DEV).view(-1, 1) % 251 - 125).to(torch.int8).expand(n, d).contiguous()
    q = torch.ones(3, d, dtype=torch.int8, device=DEV)
    b = torch.arange(n, device=DEV, dtype=torch.float32)
    y = torch.zeros(3, n, device=DEV)
    L.lora_base_product(L.BaseWeight(W, torch.ones(n, device=DEV), b), q, torch.ones(3, device=DEV), y)
    assert torch.equal(y, (W[:, 0].float() * d + b).expand(3, n))


# --------------------------------------------------------------------- apply --
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("T, d_in, d_out", [(1, 64, 48), (1, 4096, 256), (4, 1001, 77), (16, 512, 512), (64, 4096, 320),
                                            (65, 100, 40), (300, 1280, 640), (33, 17, 5)])
def test_apply(T, d_in, d_out, dtype):
    g = gen(T + d_in)
    x = (torch.randn(T, d_in, generator=g) * 3).to(dtype)
    if T > 2:
        x[1] = 0
    W, ws, b = i8((d_out, d_in), g), torch.rand(d_out, generator=g) * 0.01, torch.randn(d_out, generator=g)
    w = L.BaseWeight(W.to(DEV), ws.to(DEV), b.to(DEV))
    y = torch.full((T + 1, d_out), 5.0, dtype=dtype, device=DEV)
    ws8 = L.new_base_workspace(w, T)
    ws8.fill_(255)
    L.lora_base_apply(w, x.to(DEV), y, ws8)
    q, s = ref_quantize(x)
    ref, mag = ref_product(q, s, W, ws, b)
    assert bool(((y[:T].cpu().double() - ref).abs() <= half(dtype) * ref.abs() + 4 * V * mag).all())
    assert bool((y[T] == 5).all())


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("T", [1, 2, 40, 200])
def test_apply_on_columns_of_wider_buffers(T, dtype):
    """x and y as column ranges: their neighbours are not read (NaN) and not written."""
    g = gen(T)
    d_in, d_out = 200, 72
    xb = torch.full((T, d_in + 30), float("nan"), dtype=dtype, device=DEV)
    x = xb[:, 16:16 + d_in]
    x.copy_(torch.randn(T, d_in, generator=g).to(dtype))
    W, ws = i8((d_out, d_in), g), torch.rand(d_out, generator=g) * 0.01
    w = L.BaseWeight(W.to(DEV), ws.to(DEV))
    yb = torch.full((T, d_out + 9), 7.0, dtype=dtype, device=DEV)
    L.lora_base_apply(w, x, yb[:, 5:5 + d_out], L.new_base_workspace(w, T))
    q, s = ref_quantize(x.cpu())
    ref, mag = ref_product(q, s, W, ws, None)
    assert bool(((yb[:, 5:5 + d_out].cpu().double() - ref).abs() <= half(dtype) * ref.abs() + 4 * V * mag).all())
    assert bool((yb[:, :5] == 7).all()) and bool((yb[:, 5 + d_out:] == 7).all())


def test_nothing_to_do():
    """No rows, no tokens: nothing is launched or written."""
    w = L.BaseWeight(torch.ones(8, 16, dtype=torch.int8, device=DEV), torch.ones(8, device=DEV))
    y = torch.full((3, 8), 7.0, device=DEV)
    e = torch.empty(0, device=DEV)
    L.lora_base_product(w, torch.empty(0, 16, dtype=torch.int8, device=DEV), e, y)
    L.lora_base_apply(w, torch.empty(0, 16, device=DEV), y, L.new_base_workspace(w, 0))
    r = L.Rotary(L.lora_rotary_frequencies(8).to(DEV), 8)
    L.lora_rotary_apply(r, torch.empty(0, dtype=torch.int32, device=DEV), [torch.empty(0, 2, 8, device=DEV)])
    assert bool((y == 7).all())


def test_apply_nan_row_stays_in_its_row():
    g = gen(1)
    x = torch.randn(10, 64, generator=g)
    clean = x.clone()
    x[4, 9] = float("inf")
    w = L.BaseWeight(i8((32, 64), g).to(DEV), torch.rand(32, generator=g).to(DEV))
    out = []
    for v in (x, clean):
        y = torch.zeros(10, 32, device=DEV)
        L.lora_base_apply(w, v.to(DEV), y, L.new_base_workspace(w, 10))
        out.append(y)
    keep = torch.arange(10) != 4
    assert bool(out[0][4].isnan().all()) and torch.equal(out[0][keep], out[1][keep])


# -------------------------------------------------------------------- rotary --
def ref_rotary(x, pos, freq, rot, interleaved, inverse, m):
    w = pos.double()[:, None, None] * freq * (-1 if inverse else 1)
    c, s = torch.cos(w) * m, torch.sin(w) * m
    y, mag = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64)
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x.double()[..., i], x.double()[..., j]
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    mag[..., i] = mag[..., j] = a.abs() + b.abs()
    skip = pos < 0
    return y, mag, skip


def check_rotary(T, heads, D, rot, dtype, interleaved=False, heads_first=False, inverse=False, in_place=True, m=1.0, pad=0,
                 off=0, max_pos=10000, skip=False, seed=0):
    g = gen(seed + T + D + rot)
    freq = L.lora_rotary_frequencies(rot)
    pos = torch.randint(0, max_pos, (T,), generator=g, dtype=torch.int32)
    if skip and T > 1:
        pos[::3] = -1
    rotary = L.Rotary(freq.to(DEV), D, interleaved=interleaved, mscale=m)
    srcs, dsts, host, bufs = [], [], [], []

    def view(h, fill):
        shape = (h, T, D + pad) if heads_first else (T, h, D + pad)
        buf = torch.full((off + h * T * (D + pad) + 8,), fill, dtype=dtype, device=DEV)
        v = buf[off:off + h * T * (D + pad)].view(shape)[..., :D]
        return buf, v.transpose(0, 1) if heads_first else v

    for h in heads:
        x = torch.randn(T, h, D, generator=g).to(dtype)
        buf, v = view(h, 7.0)
        v.copy_(x)
        srcs.append(v)
        host.append(x)
        if not in_place:
            buf, v = view(h, 7.0)
        bufs.append(buf)
        dsts.append(v)
    L.lora_rotary_apply(rotary, pos.to(DEV), srcs, None if in_place else dsts, inverse=inverse)
    for x, v, s, buf in zip(host, dsts, srcs, bufs):
        y, mag, skipped = ref_rotary(x, pos, freq, rot, interleaved, inverse, float(np.float32(m)))
        got = v.cpu()
        live = ~skipped
        tol = half(dtype) * y.abs() + 6 * V * m * mag
        assert bool(((got.double() - y).abs() <= tol)[live].all())
        # values that are not part of a pair, skipped tokens and what lies between heads keep their bits
        assert torch.equal(got[live][..., rot:], x[live][..., rot:])
        assert torch.equal(got[skipped], x[skipped] if in_place else torch.full_like(x[skipped], 7.0))
        if not in_place:
            assert torch.equal(s.cpu(), x)
        v.fill_(7.0)
        assert bool((buf == 7.0).all())


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T, heads, D, rot", [(1, [1], 2, 2), (1, [32, 8], 128, 128), (3, [3], 80, 34), (64, [4, 1], 64, 64),
                                              (17, [5, 2], 96, 48), (5, [1, 1], 256, 256), (129, [2], 80, 80), (7, [3], 33, 8),
                                              (2, [2, 1], 1024, 1024), (300, [1], 16, 2), (33, [6], 72, 40), (9, [7], 40, 36)])
def test_rotary(T, heads, D, rot, interleaved, dtype):
    check_rotary(T, heads, D, rot, dtype, interleaved)
    check_rotary(T, heads, D, rot, dtype, interleaved, in_place=False, skip=True, m=1.25)
    check_rotary(T, heads, D, rot, dtype, interleaved, heads_first=True, inverse=True, skip=True)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pad, off", [(1, 0), (8, 0), (0, 1), (3, 5), (8, 8), (2, 2), (4, 4)])
def test_rotary_strides_and_alignment(pad, off, interleaved, dtype):
    for in_place in (True, False):
        check_rotary(13, [4, 2], 64, 48, dtype, interleaved, pad=pad, off=off, in_place=in_place)
        check_rotary(13, [4, 2], 64, 64, dtype, interleaved, pad=pad, off=off, in_place=in_place, heads_first=True)


def test_rotary_eight_slices():
    check_rotary(21, [1, 2, 3, 4, 5, 6, 7, 8], 64, 64, torch.bfloat16)


def test_rotary_far_positions():
    """Positions of millions keep their angles: the float64 product is off by 2^-53 of up to 3.2e5 turns and its
    reduction by as much, below 2^-33 turns."""
    check_rotary(50, [2], 64, 64, torch.float32, max_pos=2000000)


def test_rotary_values_that_pass_through_may_be_anything():
    D, rot = 16, 8
    freq = L.lora_rotary_frequencies(rot).to(DEV)
    for interleaved in (False, True):
        x = torch.ones(2, 1, D, device=DEV)
        x[0, 0, rot] = float("inf")
        x[1, 0, rot + 1] = float("nan")
        y = torch.zeros_like(x)
        L.lora_rotary_apply(L.Rotary(freq, D, interleaved=interleaved, mscale=2.0), torch.tensor([5, 6], dtype=torch.int32,
                            device=DEV), [x], [y])
        assert torch.equal(y[..., rot:].view(torch.int32), x[..., rot:].view(torch.int32))
        assert bool(y[..., :rot].isfinite().all())


def test_rotary_inverse_is_the_gradient():
    """<rotate(x), g> = <x, inverse(g)>, and differences along a direction."""
    g = gen(0)
    T, h, D, rot = 6, 3, 32, 24
    freq = L.lora_rotary_frequencies(rot).to(DEV)
    pos = torch.randint(0, 500, (T,), generator=g, dtype=torch.int32).to(DEV)
    r = L.Rotary(freq, D, mscale=1.5)
    x, dy, dx = (torch.randn(T, h, D, generator=g).to(DEV) for _ in range(3))
    fwd = lambda v: (lambda o: (L.lora_rotary_apply(r, pos, [v], [o]), o)[1])(torch.empty_like(v))  # noqa: E731
    grad = torch.empty_like(dy)
    L.lora_rotary_apply(r, pos, [dy], [grad], inverse=True)
    left, right = (fwd(x).double() * dy.double()).sum(), (x.double() * grad.double()).sum()
    # each value is off by at most 7 v m (|a| + |b|): 2 sums of 576 such, weighted by normal numbers
    bound = 7 * V * 1.5 * 2 * float((x.abs().sum() * dy.abs().max() + dy.abs().sum() * x.abs().max()))
    assert abs(float(left - right)) <= bound
    # the map is linear, so a difference over a step of 1 is exact up to the roundings of its two ends
    diff = ((fwd(x + dx).double() - fwd(x).double()) * dy.double()).sum()
    expect = ((x + dx - x).double() * grad.double()).sum()
    bound = 7 * V * 1.5 * 4 * float((x.abs() + (x + dx).abs() + dx.abs()).sum() * dy.abs().max()) * 2
    assert abs(float(diff - expect)) <= bound


def test_rotary_rows_far_apart():
    """Token strides that put later tokens beyond 4 GiB."""
    T, D = 3, 64
    st = (1 << 31) // 2 + 64
    buf = torch.empty(T * st, dtype=torch.float32, device=DEV)
    v = buf.as_strided((T, 2, D), (st, D, 1))
    x = torch.randn(T, 2, D, generator=gen(2))
    v.copy_(x)
    freq = L.lora_rotary_frequencies(D)
    pos = torch.tensor([3, 0, 77], dtype=torch.int32)
    L.lora_rotary_apply(L.Rotary(freq.to(DEV), D), pos.to(DEV), [v])
    y, mag, _ = ref_rotary(x, pos, freq, D, False, False, 1.0)
    assert bool(((v.cpu().double() - y).abs() <= V * y.abs() + 6 * V * mag).all())


def test_rotary_more_tokens_than_a_launch_takes():
    T = (1 << 24) + 5
    x = torch.ones(T, 1, 2, device=DEV)
    pos = (torch.arange(T, device=DEV) % 1000).int()
    freq = torch.tensor([0.5], dtype=torch.float64, device=DEV)
    L.lora_rotary_apply(L.Rotary(freq, 2), pos, [x])
    for lo in (0, (1 << 24) - 1000):
        w = pos[lo:].double()[:2000] * 0.5
        ref = torch.stack([torch.cos(w) - torch.sin(w), torch.cos(w) + torch.sin(w)], -1)
        assert bool(((x[lo:, 0][:2000].double() - ref).abs() <= V * ref.abs() + 12 * V).all())


@pytest.mark.parametrize("interleaved, rot", [(False, 64), (False, 36), (True, 36)])
def test_rotary_one_slice_in_place_one_not_one_broadcast(interleaved, rot):
    """In one launch: a tensor in place, one into another tensor, and one head spread to several."""
    g = gen(8)
    T, D = 50, 64
    freq = L.lora_rotary_frequencies(rot)
    pos = torch.randint(0, 900, (T,), generator=g, dtype=torch.int32)
    xs = [torch.randn(T, h, D, generator=g) for h in (3, 2, 1)]
    dev = [x.to(DEV) for x in xs]
    out = [dev[0], torch.empty(T, 2, D, device=DEV), torch.empty(T, 4, D, device=DEV)]
    L.lora_rotary_apply(L.Rotary(freq.to(DEV), D, interleaved=interleaved), pos.to(DEV),
                        [dev[0], dev[1], dev[2].expand(T, 4, D)], out)
    for x, o in zip([xs[0], xs[1], xs[2].expand(T, 4, D)], out):
        y, mag, _ = ref_rotary(x, pos, freq, rot, interleaved, False, 1.0)
        assert bool(((o.cpu().double() - y).abs() <= V * y.abs() + 6 * V * mag).all())
        assert torch.equal(o.cpu()[..., rot:], x[..., rot:])


def test_rotary_refusals_of_the_binding():
    freq = L.lora_rotary_frequencies(8).to(DEV)
    r = L.Rotary(freq, 16)
    pos = torch.zeros(2, dtype=torch.int32, device=DEV)
    x = torch.zeros(2, 3, 16, device=DEV)
    for src, dst, p in (([x[:, :, :8]], None, pos), ([x.half()], None, pos), ([x[:1]], None, pos), ([], None, pos),
                        ([x], [x, x], pos), ([x], [x.bfloat16()], pos), ([x.cpu()], None, pos), ([x], None, pos.long()),
                        ([x[:, :1].expand(2, 3, 16)], None, pos), ([x, x], None, pos), ([x] * 9, None, pos),
                        ([x.transpose(1, 2).contiguous().transpose(1, 2)], None, pos)):
        with pytest.raises(L.LoraError):
            L.lora_rotary_apply(r, p, src, dst)
    with pytest.raises(L.LoraError):
        L.Rotary(freq, 7)
    assert bool((x == 0).all())


def test_product_refusals_of_the_binding():
    W, s = torch.zeros(32, 64, dtype=torch.int8, device=DEV), torch.ones(32, device=DEV)
    w = L.BaseWeight(W, s)
    q, qs, y = torch.zeros(4, 64, dtype=torch.int8, device=DEV), torch.ones(4, device=DEV), torch.zeros(4, 32, device=DEV)
    for a in ((q[:, :63], qs, y), (q, qs[:3], y), (q, qs, y[:3]), (q, qs, y[:, :31]), (q.float(), qs, y), (q, qs, y.half()),
              (q.t().contiguous().t(), qs, y), (q.cpu(), qs, y), (q, qs.double(), y)):
        with pytest.raises(L.LoraError):
            L.lora_base_product(w, *a)
    for a in ((W.float(), s), (W, s[:31]), (W, s, s[:31]), (W, s.double()), (W.t(), s), (W[:0], s[:0])):
        with pytest.raises(L.LoraError):
            L.BaseWeight(*a)
    x = torch.zeros(4, 64, device=DEV)
    for a in ((x, y, L.new_base_workspace(w, 4)[:-256]), (x.bfloat16(), y, L.new_base_workspace(w, 4)), (x[:, :32], y, q)):
        with pytest.raises(L.LoraError):
            L.lora_base_apply(w, *a)
    with pytest.raises(L.LoraError):
        L.lora_quantize_rows(x, q[:, :32], qs)


# ------------------------------------------------------- streams, graphs, runs --
def layer(T, seed, dtype=torch.bfloat16):
    """One layer's query and key projections: base weight, LoRA pool, rotary, and a batch of requests."""
    g = gen(seed)
    d, H, K, D, n, r = 256, 4, 2, 64, 5, 16
    out = (H + K) * D
    W = torch.randn(out, d, generator=g) * 0.05
    Wq, Ws = ref_quantize(W)
    A, Bq, Bk = (torch.randn(n, r, d, generator=g) * 0.05, torch.randn(n, H * D, r, generator=g) * 0.05,
                 torch.randn(n, K * D, r, generator=g) * 0.05)
    idx = torch.randint(-1, n, (T, 1), generator=g, dtype=torch.int32)
    pos = torch.randint(0, 4000, (T,), generator=g, dtype=torch.int32)
    x = torch.randn(T, d, generator=g).to(dtype)
    return dict(d=d, H=H, K=K, D=D, n=n, Wq=Wq, Ws=Ws, A=A.to(dtype), Bq=Bq.to(dtype), Bk=Bk.to(dtype), idx=idx, pos=pos, x=x,
                freq=L.lora_rotary_frequencies(D))


class DevLayer:
    def __init__(self, m):
        dev = lambda t: t.to(DEV)  # noqa: E731
        self.m, T = m, m["x"].shape[0]
        self.w = L.BaseWeight(dev(m["Wq"]), dev(m["Ws"]))
        self.x = dev(m["x"])
        self.y = torch.zeros(T, (m["H"] + m["K"]) * m["D"], dtype=self.x.dtype, device=DEV)
        self.q, self.k = self.y[:, :m["H"] * m["D"]], self.y[:, m["H"] * m["D"]:]
        self.A, self.Bq, self.Bk = dev(m["A"]), dev(m["Bq"]), dev(m["Bk"])
        self.pool = L.Pool(self.A, self.Bq)
        self.batch = L.Batch(T, dev(m["idx"]))
        self.plan = L.new_workspace(self.batch, m["n"], DEV)
        L.lora_plan_build(self.batch, m["n"], self.plan)
        self.table, self.widths, self.aligned = L.sliced_table([(self.x, [(self.A, self.Bq, self.q), (self.A, self.Bk, self.k)])],
                                                               DEV)
        self.ws = L.new_base_workspace(self.w, T)
        self.rotary = L.Rotary(dev(m["freq"]), m["D"])
        self.pos = dev(m["pos"])
        self.heads = [v.unflatten(1, (-1, m["D"])) for v in (self.q, self.k)]

    def run(self):
        L.lora_base_apply(self.w, self.x, self.y, self.ws)
        L.lora_apply_sliced(self.pool, self.batch, self.plan, self.table, self.widths, self.aligned)
        L.lora_rotary_apply(self.rotary, self.pos, self.heads)


def ref_layer(m):
    """The layer in 64 bits, and how far off it may be: the base product is rounded to bf16 and read again by the LoRA
    step (2^-8 of it), which has the library's tolerance 1e-2 (1 + |y|); the rotation mixes the errors of a pair as it
    mixes the values (|cos|, |sin| <= 1) and rounds once more."""
    q, s = ref_quantize(m["x"])
    x = m["x"].double()
    y0 = (q.double() @ m["Wq"].double().T) * s.double()[:, None] * m["Ws"].double()
    B = torch.cat([m["Bq"], m["Bk"]], 1).double()
    y = y0.clone()
    for t, i in enumerate(m["idx"][:, 0].tolist()):
        if i >= 0:
            y[t] += x[t] @ m["A"][i].double().T @ B[i].T
    err = 2.0 ** -8 * y0.abs() + 1e-2 * (1 + y.abs())
    T, D, rot = y.shape[0], m["D"], m["D"]
    y3, e3 = y.view(T, -1, D), err.view(T, -1, D)
    out, mag, _ = ref_rotary(y3, m["pos"], m["freq"], rot, False, False, 1.0)
    e = torch.cat([e3[..., :D // 2] + e3[..., D // 2:]] * 2, -1)
    return out, e + 2.0 ** -8 * (out.abs() + e) + 6 * V * mag


@pytest.mark.parametrize("T", [1, 5, 64, 200])
def test_layer(T):
    """Quantised base product, the adapters of a mixed batch on its columns, rotary positions on the same columns."""
    m = layer(T, T)
    dl = DevLayer(m)
    dl.run()
    ref, tol = ref_layer(m)
    assert bool(((dl.y.view(T, -1, m["D"]).cpu().double() - ref).abs() <= tol).all())


def test_layers_on_two_streams():
    """Two layers at once, each on a stream of its own, give what each gives alone."""
    ls = [DevLayer(layer(100, 1)), DevLayer(layer(150, 2))]
    want = []
    for dl in ls:
        dl.run()
        want.append(dl.y.clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ls]
    for _ in range(20):
        for dl, s in zip(ls, streams):
            with torch.cuda.stream(s):
                dl.run()
    torch.cuda.synchronize()
    for dl, w in zip(ls, want):
        assert torch.equal(dl.y, w)


def test_layer_in_a_graph():
    """Captured once, replayed on new inputs, with eager work between: every replay gives what an eager run gives."""
    a, b = DevLayer(layer(40, 3)), DevLayer(layer(40, 3))
    a.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
    g = gen(9)
    for i in range(4):
        x = torch.randn(40, 256, generator=g).to(torch.bfloat16).to(DEV)
        pos = torch.randint(-1, 3000, (40,), generator=g, dtype=torch.int32).to(DEV)
        for dl in (a, b):
            dl.x.copy_(x)
            dl.pos.copy_(pos)
        graph.replay()
        b.run()
        torch.cuda.synchronize()
        assert torch.equal(a.y, b.y), i


def test_two_graphs_share_a_workspace():
    """Two captured calls on one workspace, replayed one after the other: it holds nothing between calls."""
    g = gen(4)
    w = L.BaseWeight(i8((96, 128), g).to(DEV), torch.rand(96, generator=g).to(DEV))
    ws = L.new_base_workspace(w, 64)
    xs = [torch.randn(n, 128, generator=g).to(torch.bfloat16).to(DEV) for n in (64, 7)]
    ys = [torch.zeros(len(x), 96, dtype=torch.bfloat16, device=DEV) for x in xs]
    want = []
    for x, y in zip(xs, ys):
        L.lora_base_apply(w, x, y, ws)
        want.append(y.clone())
    torch.cuda.synchronize()
    graphs = []
    for x, y in zip(xs, ys):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            L.lora_base_apply(w, x, y, ws)
        graphs.append(graph)
    for _ in range(3):
        for k in (0, 1, 1, 0):
            ys[k].zero_()
            graphs[k].replay()
            torch.cuda.synchronize()
            assert torch.equal(ys[k], want[k])


@pytest.mark.parametrize("T", [4, 64, 600])
def test_same_bits_again(T):
    dl = DevLayer(layer(T, 5))
    dl.run()
    y = dl.y.clone()
    for _ in range(3):
        dl.y.fill_(9)
        dl.run()
        assert torch.equal(dl.y, y)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("d_out, pad", [(2112, 0), (2048, 64), (2048, 3)])
def test_product_result_larger_than_the_caches(d_out, pad, dtype):
    """More than 32 MiB of results: what calls for parts of the rows give, and the columns beside them as they were."""
    g, T, d_in = torch.Generator(device=DEV).manual_seed(3), 8333, 1024
    W, q = (torch.randint(-127, 128, s, generator=g, dtype=torch.int8, device=DEV) for s in ((d_out, d_in), (T, d_in)))
    qs, sc = torch.rand(T, generator=g, device=DEV), torch.rand(d_out, generator=g, device=DEV)
    w = L.BaseWeight(W, sc)
    y = torch.full((T, d_out + pad), 9, dtype=dtype, device=DEV)
    L.lora_base_product(w, q, qs, y[:, :d_out])
    part = torch.full_like(y, 9)
    for t in range(0, T, 1000):
        L.lora_base_product(w, q[t:t + 1000], qs[t:t + 1000], part[t:t + 1000, :d_out])
    assert torch.equal(y, part)
    ref, mag = ref_product(q[-300:].cpu(), qs[-300:].cpu(), W.cpu(), sc.cpu(), None)[:2]
    assert bool(((y[-300:, :d_out].cpu().double() - ref).abs() <= half(dtype) * ref.abs() + 4 * V * mag).all())


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rot, interleaved, pad", [(128, False, 0), (128, True, 0), (70, False, 0), (128, False, 4)])
def test_rotary_result_larger_than_the_caches(rot, interleaved, pad, dtype):
    """More than 32 MiB of heads, in place and not: what calls for parts of the tokens give; a skipped token is left."""
    g, T, H, D = torch.Generator(device=DEV).manual_seed(4), 4321, 36, 128
    x = torch.randn(T, H, D + pad, generator=g, device=DEV).to(dtype)
    pos = torch.randint(-2, 5000, (T,), generator=g, dtype=torch.int32, device=DEV)
    r = L.Rotary(L.lora_rotary_frequencies(rot).to(DEV), D, interleaved=interleaved)
    y, part, own = torch.full_like(x, 9), torch.full_like(x, 9), x.clone()
    L.lora_rotary_apply(r, pos, [x[..., :D]], [y[..., :D]])
    L.lora_rotary_apply(r, pos, [own[..., :D]])
    for t in range(0, T, 500):
        L.lora_rotary_apply(r, pos[t:t + 500], [x[t:t + 500, :, :D]], [part[t:t + 500, :, :D]])
    assert torch.equal(y, part)
    keep = pos >= 0
    assert torch.equal(own[keep][..., :D], part[keep][..., :D])
    assert torch.equal(own[~keep], x[~keep])
    assert bool((y[~keep] == 9).all()) and torch.equal(own[..., D:], x[..., D:])


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_one_row_as_the_transpose_of_a_column(dtype):
    """[1][d] with strides (1, 1), which torch calls contiguous, as x, q and y of the calls that take rows."""
    g, d, n = gen(21), 200, 72
    x = torch.randn(1, d, generator=g).to(dtype)
    W, ws = i8((n, d), g), torch.rand(n, generator=g) * 0.01
    w = L.BaseWeight(W.to(DEV), ws.to(DEV))
    column = lambda k, t: torch.zeros(k, 1, dtype=t, device=DEV).t()  # noqa: E731
    xv, qv, s, y = column(d, dtype), column(d, torch.int8), torch.zeros(1, device=DEV), column(n, dtype)
    assert xv.stride() == (1, 1) and xv.is_contiguous()
    xv.copy_(x)
    L.lora_quantize_rows(xv, qv, s)
    q, qs = ref_quantize(x)
    assert torch.equal(qv.cpu(), q) and torch.equal(s.cpu(), qs)
    ref, mag = ref_product(q, qs, W, ws, None)
    tol = half(dtype) * ref.abs() + 4 * V * mag
    L.lora_base_product(w, qv, s, y)
    assert bool(((y.cpu().double() - ref).abs() <= tol).all())
    y.zero_()
    L.lora_base_apply(w, xv, y, L.new_base_workspace(w, 1))
    assert bool(((y.cpu().double() - ref).abs() <= tol).all())


PI = fractions.Fraction(31415926535897932384626433832795028841971693993751058209749445923078164062862, 10 ** 76)


@pytest.mark.parametrize("lo, hi", [(0, 1000), (1 << 30, (1 << 31) - 1)])
def test_rotary_angles_at_the_ends_of_the_positions(lo, hi):
    """Pairs (1, 0) give cosine and sine themselves: no rounding follows them.  The angle is reduced exactly here.  One
    that is off by v / 2, as a float32 below pi / 4 is, and a float32 series end below 1.4 v for cosine (v / 2 of the
    angle times sin w, the last rounding v / 2, w^2 / 2 by one rounding and its factor by a quarter) and below 1.2 v
    for sine (cos w times v / 2, v / 2, w^3 / 6 by three roundings)."""
    rot, T = 32, 400
    freq = L.lora_rotary_frequencies(rot)
    pos = torch.from_numpy(np.random.default_rng(7).integers(lo, hi, T)).int()
    pos[-1] = hi
    x = torch.zeros(T, 1, rot)
    x[..., ::2] = 1
    x = x.to(DEV)
    L.lora_rotary_apply(L.Rotary(freq.to(DEV), rot, interleaved=True), pos.to(DEV), [x])
    turns = [[fractions.Fraction(p) * fractions.Fraction(f) / (2 * PI) for f in freq.tolist()] for p in pos.tolist()]
    w = torch.tensor([[float((t - round(t)) * 2 * PI) for t in row] for row in turns], dtype=torch.float64)
    got = x.cpu().double()[:, 0]
    assert float((got[:, ::2] - torch.cos(w)).abs().max()) <= 1.4 * V
    assert float((got[:, 1::2] - torch.sin(w)).abs().max()) <= 1.4 * V


# sizes that are split into whole rounds and a rest: of 256 x 256 tiles with each of three kernels behind, of 192 x 256
SPLITS = [(13628, 592, 1826), (4135, 1296, 4039), (7751, 1168, 2062), (16997, 4096, 4096)]


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("T, d_in, d_out", TILES + SPLITS)
def test_product_in_whole_lines(T, d_in, d_out, dtype):
    """Every tile shape and the split launches, with rows of y that begin on whole 128-byte lines, where whole tiles
    leave past the caches; against the float64 product on the GPU, the columns and rows beside y as they were."""
    g = torch.Generator(device=DEV).manual_seed(T)
    rand8 = lambda n: torch.randint(-127, 128, (n, d_in), generator=g, dtype=torch.int8, device=DEV)  # noqa: E731
    q, W = rand8(T), rand8(d_out)
    qs, ws, b = (torch.rand(n, generator=g, device=DEV) * 0.02 for n in (T, d_out, d_out))
    line = 128 // torch.tensor([], dtype=dtype).element_size()
    yb = torch.full((T + 1, (d_out + line - 1) // line * line), 7.0, dtype=dtype, device=DEV)
    assert yb.data_ptr() % 128 == 0
    L.lora_base_product(L.BaseWeight(W, ws, b), q, qs, yb[:T, :d_out])
    for lo in range(0, T, 4096):
        p = (q[lo:lo + 4096].double() @ W.double().T) * qs[lo:lo + 4096, None].double() * ws.double()
        ref = p + b.double()
        y = yb[lo:min(lo + 4096, T), :d_out].double()
        bad = (y - ref).abs() > half(dtype) * ref.abs() + 4 * V * (p.abs() + b.double().abs())
        assert not bool(bad.any()), (lo, int(bad.sum()), bad.nonzero()[:4].tolist())
    assert bool((yb[T] == 7).all()) and bool((yb[:, d_out:] == 7).all())


@pytest.mark.parametrize("m", [1.0, 1.2])
@pytest.mark.parametrize("hi", [1000, 1000000, (1 << 31) - 1])
def test_rotary_cosine_and_sine_are_rounded_once(hi, m):
    """Pairs (1, 0) give m cos w and m sin w, within half a float32 step of numbers below 2^k, 2^k v / 2, and the 2e-9 at
    which the series end (0.03 v).  The angles are reduced exactly here; m is the float32 that the call gets."""
    rot, T = 32, 400
    freq = L.lora_rotary_frequencies(rot)
    pos = torch.from_numpy(np.random.default_rng(9).integers(hi // 2, hi, T)).int()
    x = torch.zeros(T, 1, rot)
    x[..., ::2] = 1
    x = x.to(DEV)
    L.lora_rotary_apply(L.Rotary(freq.to(DEV), rot, interleaved=True, mscale=m), pos.to(DEV), [x])
    turns = [[fractions.Fraction(p) * fractions.Fraction(f) / (2 * PI) for f in freq.tolist()] for p in pos.tolist()]
    w = torch.tensor([[float((t - round(t)) * 2 * PI) for t in row] for row in turns], dtype=torch.float64)
    got = x.cpu().double()[:, 0]
    for v, ref in ((got[:, ::2], torch.cos(w)), (got[:, 1::2], torch.sin(w))):
        ref = ref * float(np.float32(m))
        step = torch.where(ref.abs() < 1 - V, 1.0, 2.0)  # values from 1 to 2 have steps of 2 v
        assert bool(((v - ref).abs() <= (0.5 * step + 0.03 * m) * V).all()), float(((v - ref).abs() / step).max() / V)
